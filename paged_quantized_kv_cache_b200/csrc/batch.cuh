// batch.cuh -- the tables of a batch (block tables, slot mapping, positions,
// offsets) built on the GPU from request lengths.
#pragma once

#include "common.cuh"

namespace pqkv {

struct BatchParams {
  const int32_t* start;    // [B] tokens a request has in the cache
  const int32_t* num_new;  // [B] tokens it adds
  const int32_t* ids;      // [n_ids] block ids for this step, request after request
  int32_t* tables;         // [B][maxblk], extended in place
  int32_t* slots;          // [cap]
  int32_t* positions;      // [cap]
  int32_t* cu;             // [B + 1]
  int32_t* lens;           // [B]
  int32_t* err;
  int B, n_ids, maxblk, nb, cap;
};

cudaError_t launch_build_batch(const BatchParams& p, int sms, cudaStream_t st);

}  // namespace pqkv
