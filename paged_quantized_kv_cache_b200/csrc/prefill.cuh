// prefill.cuh -- chunked-prefill attention over the paged cache, and attention
// to an encoder's states in it (tcgen05).
#pragma once

#include <cudaTypedefs.h>

#include "common.cuh"

namespace pqkv {

constexpr int kMaxSplits = 8;  // CTAs of a cluster (the portable limit)

struct PrefillParams {
  const void* q;                // [cu_q[B]][Hq][D]
  void* out;                    // same shape and type as q
  const uint8_t* cache;
  const uint8_t* scales;
  const uint8_t* oidx;
  const uint8_t* oval;
  const int32_t* cu_q;          // [B + 1] query-token offsets
  const int32_t* seq_lens;      // [B] cached positions, the chunk's own included
  const int32_t* block_tables;  // [B][maxblk]
  int32_t* err;
  int B, Hq, Hkv, G, nb, maxblk;
  int tiles_per_seq;            // 128-row query tiles per sequence (from the longest chunk)
  float scale_log2;             // softmax scale * log2(e)
  uint64_t timeout_ns;          // limit of a wait before the CTA gives up
  uint64_t drain_ns;            // after giving up: limit of the wait for work still in flight
  // attention to an encoder's states only
  const int32_t* ranges;        // [cu_q[B]][2] positions each query token sees, or null: all
  int max_q;                    // query tokens of the longest sequence
  int splits;                   // CTAs of a cluster that share a tile pair's KV range
  // The softmax takes a scale above 0 (masked scores are -inf before they are
  // scaled): a scale below 0 turns the sign of the queries' words instead, and
  // at 0 the queries are zeros with a scale of 1.
  uint32_t q_and, q_xor;
};

cudaError_t launch_prefill(int kv_dtype, int D, bool q_bf16, const CUtensorMap& tmap16, const PrefillParams& p,
                           cudaStream_t st);
// Attention to an encoder's states: tiles of query rows on tcgen05 (cross.cu,
// map as the prefill's), or at most kFewColumns rows per KV head (cross_few.cu,
// map as the decode's; any sign of scale_log2). The launchers set p.splits.
constexpr int kFewColumns = 16;
cudaError_t launch_cross(int kv_dtype, int D, bool q_bf16, const CUtensorMap& tmap16, const PrefillParams& p, int sms,
                         cudaStream_t st);
cudaError_t launch_cross_few(int kv_dtype, int D, bool q_bf16, const CUtensorMap& tmap, const PrefillParams& p,
                             int sms, cudaStream_t st);
size_t prefill_smem_bytes(int kv_dtype, int D);

}  // namespace pqkv
