// cross.cuh -- attention of decoder tokens to an encoder's cached states.
#pragma once

#include <cudaTypedefs.h>

#include "common.cuh"
#include "tcgen05.cuh"

namespace pqkv {

// Query rows (tokens x query heads) per KV head up to which the few-rows kernel
// runs. It against the many-rows kernel, 16 sequences of 1400-1500 states, 32 / 8
// heads of 128, us: 4 rows bf16 21.2 / 25.7, FP8 18.9 / 36.3, FP4 23.6 / 40.8;
// 16 rows bf16 27.1 / 26.1, FP8 27.0 / 37.0, FP4 42.8 / 40.9; 64 sequences of
// 2048-6404 states: 4 rows bf16 163 / 201, FP8 104 / 308, FP4 137 / 363; 16 rows
// bf16 184 / 203, FP8 154 / 312, FP4 222 / 365. So 16 rows of few sequences lose
// 4-5% to the other kernel over bf16 and FP4, and win elsewhere. It has registers
// for two tiles of 8 columns and no more.
constexpr int kFewColumns = 16;

struct CrossParams {
  const void* q;                // [cu_q[B]][Hq][D]
  void* out;                    // same shape and type as q
  const uint8_t* cache;
  const uint8_t* scales;
  const uint8_t* oidx;
  const uint8_t* oval;
  const int32_t* cu_q;          // [B + 1] query-token offsets
  const int32_t* kv_lens;       // [B] states of each sequence
  const int32_t* block_tables;  // [B][maxblk]
  const int32_t* ranges;        // [cu_q[B]][2] positions each query token sees, or null: all
  int32_t* err;
  int B, Hq, Hkv, G, nb, maxblk;
  int max_q;                    // query tokens of the longest sequence
  int tiles_per_seq;            // 128-row query tiles per sequence
  int splits;                   // CTAs of a cluster, which share the states of their rows (set by the launcher)
  int by_length;                // sequences in the order of their lengths (set by the launcher)
  float scale_log2;             // softmax scale * log2(e)
  uint64_t timeout_ns;          // limit of a wait before a warp gives up
  uint64_t drain_ns;            // after giving up: limit of the wait for work still in flight
};

// Index of the b-th longest of B sequences (B at most the CTA's threads: one
// ranks a sequence; equal ones in order), in `scratch`, B + 1 words of shared
// memory that are free again on return. Every thread of the CTA calls it. With
// more CTAs than fit at once, those of the longest sequences start first, so
// that none of them is left for the end: 64 sequences of 2048-6404 FP8 states,
// one token each, 136 against 112 us.
__device__ __forceinline__ int nth_longest(const int32_t* kv_lens, int B, int b, int* scratch) {
  const int tid = threadIdx.x;
  if (tid < B) scratch[tid] = kv_lens[tid];
  __syncthreads();
  if (tid < B) {
    const int mine = scratch[tid];
    int before = 0;
    for (int i = 0; i < B; ++i) before += scratch[i] > mine || (scratch[i] == mine && i < tid);
    if (before == b) scratch[B] = tid;
  }
  __syncthreads();
  const int chosen = scratch[B];
  tc::fence_smem_to_async();  // the next to write the scratch may be a TMA copy
  __syncthreads();
  return chosen;
}

// FP8 states: O of a row is kept in units of 1 / r, and P enters its product
// with V, in f16, as p s r (s: the V scale of a key's block). The unit goes by
// the largest p s of what the row itself has seen: the scales alone, or those of
// all blocks read, would leave a row of small values beside large ones without
// bits. After a step that moved the row's max (l was multiplied by fl; `any`: the
// row has a max) and brought p s up to `need`: the new r, and what O is
// multiplied by. The unit rises when p s r would pass 2^8, and falls with l, as
// long as r is a float; r is 0 while the row has no max.
__device__ __forceinline__ float move_unit(float& r, float fl, float need, bool any) {
  constexpr float kMost = 0x1p126f;
  const float was = r;
  if (was == 0.f) {
    r = any ? fminf(1.f / need, kMost) : 0.f;
    return fl;
  }
  const bool rises = need * was > 256.f * fl;
  const float to = rises ? 1.f / need : was / fl;
  r = fminf(to, kMost);
  if (!rises && r == to) return 1.f;
  return fl > 0.f ? fl * (r / was) : 0.f;
}

// Tiles of 128 query rows on tcgen05 (cross.cu; the prefill's tensor map for
// 16-bit caches), or at most kFewColumns rows per KV head (cross_few.cu; the
// decode's tensor map).
cudaError_t launch_cross(int kv_dtype, int D, bool q_bf16, const CUtensorMap& tmap16, const CrossParams& p, int sms,
                         cudaStream_t st);
cudaError_t launch_cross_few(int kv_dtype, int D, bool q_bf16, const CUtensorMap& tmap, const CrossParams& p, int sms,
                             cudaStream_t st);
size_t cross_smem_bytes(int kv_dtype, int D);

}  // namespace pqkv
