// rope.cu -- RMS norm of every query and key head and rotary positions on one
// or several axes, in one pass between the projection and the attention;
// optionally the same pass stores keys and values into a 16-bit paged cache.
//
// Row x of D channels (one head of one token): y = x rsqrt(mean x^2 + eps) w,
// then pair i of the first rot channels turns by the token's position on the
// pair's axis: (a, b) -> (a c - b s, b c + a s), c and s from the caller's
// table; one rounding at the end. Positions on several axes (time, height,
// width) differ only in which of the token's positions a pair reads.
//
// Bound by memory: every row is read and written once, 2 D bytes each way. D / 8
// lanes hold a row, four pairs each (two 8-byte pieces, or one of 16 bytes for
// neighbouring pairs), so a rotation needs no exchange between lanes and the
// norm one tree of log2(D / 8) shuffles. A warp takes kUnroll rows per lane of
// one token, all of one kind (queries, keys or values: blockIdx.y): their loads
// are all in flight before the first sum, and the token's positions, cosines
// and sines and the kind's weights are read once for them, and for the further
// TURNS - 1 such groups that the warp takes after them in large calls.
//
// Measured (32 / 8 heads of 128, three axes): 8191 tokens 31.1 us (5.5 TB/s; the
// bytes at copy speed are 26.2), 32768 tokens 112 us (6.2 TB/s). 8191 tokens
// without norm and rotation 27.4, with the norm only 28.2, with one axis 29.9.
#include "rope.cuh"

namespace pqkv {

namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;

// Chunks of `turns` times kUnroll rows per lane that `heads` rows of a token take.
template <int D>
__host__ __device__ constexpr int chunks_of(int heads, int turns) {
  const int rows = 256 / D * kUnroll * turns;
  return (heads + rows - 1) / rows;
}

template <int D, bool BF16, bool IL, int TURNS>
__global__ void __launch_bounds__(kThreads, 8) rope_kernel(const __grid_constant__ RopeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kLanes = D / 8;       // lanes of a row
  constexpr int kRows = 32 / kLanes;  // rows a warp holds at once
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (t >= p.r.T) return;
  int chunk = blockIdx.y, heads = p.Hq;
  const int q_chunks = chunks_of<D>(p.Hq, TURNS), k_chunks = chunks_of<D>(p.Hkv, TURNS);
  const bool is_q = chunk < q_chunks;
  bool is_v = false;
  if (!is_q) {
    chunk -= q_chunks;
    heads = p.Hkv;
    is_v = chunk >= k_chunks;
    if (is_v) chunk -= k_chunks;
  }
  const int row0 = chunk * kRows * kUnroll * TURNS + lane / kLanes;
  // whether the chunk has rows from group at / kUnroll on (the same for the whole warp)
  auto more = [&](int at) { return at < kUnroll * TURNS && (chunk * kUnroll * TURNS + at) * kRows < heads; };
  const int i0 = 4 * (lane % kLanes);
  int a, b;
  pair_channels<D, IL>(i0, p.r.rot, a, b);

  int pos[kMaxAxes];
  if (!is_v) load_positions(p.r, t, pos);
  int slot = -1;
  if (!is_q && !p.k_out) slot = __ldg(p.slots + t);
  const uint16_t* src = is_q ? static_cast<const uint16_t*>(p.q) + (size_t)t * p.qs
                      : is_v ? static_cast<const uint16_t*>(p.v) + (size_t)t * p.vs
                             : static_cast<const uint16_t*>(p.k) + (size_t)t * p.ks;
  uint4 raw[kUnroll];
  const uint16_t* src_a = src + row0 * D + a;
  const uint16_t* src_b = src + row0 * D + b;
  auto load = [&](int at) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      raw[u] = row0 + (at + u) * kRows < heads
                   ? load_pairs<IL>(src_a + (at + u) * kRows * D, src_b + (at + u) * kRows * D)
                   : make_uint4(0, 0, 0, 0);
  };
  load(0);
  // where the rows go: heads of a token follow one another in an output, and lie
  // two tiles of a block apart in the cache
  uint16_t* dst;
  size_t step = D;
  if (is_q) {
    dst = static_cast<uint16_t*>(p.q_out) + (size_t)t * p.Hq * D;
  } else if (p.k_out) {
    dst = static_cast<uint16_t*>(p.k_out) + (size_t)t * p.Hkv * D;
  } else {
    if (slot >= p.nb * kBlock && !is_v && chunk == 0 && lane == 0) raise_flag(p.err, PQKV_DEVERR_SLOT);
    if (slot < 0 || slot >= p.nb * kBlock) return;
    step = 2 * kBlock * D;
    dst = reinterpret_cast<uint16_t*>(p.cache) +
          (((size_t)(slot >> 4) * p.Hkv * 2 + (is_v ? 1 : 0)) * kBlock + (slot & 15)) * D;
  }
  dst += row0 * step;
  auto put = [&](int u, uint4 out) {
    uint16_t* row = dst + u * kRows * step;
    if (row0 + u * kRows < heads) store_pairs<IL>(row + a, row + b, out);
  };
  const float* weight = is_v ? nullptr : is_q ? p.r.q_weight : p.r.k_weight;
  const bool turn = !is_v && 2 * i0 < p.r.rot;
  if (!weight && p.r.rot == 0) is_v = true;  // nothing to do to them either
  Pairs cs;
  if (!is_v && !load_angles(p.r, pos, i0, cs)) {
    if (lane == 0 && chunk == 0) raise_flag(p.err, PQKV_DEVERR_POSITION);
    for (int u = 0; u < kUnroll * TURNS; ++u) put(u, make_uint4(0, 0, 0, 0));
    return;
  }
  if (is_v) {
#pragma unroll 1
    for (int at = 0;;) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) put(at + u, raw[u]);
      at += kUnroll;
      if (!more(at)) return;
      load(at);
    }
  }
  Pairs w = {};
  if (weight) w = load_weight<IL>(weight, a, b);
  const Coefficients k = coefficients<IL>(weight != nullptr, w, turn, cs);
#pragma unroll 1
  for (int at = 0;;) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint4 out = norm_rotate<D, BF16, IL>(raw[u], weight != nullptr, p.r.eps, k);
      put(at + u, weight || turn ? out : raw[u]);
    }
    at += kUnroll;
    if (!more(at)) return;
    load(at);
  }
}

template <int D, bool BF16, bool IL, int TURNS>
cudaError_t launch_turns(const RopeParams& p, cudaStream_t st) {
  const int chunks = chunks_of<D>(p.Hq, TURNS) + p.kinds * chunks_of<D>(p.Hkv, TURNS);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.r.T + kThreads / 32 - 1) / (kThreads / 32)), (unsigned)chunks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, rope_kernel<D, BF16, IL, TURNS>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Groups of rows that a warp takes one after the other, its angles and weights
// read once for all: one while those warps are less than two rounds of the GPU,
// two from there and four from four rounds on. 32 / 8 heads of 128, three axes, us with 1, 2 and 4 groups: 1 token 2.8 / 3.5 / 5.2, 1024
// tokens 6.4 / 6.6 / 7.3, 2048 12.1 / 11.1 / 12.5, 4096 20.2 / 17.9 / 17.4, 8191
// 36.6 / 32.9 / 31.2, 32768 143 / 121 / 112. (A number known only at run time
// spills registers: 34.1 at 8191 tokens.)
template <int D, bool BF16, bool IL>
cudaError_t launch_rope_t(const RopeParams& p, int sms, cudaStream_t st) {
  const long long warps = (long long)p.r.T * (chunks_of<D>(p.Hq, 1) + p.kinds * chunks_of<D>(p.Hkv, 1));
  const long long round = (long long)sms * 8 * (kThreads / 32);
  if (warps >= 4 * round) return launch_turns<D, BF16, IL, 4>(p, st);
  if (warps >= 2 * round) return launch_turns<D, BF16, IL, 2>(p, st);
  return launch_turns<D, BF16, IL, 1>(p, st);
}

}  // namespace

cudaError_t launch_rope(bool bf16, int D, bool interleaved, const RopeParams& p, int sms, cudaStream_t st) {
  if (p.r.T == 0) return cudaSuccess;
#define PQKV_ROPE(DD, BF, IL) \
  if (D == DD && bf16 == BF && interleaved == IL) return launch_rope_t<DD, BF, IL>(p, sms, st);
  PQKV_ROPE(128, true, false)
  PQKV_ROPE(128, true, true)
  PQKV_ROPE(128, false, false)
  PQKV_ROPE(128, false, true)
  PQKV_ROPE(64, true, false)
  PQKV_ROPE(64, true, true)
  PQKV_ROPE(64, false, false)
  PQKV_ROPE(64, false, true)
#undef PQKV_ROPE
  return cudaErrorInvalidValue;
}

}  // namespace pqkv
