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
// one token at once: their loads are all in flight before the first sum, and
// the token's positions, cosines and sines are read once for them.
#include "rope.cuh"

namespace pqkv {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

template <int D, bool BF16, bool IL>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kLanes = D / 8;          // lanes of a row
  constexpr int kRows = 32 / kLanes;     // rows a warp holds at once
  constexpr int kChunk = kRows * kUnroll;
  const int lane = threadIdx.x & 31;
  const int chunks = (p.rows + kChunk - 1) / kChunk;
  const long long unit = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int t = (int)(unit / chunks);
  if (t >= p.r.T) return;
  const int row0 = (int)(unit % chunks) * kChunk + lane / kLanes;
  const int i0 = 4 * (lane % kLanes);
  int a, b;
  pair_channels<D, IL>(i0, p.r.rot, a, b);

  uint4 raw[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int row = row0 + u * kRows;
    raw[u] = make_uint4(0, 0, 0, 0);
    if (row < p.rows) {
      const uint16_t* src;
      if (row < p.Hq)
        src = static_cast<const uint16_t*>(p.q) + (size_t)t * p.qs + (size_t)row * D;
      else if (row < p.Hq + p.Hkv)
        src = static_cast<const uint16_t*>(p.k) + (size_t)t * p.ks + (size_t)(row - p.Hq) * D;
      else
        src = static_cast<const uint16_t*>(p.v) + (size_t)t * p.vs + (size_t)(row - p.Hq - p.Hkv) * D;
      raw[u] = load_pairs<IL>(src, a, b);
    }
  }
  Pairs cs;
  const bool ok = load_angles<D>(p.r, t, i0, cs);
  if (!ok && lane == 0 && row0 == 0) raise_flag(p.err, PQKV_DEVERR_POSITION);
  int slot = -1;
  if (!p.k_out && p.rows > p.Hq) {
    slot = __ldg(p.slots + t);
    if (slot >= p.nb * kBlock) {
      if (lane == 0 && row0 == 0) raise_flag(p.err, PQKV_DEVERR_SLOT);
      slot = -1;
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int row = row0 + u * kRows;
    const bool is_q = row < p.Hq, is_v = row >= p.Hq + p.Hkv;
    const float* weight = is_q ? p.r.q_weight : p.r.k_weight;
    const bool norm = weight != nullptr && !is_v;
    Pairs w = {};
    if (norm && row < p.rows) w = load_weight<IL>(weight, a, b);
    const Pairs x = unpack_pairs<BF16, IL>(raw[u]);
    const Pairs z = norm_rotate<D>(x, norm, w, p.r.eps, 2 * i0 < p.r.rot, cs);
    if (row >= p.rows) continue;
    uint4 out = is_v ? raw[u] : pack_pairs<BF16, IL>(z);
    if (!ok && !is_v) out = make_uint4(0, 0, 0, 0);
    uint16_t* dst;
    if (is_q) {
      dst = static_cast<uint16_t*>(p.q_out) + ((size_t)t * p.Hq + row) * D;
    } else if (p.k_out) {
      dst = static_cast<uint16_t*>(p.k_out) + ((size_t)t * p.Hkv + (row - p.Hq)) * D;
    } else {
      if (slot < 0) continue;
      const int h = is_v ? row - p.Hq - p.Hkv : row - p.Hq;
      dst = reinterpret_cast<uint16_t*>(p.cache) +
            ((((size_t)(slot >> 4) * p.Hkv + h) * 2 + (is_v ? 1 : 0)) * kBlock + (slot & 15)) * D;
    }
    store_pairs<IL>(dst, a, b, out);
  }
}

template <int D, bool BF16, bool IL>
cudaError_t launch_rope_t(const RopeParams& p, cudaStream_t st) {
  constexpr int kChunk = 32 / (D / 8) * kUnroll;
  const long long units = (long long)p.r.T * ((p.rows + kChunk - 1) / kChunk);
  const long long grid = (units + kThreads / 32 - 1) / (kThreads / 32);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, rope_kernel<D, BF16, IL>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(bool bf16, int D, bool interleaved, const RopeParams& p, cudaStream_t st) {
  if (p.r.T == 0 || p.rows == 0) return cudaSuccess;
#define PQKV_ROPE(DD, BF, IL) \
  if (D == DD && bf16 == BF && interleaved == IL) return launch_rope_t<DD, BF, IL>(p, st);
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
