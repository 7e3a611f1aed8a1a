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
// and sines and the kind's weights are read once for them.
//
// Measured (8191 tokens, 32 / 8 heads of 128, three axes): 36.3 us, of which the
// bytes at copy speed are 26.2; 27.3 without norm and rotation, 29.3 with the
// norm only, 32.9 with one axis: the rest is the reading of the angles.
#include "rope.cuh"

namespace pqkv {

namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;

// Chunks of kUnroll rows per lane that `heads` rows of a token take.
template <int D>
__host__ __device__ constexpr int chunks_of(int heads) {
  return (heads + 256 / D * kUnroll - 1) / (256 / D * kUnroll);
}

template <int D, bool BF16, bool IL>
__global__ void __launch_bounds__(kThreads, 8) rope_kernel(const __grid_constant__ RopeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kLanes = D / 8;       // lanes of a row
  constexpr int kRows = 32 / kLanes;  // rows a warp holds at once
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (t >= p.r.T) return;
  int chunk = blockIdx.y, heads = p.Hq;
  const bool is_q = chunk < chunks_of<D>(p.Hq);
  bool is_v = false;
  if (!is_q) {
    chunk -= chunks_of<D>(p.Hq);
    heads = p.Hkv;
    is_v = chunk >= chunks_of<D>(p.Hkv);
    if (is_v) chunk -= chunks_of<D>(p.Hkv);
  }
  const int row0 = chunk * kRows * kUnroll + lane / kLanes;
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
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    raw[u] = row0 + u * kRows < heads ? load_pairs<IL>(src_a + u * kRows * D, src_b + u * kRows * D)
                                      : make_uint4(0, 0, 0, 0);
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
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) put(u, make_uint4(0, 0, 0, 0));
    return;
  }
  if (is_v) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) put(u, raw[u]);
    return;
  }
  Pairs w = {};
  if (weight) w = load_weight<IL>(weight, a, b);
  const Coefficients k = coefficients<IL>(weight != nullptr, w, turn, cs);
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint4 out = norm_rotate<D, BF16, IL>(raw[u], weight != nullptr, p.r.eps, k);
    put(u, weight || turn ? out : raw[u]);
  }
}

template <int D, bool BF16, bool IL>
cudaError_t launch_rope_t(const RopeParams& p, cudaStream_t st) {
  const int chunks = chunks_of<D>(p.Hq) + p.kinds * chunks_of<D>(p.Hkv);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.r.T + kThreads / 32 - 1) / (kThreads / 32)), (unsigned)chunks);
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
  if (p.r.T == 0) return cudaSuccess;
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
