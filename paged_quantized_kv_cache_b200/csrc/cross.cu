// cross.cu -- attention of decoder tokens to an encoder's cached states, of a
// length of their own ("vLLM" glossary, "PagedAttention": K/V through the block
// table, one copy shared by every sequence that reads it).
//
// The kernel is the prefill's (prefill_kernel.cuh) with CROSS:
//  - a row sees positions [lo, hi) of [0, L) instead of [0, its own]: the whole
//    of the states, or the token's range. A CTA walks the tiles between the
//    first and the last position that any of its rows sees, and masks only tiles
//    that some row of a warp does not see whole.
//  - few query rows. Warpgroups and warps without rows take no part (a decode
//    step has G rows of the 256), and the KV range of a tile pair is split over
//    a cluster of up to 8 CTAs whose partial O, m and l are joined through
//    distributed shared memory: no workspace, no second launch, no order that
//    depends on timing.
#include "prefill_kernel.cuh"

namespace pqkv {

namespace {

// CTAs per tile pair: doubled while the doubled grid still fits the GPU at one
// CTA per SM and every CTA keeps a tile.
int cross_splits(long long ctas, int maxblk, int sms) {
  const int tiles = (maxblk * kBlock + kN - 1) / kN;
  int s = 1;
  while (2 * s <= kMaxSplits && ctas * 2 * s <= sms && 2 * s <= tiles) s *= 2;
  return s;
}

template <int KVF, int D, bool QBF16>
cudaError_t launch_cross_t(const CUtensorMap& tmap, PrefillParams p, int sms, cudaStream_t st) {
  auto kern = paged_prefill_kernel<KVF, D, QBF16, true>;
  constexpr int smem = PrefillGeom<KVF, D>::kSmem;
  constexpr int NWG = PrefillGeom<KVF, D>::NWG;
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  const unsigned pairs = (unsigned)(p.B * ((p.tiles_per_seq + NWG - 1) / NWG));
  p.splits = cross_splits((long long)pairs * p.Hkv, p.maxblk, sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pairs, (unsigned)p.Hkv, (unsigned)p.splits);
  cfg.blockDim = dim3(PrefillGeom<KVF, D>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = (unsigned)p.splits;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tmap, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_cross(int kv_dtype, int D, bool q_bf16, const CUtensorMap& tmap16, const PrefillParams& p, int sms,
                         cudaStream_t st) {
#define PQKV_CR(KVF, DD, QB) \
  if (kv_dtype == KVF && D == DD && q_bf16 == QB) return launch_cross_t<KVF, DD, QB>(tmap16, p, sms, st);
  PQKV_CR(PQKV_DTYPE_FP16, 128, false)
  PQKV_CR(PQKV_DTYPE_FP16, 64, false)
  PQKV_CR(PQKV_DTYPE_BF16, 128, true)
  PQKV_CR(PQKV_DTYPE_BF16, 64, true)
  PQKV_CR(PQKV_DTYPE_FP8_E4M3, 128, true)
  PQKV_CR(PQKV_DTYPE_FP8_E4M3, 128, false)
  PQKV_CR(PQKV_DTYPE_FP8_E4M3, 64, true)
  PQKV_CR(PQKV_DTYPE_FP8_E4M3, 64, false)
  PQKV_CR(PQKV_DTYPE_FP8_E5M2, 128, true)
  PQKV_CR(PQKV_DTYPE_FP8_E5M2, 128, false)
  PQKV_CR(PQKV_DTYPE_FP8_E5M2, 64, true)
  PQKV_CR(PQKV_DTYPE_FP8_E5M2, 64, false)
  PQKV_CR(PQKV_DTYPE_FP4_E2M1, 128, true)
  PQKV_CR(PQKV_DTYPE_FP4_E2M1, 128, false)
  PQKV_CR(PQKV_DTYPE_FP4_E2M1, 64, true)
  PQKV_CR(PQKV_DTYPE_FP4_E2M1, 64, false)
#undef PQKV_CR
  return cudaErrorInvalidValue;
}

}  // namespace pqkv
