// prefill.cu -- launches of the causal chunked-prefill attention (the kernel and
// its design: prefill_kernel.cuh).
#include "prefill_kernel.cuh"

namespace pqkv {

// ---- launch ------------------------------------------------------------------

template <int KVF, int D, bool QBF16>
static cudaError_t launch_prefill_t(const CUtensorMap& tmap, const PrefillParams& p, cudaStream_t st) {
  auto kern = paged_prefill_kernel<KVF, D, QBF16, false>;
  constexpr int smem = PrefillGeom<KVF, D>::kSmem;
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  cudaLaunchConfig_t cfg = {};
  constexpr int NWG = PrefillGeom<KVF, D>::NWG;
  cfg.gridDim = dim3((unsigned)(p.B * ((p.tiles_per_seq + NWG - 1) / NWG)), (unsigned)p.Hkv);
  cfg.blockDim = dim3(PrefillGeom<KVF, D>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tmap, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

size_t prefill_smem_bytes(int kv_dtype, int D) {
#define PQKV_PS(F)                                                                               \
  if (kv_dtype == F) return D == 128 ? PrefillGeom<F, 128>::kSmem : PrefillGeom<F, 64>::kSmem;
  PQKV_PS(PQKV_DTYPE_FP16)
  PQKV_PS(PQKV_DTYPE_BF16)
  PQKV_PS(PQKV_DTYPE_FP8_E4M3)
  PQKV_PS(PQKV_DTYPE_FP8_E5M2)
  PQKV_PS(PQKV_DTYPE_FP4_E2M1)
#undef PQKV_PS
  return 0;
}

cudaError_t launch_prefill(int kv_dtype, int D, bool q_bf16, const CUtensorMap& tmap16, const PrefillParams& p,
                           cudaStream_t st) {
#define PQKV_PF(KVF, DD, QB) \
  if (kv_dtype == KVF && D == DD && q_bf16 == QB) return launch_prefill_t<KVF, DD, QB>(tmap16, p, st);
  PQKV_PF(PQKV_DTYPE_FP16, 128, false)
  PQKV_PF(PQKV_DTYPE_FP16, 64, false)
  PQKV_PF(PQKV_DTYPE_BF16, 128, true)
  PQKV_PF(PQKV_DTYPE_BF16, 64, true)
  PQKV_PF(PQKV_DTYPE_FP8_E4M3, 128, true)
  PQKV_PF(PQKV_DTYPE_FP8_E4M3, 128, false)
  PQKV_PF(PQKV_DTYPE_FP8_E4M3, 64, true)
  PQKV_PF(PQKV_DTYPE_FP8_E4M3, 64, false)
  PQKV_PF(PQKV_DTYPE_FP8_E5M2, 128, true)
  PQKV_PF(PQKV_DTYPE_FP8_E5M2, 128, false)
  PQKV_PF(PQKV_DTYPE_FP8_E5M2, 64, true)
  PQKV_PF(PQKV_DTYPE_FP8_E5M2, 64, false)
  PQKV_PF(PQKV_DTYPE_FP4_E2M1, 128, true)
  PQKV_PF(PQKV_DTYPE_FP4_E2M1, 128, false)
  PQKV_PF(PQKV_DTYPE_FP4_E2M1, 64, true)
  PQKV_PF(PQKV_DTYPE_FP4_E2M1, 64, false)
#undef PQKV_PF
  return cudaErrorInvalidValue;
}

}  // namespace pqkv
