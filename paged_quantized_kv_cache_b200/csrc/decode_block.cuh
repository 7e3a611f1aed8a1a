// decode_block.cuh -- what a warp does with one 16-token block of the cache in
// shared memory, for up to 16 query rows of its KV head: scores, the product with
// the values and their dequantization in registers. Shared by the decode
// (decode.cu) and the cross attention of few tokens (cross_few.cu).
#pragma once

#include "decode.cuh"

namespace pqkv {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr float kNegInf = -INFINITY;
// The running max m is only moved (and O, l rescaled) when a block's max
// exceeds it by more than this many log2 units, so most blocks skip the
// rescale; probabilities then stay below 2^kLazy, well inside f16 / bf16.
// FP4 multiplies P by E4M3 group scales (<= 448) in f16, so it keeps P <= 16.
template <int KVF>
constexpr float lazy_of() { return KVF == PQKV_DTYPE_FP4_E2M1 ? 4.f : 8.f; }

// Zero the low (token t0) / high (token t0 + 1) half of a packed pair when the
// token lies past the end of the sequence (its bytes may hold anything).
__device__ __forceinline__ uint32_t mask_pair(uint32_t v, int t0, int valid) {
  if (t0 >= valid) v &= 0xFFFF0000u;
  if (t0 + 1 >= valid) v &= 0x0000FFFFu;
  return v;
}

__device__ __forceinline__ uint32_t f16x2_from(float a, float b) {
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// 2^x with the hardware approximation (relative error ~2^-22, denormal results flushed).
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <bool QBF16>
__device__ __forceinline__ float q_at(const void* q, size_t i) {
  if constexpr (QBF16)
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(q)[i]);
  else
    return __half2float(reinterpret_cast<const __half*>(q)[i]);
}

template <bool QBF16>
__device__ __forceinline__ void store_out(void* out, size_t i, float v) {
  if constexpr (QBF16)
    reinterpret_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else
    reinterpret_cast<__half*>(out)[i] = __float2half_rn(v);
}

// out[i], out[i + 1] = a, b in one 4-byte store (i even).
template <bool QBF16>
__device__ __forceinline__ void store_out2(void* out, size_t i, float a, float b) {
  if constexpr (QBF16)
    *reinterpret_cast<__nv_bfloat162*>(reinterpret_cast<__nv_bfloat16*>(out) + i) = __floats2bfloat162_rn(a, b);
  else
    *reinterpret_cast<__half2*>(reinterpret_cast<__half*>(out) + i) = __floats2half2_rn(a, b);
}

// Four E4M3 codes -> f16x2 of bytes (0,1) and (2,3) by the hardware conversion.
__device__ __forceinline__ void dec4_e4m3_cvt(uint32_t r, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(r));
}

// Four FP8 codes of a word -> f16x2 of bytes (0,1) and of bytes (2,3), exact.
// E5M2 codes are the high byte of the binary16 of the same value, so they are
// placed, not converted; E4M3 codes go through the hardware conversion (placing
// their bits too, as the binary16 of value x 2^-8 with three integer
// operations per pair, measured 20% slower per decode: the kernel is bound by
// instruction issue, not by the conversions).
template <int KVF>
__device__ __forceinline__ void dec4(uint32_t r, uint32_t& lo, uint32_t& hi) {
  if constexpr (KVF == PQKV_DTYPE_FP8_E5M2) {
    lo = prmt(r, 0u, 0x1404u);
    hi = prmt(r, 0u, 0x3424u);
  } else {
    dec4_e4m3_cvt(r, lo, hi);
  }
}

// Per-lane shared-memory offsets (bytes, within a stage) of the ldmatrix rows
// of one block: K reads of k-step group i and V reads of m-tile group i. The
// swizzle depends on the lane, so these are computed once per kernel.
template <int KVF, int D>
struct LdsmOffsets {
  using Gm = DecodeGeom<KVF, D>;
  // 16-bit: one x4 per 16 head dims; FP8: per 32 dims; FP4: per 64 dims
  static constexpr int kN = Gm::k16 ? D / 16 : (Gm::kFp8 ? D / 32 : D / 64);
  uint32_t k[kN], v[kN];
  __device__ __forceinline__ explicit LdsmOffsets(int lane) {
    const int mi = lane >> 3, ri = lane & 7;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      if constexpr (Gm::k16) {
        k[i] = Gm::off(((mi & 1) << 3) + ri, (2 * i + (mi >> 1)) * 16);
        v[i] = Gm::off(16 + ((mi >> 1) << 3) + ri, (2 * i + (mi & 1)) * 16);
      } else if constexpr (Gm::kFp8) {
        k[i] = Gm::off(((mi & 1) << 3) + ri, (2 * i + (mi >> 1)) * 16);
        v[i] = Gm::off(16 + ((mi & 1) << 3) + ri, (2 * i + (mi >> 1)) * 16);
      } else {
        // V: matrix mi of load i is m-tile c = 4i + mi, the 8 pair rows of
        // its half of the channels at the 16-byte column of its 16 channels
        const int c = 4 * i + mi;
        k[i] = Gm::off(((mi & 1) << 3) + ri, (2 * i + (mi >> 1)) * 16);
        v[i] = Gm::off(16 + 8 * (c / (D / 32)) + ri, 16 * (c % (D / 32)));
      }
    }
  }
};

// Row `rr` (0..15) of output m-tile `mt` -> head-dimension index. The order
// of d inside a tile follows how each format's dequantization lays out the
// V^T fragment (see block_pv).
template <int KVF>
__device__ __forceinline__ int dmap(int mt, int rr) {
  if constexpr (KVF == PQKV_DTYPE_FP16 || KVF == PQKV_DTYPE_BF16) {
    return 16 * mt + rr;
  } else {
    // FP8, FP4: tile c covers [16c, 16c + 16): row g -> 16c + 2g, row g + 8 -> 16c + 2g + 1
    return 16 * mt + 2 * (rr & 7) + (rr >> 3);
  }
}

// FP4 outlier channels: per-warp state carried from block to block. The
// outlier channels of consecutive blocks of one KV head usually agree, so the
// query fragment at the K outlier channels and the V outlier product are kept
// in registers while the channel set stays the same; the V product goes to the
// shared-memory accumulator of outlier channels only when the set changes or
// the piece ends.
template <int NT>
struct OutlierState {
  static constexpr uint32_t kNone = 0xFEFEFEFEu;  // no valid channel byte (they are < 128 or 0xFF)
  uint32_t kidx;        // K outlier channels the cached query fragments belong to
  uint32_t kq[NT];      // query fragments (B of the K outlier MMA), per column tile
  uint32_t vidx;        // V outlier channels vacc belongs to
  float vacc[NT][4];    // V outlier product (rows = slots, lanes g < 4) not yet flushed
  __device__ __forceinline__ void reset() {
    kidx = vidx = kNone;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      kq[nt] = 0;
      vacc[nt][0] = vacc[nt][1] = vacc[nt][2] = vacc[nt][3] = 0.f;
    }
  }
  // add vacc into the accumulator of outlier channels and clear it
  template <int STRIDE>
  __device__ __forceinline__ void flush(float* oext, int lane, int D) {
    const int g = lane >> 2, qd = lane & 3;
    if (vidx != kNone && g < 4) {
      const int dch = (vidx >> (8 * g)) & 0xFF;
      if (dch < D) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          oext[(8 * nt + 2 * qd) * STRIDE + dch] += vacc[nt][0];
          oext[(8 * nt + 2 * qd + 1) * STRIDE + dch] += vacc[nt][1];
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) vacc[nt][0] = vacc[nt][1] = vacc[nt][2] = vacc[nt][3] = 0.f;
  }
};

// ---------------------------------------------------------------------------
// S^T (16 tokens x 8 NT query rows) += K Q^T for one block in shared memory.
// Lane (g, qd) ends with rows (tokens) g, g + 8 and columns 8nt + 2qd, 8nt +
// 2qd + 1 of each column tile nt; the K fragments are dequantized once for all.
// ---------------------------------------------------------------------------
template <int KVF, int D, int NT>
__device__ __forceinline__ void block_scores(uint32_t tb, const uint8_t* side,
                                             const uint32_t (&qf)[NT][D / 16][2], const uint16_t* wq,
                                             const LdsmOffsets<KVF, D>& lo, int lane, float (&sc)[NT][4],
                                             OutlierState<NT>& ost) {
  using Gm = DecodeGeom<KVF, D, NT>;
  constexpr int KT = D / 16;
  const int g = lane >> 2, qd = lane & 3;
  float se[NT][4], so[NT][4];  // two independent chains per column tile
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) se[nt][i] = so[nt][i] = 0.f;
  if constexpr (Gm::k16) {
    constexpr bool kBf = (KVF == PQKV_DTYPE_BF16);
#pragma unroll
    for (int kk = 0; kk < KT; ++kk) {
      uint32_t a0, a1, a2, a3;
      ldsm_x4(tb + lo.k[kk], a0, a1, a2, a3);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (kk & 1) mma16816<kBf>(so[nt], a0, a1, a2, a3, qf[nt][kk][0], qf[nt][kk][1]);
        else mma16816<kBf>(se[nt], a0, a1, a2, a3, qf[nt][kk][0], qf[nt][kk][1]);
      }
    }
  } else if constexpr (Gm::kFp8) {
    // ldmatrix on byte data: lane (g, qd) receives bytes 4qd..4qd+3 of a token
    // row's 16-byte chunk, i.e. 4 consecutive d of one k-step.
#pragma unroll
    for (int cp = 0; cp < KT / 2; ++cp) {
      uint32_t r0, r1, r2, r3;
      ldsm_x4(tb + lo.k[cp], r0, r1, r2, r3);
      uint32_t x0l, x0h, x1l, x1h, x2l, x2h, x3l, x3h;
      dec4<KVF>(r0, x0l, x0h);
      dec4<KVF>(r1, x1l, x1h);
      dec4<KVF>(r2, x2l, x2h);
      dec4<KVF>(r3, x3l, x3h);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma16816<false>(se[nt], x0l, x1l, x0h, x1h, qf[nt][2 * cp][0], qf[nt][2 * cp][1]);
        mma16816<false>(so[nt], x2l, x3l, x2h, x3h, qf[nt][2 * cp + 1][0], qf[nt][2 * cp + 1][1]);
      }
    }
  } else {
    // FP4: one 16-byte chunk = 32 d; lane (g, qd) receives the 8 codes
    // d = 32c + 8qd .. +7 of token rows g and g + 8 and multiplies them by the
    // token's E4M3 scale of group 2c + qd/2 (the product is exact in f16).
    constexpr int SPR = D / 16;  // scale bytes per token row
    // The scale of chunk c for this lane is byte 2c + qd/2 of the token's scale
    // row: pick it from whole words and broadcast it to (s, s) in f16.
    uint32_t sa2[D / 32], sb2[D / 32];
    {
      const int a = qd >> 1;
      const uint32_t sel = (uint32_t)(a | (a << 4) | ((a + 2) << 8) | ((a + 2) << 12));
      const uint32_t* ra = reinterpret_cast<const uint32_t*>(side + g * SPR);
      const uint32_t* rb = reinterpret_cast<const uint32_t*>(side + (g + 8) * SPR);
#pragma unroll
      for (int w = 0; w < SPR / 4; ++w) {  // word w = groups 4w..4w+3 = chunks 2w, 2w+1
        dec4_e4m3_cvt(prmt(ra[w], 0u, sel), sa2[2 * w], sa2[2 * w + 1]);
        dec4_e4m3_cvt(prmt(rb[w], 0u, sel), sb2[2 * w], sb2[2 * w + 1]);
      }
    }
#pragma unroll
    for (int cp = 0; cp < D / 64; ++cp) {
      uint32_t r0, r1, r2, r3;
      ldsm_x4(tb + lo.k[cp], r0, r1, r2, r3);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = 2 * cp + e;
        const uint32_t ra = e ? r2 : r0, rb = e ? r3 : r1;
        const __half2 sa = *reinterpret_cast<const __half2*>(&sa2[c]);
        const __half2 sb = *reinterpret_cast<const __half2*>(&sb2[c]);
        uint32_t ha[4], hb[4];
        dec_e2m1x8(ra, ha);
        dec_e2m1x8(rb, hb);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          __half2 xa = __hmul2(*reinterpret_cast<__half2*>(&ha[i]), sa);
          __half2 yb = __hmul2(*reinterpret_cast<__half2*>(&hb[i]), sb);
          ha[i] = *reinterpret_cast<uint32_t*>(&xa);
          hb[i] = *reinterpret_cast<uint32_t*>(&yb);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816<false>(se[nt], ha[0], hb[0], ha[1], hb[1], qf[nt][2 * c][0], qf[nt][2 * c][1]);
          mma16816<false>(so[nt], ha[2], hb[2], ha[3], hb[3], qf[nt][2 * c + 1][0], qf[nt][2 * c + 1][1]);
        }
      }
    }
    // outlier channels (their codes are 0): S^T += Kout (16 tokens x 4 slots) Qout^T.
    // Empty slots hold +0 values and get a zero query, so they add nothing.
    {
      const uint32_t kw = *reinterpret_cast<const uint32_t*>(side + Gm::kScaleBytes + Gm::kValBytes);  // K idx
      const uint32_t* kv = reinterpret_cast<const uint32_t*>(side + Gm::kScaleBytes);  // K vals [16][4] fp16
      if (kw != ost.kidx) {  // same for the whole warp
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t b0 = 0;
          if (qd < 2) {
            const int r0i = (kw >> (16 * qd)) & 0xFF, r1i = (kw >> (16 * qd + 8)) & 0xFF;
            const uint16_t* row = wq + (8 * nt + g) * Gm::kQStride;
            const uint32_t q0 = (r0i < D) ? row[r0i] : 0u;
            const uint32_t q1 = (r1i < D) ? row[r1i] : 0u;
            b0 = q0 | (q1 << 16);
          }
          ost.kq[nt] = b0;
        }
        ost.kidx = kw;
      }
      const uint32_t a0 = (qd < 2) ? kv[g * 2 + qd] : 0u;
      const uint32_t a1 = (qd < 2) ? kv[(g + 8) * 2 + qd] : 0u;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma16816<false>(so[nt], a0, a1, 0u, 0u, ost.kq[nt], 0u);
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[nt][i] = se[nt][i] + so[nt][i];
}

// ---------------------------------------------------------------------------
// O^T (D x 8 NT query rows) += V^T P^T for one block. P^T arrives per column
// tile as two B fragments (hi and lo parts, P = P_hi + P_lo rounded to the
// operand type); the V fragments are dequantized once for all tiles.
// ---------------------------------------------------------------------------
// SPLIT: with P_lo (FP4 keeps P in f16 only; its tolerance allows it).
template <int KVF, int D, int NT, bool SPLIT = (KVF != PQKV_DTYPE_FP4_E2M1)>
__device__ __forceinline__ void block_pv(uint32_t tb, const uint8_t* side, const LdsmOffsets<KVF, D>& lo, int lane,
                                         int valid, const uint32_t (&b0)[NT], const uint32_t (&b1)[NT],
                                         const uint32_t (&c0)[NT], const uint32_t (&c1)[NT],
                                         float (&acc)[NT][D / 16][4], float* oext, OutlierState<NT>& ost) {
  using Gm = DecodeGeom<KVF, D, NT>;
  constexpr int KT = D / 16;
  constexpr bool kBf = (KVF == PQKV_DTYPE_BF16);
  const int g = lane >> 2, qd = lane & 3;
  const int t0 = 2 * qd, t1 = 2 * qd + 8;
  constexpr bool kSplitP = SPLIT;
  auto mma_pv = [&](int nt, float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
    mma16816<kBf>(d, a0, a1, a2, a3, b0[nt], b1[nt]);
    if constexpr (kSplitP) mma16816<kBf>(d, a0, a1, a2, a3, c0[nt], c1[nt]);
  };
  if constexpr (Gm::k16) {
#pragma unroll
    for (int mt = 0; mt < KT; ++mt) {
      uint32_t a0, a1, a2, a3;
      ldsm_x4_t(tb + lo.v[mt], a0, a1, a2, a3);
      if (valid < kBlock) {
        a0 = mask_pair(a0, t0, valid);
        a1 = mask_pair(a1, t0, valid);
        a2 = mask_pair(a2, t1, valid);
        a3 = mask_pair(a3, t1, valid);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_pv(nt, acc[nt][mt], a0, a1, a2, a3);
    }
  } else if constexpr (Gm::kFp8) {
    // ldmatrix.trans on byte data: lane (g, qd) receives d0 = 16c + 2g and d0 + 1
    // of tokens 2qd and 2qd + 1; one byte permute pairs the tokens per d.
#pragma unroll
    for (int cp = 0; cp < KT / 2; ++cp) {
      uint32_t r0, r1, r2, r3;
      ldsm_x4_t(tb + lo.v[cp], r0, r1, r2, r3);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t xa = prmt(e ? r2 : r0, 0u, 0x3120u);
        const uint32_t xb = prmt(e ? r3 : r1, 0u, 0x3120u);
        uint32_t a0, a1, a2, a3;
        dec4<KVF>(xa, a0, a1);
        dec4<KVF>(xb, a2, a3);
        if (valid < kBlock) {
          a0 = mask_pair(a0, t0, valid);
          a1 = mask_pair(a1, t0, valid);
          a2 = mask_pair(a2, t1, valid);
          a3 = mask_pair(a3, t1, valid);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_pv(nt, acc[nt][2 * cp + e], a0, a1, a2, a3);
      }
    }
  } else {
    // FP4: a V byte holds one channel of a token pair, so ldmatrix.trans of 8
    // pair rows hands lane (g, qd) the whole A fragment of m-tile c in one word:
    // d = 16c + 2g, 16c + 2g + 1 of tokens (2qd, 2qd + 1) and (2qd + 8, 2qd + 9).
    // m-tile c is scale group c, so the tokens' E4M3 group scales multiply P
    // (in f16: P <= 16, scale <= 448) instead of the codes.
    constexpr int SPR = D / 16;
    const uint8_t* vs = side + 16 * SPR;  // V scales [16][D/16]
    uint32_t sp[2][D / 16];               // (s(t, c), s(t + 1, c)), t = 2qd | 2qd + 8
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int ta = 2 * qd + 8 * hh;
      const uint32_t* w0 = reinterpret_cast<const uint32_t*>(vs + ta * SPR);
      const uint32_t* w1 = reinterpret_cast<const uint32_t*>(vs + (ta + 1) * SPR);
#pragma unroll
      for (int w = 0; w < SPR / 4; ++w) {
        dec4_e4m3_cvt(prmt(w0[w], w1[w], 0x5140u), sp[hh][4 * w], sp[hh][4 * w + 1]);
        dec4_e4m3_cvt(prmt(w0[w], w1[w], 0x7362u), sp[hh][4 * w + 2], sp[hh][4 * w + 3]);
      }
      if (valid < kBlock) {  // scales past the end may be NaN codes
#pragma unroll
        for (int c = 0; c < D / 16; ++c) sp[hh][c] = mask_pair(sp[hh][c], ta, valid);
      }
    }
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      uint32_t r[4];
      ldsm_x4_t(tb + lo.v[i], r[0], r[1], r[2], r[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = 4 * i + e;
        uint32_t a[4];
        dec_e2m1x8(r[e], a);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const __half2 p0 =
              __hmul2(*reinterpret_cast<const __half2*>(&b0[nt]), *reinterpret_cast<const __half2*>(&sp[0][c]));
          const __half2 p1 =
              __hmul2(*reinterpret_cast<const __half2*>(&b1[nt]), *reinterpret_cast<const __half2*>(&sp[1][c]));
          mma16816<false>(acc[nt][c], a[0], a[1], a[2], a[3], *reinterpret_cast<const uint32_t*>(&p0),
                          *reinterpret_cast<const uint32_t*>(&p1));
        }
      }
    }
    // outlier channels: Oext[n][idx_r] += (Vout^T (4 slots x 16 tokens) P^T)[r][n].
    // The result of slot r sits in lanes 4r..4r+3 (heads 2qd, 2qd+1); it stays
    // in registers while the block's V outlier channels match the previous
    // block's, and goes to the warp's shared-memory accumulator of outlier
    // channels (which follows O's rescaling and is folded into O when the piece
    // ends) when they change.
    {
      const uint32_t vw = *reinterpret_cast<const uint32_t*>(side + Gm::kScaleBytes + Gm::kValBytes + 8);  // V idx
      const uint16_t* vv = reinterpret_cast<const uint16_t*>(side + Gm::kScaleBytes + 128);    // V vals
      if (vw != ost.vidx) {  // same for the whole warp
        ost.template flush<Gm::kOStride>(oext, lane, D);
        ost.vidx = vw;
      }
      uint32_t a0 = 0, a2 = 0;
      if (g < 4) {
        a0 = (uint32_t)vv[t0 * 4 + g] | ((uint32_t)vv[(t0 + 1) * 4 + g] << 16);
        a2 = (uint32_t)vv[t1 * 4 + g] | ((uint32_t)vv[(t1 + 1) * 4 + g] << 16);
        if (valid < kBlock) {
          a0 = mask_pair(a0, t0, valid);
          a2 = mask_pair(a2, t1, valid);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_pv(nt, ost.vacc[nt], a0, 0u, a2, 0u);
    }
  }
}

}  // namespace

}  // namespace pqkv
