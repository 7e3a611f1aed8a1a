// rope.cuh -- RMS norm of query and key heads and rotary positions, in one pass
// over the projection's output; optionally with the cache write.
#pragma once

#include "common.cuh"

namespace pqkv {

constexpr int kMaxAxes = 4;

// The norm and rotation of one row (one head of one token).
struct RowParams {
  const float* q_weight;     // [D] or null: no norm of the queries
  const float* k_weight;     // [D] or null: no norm of the keys
  const int32_t* positions;  // [axes][T]
  const float* cos_sin;      // [num_pos][rot]: cosines of the rot / 2 pairs, then sines
  float eps;
  int T, num_pos, rot, axes;
  uint32_t axis[16];         // axis of each pair, a byte each
};

struct RopeParams {
  RowParams r;
  const void* q;
  const void* k;
  const void* v;
  long long qs, ks, vs;  // elements from one token to the next
  void* q_out;
  void* k_out;           // contiguous keys, or null: keys and values go to the cache
  const int32_t* slots;
  uint8_t* cache;        // 16-bit cache
  int32_t* err;
  int Hq, Hkv, nb;
  int kinds;             // 0: queries only, 1: and keys, 2: and values
};

cudaError_t launch_rope(bool bf16, int D, bool interleaved, const RopeParams& p, int sms, cudaStream_t st);

// Channels of pair i of a row of D channels whose first ROT are rotated. Half
// style: i and i + ROT / 2; interleaved: 2i and 2i + 1. The channels behind
// ROT are taken two by two as well, so that i runs over D / 2 everywhere. ROT
// is a multiple of 8: four consecutive pairs from a multiple of 4 have
// consecutive first and second channels, each four on an 8-byte boundary.
template <int D, bool IL>
__device__ __forceinline__ void pair_channels(int i, int rot, int& a, int& b) {
  if constexpr (IL) {
    a = 2 * i;
    b = 2 * i + 1;
  } else {
    const int half = rot / 2;
    a = i < half ? i : i + half;
    b = a + (i < half ? half : (D - rot) / 2);
  }
}

// Four pairs of a row, a lane's share: D / 8 lanes hold a row.
struct Pairs {
  float a[4], b[4];
};

// Raw words of a lane's four pairs of a row: half style two 8-byte pieces,
// interleaved one piece of 16 bytes.
template <bool IL>
__device__ __forceinline__ uint4 load_pairs(const uint16_t* a, const uint16_t* b) {
  if constexpr (IL) return *reinterpret_cast<const uint4*>(a);
  const uint2 x = *reinterpret_cast<const uint2*>(a), y = *reinterpret_cast<const uint2*>(b);
  return make_uint4(x.x, x.y, y.x, y.y);
}
template <bool IL>
__device__ __forceinline__ void store_pairs(uint16_t* a, uint16_t* b, uint4 w) {
  if constexpr (IL) {
    *reinterpret_cast<uint4*>(a) = w;
  } else {
    *reinterpret_cast<uint2*>(a) = make_uint2(w.x, w.y);
    *reinterpret_cast<uint2*>(b) = make_uint2(w.z, w.w);
  }
}

// A lane's weights (its four pairs' channels) of the query or key norm.
template <bool IL>
__device__ __forceinline__ Pairs load_weight(const float* w, int a, int b) {
  const float4 x = *reinterpret_cast<const float4*>(w + a);
  const float4 y = *reinterpret_cast<const float4*>(w + (IL ? a + 4 : b));
  if constexpr (IL) return Pairs{{x.x, x.z, y.x, y.z}, {x.y, x.w, y.y, y.w}};
  return Pairs{{x.x, x.y, x.z, x.w}, {y.x, y.y, y.z, y.w}};
}

// Token t's positions on the axes.
__device__ __forceinline__ void load_positions(const RowParams& r, int t, int (&pos)[kMaxAxes]) {
  const int32_t* at = r.positions + t;
#pragma unroll
  for (int x = 0; x < kMaxAxes; ++x) pos[x] = 0;
  if (r.rot == 0) return;
  pos[0] = __ldg(at);
  if (r.axes == 1) return;
#pragma unroll
  for (int x = 1; x < kMaxAxes; ++x)
    if (x < r.axes) pos[x] = __ldg(at + (size_t)x * r.T);
}

// Cosines (a) and sines (b) of pairs i0 .. i0 + 3 at these positions. False if
// one of them lies outside the table.
__device__ __forceinline__ bool load_angles(const RowParams& r, const int (&pos)[kMaxAxes], int i0, Pairs& cs) {
  cs = {};
  if (r.rot == 0) return true;
  unsigned far = (unsigned)pos[0];  // a negative position is a large one
  if (r.axes > 1) far = max(max(far, (unsigned)pos[1]), max((unsigned)pos[2], (unsigned)pos[3]));
  const bool ok = far < (unsigned)r.num_pos;
  const int half = r.rot / 2;
  if (!ok || i0 >= half) return ok;
  const uint32_t ax = r.axes > 1 ? r.axis[i0 >> 2] : 0u;
  const uint32_t first = ax & 0xFFu;
  const auto place = [&](uint32_t x) { return x == 0 ? pos[0] : x == 1 ? pos[1] : x == 2 ? pos[2] : pos[3]; };
  if (ax == first * 0x01010101u) {  // one axis for all four: two 16-byte loads
    const float* row = r.cos_sin + (size_t)place(first) * r.rot + i0;
    const float4 c = __ldg(reinterpret_cast<const float4*>(row));
    const float4 s = __ldg(reinterpret_cast<const float4*>(row + half));
    cs = Pairs{{c.x, c.y, c.z, c.w}, {s.x, s.y, s.z, s.w}};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float* row = r.cos_sin + (size_t)place((ax >> (8 * e)) & 0xFFu) * r.rot + i0 + e;
      cs.a[e] = __ldg(row);
      cs.b[e] = __ldg(row + half);
    }
  }
  return true;
}

// Two floats in one 64-bit register pair, and IEEE fp32 arithmetic on both in
// one instruction (the kernel is bound by issue before it is by memory).
typedef unsigned long long F2;
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f2_split(F2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
template <bool BF16>
__device__ __forceinline__ F2 f2_widen(uint32_t w) {
  return f2(unpack_lo(w, BF16), unpack_hi(w, BF16));
}
template <bool BF16>
__device__ __forceinline__ uint32_t f2_narrow(F2 v) {
  const float2 x = f2_split(v);
  return pack_f32x2(x.x, x.y, BF16);
}

// What a lane's pairs are multiplied by, norm weights and rotation together, for
// words in the order of load_pairs: out = (x main + partner cross) / rms, where
// the partner of a channel is the other one of its pair.
struct Coefficients {
  F2 main[4], cross[4];
};

// norm: weights w; turn: cosines and sines cs (a lane's pairs turn all or none).
template <bool IL>
__device__ __forceinline__ Coefficients coefficients(bool norm, const Pairs& w, bool turn, const Pairs& cs) {
  float ma[4], mb[4], xa[4], xb[4];  // of first channels (from the second: xa), of second channels
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float wa = norm ? w.a[e] : 1.f, wb = norm ? w.b[e] : 1.f;
    const float c = turn ? cs.a[e] : 1.f, s = turn ? cs.b[e] : 0.f;
    ma[e] = wa * c;
    xa[e] = -(wb * s);
    mb[e] = wb * c;
    xb[e] = wa * s;
  }
  Coefficients k;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (IL) {  // word i: both channels of pair i
      k.main[i] = f2(ma[i], mb[i]);
      k.cross[i] = f2(xa[i], xb[i]);
    } else {  // words 0, 1: first channels of pairs 0, 1 and 2, 3; words 2, 3: their second channels
      const int e = 2 * (i & 1);
      k.main[i] = i < 2 ? f2(ma[e], ma[e + 1]) : f2(mb[e], mb[e + 1]);
      k.cross[i] = i < 2 ? f2(xa[e], xa[e + 1]) : f2(xb[e], xb[e + 1]);
    }
  }
  return k;
}

// A lane's share of a row (words in the order of load_pairs), normed and turned
// in fp32 and rounded once. The D / 8 lanes of a row sum its squares by the same
// tree wherever a row is computed, so that every kernel built on this gives the
// same bits. Every lane of the warp calls it.
template <int D, bool BF16, bool IL>
__device__ __forceinline__ uint4 norm_rotate(uint4 raw, bool norm, float eps, const Coefficients& k) {
  const F2 x[4] = {f2_widen<BF16>(raw.x), f2_widen<BF16>(raw.y), f2_widen<BF16>(raw.z), f2_widen<BF16>(raw.w)};
  float inv = 1.f;
  if (norm) {
    const float2 s = f2_split(f2_fma(x[3], x[3], f2_fma(x[2], x[2], f2_fma(x[1], x[1], f2_mul(x[0], x[0])))));
    float ss = s.x + s.y;
#pragma unroll
    for (int o = 1; o < D / 8; o <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    inv = rsqrtf(fmaf(ss, 1.f / D, eps));
  }
  const F2 inv2 = f2(inv, inv);
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    F2 partner;
    if constexpr (IL) {
      const float2 v = f2_split(x[i]);
      partner = f2(v.y, v.x);
    } else {
      partner = x[i ^ 2];
    }
    out[i] = f2_narrow<BF16>(f2_mul(f2_fma(x[i], k.main[i], f2_mul(partner, k.cross[i])), inv2));
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

}  // namespace pqkv
