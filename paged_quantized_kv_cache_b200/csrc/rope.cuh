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

cudaError_t launch_rope(bool bf16, int D, bool interleaved, const RopeParams& p, cudaStream_t st);

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

template <bool BF16>
__device__ __forceinline__ float2 widen2(uint32_t w) {
  return make_float2(unpack_lo(w, BF16), unpack_hi(w, BF16));
}

// Raw words of a lane's four pairs of a row: half style two 8-byte pieces,
// interleaved one piece of 16 bytes.
template <bool IL>
__device__ __forceinline__ uint4 load_pairs(const uint16_t* row, int a, int b) {
  if constexpr (IL) return *reinterpret_cast<const uint4*>(row + a);
  const uint2 x = *reinterpret_cast<const uint2*>(row + a), y = *reinterpret_cast<const uint2*>(row + b);
  return make_uint4(x.x, x.y, y.x, y.y);
}
template <bool IL>
__device__ __forceinline__ void store_pairs(uint16_t* row, int a, int b, uint4 w) {
  if constexpr (IL) {
    *reinterpret_cast<uint4*>(row + a) = w;
  } else {
    *reinterpret_cast<uint2*>(row + a) = make_uint2(w.x, w.y);
    *reinterpret_cast<uint2*>(row + b) = make_uint2(w.z, w.w);
  }
}

template <bool BF16, bool IL>
__device__ __forceinline__ Pairs unpack_pairs(uint4 w) {
  const float2 x = widen2<BF16>(w.x), y = widen2<BF16>(w.y), z = widen2<BF16>(w.z), u = widen2<BF16>(w.w);
  if constexpr (IL) return Pairs{{x.x, y.x, z.x, u.x}, {x.y, y.y, z.y, u.y}};
  return Pairs{{x.x, x.y, y.x, y.y}, {z.x, z.y, u.x, u.y}};
}
template <bool BF16, bool IL>
__device__ __forceinline__ uint4 pack_pairs(const Pairs& v) {
  if constexpr (IL)
    return make_uint4(pack_f32x2(v.a[0], v.b[0], BF16), pack_f32x2(v.a[1], v.b[1], BF16),
                      pack_f32x2(v.a[2], v.b[2], BF16), pack_f32x2(v.a[3], v.b[3], BF16));
  return make_uint4(pack_f32x2(v.a[0], v.a[1], BF16), pack_f32x2(v.a[2], v.a[3], BF16),
                    pack_f32x2(v.b[0], v.b[1], BF16), pack_f32x2(v.b[2], v.b[3], BF16));
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
#pragma unroll
  for (int x = 0; x < kMaxAxes; ++x) pos[x] = (r.rot > 0 && x < r.axes) ? __ldg(r.positions + (size_t)x * r.T + t) : 0;
}

// Cosines (a) and sines (b) of pairs i0 .. i0 + 3 at these positions. False if
// one of them lies outside the table.
__device__ __forceinline__ bool load_angles(const RowParams& r, const int (&pos)[kMaxAxes], int i0, Pairs& cs) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    cs.a[e] = 1.f;
    cs.b[e] = 0.f;
  }
  if (r.rot == 0) return true;
  bool ok = true;
#pragma unroll
  for (int x = 0; x < kMaxAxes; ++x) ok = ok && pos[x] >= 0 && pos[x] < r.num_pos;
  const int half = r.rot / 2;
  if (!ok || i0 >= half) return ok;
  const uint32_t ax = r.axis[i0 >> 2];
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

// z = rotate(x rsqrt(mean x^2 + eps) w), all in fp32, without the norm or the
// rotation where they are off. The D / 8 lanes of a row sum its squares by the
// same tree wherever a row is computed, so that every kernel built on this
// gives the same bits. Every lane of the warp calls it.
template <int D>
__device__ __forceinline__ Pairs norm_rotate(const Pairs& x, bool norm, const Pairs& w, float eps, bool turn,
                                             const Pairs& cs) {
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) ss = fmaf(x.a[e], x.a[e], fmaf(x.b[e], x.b[e], ss));
#pragma unroll
  for (int o = 1; o < D / 8; o <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
  Pairs y = x;
  if (norm) {
    const float inv = rsqrtf(fmaf(ss, 1.f / D, eps));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y.a[e] = x.a[e] * inv * w.a[e];
      y.b[e] = x.b[e] * inv * w.b[e];
    }
  }
  if (!turn) return y;
  Pairs z;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    z.a[e] = fmaf(y.a[e], cs.a[e], -(y.b[e] * cs.b[e]));
    z.b[e] = fmaf(y.b[e], cs.a[e], y.a[e] * cs.b[e]);
  }
  return z;
}

}  // namespace pqkv
