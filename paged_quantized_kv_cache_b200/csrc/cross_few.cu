// cross_few.cu -- attention of a few decoder tokens per sequence (a decode step,
// a verification of some proposed tokens) to an encoder's cached states.
//
// With at most 16 query rows (tokens x query heads) per KV head the states'
// bytes bound the work, not the products, so this is the decode's way with a
// block (decode_block.cuh: rows as the columns of one or two 8-column
// mma.sync tiles, dequantization in registers), not the prefill's tcgen05
// tiles, 112 of whose 128 rows would be empty and whose dequantization into
// shared memory cannot keep up with the memory.
//
// Work decomposition. One cluster of S CTAs per (sequence, KV head): each CTA
// takes an S-th of the blocks that any of the rows sees, each warp every
// kWarps-th pair of them through a ring of its own, filled by TMA. At the end
// the warps' partial (O, m, l) are joined in shared memory, the CTAs' over
// distributed shared memory, always in the same order: no workspace, one
// launch, results that do not depend on timing. Two CTAs fit an SM, so one's
// start and end hide behind the other's stream.
//
// Measured (32 / 8 heads of 128, one token each): 64 sequences of 2048-6404
// states bf16 163 us (6.8 TB/s), FP8 104-110 us (5.1-5.3 TB/s, bound by the
// dequantization's instructions), FP4 137 us (2.5 TB/s, bound by them too); 16 of
// 1400-1500 bf16 states 21.2 us.
#include <atomic>
#include <climits>

#include "cluster.cuh"
#include "cross.cuh"
#include "decode_block.cuh"

namespace pqkv {

namespace {

constexpr int kMaxFewSplits = 16;  // CTAs of a cluster (above 8: opted into)

// What exponents are taken against when the max is m: 0 while nothing has a max,
// so that 2^(-inf - .) is 0 (-inf - -inf is NaN) and a score of NaN gives NaN.
__device__ __forceinline__ float finite(float m) { return m == -INFINITY ? 0.f : m; }

template <int KVF, int D, int NT>
struct FewGeom {
  using Gm = DecodeGeom<KVF, D, NT>;
  static constexpr int NC = Gm::kCols;
  // half of the decode's warps and stages: two CTAs per SM
  static constexpr int kWarps = Gm::k16 ? (D == 128 ? 3 : 4) : (NT == 1 ? 6 : 4);
  static constexpr int kStages = D == 128 ? 4 : 6;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kTilesBytes = kWarps * kStages * Gm::kTile;
  static constexpr int kSideBytes = kWarps * kStages * Gm::kSideStride;
  static constexpr int kBarBytes = kWarps * kStages * 8;
  static constexpr int kQBytes = Gm::kFp4 ? kWarps * NC * Gm::kQStride * 2 : 0;
  static constexpr int kOextBytes = Gm::kFp4 ? kWarps * NC * Gm::kOStride * 4 : 0;
  static constexpr int kSmem = 1024 + kTilesBytes + kSideBytes + kBarBytes + kQBytes + kOextBytes;
  // partial results, over the tiles and sides once the blocks are done with
  static constexpr int kPart = NC * (D + 2) * 4;  // O [NC][D], m [NC], l [NC]
  static_assert((kWarps + 1) * kPart <= kTilesBytes + kSideBytes, "the warps' and the CTA's partial results");
  static_assert(2 * (kSmem + 1024) <= 227 * 1024, "two CTAs per SM");
};

template <int KVF, int D, bool QBF16, int NT>
__global__ void __launch_bounds__(FewGeom<KVF, D, NT>::kThreads, 2)
    cross_few_kernel(const __grid_constant__ CUtensorMap tmap, const CrossParams p) {
  using Gm = DecodeGeom<KVF, D, NT>;
  using Fg = FewGeom<KVF, D, NT>;
  constexpr int NC = Fg::NC, NW = Fg::kWarps, NS = Fg::kStages, KT = D / 16;
  constexpr bool kBf16Mma = (KVF == PQKV_DTYPE_BF16);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // calls in a row, 64 x 4226 FP8 states: 111.7 -> 105.6 us
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sides = smem + Fg::kTilesBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sides + Fg::kSideBytes);
  uint8_t* qcopy = reinterpret_cast<uint8_t*>(bars) + Fg::kBarBytes;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, qd = lane & 3;
  const int S = p.splits, G = p.G;
  const int rank = (int)(blockIdx.x % (unsigned)S), pair = (int)(blockIdx.x / (unsigned)S);
  int b = pair / p.Hkv;
  const int h = pair - b * p.Hkv;
  if (p.by_length) b = nth_longest(p.kv_lens, p.B, b, reinterpret_cast<int*>(smem));

  const int q0 = p.cu_q[b], qn = p.cu_q[b + 1] - q0;
  const int L = p.kv_lens[b];
  const bool rejected = L < 0 || L > kBlock * p.maxblk;
  if (h == 0 && rank == 0 && tid == 0 && (qn > p.max_q || (qn > 0 && rejected))) raise_flag(p.err, PQKV_DEVERR_SEQ_LEN);
  const int nc = min(qn, p.max_q) * G;  // columns: token n / G, query head n % G
  if (nc <= 0) return;
  auto row_at = [&](int n) -> size_t { return ((size_t)(q0 + n / G) * p.Hq + (size_t)h * G + n % G) * D; };
  // positions [lo, hi) that column n sees
  auto range_of = [&](int n, int& lo, int& hi) {
    lo = hi = 0;
    if (n >= nc || rejected) return;
    hi = L;
    if (p.ranges) {
      const int2 r = __ldg(reinterpret_cast<const int2*>(p.ranges) + q0 + n / G);
      lo = max(r.x, 0);
      hi = min(r.y, L);
    }
  };
  // over all columns: the first position and the end of the last that any sees
  // (the blocks read), and what all of them see (the blocks that need no mask)
  int lo, hi;
  range_of(lane, lo, hi);
  const bool col = lane < nc, sees = col && lo < hi;
  const int any_lo = __reduce_min_sync(kFull, sees ? lo : INT_MAX);
  const int any_hi = __reduce_max_sync(kFull, sees ? hi : 0);
  const int all_lo = __reduce_max_sync(kFull, col ? lo : 0);
  const int all_hi = __reduce_min_sync(kFull, col ? hi : INT_MAX);
  const int first = any_hi > 0 ? any_lo / kBlock : 0;
  const int blocks = any_hi > 0 ? (any_hi + kBlock - 1) / kBlock - first : 0;
  if (blocks == 0) {  // the same for the whole cluster: no column sees anything
    if (rank == 0)
      for (int i = tid; i < nc * D; i += Fg::kThreads) store_out<QBF16>(p.out, row_at(i / D) + i % D, 0.f);
    return;
  }
  int2 range[NT][2];  // of this lane's columns 8nt + 2qd + c
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) range_of(8 * nt + 2 * qd + c, range[nt][c].x, range[nt][c].y);

  uint64_t* wbar = bars + warp * NS;
  uint8_t* wtile = smem + warp * NS * Gm::kTile;
  uint8_t* wside = sides + warp * NS * Gm::kSideStride;
  uint16_t* wq = reinterpret_cast<uint16_t*>(qcopy) + warp * NC * Gm::kQStride;
  float* woext = reinterpret_cast<float*>(qcopy + Fg::kQBytes) + warp * NC * Gm::kOStride;
  const LdsmOffsets<KVF, D> lofs(lane);
  if (lane == 0) {
    for (int s = 0; s < NS; ++s) mbar_init(&wbar[s], 1);
    fence_mbar_init();
  }
  if (tid == 0) prefetch_tensormap(&tmap);
  if constexpr (Gm::kFp4)
    for (int i = lane; i < NC * Gm::kOStride; i += 32) woext[i] = 0.f;
  __syncwarp();

  // ---- this warp's blocks: every NW-th pair of the CTA's share, numbered v = 0 .. V - 1 ----
  const int share = ((blocks + 1) / 2 + S - 1) / S * 2;  // whole pairs
  const int j0 = first + rank * share, n_blk = max(0, min(share, blocks - rank * share));
  const int pairs = (n_blk + 1) / 2;
  const int mine = pairs > warp ? (pairs - warp + NW - 1) / NW : 0;
  const int V = 2 * mine - ((n_blk & 1) && mine > 0 && (pairs - 1) % NW == warp ? 1 : 0);
  auto block_of = [&](int v) { return j0 + 2 * (warp + NW * (v >> 1)) + (v & 1); };
  const int32_t* table = p.block_tables + (size_t)b * p.maxblk;
  auto id_of = [&](int v) -> int { return v < V ? __ldg(table + block_of(v)) : -1; };
  // physical ids of blocks wbase + lane and, loaded ahead, wbase + 32 + lane
  int wbase = 0, ids = id_of(lane), next_ids = id_of(32 + lane);
  uint32_t phase = 0, inflight = 0, skip = 0;  // a bit per stage
  bool aborted = false;
  const uint64_t policy = l2_evict_first_policy();
  auto issue = [&](int s, int v) {
    while (v - wbase >= 32) {
      wbase += 32;
      ids = next_ids;
      next_ids = id_of(wbase + 32 + lane);
    }
    const int id = __shfl_sync(kFull, ids, v - wbase);
    const bool bad = id < 0 || id >= p.nb;
    inflight |= 1u << s;
    if (bad) skip |= 1u << s; else skip &= ~(1u << s);
    if (lane != 0) return;
    uint64_t* bar = &wbar[s];
    if (bad) {
      raise_flag(p.err, PQKV_DEVERR_BLOCK_ID);
      mbar_arrive(bar);
      return;
    }
    const size_t at = (size_t)id * p.Hkv + h;
    mbar_arrive_expect_tx(bar, Gm::kTx);
    uint8_t* dst = wtile + s * Gm::kTile;
    constexpr int kElem = Gm::k16 ? 2 : 1;
#pragma unroll
    for (int bx = 0; bx < Gm::kBoxes; ++bx)
      tma_load_2d_hint(dst + bx * 32 * Gm::kBoxRow, &tmap, bx * (Gm::kBoxRow / kElem), (int)at * 32, bar, policy);
    uint8_t* side = wside + s * Gm::kSideStride;
    if constexpr (Gm::kFp8) {
      bulk_load(side, p.scales + at * 16, 16, bar);
    } else if constexpr (Gm::kFp4) {
      bulk_load(side, p.scales + at * Gm::kScaleBytes, Gm::kScaleBytes, bar);
      bulk_load(side + Gm::kScaleBytes, p.oval + at * Gm::kValBytes, Gm::kValBytes, bar);
      bulk_load(side + Gm::kScaleBytes + Gm::kValBytes, p.oidx + at * 16, 16, bar);
    }
  };
  for (int i = 0; i < min(NS, V); ++i) issue(i, i);

  // ---- the query rows, as B fragments; a bf16 row that becomes f16 is scaled by a power of two ----
  uint32_t qf[NT][KT][2];
  float csc[NT][2];  // softmax scale (log2 units) of the lane's columns, times their row's power of two
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const bool has = 8 * nt + g < nc;
    const size_t qrow = has ? row_at(8 * nt + g) : 0;
    // k-slot order of the dequantized K fragments (block_scores)
    auto d0_of = [&](int kk) { return Gm::kFp8 ? 16 * kk + 4 * qd : 32 * (kk >> 1) + 8 * qd + 4 * (kk & 1); };
    float mul = 1.f;
    if constexpr (!Gm::k16 && QBF16) {
      float mx = 0.f;
      if (has) {
#pragma unroll
        for (int kk = 0; kk < KT; ++kk)
#pragma unroll
          for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fabsf(q_at<QBF16>(p.q, qrow + d0_of(kk) + i)));
      }
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
      mul = ldexpf(1.f, -query_exponent(mx));
    }
#pragma unroll
    for (int kk = 0; kk < KT; ++kk) {
      if constexpr (Gm::k16) {
        const uint32_t* q32 = static_cast<const uint32_t*>(p.q);
        qf[nt][kk][0] = has ? __ldg(q32 + (qrow + 16 * kk + 2 * qd) / 2) : 0u;
        qf[nt][kk][1] = has ? __ldg(q32 + (qrow + 16 * kk + 8 + 2 * qd) / 2) : 0u;
      } else {
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        if (has) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = q_at<QBF16>(p.q, qrow + d0_of(kk) + i) * mul;
        }
        qf[nt][kk][0] = f16x2_from(x[0], x[1]);
        qf[nt][kk][1] = f16x2_from(x[2], x[3]);
      }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) csc[nt][c] = p.scale_log2 / __shfl_sync(kFull, mul, (2 * qd + c) << 2);
    if constexpr (Gm::kFp4) {  // f16 copy for the outlier channels, scaled alike
      for (int n = 8 * nt; n < 8 * nt + 8; ++n) {
        const float m = __shfl_sync(kFull, mul, (n & 7) << 2);
        for (int d = lane; d < D; d += 32)
          wq[n * Gm::kQStride + d] =
              __half_as_ushort(__float2half_rn(n < nc ? q_at<QBF16>(p.q, row_at(n) + d) * m : 0.f));
      }
    }
  }
  __syncwarp();

  // ---- online softmax over this warp's blocks, two at a time ----
  float acc[NT][KT][4] = {};
  float mm[NT][2], ll[NT][2];
  float unit[NT][2] = {}, units = 0.f;  // FP8: 1 / unit of O of the lane's columns (move_unit), and the largest
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    mm[nt][0] = mm[nt][1] = kNegInf;
    ll[nt][0] = ll[nt][1] = 0.f;
  }
  OutlierState<NT> ost;
  ost.reset();
  // A stage whose wait gives up keeps its phase and its bit, for the drain.
  auto wait_stage = [&](int s) -> bool {
    const bool ok = __all_sync(kFull, mbar_wait_bounded(&wbar[s], (phase >> s) & 1u, p.timeout_ns));
    if (ok) {
      phase ^= 1u << s;
      inflight &= ~(1u << s);
    }
    return ok;
  };
  int s = 0;
  for (int v = 0; v < V; v += 2) {
    const bool two = v + 1 < V;
    const int sA = s, sB = (s + 1 == NS) ? 0 : s + 1;
    bool ok = wait_stage(sA);
    if (two) ok = wait_stage(sB) && ok;
    if (!ok) {
      if (lane == 0) raise_flag(p.err, PQKV_DEVERR_TIMEOUT);
      aborted = true;
      break;
    }
    const bool use[2] = {!((skip >> sA) & 1u), two && !((skip >> sB) & 1u)};
    const int base = kBlock * block_of(v);  // position of the first block's first token
    const uint32_t tb[2] = {smem_u32(wtile + sA * Gm::kTile), smem_u32(wtile + sB * Gm::kTile)};
    const uint8_t* sd[2] = {wside + sA * Gm::kSideStride, wside + sB * Gm::kSideStride};
    float x[2][NT][4], sk[2] = {1.f, 1.f}, sv[2] = {1.f, 1.f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) x[i][nt][0] = x[i][nt][1] = x[i][nt][2] = x[i][nt][3] = 0.f;
      if (!use[i]) continue;
      block_scores<KVF, D, NT>(tb[i], sd[i], qf, wq, lofs, lane, x[i], ost);
      if constexpr (Gm::kFp8) {
        sk[i] = reinterpret_cast<const float*>(sd[i])[0];
        sv[i] = reinterpret_cast<const float*>(sd[i])[1];
      }
    }
    // x[i][nt][e]: token base + 16 i + g + 8 (e >> 1), column 8nt + 2qd + (e & 1); log2 units
    const bool full = use[0] && use[1] && all_lo <= base && base + 2 * kBlock <= all_hi;
    float bm[NT][2];
    bool grows = false;
    constexpr float kLazy = lazy_of<KVF>();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[i][nt][e] *= csc[nt][e & 1] * sk[i];
          const int t = base + kBlock * i + g + 8 * (e >> 1);
          if (!full && (!use[i] || t < range[nt][e & 1].x || t >= range[nt][e & 1].y)) x[i][nt][e] = kNegInf;
        }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        bm[nt][c] = fmaxf(fmaxf(x[0][nt][c], x[0][nt][c + 2]), fmaxf(x[1][nt][c], x[1][nt][c + 2]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) bm[nt][c] = fmaxf(bm[nt][c], __shfl_xor_sync(kFull, bm[nt][c], o));
        grows |= bm[nt][c] > mm[nt][c] + kLazy;
      }
    }
    float fc[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) fc[nt][0] = fc[nt][1] = 1.f;
    // FP8: p is at most 2^8 (kLazy), so p s r stays within f16 as long as no s r is above 2^7
    if constexpr (Gm::kFp8) grows |= fmaxf(use[0] ? sv[0] : 0.f, use[1] ? sv[1] : 0.f) * units > 128.f;
    if (__any_sync(kFull, grows)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (bm[nt][c] > mm[nt][c] + kLazy) {
            fc[nt][c] = ex2(mm[nt][c] - bm[nt][c]);
            mm[nt][c] = bm[nt][c];
          }
          ll[nt][c] *= fc[nt][c];
        }
      if constexpr (Gm::kFp8) {
        units = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float need = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float mb = fmaxf(x[i][nt][c], x[i][nt][c + 2]);  // the max of block i alone
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) mb = fmaxf(mb, __shfl_xor_sync(kFull, mb, o));
              if (mb != kNegInf) need = fmaxf(need, ex2(mb - finite(mm[nt][c])) * sv[i]);
            }
            fc[nt][c] = move_unit(unit[nt][c], fc[nt][c], need, mm[nt][c] != kNegInf);
            if (8 * nt + 2 * qd + c < nc) units = fmaxf(units, unit[nt][c]);
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int mt = 0; mt < KT; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nt][mt][e] *= fc[nt][e & 1];
      if constexpr (Gm::kFp4) {  // the outlier channels' O follows
        __syncwarp();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          ost.vacc[nt][0] *= fc[nt][0];
          ost.vacc[nt][1] *= fc[nt][1];
#pragma unroll
          for (int mt = 0; mt < KT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              woext[(8 * nt + 2 * qd + (e & 1)) * Gm::kOStride + dmap<KVF>(mt, g + 8 * (e >> 1))] *= fc[nt][e & 1];
        }
        __syncwarp();
      }
    }
    float w[2][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) w[i][nt][e] = ex2(x[i][nt][e] - finite(mm[nt][e & 1]));
#pragma unroll
      for (int c = 0; c < 2; ++c) ll[nt][c] += (w[0][nt][c] + w[0][nt][c + 2]) + (w[1][nt][c] + w[1][nt][c + 2]);
    }
    // O^T += V^T P^T. 16-bit caches, which the memory bounds, take P = P_hi + P_lo;
    // the others, bound by instruction issue, P in f16 alone (2^-11 of p, far
    // below their codes' own steps): 64 sequences of 2048-6404 FP8 states, one
    // token each, 144 against 136 us.
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!use[i] || (Gm::kFp8 && sv[i] == 0.f)) continue;
      uint32_t b0[NT], b1[NT], c0[NT], c1[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float pr[2] = {1.f, 1.f};
        if constexpr (Gm::kFp8) {
          pr[0] = fminf(sv[i] * unit[nt][0], FLT_MAX);  // finite where every p is 0
          pr[1] = fminf(sv[i] * unit[nt][1], FLT_MAX);
        }
        const float w0 = w[i][nt][0] * pr[0], w1 = w[i][nt][1] * pr[1];
        const float w2 = w[i][nt][2] * pr[0], w3 = w[i][nt][3] * pr[1];
        const uint32_t hA = pack_f32x2(w0, w1, kBf16Mma), hB = pack_f32x2(w2, w3, kBf16Mma);
        b0[nt] = movmatrix_t(hA);
        b1[nt] = movmatrix_t(hB);
        c0[nt] = c1[nt] = 0u;
        if constexpr (Gm::k16) {
          c0[nt] = movmatrix_t(pack_f32x2(w0 - unpack_lo(hA, kBf16Mma), w1 - unpack_hi(hA, kBf16Mma), kBf16Mma));
          c1[nt] = movmatrix_t(pack_f32x2(w2 - unpack_lo(hB, kBf16Mma), w3 - unpack_hi(hB, kBf16Mma), kBf16Mma));
        }
      }
      block_pv<KVF, D, NT, Gm::k16>(tb[i], sd[i], lofs, lane, min(kBlock, L - base - kBlock * i), b0, b1, c0, c1, acc, woext, ost);
    }
    __syncwarp();
    if (v + NS < V) issue(sA, v + NS);
    if (two && v + 1 + NS < V) issue(sB, v + 1 + NS);
    s = (sB + 1 == NS) ? 0 : sB + 1;
  }
  if (aborted) {
    bool drained = true;
    for (int i = 0; i < NS; ++i)
      if ((inflight >> i) & 1u) drained = mbar_wait_bounded(&wbar[i], (phase >> i) & 1u, p.drain_ns) && drained;
    if (!drained && lane == 0) raise_flag(p.err, PQKV_DEVERR_DRAIN);
  }

  // ---- join the warps' parts in shared memory, then the CTAs' over the cluster ----
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) ll[nt][c] += __shfl_xor_sync(kFull, ll[nt][c], o);
  if constexpr (Gm::kFp4) {
    ost.template flush<Gm::kOStride>(woext, lane, D);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int mt = 0; mt < KT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[nt][mt][e] += woext[(8 * nt + 2 * qd + (e & 1)) * Gm::kOStride + dmap<KVF>(mt, g + 8 * (e >> 1))];
  }
  __syncthreads();  // every warp is done with its tiles
  float* part = reinterpret_cast<float*>(smem + warp * Fg::kPart);  // O [NC][D], m [NC], l [NC]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int n = 8 * nt + 2 * qd + c;
      const float vs = Gm::kFp8 ? (unit[nt][c] > 0.f ? 1.f / unit[nt][c] : 0.f) : 1.f;
#pragma unroll
      for (int mt = 0; mt < KT; ++mt) {
        part[n * D + dmap<KVF>(mt, g)] = acc[nt][mt][c] * vs;
        part[n * D + dmap<KVF>(mt, g + 8)] = acc[nt][mt][c + 2] * vs;
      }
      if (g == 0) {  // no max is NaN: that marks a part that a wait cut short
        part[NC * D + n] = aborted ? NAN : mm[nt][c];
        part[NC * D + NC + n] = ll[nt][c];
      }
    }
  __syncthreads();
  float* whole = reinterpret_cast<float*>(smem + NW * Fg::kPart);
  const float* parts = reinterpret_cast<const float*>(smem);
  constexpr int kStep = Fg::kPart / 4;
  auto store4 = [&](int n, int d, const float4& o, float l) {
    const float inv = l == 0.f ? 0.f : 1.f / l;  // a sum of NaN stays one
    const size_t at = row_at(n) + d;
    store_out2<QBF16>(p.out, at, o.x * inv, o.y * inv);
    store_out2<QBF16>(p.out, at + 2, o.z * inv, o.w * inv);
  };
  for (int i = tid; i < nc * (D / 4); i += Fg::kThreads) {
    const int n = i / (D / 4), d = 4 * (i % (D / 4));
    float mx = kNegInf, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    bool cut = false;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const float m = parts[k * kStep + NC * D + n];
      cut |= isnan(m);
      mx = fmaxf(mx, m);
    }
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const float f = ex2(parts[k * kStep + NC * D + n] - finite(mx));
      const float4 a = *reinterpret_cast<const float4*>(parts + k * kStep + n * D + d);
      l = fmaf(f, parts[k * kStep + NC * D + NC + n], l);
      o = make_float4(fmaf(f, a.x, o.x), fmaf(f, a.y, o.y), fmaf(f, a.z, o.z), fmaf(f, a.w, o.w));
    }
    if (S == 1) {
      if (!cut) store4(n, d, o, l);
    } else {
      *reinterpret_cast<float4*>(whole + n * D + d) = o;
      if (d == 0) {
        whole[NC * D + n] = cut ? NAN : mx;
        whole[NC * D + NC + n] = l;
      }
    }
  }
  if (S == 1) return;
  cluster_sync();
  const uint32_t at = smem_u32(whole);
  for (int i = rank * Fg::kThreads + tid; i < nc * (D / 4); i += S * Fg::kThreads) {
    const int n = i / (D / 4), d = 4 * (i % (D / 4));
    float mx = kNegInf, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    bool cut = false;
    for (int k = 0; k < S; ++k) {
      const float m = ld_peer(at + (uint32_t)(NC * D + n) * 4, k);
      cut |= isnan(m);
      mx = fmaxf(mx, m);
    }
    if (cut) continue;
    for (int k = 0; k < S; ++k) {
      const float f = ex2(ld_peer(at + (uint32_t)(NC * D + n) * 4, k) - finite(mx));
      const float4 a = ld_peer4(at + (uint32_t)(n * D + d) * 4, k);
      l = fmaf(f, ld_peer(at + (uint32_t)(NC * D + NC + n) * 4, k), l);
      o = make_float4(fmaf(f, a.x, o.x), fmaf(f, a.y, o.y), fmaf(f, a.z, o.z), fmaf(f, a.w, o.w));
    }
    store4(n, d, o, l);
  }
  cluster_sync();  // no CTA leaves while another reads its part
}

// CTAs per (sequence, KV head): doubled while the doubled grid still fits the
// GPU at two CTAs per SM and every warp keeps a pair of blocks.
int few_splits(long long pairs, int maxblk, int warps, int sms) {
  int s = 1;
  while (2 * s <= kMaxFewSplits && pairs * 2 * s <= 2LL * sms && 2 * s * 2 * warps <= maxblk) s *= 2;
  return s;
}

template <int KVF, int D, bool QBF16, int NT>
cudaError_t launch_few_t(const CUtensorMap& tmap, CrossParams p, int sms, cudaStream_t st) {
  using Fg = FewGeom<KVF, D, NT>;
  auto kern = cross_few_kernel<KVF, D, QBF16, NT>;
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Fg::kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  const long long pairs = (long long)p.B * p.Hkv;
  p.splits = few_splits(pairs, p.maxblk, Fg::kWarps, sms);
  p.by_length = pairs * p.splits > 2LL * sms && p.B <= Fg::kThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(pairs * p.splits));
  cfg.blockDim = dim3(Fg::kThreads);
  cfg.dynamicSmemBytes = Fg::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tmap, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_cross_few(int kv_dtype, int D, bool q_bf16, const CUtensorMap& tmap, const CrossParams& p,
                             int sms, cudaStream_t st) {
#define PQKV_FEW(KVF, DD, QB)                                                             \
  if (kv_dtype == KVF && D == DD && q_bf16 == QB)                                         \
    return p.max_q * p.G > 8 ? launch_few_t<KVF, DD, QB, 2>(tmap, p, sms, st)             \
                             : launch_few_t<KVF, DD, QB, 1>(tmap, p, sms, st);
  PQKV_FEW(PQKV_DTYPE_FP16, 128, false)
  PQKV_FEW(PQKV_DTYPE_FP16, 64, false)
  PQKV_FEW(PQKV_DTYPE_BF16, 128, true)
  PQKV_FEW(PQKV_DTYPE_BF16, 64, true)
  PQKV_FEW(PQKV_DTYPE_FP8_E4M3, 128, true)
  PQKV_FEW(PQKV_DTYPE_FP8_E4M3, 128, false)
  PQKV_FEW(PQKV_DTYPE_FP8_E4M3, 64, true)
  PQKV_FEW(PQKV_DTYPE_FP8_E4M3, 64, false)
  PQKV_FEW(PQKV_DTYPE_FP8_E5M2, 128, true)
  PQKV_FEW(PQKV_DTYPE_FP8_E5M2, 128, false)
  PQKV_FEW(PQKV_DTYPE_FP8_E5M2, 64, true)
  PQKV_FEW(PQKV_DTYPE_FP8_E5M2, 64, false)
  PQKV_FEW(PQKV_DTYPE_FP4_E2M1, 128, true)
  PQKV_FEW(PQKV_DTYPE_FP4_E2M1, 128, false)
  PQKV_FEW(PQKV_DTYPE_FP4_E2M1, 64, true)
  PQKV_FEW(PQKV_DTYPE_FP4_E2M1, 64, false)
#undef PQKV_FEW
  return cudaErrorInvalidValue;
}

}  // namespace pqkv
