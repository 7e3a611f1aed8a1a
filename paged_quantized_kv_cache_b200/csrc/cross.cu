// cross.cu -- attention of decoder tokens to an encoder's cached states, of a
// length of their own, on the sm_100a tensor cores (tcgen05, accumulators in
// tensor memory).
//
// "vLLM" glossary, "PagedAttention": K/V through the block table, one copy read
// by every sequence whose table names it. out = softmax(scale q K^T) V over the
// positions [lo, hi) of [0, L) that the token sees: all of them, or its range.
//
// Work decomposition. A row is (query token, query head of the GQA group); a CTA
// takes up to two tiles of 128 rows of one (sequence, KV head) and the KV tiles
// of 64 positions (4 blocks) between the first and the last position that any
// of its rows sees. With one row tile both halves of the CTA take it, one the
// even KV tiles and one the odd ("dup"), and a small grid splits the KV tiles
// over a cluster of up to 8 CTAs; the parts' O, m and l are joined through
// (distributed) shared memory. No workspace, one launch, no order that depends
// on timing. Warps have one role each, handing over by mbarriers:
//   compute warps: H groups of 4 per row tile, which take its KV tiles in turn,
//     one row per thread (its S, P and O lie in tensor-memory lane r of the row
//     tile's 256 columns): online softmax;
//   producer warps: refill rings of KV tiles, for 16-bit caches one ring of K
//     tiles (free once S is computed) and one of V tiles, each with a warp;
//   for quantized caches 8 dequantization warps: raw codes -> f16 operands;
//   an MMA warp per row tile: S(u) = Q K^T into one of two S buffers, PV(u) from
//     P(u) in tensor memory over the columns of S(u), then S(u + 2).
//
// Softmax. In the usual tile every row of a warp sees all of it or nothing and
// has a max from earlier tiles. That max then stays: exponents are taken against
// it while the scores arrive, 16 columns (a cache block) at a time, without a
// max of the tile, and only a row sum that shows a much larger score (f16 P:
// 2^15, bf16 P: 2^30) takes the tile again the general way: masks, max,
// rescaling of O and l. With H = 2 the warps of a row's
// two groups hand P over in the order of the tiles (a turn per 32 rows): the
// max is shared, and a warp whose turn comes after the max was moved takes its
// tile again.
//
// P is rounded once to the operand type (f16 2^-11, bf16 2^-8 of its value: the
// weights of a mean, whose 16-bit result is rounded as much itself): P_hi + P_lo
// as in the prefill would be half as many products again.
//
// Measured (16 sequences of 300-512 tokens over 3203-6404 bf16 states, 32 / 8
// heads of 128): 537 us, 953 TFLOP/s, when every token sees all states; 507-561 us
// with ranges that leave 37% of them visible (a CTA walks the tiles from the
// first to the last position that any of its rows sees). FP8 states: 566 us, 904
// TFLOP/s, and 589 with ranges. 8 sequences of 129-512 tokens over 1000-4096 FP4
// states: 173 us, 620 TFLOP/s (190 us with the heads as the grid's slow axis,
// where the last head's longest sequences start late). With 16-bit caches the tensor pipe bounds it: S of 64
// columns reads shared memory for most of a tile pair's time (about 1376 of
// 1700 cycles). Quantized caches: the softmax of 8 warps, 2300 cycles a tile.
//
// FP8 scales stay out of the operands: the K scale of a block multiplies its
// scores, the V scale P (move_unit). FP4 operands are exact in f16 (E2M1 x E4M3,
// fp16 outlier values).
#include <atomic>
#include <climits>

#include "attn_math.cuh"
#include "cluster.cuh"
#include "cross.cuh"

namespace pqkv {

namespace {

constexpr int kM = 128;        // rows of a tile
constexpr int kN = 64;         // KV positions of a tile (4 blocks)
constexpr int kMaxSplits = 8;  // CTAs of a cluster (the portable limit)
constexpr float kLazy = 8.f;   // the general way moves a row's max only when it grows by more (log2 units)
constexpr unsigned kFull = 0xFFFFFFFFu;

template <int KVF, int D>
struct CrossGeom {
  static constexpr bool k16 = (KVF == PQKV_DTYPE_FP16 || KVF == PQKV_DTYPE_BF16);
  static constexpr bool kFp8 = (KVF == PQKV_DTYPE_FP8_E4M3 || KVF == PQKV_DTYPE_FP8_E5M2);
  static constexpr bool kFp4 = (KVF == PQKV_DTYPE_FP4_E2M1);
  // Groups of compute warps per row tile. A tile costs a warp about as long in
  // latencies (waits, tensor memory, votes, hand-overs) as in exponents, so 16-bit
  // caches alternate two groups; quantized caches give those warps' registers to
  // the dequantization, which bounds them.
  static constexpr int H = k16 ? 2 : 1;
  static constexpr int kComputeWarps = 8 * H;
  static constexpr int kProducer = kComputeWarps;     // warp roles, in order
  static constexpr int kProducers = k16 ? 2 : 1;      // K and V, or raw tiles
  static constexpr int kMma = kProducer + kProducers; // two of them
  static constexpr int kDeq = kMma + 2;
  static constexpr int kDeqWarps = k16 ? 0 : 8;
  static constexpr int kDeqThreads = 32 * kDeqWarps;
  static constexpr int kThreads = 32 * (kDeq + kDeqWarps);
  static constexpr int NB = D / 64;                   // 128-byte boxes per operand row
  static constexpr int kQBytes = NB * kM * 128;       // Q operand of a row tile [box][128 rows][128 B]
  static constexpr int kOpBytes = NB * kN * 128;      // one K or V operand tile [box][64 rows][128 B]
  static constexpr int kRawTile = 32 * row_bytes(KVF, D);  // one block's K|V codes
  static constexpr int kScaleBytes = kFp8 ? 16 : (kFp4 ? 2 * 16 * (D / 16) : 0);
  static constexpr int kValBytes = kFp4 ? 2 * 16 * 4 * 2 : 0;
  static constexpr int kIdxBytes = kFp4 ? 16 : 0;
  static constexpr int kSide = kScaleBytes + kValBytes + kIdxBytes;
  // KV tiles in flight. A wait for a tile sees only the parity of its stage's
  // phase, so whoever waits must know that the stage's tile before has landed:
  // with an even count the halves that take the tiles in turn (dup) each keep to
  // stages of their own, and have read that tile themselves.
  static constexpr int kStages = 4;
  static_assert(kStages % 2 == 0, "a stage belongs to one half");
  static constexpr int kRawStage = k16 ? 2 * kOpBytes : 4 * (kRawTile + kSide);
  static constexpr int kStageBytes = (kRawStage + 1023) / 1024 * 1024;
  static constexpr int kKops = k16 ? 0 : 2;           // dequantized K tiles
  static constexpr int kVops = k16 ? 0 : 3;           // dequantized V tiles
  static constexpr int kMasks = 16;                   // block masks of KV tiles t % 16
  static constexpr int oQ = 0;
  static constexpr int oStage = oQ + 2 * kQBytes;
  static constexpr int oKop = oStage + kStages * kStageBytes;
  static constexpr int oVop = oKop + kKops * kOpBytes;
  static constexpr int oMisc = oVop + kVops * kOpBytes;
  static constexpr int kBars = 4 * kStages + 12 + 4 + 2 + 3 + 8 + 2 + 1;
  // FP8 scales of tile t % 8: K [8][4], V [8][4]. Tile t is dequantized once S of
  // tile t - 2 is done; with dup that leaves tile t - 4 of the same half unread.
  static constexpr int kScaleSlots = 8;
  static constexpr int oScales = oMisc + (kBars * 8 + 15) / 16 * 16;
  static constexpr int oWords = oScales + kScaleSlots * 32;
  static constexpr int kWords = kMasks + kStages + 1 + 2 + 8 + 2 + 1;
  static constexpr int oRows = oWords + (kWords * 4 + 15) / 16 * 16;  // H = 2: max, and sum of each group, of every row
  static constexpr int kSmem = oRows + (H == 2 ? 3 * 2 * kM * 4 : 0) + 1024;  // + alignment slack
  static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
  static_assert(2 * kM * (D * 4 + 8) <= oMisc, "partial O, m and l over the queries, stages and operands");
};

// The tcgen05 loads, stores and allocations and the named barriers want their
// warp converged; waits and loops whose lanes may part come before many of
// them, so each such place has a __syncwarp first.
template <int N>
__device__ __forceinline__ void deq_sync() {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}

// And-reduction over the `n` threads (a multiple of 32) of named barrier `id`.
__device__ __forceinline__ bool bar_all(int id, int n, bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbar.red.and.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

// Exponents of a row's 64 scores (at t_s) in log2 units, x cj + nm: P, times
// vr, goes to pk as pairs of the operand type, its sum (before vr) is returned.
// kMasked: columns outside `cols` (a bit each) give 0.
template <bool kMasked, bool kFp8, bool kBf16>
__device__ __forceinline__ float exponents(uint32_t t_s, float nm, const float (&cj)[4], const float (&vr)[4],
                                           uint64_t cols, uint32_t (&pk)[32]) {
  float ra[2] = {0.f, 0.f}, rb[2] = {0.f, 0.f};
  uint32_t x[2][16];
  tc::tmem_ld16_start(t_s, x[0]);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (kMasked) __syncwarp();
    tc::tmem_ld_wait(x[j & 1]);
    if (j < 3) tc::tmem_ld16_start(t_s + 16 * (j + 1), x[(j + 1) & 1]);
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
      float ya, yb;
      fma2(ya, yb, __uint_as_float(x[j & 1][c]), __uint_as_float(x[j & 1][c + 1]), cj[j], cj[j], nm, nm);
      if constexpr (kMasked) {
        if (!((cols >> (16 * j + c)) & 1)) ya = -INFINITY;
        if (!((cols >> (16 * j + c + 1)) & 1)) yb = -INFINITY;
      }
      float pa = ex2(ya), pb = ex2(yb);
      const int i = (c >> 1) & 1;
      add2(ra[i], rb[i], ra[i], rb[i], pa, pb);
      if constexpr (kFp8) mul2(pa, pb, pa, pb, vr[j], vr[j]);
      pk[8 * j + (c >> 1)] = pack_f32x2(pa, pb, kBf16);
    }
  }
  return (ra[0] + ra[1]) + (rb[0] + rb[1]);
}

// The largest of a row's scores x cj (kMasked: of those in `cols`); kPerBlock:
// mx[j] is that of block j.
template <bool kMasked, bool kPerBlock>
__device__ __forceinline__ float largest(uint32_t t_s, const float (&cj)[4], uint64_t cols, float (&mx)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) mx[j] = -INFINITY;
  uint32_t x[2][16];
  tc::tmem_ld16_start(t_s, x[0]);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (kMasked) __syncwarp();
    tc::tmem_ld_wait(x[j & 1]);
    if (j < 3) tc::tmem_ld16_start(t_s + 16 * (j + 1), x[(j + 1) & 1]);
#pragma unroll
    for (int c = 0; c < 16; ++c)
      if (!kMasked || ((cols >> (16 * j + c)) & 1)) {
        float& most = mx[kPerBlock ? j : c & 3];
        most = fmaxf(most, __uint_as_float(x[j & 1][c]) * cj[j]);
      }
  }
  return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}

template <int KVF, int D, bool QBF16>
__global__ void __launch_bounds__(CrossGeom<KVF, D>::kThreads, 1)
    paged_cross_kernel(const __grid_constant__ CUtensorMap tmap, const __grid_constant__ CrossParams p) {
  using Gm = CrossGeom<KVF, D>;
  constexpr int H = Gm::H;
  constexpr bool kBfMma = (KVF == PQKV_DTYPE_BF16);  // operand type: bf16 for a bf16 cache, else f16
  constexpr uint32_t kIdescS = tc::f16_idesc(kBfMma, kM, kN, false);
  constexpr uint32_t kIdescPV = tc::f16_idesc(kBfMma, kM, D, true);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sKop = smem + Gm::oKop;
  uint8_t* sVop = smem + Gm::oVop;
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(smem + Gm::oMisc);  // [kStages] tile (16-bit: its K) landed
  uint64_t* bar_empty = bar_full + Gm::kStages;                         // [kStages] its stage free again
  uint64_t* bar_vfull = bar_empty + Gm::kStages;                        // 16-bit: the same for V
  uint64_t* bar_vempty = bar_vfull + Gm::kStages;
  uint64_t* bar_s = bar_vempty + Gm::kStages;     // [2][2] row tile w's S(u) computed (buffer u % 2)
  uint64_t* bar_p = bar_s + 4;                   // [2][2] its P(u) in tensor memory (one arrival per warp)
  uint64_t* bar_pv = bar_p + 4;                  // [2][2] its PV(u) computed
  uint64_t* bar_op = bar_pv + 4;                 // [4] quantized: operands, mask and scales of tile t ready
  uint64_t* bar_kfree = bar_op + 4;              // [2] quantized: every S(t) done (kop[t % 2])
  uint64_t* bar_vfree = bar_kfree + 2;           // [3] quantized: every PV(t) done (vop[t % 3])
  uint64_t* bar_turn = bar_vfree + 3;            // [2][4] H = 2: tile u of these 32 rows handed over (phase u)
  uint64_t* bar_drain = bar_turn + 8;            // [2] every product an MMA warp issued has completed
  uint64_t* bar_q = bar_drain + 2;               // the Q tiles are there (one arrival per compute warp)
  float* tile_sk = reinterpret_cast<float*>(smem + Gm::oScales);  // [kScaleSlots][4] FP8 K scales
  float* tile_sv = tile_sk + 4 * Gm::kScaleSlots;                 // [kScaleSlots][4] FP8 V scales
  volatile int* tile_mask = reinterpret_cast<volatile int*>(smem + Gm::oWords);  // [kMasks] blocks of tile t that hold data
  volatile int* stage_mask = tile_mask + Gm::kMasks;  // [kStages] quantized: the same, of a raw stage
  volatile int* abort_flag = stage_mask + Gm::kStages;
  volatile int* n_issued = abort_flag + 1;       // [2] tiles that the producers started
  volatile int* row_moves = n_issued + 2;        // [2][4] H = 2: how often the max of these 32 rows was moved
  int* span = const_cast<int*>(row_moves) + 8;   // [2] positions that rows of the CTA see
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(span + 2);
  float* row_max = reinterpret_cast<float*>(smem + Gm::oRows);  // [2][128] H = 2
  float* row_sum = row_max + 2 * kM;                            // [2 groups][2][128] H = 2

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // 4 sequences of 3-40 tokens: 11.7 -> 11.4 us
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);  // the same register for the whole warp
  const int h = blockIdx.x % (unsigned)p.Hkv, rank = blockIdx.z;  // all heads of the longest sequence first
  const int G = p.G, TOK = kM / G;
  const int ctas = (p.tiles_per_seq + 1) / 2;
  const int pair = blockIdx.x / (unsigned)p.Hkv;
  int b = pair / ctas;
  const int mt0 = 2 * (pair % ctas);  // first row tile
  if (p.by_length) b = nth_longest(p.kv_lens, p.B, b, reinterpret_cast<int*>(smem));
  const int q0 = p.cu_q[b], qn = p.cu_q[b + 1] - q0;
  const int L = p.kv_lens[b];
  if (mt0 == 0 && h == 0 && rank == 0 && tid == 0 && qn > (long long)p.tiles_per_seq * TOK)
    raise_flag(p.err, PQKV_DEVERR_SEQ_LEN);  // rows past max_q_len are not computed
  if (qn <= 0 || mt0 * TOK >= qn) return;
  const bool rejected = L < 0 || L > kBlock * p.maxblk;
  if (rejected && mt0 == 0 && h == 0 && rank == 0 && tid == 0) raise_flag(p.err, PQKV_DEVERR_SEQ_LEN);

  const int n_rows = min(min(qn - mt0 * TOK, 2 * TOK) * G, min(p.tiles_per_seq - mt0, 2) * kM);
  // compute warps: half of the CTA (0, 1), group (0 .. H - 1), quarter of the tile's lanes
  const bool is_compute = warp < Gm::kComputeWarps;
  const int wg = (warp >> 2) & 1, group = warp >> 3, quad = warp & 3;
  const int r = 32 * quad + lane;
  const bool one_tile = n_rows <= kM;
  const int row = (one_tile ? 0 : wg * kM) + r;           // row of this thread in the CTA's rows
  const bool row_ok = is_compute && row < n_rows;
  const int my_token = q0 + mt0 * TOK + (row_ok ? row / G : 0);
  const size_t orow = ((size_t)my_token * p.Hq + (size_t)h * G + row % G) * D;
  // warps of half w's row tile that hold rows
  auto warps_of = [&](int w) { return min(4, (n_rows - (one_tile ? 0 : w * kM) + 31) / 32); };

  // ---- positions that the rows see; the KV tiles of this CTA ----
  int my_lo = 0, my_hi = 0, lo = 0, hi = rejected ? 0 : L;
  if (p.ranges && !rejected) {
    if (tid == 0) {
      span[0] = L;
      span[1] = 0;
    }
    __syncthreads();
    if (row_ok) {
      const int2 r2 = __ldg(reinterpret_cast<const int2*>(p.ranges) + my_token);
      my_lo = max(r2.x, 0);
      my_hi = min(r2.y, L);
    }
    if (is_compute) {
      const bool sees = row_ok && my_lo < my_hi;
      const int a = __reduce_min_sync(kFull, sees ? my_lo : INT_MAX), z = __reduce_max_sync(kFull, sees ? my_hi : 0);
      if (lane == 0 && z > 0) {
        atomicMin(&span[0], a);
        atomicMax(&span[1], z);
      }
    }
    __syncthreads();
    lo = span[0];
    hi = span[1];
  } else if (row_ok) {
    my_hi = hi;
  }
  const int first = lo / kN, tiles = max(0, (hi + kN - 1) / kN - first);
  if (tiles == 0) {  // the same for every CTA of the cluster: no row sees anything
    if (row_ok && rank == 0 && group == 0 && (!one_tile || wg == 0)) {
      uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + orow);
      for (int c = 0; c < D / 8; ++c) o[c] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const int share = (tiles + p.splits - 1) / p.splits;
  const int t0 = first + rank * share;                        // tile 0 of this CTA
  const int T = max(0, min(share, tiles - rank * share));
  // one row tile: the halves of the CTA take the KV tiles in turn, half w tiles
  // w, w + 2, ... (the second half has none if there is one KV tile)
  const bool dup = one_tile && share > 1;
  const int pshift = dup ? 1 : 0, par = 1 << pshift;
  const int consumers = one_tile ? 1 : 2;  // MMA warps that read a KV tile
  auto tiles_of = [&](int w) { return dup ? (T - w + 1) >> 1 : (one_tile && w > 0 ? 0 : T); };
  const int32_t* table = p.block_tables + (size_t)b * p.maxblk;
  constexpr int ns = Gm::kStages;
  auto stage_at = [&](int s) -> uint8_t* { return smem + Gm::oStage + s * Gm::kStageBytes; };
  auto stage_of = [&](int t) { return t % ns; };
  auto lap_of = [&](int t) { return (uint32_t)(t / ns) & 1u; };

  // ---- setup: tensor memory, barriers ----
  __syncwarp();
  if (warp == 0) tc::tmem_alloc(tmem_slot, 512);
  if (tid == 32 * Gm::kProducer) {
    if constexpr (Gm::k16) prefetch_tensormap(&tmap);
    for (int s = 0; s < Gm::kStages; ++s) {
      mbar_init(&bar_full[s], 1);
      mbar_init(&bar_empty[s], Gm::k16 ? consumers : 1);  // 16-bit: each MMA warp's commit; else dequantized
      mbar_init(&bar_vfull[s], 1);
      mbar_init(&bar_vempty[s], consumers);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar_s[i], 1);
      mbar_init(&bar_p[i], max(1, warps_of(i >> 1)));
      mbar_init(&bar_pv[i], 1);
      mbar_init(&bar_op[i], 1);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(&bar_turn[i], 1);
      row_moves[i] = 0;
    }
    for (int i = 0; i < 2; ++i) mbar_init(&bar_kfree[i], consumers);
    for (int i = 0; i < 3; ++i) mbar_init(&bar_vfree[i], consumers);
    for (int i = 0; i < 2; ++i) mbar_init(&bar_drain[i], 1);
    mbar_init(bar_q, Gm::kComputeWarps);
    *abort_flag = 0;
    n_issued[0] = n_issued[1] = 0;
    fence_mbar_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  float m = -INFINITY, l = 0.f, unit = 0.f;  // this row's max, sum (of this thread's tiles), FP8: 1 / unit of O
  bool aborted = false;

  if (warp >= Gm::kProducer && warp < Gm::kMma) {
    // ================= producers: KV tiles (16-bit: K, and V) into the stage rings =================
    // A lane per copy of a tile (copy `what` of block j), its block ids read two
    // tiles ahead: read and issued one after the other by one thread, a tile
    // took 1450 cycles.
    constexpr int kCopies = Gm::k16 ? Gm::NB : (Gm::kFp8 ? 2 : 4);  // per block
    const int kv = warp - Gm::kProducer;  // 16-bit: 0 = K, 1 = V
    uint64_t* full = kv ? bar_vfull : bar_full;
    uint64_t* empty = kv ? bar_vempty : bar_empty;
    const int j = lane / kCopies, what = lane % kCopies;
    const int hi_blk = (hi + kBlock - 1) / kBlock;  // blocks from here on are not read
    auto id_of = [&](int t) {
      const int blk = 4 * (t0 + t) + j;
      return j < 4 && t < T && blk < hi_blk ? __ldg(table + blk) : -1;
    };
    int id = id_of(0), id1 = id_of(1), id2 = id_of(2);
    int t = 0, s = 0;
    uint32_t lap = 0;
    for (; t < T; ++t) {
      if (t >= ns && !__all_sync(kFull, mbar_test_wait(&empty[s], lap ^ 1u) ||
                                            mbar_wait_bounded(&empty[s], lap ^ 1u, p.timeout_ns)))
        break;
      if (*abort_flag) break;
      const bool inside = j < 4 && 4 * (t0 + t) + j < hi_blk, good = inside && id >= 0 && id < p.nb;
      if (inside && !good && what == 0) raise_flag(p.err, PQKV_DEVERR_BLOCK_ID);
      const uint32_t votes = __ballot_sync(kFull, good && what == 0);
      if (lane == 0) {
        int mask = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) mask |= ((votes >> (i * kCopies)) & 1) << i;
        // published to the consumers by the stage's barrier
        if (!Gm::k16) stage_mask[s] = mask;
        else if (kv == 0) tile_mask[t % Gm::kMasks] = mask;
        constexpr uint32_t kBytes = Gm::k16 ? (uint32_t)Gm::NB * kBlock * 128u : (uint32_t)(Gm::kRawTile + Gm::kSide);
        mbar_arrive_expect_tx(&full[s], (uint32_t)__popc(mask) * kBytes);
      }
      __syncwarp();
      if (good) {
        uint8_t* st = stage_at(s);
        const size_t pair = (size_t)id * p.Hkv + h;
        if constexpr (Gm::k16) {
          tma_load_2d(st + kv * Gm::kOpBytes + what * kN * 128 + j * kBlock * 128, &tmap, what * 64,
                      (int)pair * 32 + 16 * kv, &full[s]);
        } else {
          uint8_t* side = st + 4 * Gm::kRawTile + j * Gm::kSide;
          if (what == 0)
            bulk_load(st + j * Gm::kRawTile, p.cache + pair * Gm::kRawTile, Gm::kRawTile, &full[s]);
          else if (what == 1)
            bulk_load(side, p.scales + pair * Gm::kScaleBytes, Gm::kScaleBytes, &full[s]);
          else if (what == 2)
            bulk_load(side + Gm::kScaleBytes, p.oval + pair * Gm::kValBytes, Gm::kValBytes, &full[s]);
          else
            bulk_load(side + Gm::kScaleBytes + Gm::kValBytes, p.oidx + pair * 16, 16, &full[s]);
        }
      }
      id = id1;
      id1 = id2;
      id2 = id_of(t + 3);
      if (++s == ns) {
        s = 0;
        lap ^= 1u;
      }
    }
    if (lane == 0) n_issued[kv] = t;
  } else if (warp >= Gm::kMma && warp < Gm::kMma + 2) {
    // ================= MMA warp of half w: its products, KV tiles t = w0 + u par =================
    // Order: PV(u) once P(u) is in tensor memory, then S(u + 2) into the buffer
    // that P(u) occupied, once PV(u) has read it. S(0) and S(1) come first, so
    // the half finds the scores of its next tile computed.
    // The whole warp walks the tiles, so that addresses stay in uniform
    // registers; one thread of it issues.
    const int w = warp - Gm::kMma, w0 = dup ? w : 0, U = tiles_of(w);
    bool good = true;
    // both barriers' phases are complete
    auto wait = [&](uint64_t* bar, uint32_t parity, uint64_t* bar2, uint32_t parity2) {
      const bool a = mbar_test_wait(bar, parity), a2 = mbar_test_wait(bar2, parity2);
      good = __all_sync(kFull, (a || mbar_wait_bounded(bar, parity, p.timeout_ns)) &&
                                   (a2 || mbar_wait_bounded(bar2, parity2, p.timeout_ns))) &&
             good;
    };
    // tiles in order: those whose S is issued next (k) and whose PV is (v), with
    // their places in the rings
    struct Place {
      int t, s;
      uint32_t lap;
    };
    auto next = [&](Place& x) {
      x.t += par;
      x.s += par;
      if (x.s >= ns) {
        x.s -= ns;
        x.lap ^= 1u;
      }
    };
    Place k{w0, w0, 0}, v{w0, w0, 0};
    // K (with it, quantized, V) of tile k.t is there
    auto k_bar = [&]() { return Gm::k16 ? &bar_full[k.s] : &bar_op[k.t & 3]; };
    auto k_parity = [&]() { return Gm::k16 ? k.lap : (uint32_t)(k.t >> 2) & 1u; };
    const uint32_t base = smem_u32(smem);
    const uint32_t qa = base + Gm::oQ + (one_tile ? 0 : w) * Gm::kQBytes;
    const bool issuer = tc::elect_one();
    auto stage_addr = [&](int s) -> uint32_t { return base + Gm::oStage + s * Gm::kStageBytes; };
    const uint64_t q_desc = tc::sw128_desc(qa, 16, 1024);
    auto issue_s = [&](int u) {
      tc::fence_after_sync();
      const uint32_t d = tmem + 256u * w + D + 64 * (u & 1);
      const uint32_t ka = Gm::k16 ? stage_addr(k.s) : base + Gm::oKop + (k.t & 1) * Gm::kOpBytes;
      const uint64_t k_desc = tc::sw128_desc(ka, 16, 1024);
      if (issuer) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)  // addresses in units of 16 bytes; no field overflows (shared memory)
          tc::mma_ss(d, q_desc + (kk >> 2) * (kM * 8) + (kk & 3) * 2, k_desc + (kk >> 2) * (kN * 8) + (kk & 3) * 2,
                     kIdescS, kk > 0);
        tc::commit(&bar_s[2 * w + (u & 1)]);
        tc::commit(Gm::k16 ? &bar_empty[k.s] : &bar_kfree[k.t & 1]);  // K may be refilled
      }
      next(k);
    };
    auto issue_pv = [&](int u) {
      tc::fence_after_sync();
      const uint32_t va = Gm::k16 ? stage_addr(v.s) + Gm::kOpBytes : base + Gm::oVop + (v.t % 3) * Gm::kOpBytes;
      const uint64_t v_desc = tc::sw128_desc(va, kN * 128, 1024);
      const uint32_t o = tmem + 256u * w, pa = o + D + 64 * (u & 1);
      if (issuer) {
#pragma unroll
        for (int kk = 0; kk < kN / 16; ++kk)
          tc::mma_ts(o, pa + kk * 8, v_desc + kk * 128, kIdescPV, u > 0 || kk > 0);
        tc::commit(&bar_pv[2 * w + (u & 1)]);
        tc::commit(Gm::k16 ? &bar_vempty[v.s] : &bar_vfree[v.t % 3]);  // V may be refilled
      }
      next(v);
    };
    for (int u = 0; u < min(2, U) && good; ++u) {
      wait(k_bar(), k_parity(), bar_q, 0);
      if (good) issue_s(u);
    }
    for (int u = 0; u < U && good; ++u) {
      uint64_t* p_bar = &bar_p[2 * w + (u & 1)];
      const uint32_t p_parity = (uint32_t)(u >> 1) & 1u;
      wait(p_bar, p_parity, Gm::k16 ? &bar_vfull[v.s] : p_bar, Gm::k16 ? v.lap : p_parity);
      if (!good) break;
      issue_pv(u);
      if (u + 2 < U) {
        wait(&bar_pv[2 * w + (u & 1)], p_parity, k_bar(), k_parity());
        if (good) issue_s(u + 2);
      }
    }
    if (!good && lane == 0) {
      *abort_flag = 1;
      raise_flag(p.err, PQKV_DEVERR_TIMEOUT);
    }
    // every product issued completes before tensor memory is released
    if (issuer) tc::commit(&bar_drain[w]);
    if (!mbar_wait_bounded(&bar_drain[w], 0, p.drain_ns) && lane == 0) raise_flag(p.err, PQKV_DEVERR_DRAIN);
  } else if (!is_compute) {
    // ================= dequantization warps (quantized caches) =================
    // Tile t: raw codes landed, the operand buffers free again (every S(t - 2)
    // read kop[t % 2], every PV(t - 3) vop[t % 3]), then the codes become f16
    // operands; bar_op[t % 4] hands them, the tile's block mask and FP8 scales
    // over, and the raw stage goes back to the producer. The warps leave
    // together, at a consensus.
    if constexpr (!Gm::k16) {
      const int dq = tid - 32 * Gm::kDeq;
      bool ok = true;
      for (int t = 0; t < T; ++t) {
        const int s = stage_of(t);
        ok = mbar_wait_bounded(&bar_full[s], lap_of(t), p.timeout_ns) && ok;
        if (t >= 2) ok = mbar_wait_bounded(&bar_kfree[t & 1], (uint32_t)((t >> 1) - 1) & 1u, p.timeout_ns) && ok;
        if (t >= 3) ok = mbar_wait_bounded(&bar_vfree[t % 3], (uint32_t)((t / 3) - 1) & 1u, p.timeout_ns) && ok;
        ok = bar_all(1, Gm::kDeqThreads, ok);
        if (!ok) break;
        const int mask = stage_mask[s];
        const int base = (t0 + t) * kN;
        uint8_t* st = stage_at(s);
        uint8_t* kop = sKop + (t & 1) * Gm::kOpBytes;
        uint8_t* vop = sVop + (t % 3) * Gm::kOpBytes;
        constexpr int CPR = D / 8;  // 16-byte operand chunks per row
        constexpr int kRounds = kN * CPR / Gm::kDeqThreads;  // a compile-time count: fully unrolled
        static_assert(kN * CPR % Gm::kDeqThreads == 0, "whole rounds");
#pragma unroll
        for (int k = 0; k < kRounds; ++k) {
          const int u = dq + k * Gm::kDeqThreads;
          const int rr = u / CPR, c = u % CPR, j = rr >> 4, tr = rr & 15;
          uint32_t kf[4] = {0, 0, 0, 0}, vf[4] = {0, 0, 0, 0};
          if (((mask >> j) & 1) && base + rr < L) {
            const uint8_t* tile = st + j * Gm::kRawTile;
            if constexpr (Gm::kFp8) {
              const uint2 kc = *reinterpret_cast<const uint2*>(tile + tr * D + 8 * c);
              const uint2 vc = *reinterpret_cast<const uint2*>(tile + (16 + tr) * D + 8 * c);
              kf[0] = dec_fp8x2<KVF>(kc.x);
              kf[1] = dec_fp8x2<KVF>(kc.x >> 16);
              kf[2] = dec_fp8x2<KVF>(kc.y);
              kf[3] = dec_fp8x2<KVF>(kc.y >> 16);
              vf[0] = dec_fp8x2<KVF>(vc.x);
              vf[1] = dec_fp8x2<KVF>(vc.x >> 16);
              vf[2] = dec_fp8x2<KVF>(vc.y);
              vf[3] = dec_fp8x2<KVF>(vc.y >> 16);
            } else {
              const uint8_t* side = st + 4 * Gm::kRawTile + j * Gm::kSide;
              constexpr int SPR = D / 16;  // scale bytes per token row
              // K: row tr, channels 8c..8c+7 = 4 bytes, channel 2i in the low nibble
              dec_e2m1x8(*reinterpret_cast<const uint32_t*>(tile + tr * (D / 2) + 4 * c), kf);
              // V: token-pair rows; this token's nibble of channels 8c..8c+7
              const int hh = (8 * c) / (D / 2);
              const int pr = tr < 8 ? (tr & ~1) : (((tr - 8) & ~1) + 1);
              const uint2 wv =
                  *reinterpret_cast<const uint2*>(tile + (16 + 8 * hh + pr) * (D / 2) + (8 * c) % (D / 2));
              const uint32_t x0 = ((tr & 1) ? (wv.x >> 4) : wv.x) & 0x0F0F0F0Fu;
              const uint32_t x1 = ((tr & 1) ? (wv.y >> 4) : wv.y) & 0x0F0F0F0Fu;
              dec_e2m1x8(prmt(x0 | (x0 >> 4), x1 | (x1 >> 4), 0x6420u), vf);
              const __half2 sk = scale2(side[tr * SPR + (c >> 1)]);
              const __half2 sv = scale2(side[16 * SPR + tr * SPR + (c >> 1)]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                kf[i] = hmul2u(kf[i], sk);
                vf[i] = hmul2u(vf[i], sv);
              }
            }
          }
          const uint32_t off = (c >> 3) * (kN * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4);
          *reinterpret_cast<uint4*>(kop + off) = make_uint4(kf[0], kf[1], kf[2], kf[3]);
          *reinterpret_cast<uint4*>(vop + off) = make_uint4(vf[0], vf[1], vf[2], vf[3]);
        }
        if constexpr (Gm::kFp4) {
          // outlier channels (their codes are 0): write the fp16 values over them;
          // item = (block j, K|V, slot, eighth of the tokens)
          deq_sync<Gm::kDeqThreads>();
          static_assert(Gm::kDeqThreads == 256, "an item per thread");
          const int j = dq >> 6, kv = (dq >> 5) & 1, slot = (dq >> 3) & 3, eighth = dq & 7;
          if ((mask >> j) & 1) {
            const uint8_t* side = st + 4 * Gm::kRawTile + j * Gm::kSide;
            const int ch = side[Gm::kScaleBytes + Gm::kValBytes + 8 * kv + slot];
            if (ch < D) {
              const uint16_t* val = reinterpret_cast<const uint16_t*>(side + Gm::kScaleBytes) + kv * 64;
              uint8_t* op = kv ? vop : kop;
              const int c = ch >> 3;
#pragma unroll
              for (int q4 = 0; q4 < 2; ++q4) {
                const int tr = 2 * eighth + q4, rr = 16 * j + tr;
                if (base + rr < L)
                  *reinterpret_cast<uint16_t*>(op + (c >> 3) * (kN * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4) +
                                               (ch & 7) * 2) = val[tr * 4 + slot];
              }
            }
          }
        }
        if constexpr (Gm::kFp8) {
          if (dq < 4) {
            const bool okb = (mask >> dq) & 1;
            const float* sc = reinterpret_cast<const float*>(st + 4 * Gm::kRawTile + dq * Gm::kSide);
            tile_sk[(t % Gm::kScaleSlots) * 4 + dq] = okb ? sc[0] : 0.f;
            tile_sv[(t % Gm::kScaleSlots) * 4 + dq] = okb ? sc[1] : 0.f;
          }
        }
        if (dq == 0) tile_mask[t % Gm::kMasks] = mask;
        tc::fence_smem_to_async();
        deq_sync<Gm::kDeqThreads>();  // every thread's part is written
        if (dq == 0) {
          mbar_arrive(&bar_empty[s]);  // a raw stage is free as soon as it is dequantized
          mbar_arrive(&bar_op[t & 3]);
        }
      }
      if (!ok && dq == 0) {
        *abort_flag = 1;
        raise_flag(p.err, PQKV_DEVERR_TIMEOUT);
      }
    }
  } else {
    // ================= compute warps: row r of half wg, its tiles u = group, group + H, ... =================
    // softmax scale in log2 units of this thread's row, times 2^e when the row's
    // bf16 query was scaled by 2^-e before narrowing to f16 (quantized caches)
    float sl2 = p.scale_log2;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + orow);
    float qmul = 1.f;
    if constexpr (!Gm::k16 && QBF16) {
      // the power of two 2^-e that brings the row's largest |q| into
      // [2^13, 2^14): exact, and far from both ends of the f16 range
      float mx = 0.f;
      if (row_ok) {
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = __ldg(src + c);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
        }
      }
      const int ex = query_exponent(mx);
      qmul = ldexpf(1.f, -ex);
      sl2 = p.scale_log2 * ldexpf(1.f, ex);
    }
    if (!one_tile || wg == 0) {
      // this thread's share of its row of the Q tile, converted to the operand
      // type, 16-byte chunks swizzled; rows past the end are zeros
      uint8_t* sQ = smem + Gm::oQ + (one_tile ? 0 : wg) * Gm::kQBytes;
#pragma unroll 4
      for (int c = group * (D / 8 / H); c < (group + 1) * (D / 8 / H); ++c) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row_ok) v = __ldg(src + c);
        if constexpr (!Gm::k16 && QBF16) {
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = to_f16x2(__uint_as_float(w[i] << 16) * qmul, __uint_as_float(w[i] & 0xFFFF0000u) * qmul);
          v = make_uint4(w[0], w[1], w[2], w[3]);
        }
        *reinterpret_cast<uint4*>(sQ + (c >> 3) * (kM * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
      }
    }
    tc::fence_smem_to_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_q);
    const uint32_t t_row = tmem + 256u * wg + ((uint32_t)(32 * quad) << 16);
    uint64_t* my_s = bar_s + 2 * wg;
    uint64_t* my_p = bar_p + 2 * wg;
    uint64_t* my_pv = bar_pv + 2 * wg;
    uint64_t* my_turn = bar_turn + 4 * wg + quad;
    // a warp without rows has only zeros to leave in the Q tile
    const int w0 = dup ? wg : 0, U = quad < warps_of(wg) ? tiles_of(wg) : 0;
    bool ok = true;      // no wait of this thread has timed out
    int moves = 0;       // H = 2: moves of the max that this warp has followed
    // tiles [whole_lo, whole_hi) of the CTA lie inside this row's range, tiles
    // below none_hi and from none_lo on outside it; those below t_full end
    // inside the states
    int whole_lo = 0, whole_hi = 0, none_hi = INT_MAX, none_lo = 0;
    const int t_full = L / kN - t0;
    if (row_ok && my_lo < my_hi) {
      whole_lo = (my_lo + kN - 1) / kN - t0;
      whole_hi = my_hi / kN - t0;
      none_hi = my_lo / kN - t0;
      none_lo = (my_hi + kN - 1) / kN - t0;
    }
    // largest row sum of a tile: f16 P fits its type; bf16 P leaves values below
    // 2^70 room in the sums over 2^25 tiles
    constexpr float kMost = kBfMma ? 0x1p30f : 0x1p15f;
    // the max was moved by the row's other group: l follows
    auto follow = [&]() {
      const float to = row_max[wg * kM + r];
      l *= m == to ? 1.f : ex2(m - to);  // 0 when m was -inf (and l 0)
      m = to;
    };

    for (int u = group; u < U; u += H) {
      const int t = w0 + (u << pshift);
      const uint32_t t_s = t_row + D + 64 * (u & 1);
      ok = (mbar_test_wait(&my_s[u & 1], (uint32_t)(u >> 1) & 1u) ||
            mbar_wait_bounded(&my_s[u & 1], (uint32_t)(u >> 1) & 1u, p.timeout_ns)) && ok;
      // S(u) done: its MMA warp saw the tile's operands, mask and scales, so they are visible here too
      const int mask = tile_mask[t % Gm::kMasks];
      const bool none = t < none_hi || t >= none_lo;
      // every row of the warp sees all of the tile or nothing
      const bool plain = __all_sync(kFull, ok && mask == 0xF && t < t_full && (none || (t >= whole_lo && t < whole_hi)));
      tc::fence_after_sync();
      float cj[4], vr[4];  // a row that sees nothing of a plain tile gets arguments of 0 x - inf
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        cj[j] = none ? 0.f : sl2;
        vr[j] = 1.f;
      }
      float most_v = 1.f;  // FP8: the largest factor of P, or 1
      if constexpr (Gm::kFp8) {
        const float4 k4 = *reinterpret_cast<const float4*>(tile_sk + (t % Gm::kScaleSlots) * 4);
        const float4 v4 = *reinterpret_cast<const float4*>(tile_sv + (t % Gm::kScaleSlots) * 4);
        const float k[4] = {k4.x, k4.y, k4.z, k4.w}, v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          cj[j] *= k[j];
          vr[j] = none ? 0.f : v[j] * unit;  // a block without data has scale 0
          most_v = fmaxf(most_v, vr[j]);
        }
      }
      uint32_t pk[32];
      float sum = 0.f;
      // the usual way, against the max as this warp knows it
      auto usual = [&]() -> bool {
        if (!__all_sync(kFull, plain && (none || m != -INFINITY))) return false;
        sum = exponents<false, Gm::kFp8, kBfMma>(t_s, none ? -INFINITY : -m, cj, vr, 0, pk);
        return __all_sync(kFull, sum * most_v <= kMost);
      };
      bool done = usual();
      if constexpr (H == 2) {
        // this warp's turn: the tile before has been handed over
        if (u > 0)
          ok = (mbar_test_wait(my_turn, (uint32_t)(u - 1) & 1u) ||
                mbar_wait_bounded(my_turn, (uint32_t)(u - 1) & 1u, p.timeout_ns)) && ok;
        if (row_moves[wg * 4 + quad] != moves) {
          moves = row_moves[wg * 4 + quad];
          follow();
          done = usual();
        }
      }
      if (!__all_sync(kFull, done && ok)) {
        // ---- the general way: masks, max, rescaling ----
        if (!__all_sync(kFull, ok)) {
          aborted = true;
          break;
        }
        const int base = (t0 + t) * kN;
        if constexpr (Gm::k16) {
          // V rows without valid data (past the states, or a block not loaded)
          // are zeroed: P is 0 there, and 0 x NaN would poison O. Each row tile's
          // warps zero them (the same zeros) before their P is handed over.
          if (mask != 0xF || t >= t_full) {
            ok = mbar_wait_bounded(&bar_vfull[stage_of(t)], lap_of(t), p.timeout_ns) && ok;
            uint8_t* v_op = stage_at(stage_of(t)) + Gm::kOpBytes;
            const int step = 32 * warps_of(wg);
            for (int i = r; i < kN * Gm::NB * 8; i += step) {
              const int rr = i / (Gm::NB * 8), k = i % (Gm::NB * 8);
              if (((mask >> (rr >> 4)) & 1) && base + rr < L) continue;
              *reinterpret_cast<uint4*>(v_op + (k >> 3) * kN * 128 + rr * 128 + ((k & 7) << 4)) =
                  make_uint4(0, 0, 0, 0);
            }
            tc::fence_smem_to_async();
          }
        }
        // columns that the row sees, in blocks that hold data
        uint64_t cols = 0;
        {
          const int a = min(max(my_lo - base, 0), kN), z = min(max(my_hi - base, 0), kN);
          if (row_ok && a < z) cols = (z - a == 64 ? ~0ull : ((1ull << (z - a)) - 1)) << a;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (!((mask >> j) & 1)) cols &= ~(0xFFFFull << (16 * j));
        }
        // a row that sees nothing of a plain tile goes by its mask: 0 x a key's NaN
        // or infinity is what brought it here
        const bool whole = __all_sync(kFull, plain && !none);
        float mb[4];
        const float mx = whole ? largest<false, Gm::kFp8>(t_s, cj, 0, mb) : largest<true, Gm::kFp8>(t_s, cj, cols, mb);
        float fo = 1.f;  // rescale of l and O for a larger row max
        if (mx > m + kLazy && !none) {
          fo = ex2(m - mx);  // 0 when m was -inf
          m = mx;
        }
        l *= fo;
        if constexpr (Gm::kFp8) {
          const float4 v4 = *reinterpret_cast<const float4*>(tile_sv + (t % Gm::kScaleSlots) * 4);
          const float v[4] = {v4.x, v4.y, v4.z, v4.w};
          float need = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            vr[j] = ((cols >> (16 * j)) & 0xFFFF) ? v[j] : 0.f;  // blocks that the row sees
            need = fmaxf(need, ex2(mb[j] - (m == -INFINITY ? 0.f : m)) * vr[j]);
          }
          fo = move_unit(unit, fo, need, m != -INFINITY);
#pragma unroll
          for (int j = 0; j < 4; ++j) vr[j] = fminf(vr[j] * unit, FLT_MAX);  // finite where every p is 0
        }
        __syncwarp();
        if (whole)
          sum = exponents<false, Gm::kFp8, kBfMma>(t_s, -m, cj, vr, 0, pk);
        else
          sum = exponents<true, Gm::kFp8, kBfMma>(t_s, m == -INFINITY ? 0.f : -m, cj, vr, cols, pk);
        // O is rescaled once PV(u - 1) is done, before PV(u) is issued (which waits for P(u))
        if (u > 0 && __any_sync(kFull, fo != 1.f)) {
          ok = mbar_wait_bounded(&my_pv[(u - 1) & 1], (uint32_t)((u - 1) >> 1) & 1u, p.timeout_ns) && ok;
          __syncwarp();
          tc::fence_after_sync();
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t o[32];
            tc::tmem_ld32(t_row + c0, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fo);
            tc::tmem_st32(t_row + c0, o);
          }
        }
        if constexpr (H == 2) {
          row_max[wg * kM + r] = m;
          ++moves;
          if (lane == 0) row_moves[wg * 4 + quad] = moves;
        }
      }
      l += sum;
      // P over this row's columns of S, then the warp's share is handed over
      __syncwarp();
      tc::tmem_st32(t_s, pk);
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&my_p[u & 1]);
        if constexpr (H == 2) mbar_arrive(my_turn);
      }
    }

    if (!aborted && U > 0) {
      // PV(U - 2) first: a group whose last tile that is knows of PV(U - 4) only,
      // and the parity that it then waits for is that of PV(U - 3) done
      if (U > 1) ok = mbar_wait_bounded(&my_pv[U & 1], (uint32_t)((U - 2) >> 1) & 1u, p.timeout_ns) && ok;
      ok = mbar_wait_bounded(&my_pv[(U - 1) & 1], (uint32_t)((U - 1) >> 1) & 1u, p.timeout_ns) && ok;
      aborted = !__all_sync(kFull, ok);
    }
    if (aborted && lane == 0) {
      *abort_flag = 1;
      raise_flag(p.err, PQKV_DEVERR_TIMEOUT);
    }
    // every tile of the half is handed over: the max is final
    if constexpr (H == 2) {
      if (!aborted && U > 0 && row_moves[wg * 4 + quad] != moves) follow();
      row_sum[(group * 2 + wg) * kM + r] = l;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (*abort_flag) {  // copies in flight land before the CTA goes on
    if (tid == 0) {
      bool drained = true;
      for (int kv = 0; kv < Gm::kProducers; ++kv)
        for (int t = max(0, n_issued[kv] - ns); t < n_issued[kv]; ++t)
          drained = mbar_wait_bounded(kv ? &bar_vfull[stage_of(t)] : &bar_full[stage_of(t)], lap_of(t), p.drain_ns) &&
                    drained;
      if (!drained) raise_flag(p.err, PQKV_DEVERR_DRAIN);
    }
    __syncthreads();
  }
  tc::fence_after_sync();
  // the groups of a row share out its channels
  const uint32_t t_row = tmem + 256u * wg + ((uint32_t)(32 * quad) << 16);
  const bool holds_row = is_compute && quad < warps_of(wg) && (dup || !one_tile || wg == 0);
  if (H == 2 && holds_row) l = row_sum[wg * kM + r] + row_sum[(2 + wg) * kM + r];
  // Partial results in shared memory (the stages and operands are done with):
  // chunk c (16 bytes) of row `slot` lies at c ^ slot, so that 32 rows' equal
  // chunks fall in different banks.
  constexpr int kChunks = D / 4;  // 16-byte pieces of a row of O
  float2* s_stat = reinterpret_cast<float2*>(smem + 2 * kM * D * 4);
  auto chunk_at = [&](int slot, int c) { return (uint32_t)(slot * kChunks + (c ^ (slot & (kChunks - 1)))) * 16; };
  auto leave_part = [&]() {  // this thread's channels of its row, and m and l
    const int slot = wg * kM + r;
    if (group == 0) s_stat[slot] = make_float2(*abort_flag ? NAN : m, l);  // no max is NaN: a part that a wait cut short
    __syncwarp();
    if (tiles_of(wg) > 0) {
      const float vs = Gm::kFp8 ? (unit > 0.f ? 1.f / unit : 0.f) : 1.f;
#pragma unroll 1
      for (int c0 = group * (D / H); c0 < (group + 1) * (D / H); c0 += 32) {
        uint32_t o[32];
        tc::tmem_ld32(t_row + c0, o);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<float4*>(smem + chunk_at(slot, c0 / 4 + k)) =
              make_float4(__uint_as_float(o[4 * k]) * vs, __uint_as_float(o[4 * k + 1]) * vs,
                          __uint_as_float(o[4 * k + 2]) * vs, __uint_as_float(o[4 * k + 3]) * vs);
      }
    }
    tc::fence_before_sync();
  };
  if (p.splits == 1) {
    // the second half of a CTA that shares a row tile (dup) leaves its part to the first
    if (dup && wg == 1 && holds_row) leave_part();
    if (dup) __syncthreads();
    if (holds_row && (!dup || wg == 0) && !*abort_flag) {
      float2 st = make_float2(-INFINITY, 0.f);
      if (dup) st = s_stat[kM + r];
      const float mx = fmaxf(m, st.x);
      const float f = m == -INFINITY ? 0.f : ex2(m - mx), f2 = st.x == -INFINITY ? 0.f : ex2(st.x - mx);
      const float sum = f * l + f2 * st.y, inv = sum == 0.f ? 0.f : 1.f / sum;  // a sum of NaN stays one
      const float a = f * inv * (Gm::kFp8 ? (unit > 0.f ? 1.f / unit : 0.f) : 1.f), a2 = f2 * inv;
      uint16_t* dst = static_cast<uint16_t*>(p.out) + orow;
#pragma unroll 1
      for (int c0 = group * (D / H); c0 < (group + 1) * (D / H); c0 += 32) {
        uint32_t o[32];
        __syncwarp();
        tc::tmem_ld32(t_row + c0, o);
        if (!row_ok) continue;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(o[8 * k + i]) * a;
          if (a2 > 0.f) {  // a half without tiles leaves no O
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float4 w = *reinterpret_cast<const float4*>(smem + chunk_at(kM + r, c0 / 4 + 2 * k + i));
              v[4 * i] = fmaf(w.x, a2, v[4 * i]);
              v[4 * i + 1] = fmaf(w.y, a2, v[4 * i + 1]);
              v[4 * i + 2] = fmaf(w.z, a2, v[4 * i + 2]);
              v[4 * i + 3] = fmaf(w.w, a2, v[4 * i + 3]);
            }
          }
          *reinterpret_cast<uint4*>(dst + c0 + 8 * k) =
              make_uint4(pack_f32x2(v[0], v[1], QBF16), pack_f32x2(v[2], v[3], QBF16), pack_f32x2(v[4], v[5], QBF16),
                         pack_f32x2(v[6], v[7], QBF16));
        }
      }
      tc::fence_before_sync();
    }
    __syncthreads();  // tensor memory is read
  } else {
    // Parts of the same rows: the CTAs of the cluster, and the halves of each
    // (dup). Each leaves its O, m and l in shared memory, then the CTAs share out
    // the rows, a group of lanes joining a row from all parts.
    if (holds_row) leave_part();
    cluster_sync();
    const uint32_t part_at = smem_u32(smem), stat_at = smem_u32(s_stat);
    constexpr int kRowsPerWarp = 32 / kChunks;  // 32 (D = 128) or 16 lanes a row
    constexpr int kWarps = Gm::kThreads / 32;
    const int c = lane % kChunks;
    // a group of kChunks lanes per row: lane k holds the statistics of part k =
    // s par + e (half e of CTA s), then every lane adds up its chunk of all parts
    const int parts = p.splits << pshift;  // at most 16
    for (int i0 = (rank * kWarps + warp) * kRowsPerWarp; i0 < n_rows; i0 += p.splits * kWarps * kRowsPerWarp) {
      const int i = min(i0 + lane / kChunks, n_rows - 1);
      float2 st = make_float2(-INFINITY, 0.f);
      if (c < parts) st = ld_peer2(stat_at + (uint32_t)(i + (c & (par - 1)) * kM) * 8, c >> pshift);
      // rows of which a part was cut short are left as they are
      const unsigned cut = __ballot_sync(kFull, isnan(st.x)) & (kChunks == 32 ? kFull : 0xFFFFu << (lane & 16));
      float mx = st.x;
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o, 16));
      // a part without tiles leaves no O and counts nothing (its sum is 0); a
      // part's sum of NaN makes the row NaN, whatever its max
      float w = st.x == -INFINITY ? 0.f : ex2(st.x - mx);
      float sum = w * st.y;
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o, 16);
      sum = __shfl_sync(kFull, sum, 0, kChunks);
      w = sum == 0.f ? 0.f : w / sum;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int k = 0; k < parts; ++k) {
        const int at = i + (k & (par - 1)) * kM;
        const float4 o = ld_peer4(part_at + chunk_at(at, c), k >> pshift);
        const float f = __shfl_sync(kFull, w, k, kChunks);
        if (f != 0.f)
          acc = make_float4(fmaf(f, o.x, acc.x), fmaf(f, o.y, acc.y), fmaf(f, o.z, acc.z), fmaf(f, o.w, acc.w));
      }
      if (i0 + lane / kChunks >= n_rows || cut) continue;
      uint16_t* dst = static_cast<uint16_t*>(p.out) +
                      ((size_t)(q0 + mt0 * TOK + i / G) * p.Hq + (size_t)h * G + i % G) * D + 4 * c;
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack_f32x2(acc.x, acc.y, QBF16), pack_f32x2(acc.z, acc.w, QBF16));
    }
    cluster_sync();  // no CTA leaves while another reads its parts
  }
  if (warp == 0) {
    __syncwarp();
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// CTAs per row-tile pair: doubled while the doubled grid still fits the GPU at
// one CTA per SM and every CTA keeps two tiles, one for each of its halves
// (4 sequences of 3-40 tokens over 1-577 states: 12.2 us; 12.7 without splits,
// 14.5 and 17.5 when a CTA keeps four and eight tiles).
int cross_splits(long long ctas, int maxblk, int sms) {
  const int tiles = (maxblk * kBlock + kN - 1) / kN;
  int s = 1;
  while (2 * s <= kMaxSplits && ctas * 2 * s <= sms && 2 * s * 2 <= tiles) s *= 2;
  return s;
}

template <int KVF, int D, bool QBF16>
cudaError_t launch_cross_t(const CUtensorMap& tmap, CrossParams p, int sms, cudaStream_t st) {
  using Gm = CrossGeom<KVF, D>;
  auto kern = paged_cross_kernel<KVF, D, QBF16>;
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Gm::kSmem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  const unsigned ctas = (unsigned)p.B * (unsigned)((p.tiles_per_seq + 1) / 2) * (unsigned)p.Hkv;
  p.splits = cross_splits(ctas, p.maxblk, sms);
  p.by_length = p.B > 1 && p.B <= Gm::kThreads && ctas > (unsigned)sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, (unsigned)p.splits);
  cfg.blockDim = dim3(Gm::kThreads);
  cfg.dynamicSmemBytes = Gm::kSmem;
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

size_t cross_smem_bytes(int kv_dtype, int D) {
#define PQKV_CS(F) \
  if (kv_dtype == F) return D == 128 ? CrossGeom<F, 128>::kSmem : CrossGeom<F, 64>::kSmem;
  PQKV_CS(PQKV_DTYPE_FP16)
  PQKV_CS(PQKV_DTYPE_BF16)
  PQKV_CS(PQKV_DTYPE_FP8_E4M3)
  PQKV_CS(PQKV_DTYPE_FP8_E5M2)
  PQKV_CS(PQKV_DTYPE_FP4_E2M1)
#undef PQKV_CS
  return 0;
}

cudaError_t launch_cross(int kv_dtype, int D, bool q_bf16, const CUtensorMap& tmap16, const CrossParams& p, int sms,
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
