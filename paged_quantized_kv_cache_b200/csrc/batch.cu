// batch.cu -- block tables, slot mapping, positions and offsets of a batch,
// from request lengths that are on the GPU.
//
// "vLLM" glossary, "PagedAttention" (logical to physical blocks) and
// "Continuous batching" (every iteration has another batch): request b holds
// s_b tokens and adds n_b. It needs ceil((s_b + n_b) / 16) - ceil(s_b / 16) new
// blocks, the next ones of the step's flat id list; token s_b + i takes row
// N_b + i of the batch (N, M: exclusive sums of new tokens and new blocks) and
// slot 16 table_b[p / 16] + p % 16.
//
// One launch, no workspace: every CTA sums the lengths of all requests into
// shared memory for itself (at most 4096 pairs, from L2), then the CTAs share
// out the rows and the new blocks, a thread finding the request of its first row
// by bisection.
// A row reads its block id from the id list, or from the one table entry that
// holds the request's open block (which no thread writes), so no CTA waits for
// another's table entries. Latency bounds it: 2.3 us on the device for 16
// requests of one token, 5.3 us for 512 prompts (2.8 MB of results), 17 us for
// 4096 requests, most of it the sums.
#include "batch.cuh"

namespace pqkv {

namespace {

constexpr int kThreads = 256;
constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ int blocks_of(int tokens) { return (tokens + kBlock - 1) / kBlock; }

// Lengths of request i: its start and new tokens, zero new ones (and false) if
// they are negative or do not fit a table row.
__device__ __forceinline__ bool lengths(const BatchParams& p, int i, int& s, int& n) {
  s = p.start[i];
  n = p.num_new[i];
  const bool ok = s >= 0 && n >= 0 && (long long)s + n <= (long long)kBlock * p.maxblk;
  if (!ok) s = n = 0;
  return ok;
}

// Largest b in [0, B) with cum[b] <= i, for cum[0] = 0 <= i < cum[B]: the
// request that row (or new block) i belongs to.
__device__ __forceinline__ int owner(const int* cum, int B, int i) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// ROWS: consecutive rows of the batch that a thread takes, from one bisection on.
template <int ROWS>
__global__ void __launch_bounds__(kThreads) build_batch_kernel(const BatchParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ int smem[];
  int* tok = smem;            // [B + 1] first row of each request
  int* blk = smem + p.B + 1;  // [B + 1] first new block of each request
  __shared__ long long warp_tok[kThreads / 32], warp_blk[kThreads / 32];
  __shared__ int total_tok, total_blk;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int lo = min(p.B, tid * per), hi = min(p.B, lo + per);

  // sums in 64 bits: 4096 requests of up to 2^31 tokens
  long long t = 0, m = 0;
#pragma unroll 4
  for (int i = lo; i < hi; ++i) {
    int s, n;
    lengths(p, i, s, n);
    t += n;
    m += blocks_of(s + n) - blocks_of(s);
  }
  long long ti = t, mi = m;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(kFull, ti, o), b = __shfl_up_sync(kFull, mi, o);
    if (lane >= o) {
      ti += a;
      mi += b;
    }
  }
  if (lane == 31) {
    warp_tok[warp] = ti;
    warp_blk[warp] = mi;
  }
  if (tid == 0) {
    total_tok = total_blk = 0;
    tok[0] = blk[0] = 0;
  }
  __syncthreads();
  t = ti - t;
  m = mi - m;
  for (int w = 0; w < warp; ++w) {
    t += warp_tok[w];
    m += warp_blk[w];
  }
  // Requests fit from the first one up to the one whose rows or blocks pass
  // what there is; it and all behind it are left out whole (both sums only
  // grow, so whether a request fits needs no other thread's answer).
  int bits = 0, my_tok = 0, my_blk = 0;
#pragma unroll 4
  for (int i = lo; i < hi; ++i) {
    int s, n;
    if (!lengths(p, i, s, n)) bits |= PQKV_DEVERR_SEQ_LEN;
    t += n;
    m += blocks_of(s + n) - blocks_of(s);
    const bool fits = t <= p.cap && m <= p.n_ids;
    if (!fits) bits |= PQKV_DEVERR_CAPACITY;
    tok[i + 1] = fits ? (int)t : -1;
    blk[i + 1] = fits ? (int)m : -1;
    if (fits) {
      my_tok = (int)t;
      my_blk = (int)m;
    }
    if (blockIdx.x == 0) p.lens[i] = fits ? s + n : 0;
  }
  if (bits && blockIdx.x == 0) raise_flag(p.err, bits);
  my_tok = __reduce_max_sync(kFull, my_tok);
  my_blk = __reduce_max_sync(kFull, my_blk);
  if (lane == 0) {
    atomicMax(&total_tok, my_tok);
    atomicMax(&total_blk, my_blk);
  }
  __syncthreads();
  const int T = total_tok, M = total_blk;
  for (int i = lo; i < hi; ++i) {
    if (tok[i + 1] < 0) {
      tok[i + 1] = T;
      blk[i + 1] = M;
    }
    if (blockIdx.x == 0) p.cu[i + 1] = tok[i + 1];
  }
  if (blockIdx.x == 0 && tid == 0) p.cu[0] = 0;
  __syncthreads();

  const int step = gridDim.x * kThreads;
  for (long long i = (long long)blockIdx.x * kThreads + tid; i < M; i += step) {
    const int b = owner(blk, p.B, (int)i);
    const int id = p.ids[i];
    const bool ok = id >= 0 && id < p.nb;
    if (!ok) raise_flag(p.err, PQKV_DEVERR_BLOCK_ID);
    p.tables[(size_t)b * p.maxblk + blocks_of(p.start[b]) + ((int)i - blk[b])] = ok ? id : -1;
  }
  const bool wide = ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions)) & 15u) == 0;
  for (long long i0 = ((long long)blockIdx.x * kThreads + tid) * ROWS; i0 < p.cap;
       i0 += (long long)step * ROWS) {
    int slot[ROWS], pos[ROWS];
    int b = i0 < T ? owner(tok, p.B, (int)i0) : 0;
#pragma unroll
    for (int e = 0; e < ROWS; ++e) {
      slot[e] = -1;
      pos[e] = 0;
      const int i = (int)min(i0 + e, (long long)T);
      if (i >= T) continue;
      if (e > 0)
        while (i >= tok[b + 1]) ++b;  // tok[B] = T
      const int s = p.start[b];
      pos[e] = s + (i - tok[b]);
      const int j = pos[e] / kBlock, have = blocks_of(s);
      const int id = j < have ? p.tables[(size_t)b * p.maxblk + j] : p.ids[blk[b] + j - have];
      if (id >= 0 && id < p.nb)
        slot[e] = id * kBlock + pos[e] % kBlock;
      else
        raise_flag(p.err, PQKV_DEVERR_BLOCK_ID);
    }
    if (ROWS == 4 && wide && i0 + ROWS <= p.cap) {
      *reinterpret_cast<int4*>(p.slots + i0) = make_int4(slot[0], slot[1 % ROWS], slot[2 % ROWS], slot[3 % ROWS]);
      *reinterpret_cast<int4*>(p.positions + i0) = make_int4(pos[0], pos[1 % ROWS], pos[2 % ROWS], pos[3 % ROWS]);
    } else {
#pragma unroll
      for (int e = 0; e < ROWS; ++e)
        if (i0 + e < p.cap) {
          p.slots[i0 + e] = slot[e];
          p.positions[i0 + e] = pos[e];
        }
    }
  }
}

template <int ROWS>
cudaError_t launch_rows(const BatchParams& p, int sms, cudaStream_t st) {
  const long long rows = ((long long)p.cap + ROWS - 1) / ROWS;
  const long long items = rows > p.n_ids ? rows : p.n_ids;
  const long long need = (items + kThreads - 1) / kThreads;
  const int grid = (int)(need < 1 ? 1 : need < 4LL * sms ? need : 4LL * sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 2 * (size_t)(p.B + 1) * sizeof(int);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, build_batch_kernel<ROWS>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// Four rows a thread where one each would make a second round of the CTAs that
// fit, or the CTAs' sums of many lengths (a CTA sums all B) would take as long;
// us with one and four: 16 rows 2.9 / 3.9, 96 requests of 25 thousand rows 3.8 /
// 4.5, 200 of 102 thousand 4.2 / 4.8, 400 of 205 thousand 7.3 / 5.3, 512 of 328
// thousand 8.6 / 5.6; 4096 requests of 4 thousand rows 17.5 / 19.1, of 82
// thousand 30.8 / 18.2, of 133 thousand 52.7 / 18.2.
cudaError_t launch_build_batch(const BatchParams& p, int sms, cudaStream_t st) {
  return p.cap * (1 + p.B / 512.0) > 4.0 * sms * kThreads ? launch_rows<4>(p, sms, st) : launch_rows<1>(p, sms, st);
}

}  // namespace pqkv
