// Forking, freeing, reserving and compacting the pages of a cache.
//
// The state is a page table [B][columns], lengths [B] and, per page, how many
// entries of the table name it: refs[p] = sum over (b, j) of [table[b][j] == p],
// 0 where p is free.  There is no list of free pages: changes of the counts are
// integer additions, which commute, and new pages are the lowest free ids, so
// nothing depends on the order in which threads get to run.
#include <algorithm>

#include "pages.cuh"

namespace wedlm {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ bool is_page(int e, int N) { return e >= 0 && e < N; }

// ---------------------------------------------------------------------------
// the old state to the new arrays
// ---------------------------------------------------------------------------
__device__ __forceinline__ void copy_ints(const int32_t* __restrict__ from,
                                          int32_t* __restrict__ to, long long n, long long at,
                                          long long step) {
  if (!((reinterpret_cast<uintptr_t>(from) | reinterpret_cast<uintptr_t>(to)) & 15)) {
    for (long long i = at; i < n / 4; i += step)
      reinterpret_cast<int4*>(to)[i] = reinterpret_cast<const int4*>(from)[i];
    for (long long i = n / 4 * 4 + at; i < n; i += step) to[i] = from[i];
  } else {
    for (long long i = at; i < n; i += step) to[i] = from[i];
  }
}

__global__ void __launch_bounds__(kThreads) page_state_copy_kernel(PageArrays S, bool table) {
  pdl_wait();
  pdl_trigger();  // what follows waits before it reads
  const long long at = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long step = (long long)gridDim.x * kThreads;
  if (S.refs != S.new_refs) copy_ints(S.refs, S.new_refs, S.N, at, step);
  if (table && S.table != S.new_table)
    copy_ints(S.table, S.new_table, (long long)S.B * S.cols, at, step);
}

// Small states are copied by the kernel that changes them, run as one cluster: a launch
// less is 2 to 3 us less of host time, which is what a small call is bound by (one row of 8
// over 273 columns 8.2 us a call from Python, captured 4.4; with a copy ahead 11.3 and 3.8)
constexpr int kFewInts = 1 << 16, kFewBlocks = 8, kFewThreads = 1024;

// Counts to their new place; no thread of the cluster changes one before it has
// passed cluster_wait.
__device__ __forceinline__ void copy_refs(const PageArrays& S) {
  copy_ints(S.refs, S.new_refs, S.N, (long long)blockIdx.x * blockDim.x + threadIdx.x,
            (long long)gridDim.x * blockDim.x);
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
struct ForkArgs {
  PageArrays S;
  bool copy;     // the counts, in a cluster
  int n, width;  // width: columns of a strip
  const int32_t *src, *dst, *lens;
};

// Entries are copied and, where they change, counted: 4 bytes read, 4 written and at most two
// atomic additions an entry, none where the row it names had the same page (a beam's shared
// prefix).  Bound by latency: pairs, entries, counts in a chain.  256 rows over 2053
// columns, 8 to a beam: 5.2 us captured, 0.7 of them the bytes.
//
// In place a block has a strip of columns of all pairs: it reads the strip's source
// entries into shared memory before it writes any.  The same 256 rows take 38 us this way (65 strips,
// 32 entries a thread twice, each behind the loads of its pair), one row of 8 over 273
// columns 2.8.  Into a new table 256 threads have
// a strip of kForkRows rows and write straight through.  The first block sees to
// the lengths.
constexpr int kForkRows = 32, kStrip = 32;  // a whole line of a row

__global__ void __launch_bounds__(kFewThreads) fork_kernel(const __grid_constant__ ForkArgs A) {
  extern __shared__ int sm[];
  const PageArrays& S = A.S;
  int* pair_of = sm;        // [B] the pair whose dst this row is, n: none
  int* stage = sm + S.B;    // [n][width] or the new lengths [B]
  const bool first = blockIdx.x == 0;
  const bool in_place = S.table == S.new_table;
  for (int b = threadIdx.x; b < S.B; b += blockDim.x) pair_of[b] = A.n;
  pdl_wait();
  if (A.copy) copy_refs(S);  // under way while the pairs are read
  __syncthreads();
  for (int i = threadIdx.x; i < A.n; i += blockDim.x) {
    const int s = A.src[i], d = A.dst[i];
    if (s >= -1 && s < S.B && d >= 0 && d < S.B) atomicMin(&pair_of[d], i);
    else if (first) set_err(S.err, WEDLM_DEV_BAD_ROW);
  }
  __syncthreads();
  // the entry that pair i puts into column c
  auto taken = [&](int i, int c) {
    const int s = A.src[i];
    if (s < 0) return -1;
    if (A.lens) {
      const int len = max(A.lens[i], 0);
      if (c >= len / kPageBlock + (len % kPageBlock != 0)) return -1;
    }
    const int e = S.table[(size_t)s * S.cols + c];
    if (e >= S.N) set_err(S.err, WEDLM_DEV_BAD_PAGE);
    return is_page(e, S.N) ? e : -1;
  };
  // pages named before and after keep their count
  auto recount = [&](int was, int now) {
    if (was == now) return;
    if (is_page(was, S.N)) atomicAdd(&S.new_refs[was], -1);
    if (now >= 0) atomicAdd(&S.new_refs[now], 1);
  };
  if (A.copy) cluster_wait();
  if (in_place) {
    const int c0 = blockIdx.x * A.width, cw = min(A.width, S.cols - c0);
    for (int k = threadIdx.x; k < A.n * A.width; k += blockDim.x) {
      const int i = k / A.width, c = k % A.width, d = A.dst[i];
      // a pair that is left out is no row's
      if (c < cw && d >= 0 && d < S.B && pair_of[d] == i) stage[k] = taken(i, c0 + c);
    }
    __syncthreads();
    for (int k = threadIdx.x; k < A.n * A.width; k += blockDim.x) {
      const int i = k / A.width, c = k % A.width, d = A.dst[i];
      if (c >= cw || d < 0 || d >= S.B || pair_of[d] != i) continue;
      int32_t* at = S.new_table + (size_t)d * S.cols + c0 + c;
      const int was = *at;
      recount(was, stage[k]);
      *at = stage[k];
    }
  } else {
    const int strips = (S.cols + kStrip - 1) / kStrip;
    const int items = strips * ((S.B + kForkRows - 1) / kForkRows), teams = blockDim.x / kThreads;
    const int team = threadIdx.x / kThreads, t = threadIdx.x % kThreads;
    for (int it = blockIdx.x * teams + team; it < items; it += gridDim.x * teams) {
      const int c = it % strips * kStrip + t % kStrip, r0 = it / strips * kForkRows;
      const int r1 = min(S.B, r0 + kForkRows);
      if (c >= S.cols) continue;
#pragma unroll 4
      for (int b = r0 + t / kStrip; b < r1; b += kThreads / kStrip) {
        const size_t at = (size_t)b * S.cols + c;
        const int was = S.table[at], i = pair_of[b];
        int now = was;
        if (i < A.n) {
          now = taken(i, c);
          recount(was, now);
        }
        S.new_table[at] = now;
      }
    }
  }
  if (!first) return;
  __syncthreads();
  for (int i = threadIdx.x; i < A.n; i += blockDim.x) {
    const int s = A.src[i], d = A.dst[i];
    if (s >= -1 && s < S.B && d >= 0 && d < S.B && pair_of[d] != i) set_err(S.err, WEDLM_DEV_BAD_ROW);
  }
  // every length is read before one is written
  for (int b = threadIdx.x; b < S.B; b += blockDim.x) {
    const int i = pair_of[b];
    int len = 0;
    if (i < A.n) {
      const int s = A.src[i];
      if (s >= 0) {
        len = S.seq_len[s];
        if (A.lens) {
          const int want = A.lens[i];
          if (want < 0 || want > len) set_err(S.err, WEDLM_DEV_BAD_SEQLEN);
          len = min(max(want, 0), len);
        }
      }
    } else {
      len = S.seq_len[b];
    }
    stage[b] = len;
  }
  __syncthreads();
  for (int b = threadIdx.x; b < S.B; b += blockDim.x) S.new_len[b] = stage[b];
}

// ---------------------------------------------------------------------------
// free
// ---------------------------------------------------------------------------
// As fork: bound by latency and, where many rows give up one page, by the additions to its
// count.  256 rows over 2053 columns, half of them dropped, 8 to a page: 5.8 us.
struct FreeArgs {
  PageArrays S;
  bool copy;  // the counts, in a cluster
  const int32_t* keep;
};

constexpr int kFreeCols = 4 * kThreads;  // columns of 256 threads

__global__ void __launch_bounds__(kFewThreads) free_kernel(const __grid_constant__ FreeArgs A) {
  const PageArrays& S = A.S;
  pdl_wait();
  if (A.copy) copy_refs(S);
  bool wait = A.copy;
  const bool in_place = S.table == S.new_table;
  const int pieces = (S.cols + kFreeCols - 1) / kFreeCols, teams = blockDim.x / kThreads;
  const int team = threadIdx.x / kThreads, t = threadIdx.x % kThreads;
  const long long items = (long long)S.B * pieces;
  for (long long it = (long long)blockIdx.x * teams + team; it < items; it += gridDim.x * teams) {
    const int b = (int)(it / pieces), c0 = (int)(it % pieces) * kFreeCols + t;
    const size_t row = (size_t)b * S.cols;
    const int keep = A.keep[b];
    int e[4];  // in flight together
#pragma unroll
    for (int k = 0; k < 4; ++k) e[k] = c0 + k * kThreads < S.cols ? S.table[row + c0 + k * kThreads] : -1;
    if (c0 == 0) {
      const int len = S.seq_len[b];
      if (keep < 0) set_err(S.err, WEDLM_DEV_BAD_SEQLEN);
      S.new_len[b] = keep < 0 ? len : min(len, keep);
    }
    const int cut = keep < 0 ? INT32_MAX : keep / kPageBlock + (keep % kPageBlock != 0);
    if (wait) cluster_wait();
    wait = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c0 + k * kThreads;
      if (c >= S.cols || (in_place && c < cut)) continue;
      if (c >= cut && e[k] >= 0 && (e[k] >= S.N || atomicAdd(&S.new_refs[e[k]], -1) < 1))
        set_err(S.err, WEDLM_DEV_BAD_PAGE);
      S.new_table[row + c] = c >= cut ? -1 : e[k];
    }
  }
  if (wait) cluster_wait();
}

// ---------------------------------------------------------------------------
// copies of pages
// ---------------------------------------------------------------------------
// Bound by DRAM: 240 pages of 64 KB in 36 layers (1.1 GB read and written) take 175 us,
// 6.5 TB/s, 0.95 of a plain copy's rate.  A block's item is 16 KB, four 16-byte loads of
// each thread ahead of the stores; eight blocks an SM.
constexpr int kCopyVec = 4;                            // 16-byte loads of a thread in flight
constexpr int kCopyChunk = kThreads * kCopyVec * 16;   // bytes of a block's item

// this block's share of `count` pages in all layers, in items of kCopyChunk bytes
__device__ void copy_pages(const PagePools& P, const int2* pairs, int count) {
  const int chunks = (int)((P.page_bytes + kCopyChunk - 1) / kCopyChunk);
  const long long items = (long long)count * P.n_layers * chunks;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int k = (int)(it % chunks);
    const long long rest = it / chunks;
    const int2 pr = pairs[rest / P.n_layers];
    char* pool = static_cast<char*>(P.p[rest % P.n_layers]);
    const int64_t base = (int64_t)k * kCopyChunk + threadIdx.x * 16;
    const char* from = pool + pr.x * P.page_bytes + base;
    char* to = pool + pr.y * P.page_bytes + base;
    uint4 v[kCopyVec];
#pragma unroll
    for (int j = 0; j < kCopyVec; ++j)
      if (base + j * kThreads * 16 < P.page_bytes)
        v[j] = *reinterpret_cast<const uint4*>(from + j * kThreads * 16);
#pragma unroll
    for (int j = 0; j < kCopyVec; ++j)
      if (base + j * kThreads * 16 < P.page_bytes)
        *reinterpret_cast<uint4*>(to + j * kThreads * 16) = v[j];
  }
}

__global__ void __launch_bounds__(kThreads)
copy_pages_kernel(const __grid_constant__ PagePools P, const int2* pairs, const int* count) {
  pdl_wait();
  copy_pages(P, pairs, *count);
}

// ---------------------------------------------------------------------------
// plans: sums and ranks over the counts.  One block, or a cluster where there are many
// pages to look at: what an SM takes from L2 (about 90 GB/s) is what bounds it then, the
// chain of loads (lengths, entries, counts, free pages) otherwise.  Captured calls that copy
// next to nothing: reserve for 64 rows among 8000 pages 7.4 us, 106000 10.2, 1000000 16;
// compact 5.8, 10.8 and 47.5.  At 16384 pages a block and a cluster are even.
// ---------------------------------------------------------------------------
constexpr int kPlan = 1024, kPlanWarps = kPlan / 32;
constexpr int kFewPages = 2048;     // that a plan lists in shared memory
constexpr int kScan = 8;            // counts of a thread in flight
constexpr int kManyPages = 1 << 14, kPlanBlocks = 8;
// Sums stop at kSumCap.  Needs of 1024 rows of up to 2^26 columns add up to 2^36, but what
// is beyond the number of pages is all the same; min(a + b, cap) is associative, so that a
// sum below the cap is exact and one beyond it is the cap, in any order.
constexpr int kSumCap = kMaxPages + 1;

// inclusive sum over the warp, values 0..kSumCap
__device__ __forceinline__ int warp_incl(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = min(v + u, kSumCap);
  }
  return v;
}

// the same over the block's threads; `sums` [kPlanWarps + 1], the total in the last
__device__ int block_incl(int v, int* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_incl(v);
  __syncthreads();
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    const int s = warp_incl(sums[lane]);
    __syncwarp();
    sums[lane] = s;
    if (lane == 31) sums[kPlanWarps] = s;
  }
  __syncthreads();
  return min(v + (warp ? sums[warp - 1] : 0), kSumCap);
}

// all threads of the cluster; what they wrote is seen by all of it
__device__ __forceinline__ void plan_sync() {
  if (gridDim.x == 1) {
    __syncthreads();
  } else {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  }
}
// a shared int of another block of the cluster
__device__ __forceinline__ int of_block(const int* p, int rank) {
  if (gridDim.x == 1) return *p;
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p);
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(a) : "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// the pages of a warp: a run of neighbours
__device__ __forceinline__ void segment(int n, int& p0, int& p1) {
  const int warps = gridDim.x * kPlanWarps, warp = blockIdx.x * kPlanWarps + (threadIdx.x >> 5);
  const int seg = ((n + warps - 1) / warps + 31) / 32 * 32;
  p0 = (int)min((long long)n, (long long)warp * seg);
  p1 = (int)min((long long)n, (long long)p0 + seg);
}

// f(p, refs[p]) for pages p0..p1-1 in steps of a warp, in order; the same p0, p1 and
// `more` in all its lanes; p >= p1 has no page
template <typename M, typename F>
__device__ __forceinline__ void scan_refs(const int32_t* refs, int p0, int p1, M more, F f) {
  const int lane = threadIdx.x & 31;
  for (int q = p0; q < p1 && more(); q += 32 * kScan) {
    int r[kScan];
#pragma unroll
    for (int k = 0; k < kScan; ++k) r[k] = q + 32 * k + lane < p1 ? refs[q + 32 * k + lane] : 0;
#pragma unroll
    for (int k = 0; k < kScan; ++k) f(q + 32 * k + lane, r[k]);
  }
}

// put(rank, p) for the pages p of p0..p1-1 that `hit` holds for, ranks ascending from `rank`
template <typename F, typename G>
__device__ __forceinline__ void rank_refs(const int32_t* refs, int p0, int p1, int rank, int most,
                                          F hit, G put) {
  const int lane = threadIdx.x & 31;
  scan_refs(refs, p0, p1, [&] { return rank < most; }, [&](int p, int r) {
    const bool h = p < p1 && hit(r);
    const unsigned m = __ballot_sync(0xffffffffu, h);
    if (h) put(rank + __popc(m & ((1u << lane) - 1)), p);
    rank += __popc(m);
  });
}

// Where this warp's values start in the cluster's order, and the cluster's total.
// `sums` [kPlanWarps + 1]; `total` a shared int that the other blocks read: not written
// again before a plan_sync.
struct PlanRank {
  int at, total;
};
__device__ PlanRank plan_rank(int of_warp, int* sums, int* total) {
  const int lane = threadIdx.x & 31;
  const int upto = block_incl(lane == 0 ? of_warp : 0, sums);
  PlanRank r;
  r.at = __shfl_sync(0xffffffffu, upto, 0) - of_warp;
  if (threadIdx.x == 0) *total = sums[kPlanWarps];
  plan_sync();
  const int t = lane < (int)gridDim.x ? of_block(total, lane) : 0;
  r.at += __reduce_add_sync(0xffffffffu, lane < (int)blockIdx.x ? t : 0);
  r.total = __reduce_add_sync(0xffffffffu, t);
  return r;
}

// ---------------------------------------------------------------------------
// reserve
// ---------------------------------------------------------------------------
struct ReserveArgs {
  PageArrays S;
  bool copy;  // the state to the new arrays: here, else it has been copied
  int rows;
  const int32_t* counts;
  int32_t *granted, *n_free;
  int *list, *dropped;  // [N] free pages handed out, and what each replaces (-1: nothing)
  int2* pairs;          // [B] pages to be copied
  int* n_pairs;
};

// A thread sees to the columns of a row while they are few (all loads of all rows in
// flight together), a warp otherwise.
constexpr int kShort = 4;

// The first block sees to the rows, all of them to the counts.
__global__ void __launch_bounds__(kPlan) reserve_plan_kernel(const __grid_constant__ ReserveArgs A) {
  __shared__ int s_first[kReserveMaxBatch], s_end[kReserveMaxBatch], s_need[kReserveMaxBatch];
  __shared__ __align__(16) int s_cand[kReserveMaxBatch];
  __shared__ unsigned char s_part[kReserveMaxBatch], s_keep[kReserveMaxBatch];
  __shared__ int s_sums[kPlanWarps + 1], s_total, s_taken, s_freed, s_pairs;
  __shared__ int s_list[kFewPages], s_dropped[kFewPages];
  const PageArrays& S = A.S;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool lead = blockIdx.x == 0;
  pdl_wait();
  pdl_trigger();  // the copies wait for all of this before they read
  if (tid == 0) s_taken = s_freed = s_pairs = 0;
  // What is read below is the old state, so nothing waits for these.  In place the two
  // are one, which is why nothing is written before every row has been walked.
  if (A.copy) {
    const long long at = (long long)blockIdx.x * kPlan + tid, step = (long long)gridDim.x * kPlan;
    if (S.refs != S.new_refs) copy_ints(S.refs, S.new_refs, S.N, at, step);
    if (S.table != S.new_table) copy_ints(S.table, S.new_table, (long long)S.B * S.cols, at, step);
  }
  bool served = true, keep = false;
  int need = 0, first = 0, end = 0, e[kShort], uses[kShort];
  bool part = false, brief = false;
  if (lead) {
    // columns that the rows fall into; none where a sequence asks for nothing
    if (tid < S.B) {
      const int len = S.seq_len[tid];
      int n = A.counts ? A.counts[tid] : A.rows;
      if (len < 0 || n < 0 || n > A.rows) set_err(S.err, WEDLM_DEV_BAD_SEQLEN);
      n = max(0, min(n, A.rows));
      first = end = len < 0 ? 0 : len / kPageBlock;
      if (len < 0) {
        served = false;
      } else if (n > 0) {
        const long long to = ((long long)len + n + kPageBlock - 1) / kPageBlock;
        if (to > S.cols) {
          served = false;
          set_err(S.err, WEDLM_DEV_CAPACITY);
        } else {
          end = (int)to;
        }
      }
      part = end > first && len % kPageBlock != 0;
      brief = end - first <= kShort;
      s_first[tid] = first;
      s_end[tid] = end;
      s_part[tid] = part;
      // what its columns lack
      if (brief) {
        const int32_t* row = S.table + (size_t)tid * S.cols + first;
        int cand = -1;
        bool bad = false;
#pragma unroll
        for (int k = 0; k < kShort; ++k) e[k] = first + k < end ? row[k] : 0;
#pragma unroll
        for (int k = 0; k < kShort; ++k)
          uses[k] = first + k < end && is_page(e[k], S.N) ? S.refs[e[k]] : 0;
#pragma unroll
        for (int k = 0; k < kShort; ++k)
          if (first + k < end) {
            bad |= e[k] >= S.N || (e[k] >= 0 && uses[k] < 1);
            need += e[k] < 0 || uses[k] > 1;
          }
        if (part && uses[0] > 1) cand = e[0];
        if (bad) set_err(S.err, WEDLM_DEV_BAD_PAGE);
        s_need[tid] = bad ? -1 : need;  // -1: not served
        s_cand[tid] = bad ? -1 : cand;
      }
    }
    if (tid >= S.B && tid < (S.B + 3) / 4 * 4) s_cand[tid] = -1;
    if (__syncthreads_or(tid < S.B && !brief)) {
      for (int b = warp; b < S.B; b += kPlanWarps) {
        if (s_end[b] - s_first[b] <= kShort) continue;
        const int32_t* row = S.table + (size_t)b * S.cols;
        int n = 0, bad = 0, cand = -1;
        for (int c = s_first[b] + lane; c < s_end[b]; c += 32) {
          const int p = row[c], u = is_page(p, S.N) ? S.refs[p] : 0;
          if (p >= S.N || (p >= 0 && u < 1)) bad = 1;
          n += p < 0 || u > 1;
          if (c == s_first[b] && s_part[b] && u > 1) cand = p;
        }
        n = __reduce_add_sync(0xffffffffu, n);
        bad = __any_sync(0xffffffffu, bad);
        cand = __reduce_max_sync(0xffffffffu, cand);
        if (lane == 0) {
          if (bad) set_err(S.err, WEDLM_DEV_BAD_PAGE);
          s_need[b] = bad ? -1 : n;
          s_cand[b] = bad ? -1 : cand;
        }
      }
      __syncthreads();
    }
    // of owners that all write their page the last keeps it
    if (tid < S.B) {
      const int p = s_cand[tid];
      if (p >= 0) {
        int same = 0, last = 0;
        for (int b = 0; b < S.B; b += 4) {
          const int4 q = *reinterpret_cast<const int4*>(s_cand + b);
          same += (q.x == p) + (q.y == p) + (q.z == p) + (q.w == p);
          last = q.w == p ? b + 3 : q.z == p ? b + 2 : q.y == p ? b + 1 : q.x == p ? b : last;
        }
        keep = same == S.refs[p] && last == tid;
      }
      need = s_need[tid];
      if (need < 0) served = false;
      need = max(need, 0) - keep;
      s_keep[tid] = keep;
    }
  }
  int p0, p1, here = 0;
  segment(S.N, p0, p1);
  scan_refs(S.refs, p0, p1, [] { return true; }, [&](int p, int r) { here += p < p1 && r == 0; });
  here = __reduce_add_sync(0xffffffffu, here);
  const PlanRank rank = plan_rank(here, s_sums, &s_total);
  const int n_free = rank.total;
  if (lead) {
    const int upto = block_incl(need, s_sums);
    if (tid < S.B) {
      const bool ok = served && (upto <= n_free || (need == 0 && !keep));
      if (served && !ok) set_err(S.err, WEDLM_DEV_CAPACITY);
      if (ok && need) atomicMax(&s_taken, upto);
      if (A.granted) A.granted[tid] = ok;
      s_need[tid] = ok ? need : 0;
      s_cand[tid] = upto - need;  // the rank of its first page
    }
  }
  plan_sync();
  const int taken = of_block(&s_taken, 0);
  // a single block lists a few pages in its own memory
  const bool few = gridDim.x == 1 && taken <= kFewPages;
  int* list = few ? s_list : A.list;
  int* dropped = few ? s_dropped : A.dropped;
  rank_refs(S.refs, p0, p1, rank.at, taken, [](int r) { return r == 0; },
            [&](int r, int p) { if (r < taken) list[r] = p; });
  plan_sync();
  if (!lead) return;
  // the counts stay as they were until every row has been walked
  auto give = [&](int b, int c, int p, int r, bool partly) {  // column c held p
    const int q = list[r];
    S.new_table[(size_t)b * S.cols + c] = q;
    dropped[r] = p < 0 ? -1 : p;
    if (partly && p >= 0) A.pairs[atomicAdd(&s_pairs, 1)] = make_int2(p, q);
  };
  if (tid < S.B && brief && s_need[tid]) {
    int at = s_cand[tid];
#pragma unroll
    for (int k = 0; k < kShort; ++k)
      if (first + k < end && !(k == 0 && keep) && (e[k] < 0 || uses[k] > 1))
        give(tid, first + k, e[k], at++, k == 0 && part);
  }
  if (__syncthreads_or(tid < S.B && !brief)) {
    for (int b = warp; b < S.B; b += kPlanWarps) {
      if (s_need[b] == 0 || s_end[b] - s_first[b] <= kShort) continue;
      int at = s_cand[b];
      for (int c0 = s_first[b]; c0 < s_end[b]; c0 += 32) {
        const int c = c0 + lane;
        const int p = c < s_end[b] ? S.table[(size_t)b * S.cols + c] : 0;
        const bool partly = c == s_first[b] && s_part[b];
        const bool want = c < s_end[b] && !(partly && s_keep[b]) && (p < 0 || S.refs[p] > 1);
        const unsigned m = __ballot_sync(0xffffffffu, want);
        if (want) give(b, c, p, at + __popc(m & ((1u << lane) - 1)), partly);
        at += __popc(m);
      }
    }
  }
  __syncthreads();
  for (int r = tid; r < taken; r += kPlan) {
    S.new_refs[list[r]] = 1;
    const int p = dropped[r];
    if (p >= 0 && atomicAdd(&S.new_refs[p], -1) == 1) atomicAdd(&s_freed, 1);
  }
  __syncthreads();
  if (tid == 0) {
    *A.n_pairs = s_pairs;
    if (A.n_free) *A.n_free = n_free - taken + s_freed;
  }
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------
struct CompactArgs {
  PageArrays S;
  int max_moves;
  int32_t *map, *n_live;
  int2* pairs;  // [N/2] source and destination
  int* n_pairs;
};

__global__ void __launch_bounds__(kPlan) compact_plan_kernel(const __grid_constant__ CompactArgs A) {
  __shared__ int s_sums[kPlanWarps + 1], s_total, s_low;
  const PageArrays& S = A.S;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) s_low = 0;
  pdl_wait();
  pdl_trigger();  // the moves wait for all of this before they read
  int p0, p1, lives = 0;
  segment(S.N, p0, p1);
  scan_refs(S.refs, p0, p1, [] { return true; }, [&](int p, int r) { lives += p < p1 && r != 0; });
  lives = __reduce_add_sync(0xffffffffu, lives);
  const PlanRank live = plan_rank(lives, s_sums, &s_total);
  const int n = live.total;
  // the pages in use below n, counted by the warp that n falls to
  const int mid = max(p0, min(p1, n));
  if (p0 < n && n <= p1) {
    int low = mid == p1 ? lives : 0;
    if (mid < p1) {
      scan_refs(S.refs, p0, mid, [] { return true; }, [&](int p, int r) { low += p < mid && r != 0; });
      low = __reduce_add_sync(0xffffffffu, low);
    }
    if (lane == 0) s_low = live.at + low;
  }
  plan_sync();
  const int low = __reduce_add_sync(0xffffffffu, lane < (int)gridDim.x ? of_block(&s_low, lane) : 0);
  // as many free pages below n as pages in use from n on
  const int all = n - low, moves = min(all, A.max_moves);
  rank_refs(S.refs, p0, mid, p0 - live.at, moves, [](int r) { return r == 0; },
            [&](int r, int p) { if (r < moves) A.pairs[r].y = p; });
  rank_refs(S.refs, mid, p1, p0 >= n ? live.at - low : 0, all, [](int r) { return r != 0; },
            [&](int r, int p) { if (all - 1 - r < moves) A.pairs[all - 1 - r].x = p; });
  scan_refs(S.refs, p0, p1, [] { return true; }, [&](int p, int r) {
    if (p < p1) {
      A.map[p] = r != 0 ? p : -1;
      S.new_refs[p] = r;
    }
  });
  plan_sync();
  for (int k = blockIdx.x * kPlan + threadIdx.x; k < moves; k += gridDim.x * kPlan) {
    const int2 m = A.pairs[k];
    const int r = S.new_refs[m.x];
    A.map[m.x] = m.y;
    S.new_refs[m.y] = r;
    S.new_refs[m.x] = 0;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *A.n_pairs = moves;
    if (A.n_live) *A.n_live = n;
  }
}

__global__ void __launch_bounds__(kThreads)
compact_move_kernel(const __grid_constant__ PagePools P, PageArrays S, const int32_t* map,
                    const int2* pairs, const int* count) {
  pdl_wait();
  const long long n = (long long)S.B * S.cols;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < n;
       i += (long long)gridDim.x * kThreads) {
    const int e = S.table[i];
    int to = e;
    if (e >= 0) {
      to = e < S.N ? map[e] : -1;
      if (to < 0) set_err(S.err, WEDLM_DEV_BAD_PAGE);
    }
    S.new_table[i] = to;
  }
  copy_pages(P, pairs, *count);
}

}  // namespace

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
namespace {
bool bad4(const void* p) { return !p || (reinterpret_cast<uintptr_t>(p) & 3); }
bool odd4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3); }
bool meet(const PageSpan& a, const PageSpan& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x && y && x < y + 4 * (uintptr_t)b.n && y < x + 4 * (uintptr_t)a.n;
}
size_t align256(size_t n) { return (n + 255) / 256 * 256; }
int copy_grid(int sms, int64_t items) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(items, 8 * (int64_t)sms));
}
int64_t copy_items(const wedlm_page_pools& p, int64_t pages) {
  return pages * p.n_layers * ((p.page_bytes + kCopyChunk - 1) / kCopyChunk);
}
}  // namespace

bool page_state_ok(const wedlm_page_state& s, int max_batch, bool uses_len, bool new_len,
                   std::initializer_list<PageSpan> inputs, std::initializer_list<PageSpan> outputs) {
  if (s.batch < 1 || s.batch > max_batch || s.max_pages_per_seq < 1 ||
      s.max_pages_per_seq > kMaxColumns || s.num_pages < 1 || s.num_pages > kMaxPages ||
      bad4(s.page_table) || bad4(s.page_refs) || bad4(s.new_page_table) ||
      bad4(s.new_page_refs) || (uses_len && bad4(s.seq_len)) || (new_len && bad4(s.new_seq_len)) ||
      odd4(s.error))
    return false;
  const int64_t cells = (int64_t)s.batch * s.max_pages_per_seq;
  const PageSpan in[3] = {{s.page_table, cells},
                          {uses_len ? s.seq_len : nullptr, s.batch},
                          {s.page_refs, s.num_pages}};
  const PageSpan out[3] = {{s.new_page_table, cells},
                           {new_len ? s.new_seq_len : nullptr, s.batch},
                           {s.new_page_refs, s.num_pages}};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 3; ++j)
      if ((meet(out[i], in[j]) && !(i == j && out[i].p == in[j].p)) ||
          (i < j && meet(out[i], out[j])))
        return false;
    for (const PageSpan& x : inputs)
      if (meet(out[i], x)) return false;
    for (const PageSpan& x : outputs)
      if (meet(out[i], x) || meet(in[i], x)) return false;
  }
  for (const PageSpan& x : inputs)
    if (odd4(x.p)) return false;
  for (const PageSpan& x : outputs) {
    if (odd4(x.p)) return false;
    for (const PageSpan& y : inputs)
      if (meet(x, y)) return false;
    for (const PageSpan& y : outputs)
      if (&x != &y && meet(x, y)) return false;
  }
  return true;
}

bool page_pools_ok(const wedlm_page_pools& p, bool sizes_only) {
  if (p.n_layers < 1 || p.n_layers > kMaxLayers || p.page_bytes < 16 || p.page_bytes % 16 ||
      p.page_bytes > INT32_MAX)
    return false;
  if (sizes_only) return true;
  if (!p.kv_pools)
    return p.base && !(reinterpret_cast<uintptr_t>(p.base) & 15) && p.layer_stride >= 0 &&
           p.layer_stride % 16 == 0;
  for (int l = 0; l < p.n_layers; ++l)
    if (!p.kv_pools[l] || (reinterpret_cast<uintptr_t>(p.kv_pools[l]) & 15)) return false;
  return true;
}

bool page_pools_apart(const wedlm_page_pools& p, const wedlm_page_state& s, bool uses_len,
                      std::initializer_list<PageSpan> others) {
  const uintptr_t bytes = (uintptr_t)s.num_pages * (uintptr_t)p.page_bytes;
  auto pool = [&](int l) {
    return p.kv_pools ? reinterpret_cast<uintptr_t>(p.kv_pools[l])
                      : reinterpret_cast<uintptr_t>(p.base) + l * (uintptr_t)p.layer_stride;
  };
  uintptr_t low = pool(0), high = low;
  for (int l = 1; l < p.n_layers; ++l) {
    const uintptr_t a = pool(l);
    // one that layers share, or none of another's; below or above all others mostly
    for (int k = a < high + bytes && low < a + bytes ? 0 : l; k < l; ++k)
      if (a != pool(k) && a < pool(k) + bytes && pool(k) < a + bytes) return false;
    low = std::min(low, a);
    high = std::max(high, a);
  }
  auto apart = [&](const void* x, int64_t ints) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = a + 4 * (uintptr_t)ints;
    if (!a || b <= low || a >= high + bytes) return true;  // outside of all of them: most are
    for (int l = 0; l < p.n_layers; ++l)
      if (a < pool(l) + bytes && pool(l) < b) return false;
    return true;
  };
  const int64_t cells = (int64_t)s.batch * s.max_pages_per_seq;
  bool ok = apart(s.page_table, cells) && apart(s.new_page_table, cells) &&
            apart(s.page_refs, s.num_pages) && apart(s.new_page_refs, s.num_pages) &&
            apart(s.error, 1) && (!uses_len || apart(s.seq_len, s.batch));
  for (const PageSpan& x : others) ok = ok && apart(x.p, x.n);
  return ok;
}

PageArrays page_arrays(const wedlm_page_state& s) {
  PageArrays S;
  S.B = s.batch;
  S.cols = s.max_pages_per_seq;
  S.N = s.num_pages;
  S.table = s.page_table;
  S.seq_len = s.seq_len;
  S.refs = s.page_refs;
  S.new_table = s.new_page_table;
  S.new_len = s.new_seq_len;
  S.new_refs = s.new_page_refs;
  S.err = s.error;
  return S;
}

PagePools page_pools(const wedlm_page_pools& p) {
  PagePools P;
  P.n_layers = p.n_layers;
  P.page_bytes = p.page_bytes;
  for (int l = 0; l < p.n_layers; ++l)
    P.p[l] = p.kv_pools ? p.kv_pools[l] : static_cast<char*>(p.base) + l * p.layer_stride;
  return P;
}

// int32 values of the state that have to be copied
int64_t page_state_ints(const PageArrays& S, bool table) {
  return (S.refs != S.new_refs ? S.N : 0) +
         (table && S.table != S.new_table ? (int64_t)S.B * S.cols : 0);
}

cudaError_t launch_page_state_copy(const PageArrays& S, bool table, cudaStream_t st) {
  const int64_t n = page_state_ints(S, table);
  if (n == 0) return cudaSuccess;
  const int sms = device_sms();
  if (sms < 1) return cudaErrorNoDevice;
  const int grid = (int)std::min<int64_t>(4 * (int64_t)sms, (n + 4 * kThreads - 1) / (4 * kThreads));
  return launch_pdl(page_state_copy_kernel, dim3(grid), dim3(kThreads), 0, st, S, table);
}

namespace {
// A kernel over `items` pieces of a new state, 256 threads each: with the counts to be
// copied first, as one cluster that does it while the state is small, behind a copy
// otherwise.
template <typename Args>
cudaError_t launch_over_state(void (*kernel)(Args), Args& A, int64_t items, size_t smem,
                              cudaStream_t st) {
  const int64_t cells = (int64_t)A.S.B * A.S.cols;
  A.copy = A.S.refs != A.S.new_refs && A.S.N + cells <= kFewInts;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (A.copy) {
    const int teams = kFewThreads / kThreads;
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(kFewBlocks, (items + teams - 1) / teams));
    cfg.blockDim = dim3(kFewThreads);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cfg.gridDim.x;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  } else {
    const cudaError_t e = launch_page_state_copy(A.S, false, st);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(items, 1 << 20));
    cfg.blockDim = dim3(kThreads);
  }
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, A);
}
}  // namespace

}  // namespace wedlm

using namespace wedlm;

namespace {
// a block a strip, all of whose pairs it stages
cudaError_t launch_in_place(ForkArgs& A, int64_t strips, size_t smem, cudaStream_t st) {
  A.copy = false;
  const cudaError_t e = launch_page_state_copy(A.S, false, st);
  if (e != cudaSuccess) return e;
  return launch_pdl(fork_kernel, dim3((unsigned)strips), dim3(kThreads), smem, st, A);
}
}  // namespace

extern "C" int wedlm_fork_pages(const wedlm_fork_args* a, void* stream) {
  if (!a || a->n < 1 || a->n > a->state.batch || bad4(a->src) || bad4(a->dst) ||
      !page_state_ok(a->state, kPageMaxBatch, true, true,
                     {{a->src, a->n}, {a->dst, a->n}, {a->lens, a->n}}, {}))
    return WEDLM_ERR_INVALID_ARG;
  ForkArgs A;
  A.S = page_arrays(a->state);
  A.n = a->n;
  A.src = a->src;
  A.dst = a->dst;
  A.lens = a->lens;
  const bool in_place = A.S.table == A.S.new_table;
  // in place a block holds its strip of all pairs, 8 columns (a sector) of them where 32
  // would not fit shared memory
  A.width = in_place && A.n > 1024 ? 8 : kStrip;
  const size_t smem = sizeof(int) * (A.S.B + std::max<size_t>(A.S.B, in_place ? (size_t)A.n * A.width : 0));
  const int64_t strips = (A.S.cols + A.width - 1) / A.width;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((smem > 40 << 10 &&  // beyond what a kernel has without asking
       ensure_dyn_smem(reinterpret_cast<const void*>(fork_kernel),
                       sizeof(int) * (kPageMaxBatch + 8 * kPageMaxBatch)) != cudaSuccess) ||
      (in_place ? launch_in_place(A, strips, smem, st)
                : launch_over_state(fork_kernel, A, strips * ((A.S.B + kForkRows - 1) / kForkRows),
                                    smem, st)) != cudaSuccess)
    return WEDLM_ERR_CUDA;
  return WEDLM_OK;
}

extern "C" int wedlm_free_pages(const wedlm_free_args* a, void* stream) {
  if (!a || bad4(a->keep_len)) return WEDLM_ERR_INVALID_ARG;
  // keep_len may be the lengths themselves: they then stay what they are
  const PageSpan keep = {a->keep_len == a->state.seq_len ? nullptr : a->keep_len, a->state.batch};
  if (!page_state_ok(a->state, kPageMaxBatch, true, true, {keep}, {})) return WEDLM_ERR_INVALID_ARG;
  FreeArgs A;
  A.S = page_arrays(a->state);
  A.keep = a->keep_len;
  const int64_t items = (int64_t)A.S.B * ((A.S.cols + kFreeCols - 1) / kFreeCols);
  if (launch_over_state(free_kernel, A, items, 0, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return WEDLM_ERR_CUDA;
  return WEDLM_OK;
}

namespace {
// a block that plans, or a cluster of them
template <typename Args>
cudaError_t launch_plan(void (*kernel)(Args), const Args& A, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(A.S.N >= kManyPages ? kPlanBlocks : 1);
  cfg.blockDim = dim3(kPlan);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cfg.gridDim.x;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cfg.gridDim.x > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, A);
}

struct PageSpace {
  size_t list, dropped, pairs, count, bytes;
};

PageSpace reserve_space(const wedlm_reserve_args& a) {
  PageSpace w;
  w.list = 0;
  w.dropped = align256(4 * (size_t)a.state.num_pages);
  w.pairs = 2 * w.dropped;
  w.count = w.pairs + align256(8 * (size_t)a.state.batch);
  w.bytes = w.count + 256;
  return w;
}

PageSpace compact_space(const wedlm_compact_args& a) {
  PageSpace w;
  w.list = w.dropped = 0;  // the map, where the caller wants none
  w.pairs = align256(4 * (size_t)a.state.num_pages);
  w.count = w.pairs + align256(4 * (size_t)a.state.num_pages);
  w.bytes = w.count + 256;
  return w;
}

bool reserve_sizes(const wedlm_reserve_args& a) {
  const wedlm_page_state& s = a.state;
  return s.batch >= 1 && s.batch <= kReserveMaxBatch && s.max_pages_per_seq >= 1 &&
         s.max_pages_per_seq <= kMaxColumns && s.num_pages >= 1 && s.num_pages <= kMaxPages &&
         a.rows >= 0 && page_pools_ok(a.pools, true);
}

bool compact_sizes(const wedlm_compact_args& a) {
  const wedlm_page_state& s = a.state;
  return s.batch >= 1 && s.batch <= kPageMaxBatch && s.max_pages_per_seq >= 1 &&
         s.max_pages_per_seq <= kMaxColumns && s.num_pages >= 1 && s.num_pages <= kMaxPages &&
         a.max_moves >= -1 && page_pools_ok(a.pools, true);
}
}  // namespace

extern "C" size_t wedlm_reserve_pages_workspace(const wedlm_reserve_args* a) {
  return a && reserve_sizes(*a) ? reserve_space(*a).bytes : 0;
}

extern "C" int wedlm_reserve_pages(const wedlm_reserve_args* a, void* stream) {
  if (!a || !reserve_sizes(*a) || !page_pools_ok(a->pools, false) || !a->workspace ||
      (reinterpret_cast<uintptr_t>(a->workspace) & 255))
    return WEDLM_ERR_INVALID_ARG;
  const PageSpace w = reserve_space(*a);
  if (!page_state_ok(a->state, kReserveMaxBatch, true, false, {{a->counts, a->state.batch}},
                     {{a->granted, a->state.batch},
                      {a->n_free, 1},
                      {a->workspace, (int64_t)(w.bytes / 4)}}) ||
      !page_pools_apart(a->pools, a->state, true,
                        {{a->counts, a->state.batch},
                         {a->granted, a->state.batch},
                         {a->n_free, 1},
                         {a->workspace, (int64_t)(w.bytes / 4)}}))
    return WEDLM_ERR_INVALID_ARG;
  if (a->workspace_bytes < w.bytes) return WEDLM_ERR_CAPACITY;
  const int sms = device_sms();
  if (sms < 1) return WEDLM_ERR_CUDA;
  char* ws = static_cast<char*>(a->workspace);
  ReserveArgs A;
  A.S = page_arrays(a->state);
  A.rows = a->rows;
  A.counts = a->counts;
  A.granted = a->granted;
  A.n_free = a->n_free;
  A.list = reinterpret_cast<int*>(ws + w.list);
  A.dropped = reinterpret_cast<int*>(ws + w.dropped);
  A.pairs = reinterpret_cast<int2*>(ws + w.pairs);
  A.n_pairs = reinterpret_cast<int*>(ws + w.count);
  const PagePools P = page_pools(a->pools);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int grid = copy_grid(sms, copy_items(a->pools, A.S.B));
  A.copy = page_state_ints(A.S, true) <= kFewInts / 2;  // by the block that plans
  if ((!A.copy && launch_page_state_copy(A.S, true, st) != cudaSuccess) ||
      launch_plan(reserve_plan_kernel, A, st) != cudaSuccess ||
      launch_pdl(copy_pages_kernel, dim3(grid), dim3(kThreads), 0, st, P, A.pairs, A.n_pairs) !=
          cudaSuccess)
    return WEDLM_ERR_CUDA;
  return WEDLM_OK;
}

extern "C" size_t wedlm_compact_pages_workspace(const wedlm_compact_args* a) {
  return a && compact_sizes(*a) ? compact_space(*a).bytes : 0;
}

extern "C" int wedlm_compact_pages(const wedlm_compact_args* a, void* stream) {
  if (!a || !compact_sizes(*a) || !page_pools_ok(a->pools, false) || !a->workspace ||
      (reinterpret_cast<uintptr_t>(a->workspace) & 255))
    return WEDLM_ERR_INVALID_ARG;
  const PageSpace w = compact_space(*a);
  if (!page_state_ok(a->state, kPageMaxBatch, false, false, {},
                     {{a->page_map, a->state.num_pages},
                      {a->n_live, 1},
                      {a->workspace, (int64_t)(w.bytes / 4)}}) ||
      !page_pools_apart(a->pools, a->state, false,
                        {{a->page_map, a->state.num_pages},
                         {a->n_live, 1},
                         {a->workspace, (int64_t)(w.bytes / 4)}}))
    return WEDLM_ERR_INVALID_ARG;
  if (a->workspace_bytes < w.bytes) return WEDLM_ERR_CAPACITY;
  const int sms = device_sms();
  if (sms < 1) return WEDLM_ERR_CUDA;
  char* ws = static_cast<char*>(a->workspace);
  CompactArgs A;
  A.S = page_arrays(a->state);
  A.max_moves = a->max_moves < 0 ? INT32_MAX : a->max_moves;
  A.map = a->page_map ? a->page_map : reinterpret_cast<int32_t*>(ws + w.list);
  A.n_live = a->n_live;
  A.pairs = reinterpret_cast<int2*>(ws + w.pairs);
  A.n_pairs = reinterpret_cast<int*>(ws + w.count);
  const PagePools P = page_pools(a->pools);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t cells = ((int64_t)A.S.B * A.S.cols + kThreads - 1) / kThreads;
  const int grid = copy_grid(sms, std::max(cells, copy_items(a->pools, A.S.N / 2)));
  if (launch_plan(compact_plan_kernel, A, st) != cudaSuccess ||
      launch_pdl(compact_move_kernel, dim3(grid), dim3(kThreads), 0, st, P, A.S,
                 (const int32_t*)A.map, (const int2*)A.pairs, (const int*)A.n_pairs) != cudaSuccess)
    return WEDLM_ERR_CUDA;
  return WEDLM_OK;
}
