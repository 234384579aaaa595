// The work split that the shared-prefix attention kernels and their merge
// agree on.
//
// The query rows of one kv head h are numbered token * G + g (token = b*W + p,
// G q heads per kv head).  A unit is up to `urows` rows of one kv head and the
// keys they attend to in one of two ranges:
//   shared units: consecutive rows of the whole batch x the shared pages;
//   private units: consecutive rows of one sequence x its own pages past the
//   shared ones, followed by the pages of its window block.
// A unit's keys come in tiles of 8 pages (128 keys).  All units' tiles are
// laid end to end (shared units first, kv head by kv head) and every block
// takes a contiguous share of about equal cost: a unit costs `ucost` to start
// and finish plus shared_cost or private_cost per tile.  The tiles of one unit
// inside one block are a segment; it leaves an unnormalised partial (O, m, l)
// in slot unit + block of its range.  Along the tile order neither index
// decreases and one grows from a segment to the next, so slots are distinct.
// The blocks that hold a unit's first and last tile record themselves, and
// the merge walks the slots in between, in order.
#pragma once
#include "internal.h"

namespace wedlm {

constexpr int kSharedTile = 128;                            // keys per tile
constexpr int kSharedTilePages = kSharedTile / kPageBlock;  // 8
constexpr int kSharedMaxBatch = 1024;
constexpr int kSharedMaxGrid = 256;

struct SharedArgs {
  int B, W, Wp, G, nkv, nsp;      // nsp: shared pages
  int max_pages, num_pages;
  float scale_log2;               // log2(e) / sqrt(head_dim)
  const void *q, *pool, *kv_win;
  const int32_t *shared, *page_table, *seq_len;
  void* o;
  int* err;
  // split
  int srows, sblocks;             // rows per shared unit, shared units per kv head
  int prows, pblocks;             // rows per private unit, units per (sequence, kv head)
  int ucost, shared_cost, private_cost, min_share;
  int grid;
  // workspace
  float4 *part_s, *part_p;        // [slot][hd/4][rows of a unit] partial O
  float2 *ml_s, *ml_p;            // [slot][rows of a unit] running max (log2 units), row sum
  int2* unit_blocks;              // [unit] blocks of the first and last tile
};

// cached length of sequence b as the kernels see it, and the pages of it that
// come from the shared list (all of them or none)
struct SeqSpan { int len, shared; };
__device__ __forceinline__ SeqSpan seq_span(const SharedArgs& A, int b, bool tell) {
  int L = A.seq_len[b];
  if (L < 0) {
    if (tell) set_err(A.err, WEDLM_DEV_BAD_SEQLEN);
    L = 0;
  } else if (L > A.max_pages * kPageBlock) {
    if (tell) set_err(A.err, WEDLM_DEV_CAPACITY);
    L = A.max_pages * kPageBlock;
  }
  return {L, L >= A.nsp * kPageBlock ? A.nsp : 0};
}
__device__ __forceinline__ int own_pages(const SeqSpan& s) {
  return (s.len + kPageBlock - 1) / kPageBlock - s.shared;
}
__device__ __forceinline__ int own_tiles(const SharedArgs& A, const SeqSpan& s) {
  return (own_pages(s) + A.Wp / kPageBlock + kSharedTilePages - 1) / kSharedTilePages;
}

// The split, built once per block by all of its threads.  s_w: B + 1 words of
// shared memory, the weighted start of each sequence's private units.
struct SharedSplit {
  long long shared_unit;  // weight of one shared unit (0: nobody shares)
  long long shared_total, total;
  int shared_tiles, blocks;
};
__device__ inline SharedSplit shared_split(const SharedArgs& A, long long* s_w, int* s_any) {
  if (threadIdx.x == 0) *s_any = 0;
  __syncthreads();
  for (int b = threadIdx.x; b < A.B; b += blockDim.x) {
    const SeqSpan sp = seq_span(A, b, blockIdx.x == 0);
    if (sp.shared) *s_any = 1;
    s_w[b] = (long long)A.nkv * A.pblocks *
             (A.ucost + (long long)own_tiles(A, sp) * A.private_cost);
  }
  __syncthreads();
  if (threadIdx.x < 32) {  // exclusive prefix sums, in place
    const int lane = threadIdx.x, per = (A.B + 31) / 32;
    const int b0 = min(A.B, lane * per), b1 = min(A.B, b0 + per);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) sum += s_w[b];
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    long long acc = incl - sum;
    for (int b = b0; b < b1; ++b) {
      const long long x = s_w[b];
      s_w[b] = acc;
      acc += x;
    }
    if (lane == 31) s_w[A.B] = incl;
  }
  __syncthreads();
  SharedSplit S;
  S.shared_tiles = *s_any ? (A.nsp + kSharedTilePages - 1) / kSharedTilePages : 0;
  S.shared_unit = S.shared_tiles ? A.ucost + (long long)S.shared_tiles * A.shared_cost : 0;
  S.shared_total = S.shared_unit * A.nkv * A.sblocks;
  S.total = S.shared_total + s_w[A.B];
  // a share holds at least one tile start wherever it lies inside a unit
  S.blocks = (int)max(1LL, min((long long)A.grid, S.total / A.min_share));
  return S;
}

// One segment: tiles t0 .. t1-1 of a unit.
struct SharedSeg {
  int unit;       // index over all units (shared ones first)
  int b;          // sequence of a private unit, -1: shared
  int kvh, blk;   // kv head, row block
  int t0, t1, T;  // tiles of the segment, of the unit
};

// Walks the segments of one block in tile order.
struct SharedWalk {
  long long w, w1;  // weighted position, end of the share
  __device__ void init(const SharedSplit& S, int block) {
    w = block * S.total / S.blocks;
    w1 = (block + 1) * S.total / S.blocks;
  }
  // tile t of a unit starts ucost + t * cost after the unit; a block owns the
  // tiles that start in its share
  __device__ bool next(const SharedArgs& A, const SharedSplit& S, const long long* s_w,
                       SharedSeg& g) {
    while (w < w1) {
      long long u0, uw;
      int cost;
      if (w < S.shared_total) {
        const int u = (int)(w / S.shared_unit);
        u0 = u * S.shared_unit;
        uw = S.shared_unit;
        g.unit = u;
        g.b = -1;
        g.kvh = u / A.sblocks;
        g.blk = u % A.sblocks;
        g.T = S.shared_tiles;
        cost = A.shared_cost;
      } else {
        const long long r = w - S.shared_total;
        int lo = 0, hi = A.B - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (s_w[mid] <= r) lo = mid; else hi = mid - 1;
        }
        const int per = A.nkv * A.pblocks;
        uw = (s_w[lo + 1] - s_w[lo]) / per;
        const int k = (int)((r - s_w[lo]) / uw);
        u0 = S.shared_total + s_w[lo] + k * uw;
        g.unit = A.nkv * A.sblocks + lo * per + k;
        g.b = lo;
        g.kvh = k / A.pblocks;
        g.blk = k % A.pblocks;
        cost = A.private_cost;
        g.T = (int)((uw - A.ucost) / cost);
      }
      const long long first = w - u0 - A.ucost, end = w1 - u0 - A.ucost;
      g.t0 = first <= 0 ? 0 : (int)((first + cost - 1) / cost);
      g.t1 = end <= 0 ? 0 : (int)min((long long)g.T, (end + cost - 1) / cost);
      w = u0 + uw;
      if (g.t0 < g.t1) return true;
    }
    return false;
  }
};

// slot of a segment in its range's partials
__device__ __forceinline__ int seg_slot(const SharedArgs& A, int unit, int block) {
  const int ns = A.nkv * A.sblocks;
  return (unit < ns ? unit : unit - ns) + block;
}

// one thread of the block records the unit's first and last block
__device__ __forceinline__ void record_unit(const SharedArgs& A, const SharedSeg& g) {
  if (g.t0 == 0) A.unit_blocks[g.unit].x = blockIdx.x;
  if (g.t1 == g.T) A.unit_blocks[g.unit].y = blockIdx.x;
}

// Page `j` of a unit (its keys 16j .. 16j+15): cached pages first, then the
// window block's.  Sets the 16-token K (kv = 0) or V block of kv head kvh, or
// null for a page id out of range (recorded in the error word).
template <typename T>
__device__ __forceinline__ const T* unit_page(const SharedArgs& A, const SharedSeg& g,
                                              const SeqSpan& sp, int n_own, int j, int kv, int hd) {
  const size_t blockn = (size_t)kPageBlock * hd;
  if (g.b >= 0 && j >= n_own)
    return static_cast<const T*>(A.kv_win) +
           (((size_t)g.b * 2 + kv) * A.nkv + g.kvh) * A.Wp * hd + (size_t)(j - n_own) * blockn;
  const int id = g.b < 0 ? A.shared[j]
                         : A.page_table[(size_t)g.b * A.max_pages + sp.shared + j];
  if (id < 0 || id >= A.num_pages) {
    set_err(A.err, WEDLM_DEV_BAD_PAGE);
    return nullptr;
  }
  return static_cast<const T*>(A.pool) + (((size_t)id * 2 + kv) * A.nkv + g.kvh) * blockn;
}

// fp32: urows query rows per unit, whatever tokens they belong to
constexpr int kSimtRows = 64;
cudaError_t launch_shared_attention_simt(const SharedArgs& A, int hd, cudaStream_t st);
// bf16: units of 2 * TPB tokens, TPB = 128 / G
cudaError_t launch_shared_attention_tc(const SharedArgs& A, int hd, int TPB, cudaStream_t st);
cudaError_t launch_shared_merge(const SharedArgs& A, int hd, bool is_bf16, cudaStream_t st);

}  // namespace wedlm
