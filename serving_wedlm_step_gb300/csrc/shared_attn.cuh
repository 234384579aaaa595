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
#include <atomic>

#include "internal.h"

namespace wedlm {

// Raise a kernel's dynamic shared-memory limit on the current device, once per
// (kernel, device); throws nothing.  `done` is the kernel's own word.
inline cudaError_t raise_smem(std::atomic<uint64_t>& done, const void* kernel, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

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
__device__ __forceinline__ SeqSpan seq_span(const SharedArgs& A, int b) {
  const int L = max(0, min(A.seq_len[b], A.max_pages * kPageBlock));
  return {L, L >= A.nsp * kPageBlock ? A.nsp : 0};
}
// records a length that seq_span has to change
__device__ __forceinline__ void check_len(const SharedArgs& A, int b) {
  const int L = A.seq_len[b];
  if (L < 0 || L > A.max_pages * kPageBlock)
    set_err(A.err, L < 0 ? WEDLM_DEV_BAD_SEQLEN : WEDLM_DEV_CAPACITY);
}
__device__ __forceinline__ int own_pages(const SeqSpan& s) {
  return (s.len + kPageBlock - 1) / kPageBlock - s.shared;
}
__device__ __forceinline__ int own_tiles(const SharedArgs& A, const SeqSpan& s) {
  return (own_pages(s) + A.Wp / kPageBlock + kSharedTilePages - 1) / kSharedTilePages;
}

// One segment: tiles t0 .. t1-1 of a unit of T tiles.
struct SharedSeg {
  int unit;             // index over all units (shared ones first)
  int b;                // sequence of a private unit, -1: shared
  int kvh, blk;         // kv head, row block
  int t0, t1, T;
  SeqSpan sp;           // of sequence b
};

// Walks the segments of this block in tile order; one warp runs it, all lanes
// alike.  Tile t of a unit starts ucost + t * cost after the unit, and a block
// owns the tiles that start in its share of the total weight.  The host keeps
// the total below 2^31, so that the divisions are 32 bits wide: the planner runs
// before the first copy can start.
struct SharedWalk {
  int u0, w0, w1;        // weighted start of the next unit, the block's share
  int shared_tiles, u, b, k;  // next unit: shared unit u, or unit k of sequence b
  int uw;                // weight of a unit of the range at hand
  SeqSpan sp;

  __device__ void init(const SharedArgs& A) {
    const int lane = threadIdx.x & 31, units = A.nkv * A.pblocks;
    const int per = (A.B + 31) / 32, b0 = min(A.B, lane * per), b1 = min(A.B, b0 + per);
    int sum = 0, any = 0;
#pragma unroll 1
    for (int i = b0; i < b1; i += 4) {
      SeqSpan s[4];  // four loads in flight
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] = seq_span(A, min(i + k, b1 - 1));
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k < b1) {
          any |= s[k].shared;
          sum += A.ucost + own_tiles(A, s[k]) * A.private_cost;
        }
    }
    sum *= units;
    if (blockIdx.x == 0)
#pragma unroll 1
      for (int i = b0; i < b1; ++i) check_len(A, i);
    any = __any_sync(0xffffffffu, any);
    int incl = sum;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    // nothing to do for the shared pages when no sequence takes part
    shared_tiles = any ? (A.nsp + kSharedTilePages - 1) / kSharedTilePages : 0;
    uw = A.ucost + shared_tiles * A.shared_cost;
    const int shared_total = any ? uw * A.nkv * A.sblocks : 0;
    const unsigned total = shared_total + __shfl_sync(0xffffffffu, incl, 31);
    // a share is never shorter than min_share >= a tile, so that it holds a
    // tile's start wherever it lies inside a unit
    const unsigned blocks = max(1u, min((unsigned)A.grid, total / (unsigned)A.min_share));
    const unsigned share = total / blocks, extra = total - share * blocks;
    w0 = blockIdx.x * share + min(blockIdx.x, extra);
    w1 = w0 + share + (blockIdx.x < extra ? 1 : 0);
    u = b = k = u0 = 0;
    if (blockIdx.x >= blocks) {
      b = A.B;
      u = A.nkv * A.sblocks;
    } else if (w0 < shared_total) {
      u = (unsigned)w0 / (unsigned)uw;
      u0 = u * uw;
    } else {  // the first sequence of the lane in whose range the share starts
      u = A.nkv * A.sblocks;
      const int owner = __ffs(__ballot_sync(0xffffffffu, incl > w0 - shared_total)) - 1;
      b = owner * per;
      u0 = shared_total + __shfl_sync(0xffffffffu, incl - sum, owner);
    }
  }
  __device__ bool next(const SharedArgs& A, SharedSeg& g) {
#pragma unroll 1
    while (true) {
      int cost = A.shared_cost;
      if (shared_tiles && u < A.nkv * A.sblocks) {
        g.unit = u;
        g.b = -1;
        g.kvh = u / A.sblocks;
        g.blk = u - g.kvh * A.sblocks;
        g.T = shared_tiles;
        g.sp = SeqSpan{0, 0};
        if (u0 >= w1) return false;
        ++u;
      } else {
        if (b >= A.B || u0 >= w1) return false;
        const int units = A.nkv * A.pblocks;
        if (k == 0) {  // a sequence's first unit: skip to where the share starts
          sp = seq_span(A, b);
          uw = A.ucost + own_tiles(A, sp) * A.private_cost;
          if (u0 < w0) k = min(units, (w0 - u0) / uw);
          u0 += k * uw;
        }
        const bool here = k < units;
        if (here) {
          g.unit = A.nkv * A.sblocks + b * units + k;
          g.b = b;
          g.kvh = k / A.pblocks;
          g.blk = k - g.kvh * A.pblocks;
          g.sp = sp;
          g.T = own_tiles(A, sp);
          ++k;
        }
        cost = A.private_cost;
        if (k == units) {
          k = 0;
          ++b;
        }
        if (!here) continue;  // the whole sequence lies before the share
      }
      const int start = u0 + A.ucost;
      u0 = start + g.T * cost;
      g.t0 = w0 <= start ? 0 : min(g.T, (w0 - start + cost - 1) / cost);
      g.t1 = w1 <= start ? 0 : min(g.T, (w1 - start + cost - 1) / cost);
      if (g.t0 < g.t1) return true;
    }
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

// Page `j` of a unit (its keys 16j .. 16j+15): n_own cached pages, then the
// window block's.  own_page_id: the id of a cached one, as the table has it.
__device__ __forceinline__ int own_page_id(const SharedArgs& A, int b, int shared, int j) {
  return b < 0 ? __ldg(A.shared + j) : __ldg(A.page_table + (size_t)b * A.max_pages + shared + j);
}
template <typename T>
__device__ __forceinline__ const T* cached_block(const SharedArgs& A, int id, int kv, int kvh,
                                                 int hd) {
  return static_cast<const T*>(A.pool) + (((size_t)id * 2 + kv) * A.nkv + kvh) * kPageBlock * hd;
}
template <typename T>
__device__ __forceinline__ const T* window_block(const SharedArgs& A, int b, int j, int kv, int kvh,
                                                 int hd) {
  return static_cast<const T*>(A.kv_win) +
         ((((size_t)b * 2 + kv) * A.nkv + kvh) * A.Wp + j * kPageBlock) * hd;
}

// fp32: urows query rows per unit, whatever tokens they belong to
constexpr int kSimtRows = 64;
constexpr int kSimtFewRows = 16;  // units of at most so many rows take smaller tiles
cudaError_t launch_shared_attention_simt(const SharedArgs& A, int hd, cudaStream_t st);
// bf16: units of 2 * TPB tokens, TPB = 128 / G
cudaError_t launch_shared_attention_tc(const SharedArgs& A, int hd, int TPB, cudaStream_t st);
cudaError_t launch_shared_merge(const SharedArgs& A, int hd, bool is_bf16, cudaStream_t st);

}  // namespace wedlm
