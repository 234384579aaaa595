// Shared-prefix window attention on the 5th-generation tensor cores (bf16).
//
// A block (one per SM) holds two streams, A and B: 128 query rows each of Q, S,
// P and O.  A unit (a range of query rows of one kv head, see shared_attn.cuh)
// takes them in one of two ways:
//   pair:  more than one row block (TPB = 128/G tokens, at most 128 rows): A
//          takes the first, B the second, and both read every K/V tile, so a
//          tile's 64 KB feed 256 rows;
//   split: one row block: A takes the even key tiles, B the odd ones, and the
//          two (m, l, O) are joined before they leave the block.
// While one stream's softmax runs, the tensor core works for the other.
//
// One tile of one stream (128 keys):
//   S = Q K^T   (tcgen05.mma, A = Q and B = K from shared memory) -> TMEM S
//   P = 2^(S * scale - m), bf16, written over the first half of S (softmax)
//   O += P V    (A = P from TMEM, B = V from shared memory)       -> TMEM O
// P holds bf16 because the MMA takes both operands in one type; its rounding is
// as large as that of the output.  The running maximum m is raised only when a
// tile exceeds it by 2^8; until then the exponentials are taken against the
// stale one, which the division by l (held in 32 bits, like m and O) undoes.
//
// TMEM (512 columns): S/P of A at 0, of B at 128, O of A at 256, of B at 384.
// Each stream has its own issuing warp: P V of one tile, then S of the next, back
// to back.  The tensor core takes a thread's MMAs in order, so S may follow P V
// into the columns that P V reads, and S's barrier says that O is up to date too;
// and its queue is short, so what one issuer spends on waits and descriptors is
// time the other's MMAs run.
//
// What bounds it: the softmax.  A tile's takes its eight warps 1,340 cycles, and the
// warps take the streams' tiles in turn, so a round of two tiles is 2,680; the MMAs
// of a round are 2,048 with heads of 128 and 1,024 with heads of 64.  64 x 32 rows of
// 32 heads over 16384 shared positions: heads of 128 401 us, 1457 TFLOP/s (425 us
// in a run of half a second, where the power limit takes the SMs from 2070 to some
// 1880 MHz), heads of 64 361 us, 809 TFLOP/s.
//
// Single-thread instructions sit under elect.sync: under a comparison of the lane
// number an MMA took 90-110 cycles to issue, under elect.sync it runs at the
// tensor core's 64 (128 x 128 x 16).
//
// Code size: an SM holds about 64 KB of instructions; beyond that a 128-byte line
// costs 1300 cycles (measured with straight-line code).  An unrolled schedule made
// this kernel 140 KB, and masking one tile took 10,000 cycles.  So every role is a
// flat loop with its MMAs, copies and waits written once, and only the softmax of
// a tile is unrolled.
//
// Warps (384 threads): 0-7 softmax, A's and B's tiles in turn, half of a tile's
// keys each (a warpgroup per stream took 1,400 cycles from S to P, which the other
// stream's 1,024 cycles of MMA did not cover); 8 copies Q (TMA boxes) and K, 10
// copies V (4 KiB bulk copies of whole pages, already in the 8x8-tile operand
// layout; one warp for both took 1,900 cycles a tile) and plans: it walks the split
// and publishes the segments ahead of their use; 9 and 11 issue the MMAs of A and B.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "shared_attn.cuh"
#include "tc_ptx.cuh"

namespace wedlm {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;
constexpr float kRaise = 8.f;            // log2 units

template <int HD> struct Cfg {
  static constexpr uint32_t kPage = kPageBlock * HD * 2;
  static constexpr uint32_t kTileBytes = kSharedTile * HD * 2;
  static constexpr uint32_t kQBytes = 128 * HD * 2;
  // tiles in flight: what fits beside Q; K is needed before V
  static constexpr int kK = HD == 128 ? 3 : 4, kV = HD == 128 ? 2 : 4;
  static constexpr uint32_t kData = 2 * kQBytes + (kK + kV) * kTileBytes;
};

// A segment as the planner publishes it; n = 0 ends the list.
struct __align__(16) Seg {
  int b, kvh, shared;     // sequence (-1: shared unit), kv head, pages it skips
  int n_own, own_keys;    // cached pages of the range, keys in them (private)
  int pages;              // pages of the unit: cached, then the window's
  int t0, t1, n, nB;      // tiles; tiles of stream A, of stream B
  int pair;
  int tok0, ntok;         // first query token, tokens
  int w0;                 // window row of the first token (private)
  int slot, pad;
};
constexpr int kSegs = 4;  // segments published ahead

__device__ __forceinline__ int seg_tile(const Seg& g, int x, int j) {
  return g.t0 + (g.pair ? j : 2 * j + x);
}
__device__ __forceinline__ int tile_pages(const Seg& g, int t) {
  return min(kSharedTilePages, g.pages - t * kSharedTilePages);
}

// one lane of a converged warp, known as such to the compiler
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}
// D[tmem] (+)= A[tmem] * B[smem desc]: A's lane is its row, each 32-bit column
// two consecutive K elements
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void load_q_box(void* dst, const CUtensorMap* m, uint64_t* bar, int c0,
                                           int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
#define R8(a, i) "=f"(a[i]), "=f"(a[i + 1]), "=f"(a[i + 2]), "=f"(a[i + 3]), "=f"(a[i + 4]), \
                 "=f"(a[i + 5]), "=f"(a[i + 6]), "=f"(a[i + 7])
// 32 lanes x 64 columns, complete on return (load and wait in one statement, so
// that no use can move in between)
__device__ __forceinline__ void ld64(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, "
      "[%64];\n\ttcgen05.wait::ld.sync.aligned;"
      : R8(v, 0), R8(v, 8), R8(v, 16), R8(v, 24), R8(v, 32), R8(v, 40), R8(v, 48), R8(v, 56)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void ld16(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : R8(v, 0), R8(v, 8)
      : "r"(taddr)
      : "memory");
}
#undef R8
#define W8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), \
                 "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      W8(r, 0), W8(r, 8)
      : "memory");
}
#undef W8
// two 32-bit lanes at once
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max64(const float* v) {
  float mx[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    mx[k] = fmaxf(v[k], v[k + 4]);
#pragma unroll
    for (int c = 8; c < 64; c += 8) mx[k] = fmaxf(mx[k], fmaxf(v[c + k], v[c + k + 4]));
  }
  return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}
// p = 2^(v * sc + nm) of 32 columns to 16 columns of bf16 pairs; their sum
__device__ __forceinline__ float exp32(uint32_t taddr, const float* v, float sc, float nm) {
  const uint64_t sc2 = pack2(sc, sc), nm2 = pack2(nm, nm);
  uint64_t ps[2] = {0, 0};
  uint32_t pk[16];
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    float p0, p1;
    unpack2(fma2(pack2(v[c], v[c + 1]), sc2, nm2), p0, p1);
    p0 = ex2_approx(p0);
    p1 = ex2_approx(p1);
    ps[(c >> 1) & 1] = add2(ps[(c >> 1) & 1], pack2(p0, p1));
    const __nv_bfloat162 b2 = __floats2bfloat162_rn(p0, p1);
    pk[c >> 1] = *reinterpret_cast<const uint32_t*>(&b2);
  }
  st16(taddr, pk);
  float s0, s1;
  unpack2(add2(ps[0], ps[1]), s0, s1);
  return s0 + s1;
}
__device__ __forceinline__ void wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

template <int HD> struct Ctl {
  uint64_t k_full[Cfg<HD>::kK], k_empty[Cfg<HD>::kK], v_full[Cfg<HD>::kV], v_empty[Cfg<HD>::kV];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_done[2];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t pair[4], fin;  // pair: the two softmax warps of a row
  Seg seg[kSegs];
  const bf16* src[2][kSharedTilePages];  // a tile's pages: K, V
  float red[2][2][128];                  // [half][row]: row max of a tile; at the end, row sums
  int raise[2][4];                       // [tile parity]: last tile that raised a maximum
  int issued[4];                         // copies of K, V, Q buffer 0 and 1 started
  int abort;
  uint32_t tmem;
};

// the slow half of a wait, written once; false when this or another wait expired
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, int* err,
                                     volatile int* abort) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (int n = 1; !mbar_try_wait(bar, parity); ++n) {
    if (*abort) return false;
    if (n & 4095) continue;
    if (!t0) t0 = global_ns();
    if (global_ns() - t0 > kWaitNs) {
      set_err(err, WEDLM_DEV_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
  return true;
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
shared_attn_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ SharedArgs A,
                      int TPB) {
  using C = Cfg<HD>;
  // no static shared memory: the data starts on a 1024-byte boundary, as the
  // swizzled rows of Q need, and fills the SM's 227 KB up to the control block
  extern __shared__ __align__(1024) uint8_t base[];
  uint8_t* k_ring = base + 2 * C::kQBytes;
  uint8_t* v_ring = k_ring + C::kK * C::kTileBytes;
  Ctl<HD>& ctl = *reinterpret_cast<Ctl<HD>*>(base + C::kData);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = A.G;

  if (threadIdx.x == 32) {
    for (int i = 0; i < C::kK; ++i) {
      mbar_init(&ctl.k_full[i], 1);
      mbar_init(&ctl.k_empty[i], 2);  // both issuers
    }
    for (int i = 0; i < C::kV; ++i) {
      mbar_init(&ctl.v_full[i], 1);
      mbar_init(&ctl.v_empty[i], 2);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&ctl.q_full[x], 1);
      mbar_init(&ctl.q_empty[x], 2);
      mbar_init(&ctl.s_full[x], 1);
      mbar_init(&ctl.p_full[x], 8);
      mbar_init(&ctl.o_done[x], 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&ctl.seg_full[i], 1);
      mbar_init(&ctl.seg_empty[i], 12);  // copiers, issuers, 8 softmax warps
      mbar_init(&ctl.pair[i], 2);
      ctl.issued[i] = ctl.raise[0][i] = ctl.raise[1][i] = 0;
    }
    mbar_init(&ctl.fin, 2);
    ctl.abort = 0;
    mbar_fence_init();
  }
  if (warp == 0) {
    tmem_alloc(&ctl.tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  // warp-wide and bounded (2 s): what follows is executed by the whole warp together
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) ok = wait_on(bar, parity, A.err, &ctl.abort);
    return __all_sync(0xffffffffu, ok);
  };
  // next published segment, into registers (warp-wide); false after the last
  int seg_i = 0, pub_i = 0;
  uint32_t seg_ph = 0, pub_ph = 0;
  auto get = [&](Seg& g) -> bool {
    if (!wait(&ctl.seg_full[seg_i], seg_ph)) return false;
    g = ctl.seg[seg_i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl.seg_empty[seg_i]);
    if (++seg_i == kSegs) {
      seg_i = 0;
      seg_ph ^= 1u;
    }
    return g.n > 0;
  };

  pdl_wait();  // nothing of an earlier kernel is read before
  pdl_trigger();
  if (warp == 8 || warp == 10) {
    // ---------------- copiers: Q and K (8), V (10); 10 plans too ----------------
    const int kv = warp == 10;
    uint64_t* full = kv ? ctl.v_full : ctl.k_full;
    uint64_t* empty = kv ? ctl.v_empty : ctl.k_empty;
    uint8_t* ring = kv ? v_ring : k_ring;
    const int NS = kv ? C::kV : C::kK;
    const uint64_t keep = l2_evict_last_policy(), once = l2_evict_first_policy();
    SharedWalk walk;
    bool planned = true;  // the whole list is published
    // publish the next segment of the block's share, or the end of the list; this
    // warp keeps one segment ahead of the one it copies
    auto publish = [&]() -> bool {
      SharedSeg u;
      const bool more = __shfl_sync(0xffffffffu, walk.next(A, u), 0);
      Seg g = {};
      if (more) {
        const int n = u.t1 - u.t0;
        g.b = u.b;
        g.kvh = u.kvh;
        g.shared = u.sp.shared;
        g.t0 = u.t0;
        g.t1 = u.t1;
        g.w0 = u.blk * 2 * TPB;
        if (u.b < 0) {
          g.tok0 = g.w0;
          g.ntok = min(2 * TPB, A.B * A.W - g.tok0);
          g.pages = A.nsp;
        } else {
          g.tok0 = u.b * A.W + g.w0;
          g.ntok = min(2 * TPB, A.W - g.w0);
          g.n_own = own_pages(u.sp);
          g.own_keys = u.sp.len - u.sp.shared * kPageBlock;
          g.pages = g.n_own + A.Wp / kPageBlock;
        }
        g.pair = g.ntok > TPB;
        g.n = g.pair ? n : (n + 1) / 2;
        g.nB = g.pair ? n : n / 2;
        g.slot = seg_slot(A, u.unit, blockIdx.x);
      }
      planned = !more;
      if (!wait(&ctl.seg_empty[pub_i], pub_ph ^ 1u)) return false;
      if (lane == 0) {
        ctl.seg[pub_i] = g;
        mbar_arrive(&ctl.seg_full[pub_i]);
        if (more) record_unit(A, u);
      }
      __syncwarp();
      if (++pub_i == kSegs) {
        pub_i = 0;
        pub_ph ^= 1u;
      }
      return true;
    };
    if (kv) {
      walk.init(A);
      planned = false;
    } else if (elect_one()) {
      tma_prefetch_desc(&mq);
    }
    int st = 0, issued = 0, nq0 = 0, nq1 = 0, flip = 0;
    uint32_t ph = 1;
    // this lane's page id of a tile, loaded a tile ahead of its use
    auto id_of = [&](const Seg& g, int t) -> int {
      const int j = t * kSharedTilePages + lane;
      return lane < kSharedTilePages && t < g.t1 && j < (g.b < 0 ? g.pages : g.n_own)
                 ? own_page_id(A, g.b, g.shared, j)
                 : -1;
    };
    Seg g;
    bool ok = true;
#pragma unroll 1
    for (bool first = true; ok; first = false) {
      if (!planned && !(ok = publish())) break;
      if (first) {
        if (!get(g)) break;
        continue;
      }
      // Q: A's and B's row block, or one buffer in turn for both
#pragma unroll 1
      for (int x = 0; !kv && x < 1 + g.pair; ++x) {
        const int buf = g.pair ? x : flip;
        const int nq = buf ? nq1++ : nq0++;
        if (!(ok = wait(&ctl.q_empty[buf], (uint32_t)(nq & 1) ^ 1u))) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&ctl.q_full[buf], (uint32_t)(min(TPB, A.B * A.W) * G) * HD * 2);
#pragma unroll 1
          for (int c = 0; c < HD / 64; ++c)
            load_q_box(base + buf * C::kQBytes + c * 128 * 128, &mq, &ctl.q_full[buf], 64 * c,
                       g.kvh * G, g.tok0 + x * TPB);
          ctl.issued[2 + buf] = nq + 1;
        }
        __syncwarp();
      }
      if (!g.pair) flip ^= 1;
      int next_id = ok ? id_of(g, g.t0) : -1;
#pragma unroll 1
      for (int t = g.t0; ok && t < g.t1; ++t) {
        const int np = tile_pages(g, t), j = t * kSharedTilePages + lane, id = next_id;
        next_id = id_of(g, t + 1);
        const bf16* src = nullptr;
        if (lane < np) {
          if (g.b >= 0 && j >= g.n_own)
            src = window_block<bf16>(A, g.b, j - g.n_own, kv, g.kvh, HD);
          else if (id >= 0 && id < A.num_pages)
            src = cached_block<bf16>(A, id, kv, g.kvh, HD);
          else
            set_err(A.err, WEDLM_DEV_BAD_PAGE);
        }
        if (lane < kSharedTilePages) ctl.src[kv][lane] = src;
        const unsigned have = __ballot_sync(0xffffffffu, src != nullptr);
        if (!(ok = wait(&empty[st], ph))) break;
        uint8_t* dst = ring + st * C::kTileBytes;
        uint64_t* bar = &full[st];
        if (__popc(have) < np) {  // page ids out of range read as zeros
#pragma unroll 1
          for (int e = lane; e < np * (int)C::kPage / 16; e += 32)
            if (!(have >> (e / (C::kPage / 16)) & 1))
              reinterpret_cast<uint4*>(dst)[e] = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (elect_one()) {
          mbar_arrive_expect_tx(bar, (uint32_t)__popc(have) * C::kPage);
          const uint64_t pol = g.b < 0 ? keep : once;
          if (have == (1u << kSharedTilePages) - 1) {
            const bf16* sp[kSharedTilePages];
#pragma unroll
            for (int p = 0; p < kSharedTilePages; ++p) sp[p] = ctl.src[kv][p];
#pragma unroll
            for (int p = 0; p < kSharedTilePages; ++p)
              bulk_load(dst + p * C::kPage, sp[p], C::kPage, bar, pol);
          } else {
#pragma unroll 1
            for (int p = 0; p < kSharedTilePages; ++p)
              if (have >> p & 1) bulk_load(dst + p * C::kPage, ctl.src[kv][p], C::kPage, bar, pol);
          }
          ctl.issued[kv] = ++issued;
        }
        __syncwarp();
        if (++st == NS) {
          st = 0;
          ph ^= 1u;
        }
      }
      if (!ok || !get(g)) break;
    }
  } else if (warp == 9 || warp == 11) {
    // ---------------- MMA issuers ----------------
    // Q: rows of 64 dims, 128-byte swizzle (16 KB a half; 16 dims are 32 bytes); K:
    // 8-dim groups 128 B and 8-token groups HD*16 B apart (K-major); V: 8-token
    // groups HD*16 B, 8-dim groups 128 B apart (MN-major)
    const int x = warp == 11;
    const uint64_t dq0 = sdesc_sw128(smem_u32(base));
    const uint64_t dk0 = sdesc_noswz(smem_u32(k_ring), 128, HD * 16);
    const uint64_t dv0 = sdesc_noswz(smem_u32(v_ring), HD * 16, 128);
    const uint32_t idPV = idesc_bf16_m128(HD) | (1u << 16);
    const uint32_t dS = tmem + kColS + (uint32_t)(x * 128), dO = tmem + kColO + (uint32_t)(x * 128);
    Seg g;
    int j = -1;             // tile of this stream in the segment
    int base_n = 0;         // tiles of the block before the segment
    int nq0 = 0, nq1 = 0, flip = 0;
    // Both issuers follow every K and V tile and every Q of the block in order,
    // and release what the other one uses as soon as it is there: a barrier's
    // parity tells two neighbouring phases apart, so a reader may not skip any.
    int kpos = 0, vpos = 0, kst = 0, vst = 0;
    uint32_t kph = 0, vph = 0;
    auto wait_k = [&]() { return wait(&ctl.k_full[kst], kph); };
    auto wait_v = [&]() { return wait(&ctl.v_full[vst], vph); };
    auto next_k = [&]() {
      ++kpos;
      if (++kst == C::kK) {
        kst = 0;
        kph ^= 1u;
      }
    };
    auto next_v = [&]() {
      ++vpos;
      if (++vst == C::kV) {
        vst = 0;
        vph ^= 1u;
      }
    };
    // the tile whose P V is due: its number, pages, whether O starts or is complete
    // with it, the ends of its cached keys and of the window in it
    int pn = -1, pnp = 0, pfirst = 0, plast = 0, pc0 = 0, pc1 = 0;
    uint32_t pph = 0;
    bool have = get(g), ok = true;
#pragma unroll 1
    while (true) {
      // This stream's next tile, or none in this round: one segment on at most, for
      // the planner publishes only a few ahead of the slowest reader, which may be
      // waiting for the P V due here.
      ++j;
      if (have && j >= max(1, x ? g.nB : g.n)) {
        base_n += g.t1 - g.t0;
        if (g.pair || !flip) ++nq0;
        if (g.pair || flip) ++nq1;
        if (!g.pair) flip ^= 1;
        j = 0;
        have = get(g);
      }
      if (!have && pn < 0) break;
      const bool tile = have && j < (x ? g.nB : g.n);
      const int buf = g.pair ? x : flip;
      if (have && j == 0) {  // a new segment's Q
        if (!(ok = wait(&ctl.q_full[buf], (uint32_t)((buf ? nq1 : nq0) & 1)))) break;
        if (!tile && lane == 0) mbar_arrive(&ctl.q_empty[buf]);
        if (g.pair) {
          if (!(ok = wait(&ctl.q_full[buf ^ 1], (uint32_t)((buf ? nq0 : nq1) & 1)))) break;
          if (lane == 0) mbar_arrive(&ctl.q_empty[buf ^ 1]);
        }
        __syncwarp();
      }
      const int t = tile ? seg_tile(g, x, j) : 0, np = tile ? tile_pages(g, t) : 0;
      const int n = base_n + t - g.t0;
      // V up to the tile that is due, then K up to the next tile
      const int vto = pn >= 0 ? pn : base_n;
#pragma unroll 1
      while (vpos < vto && (ok = wait_v())) {
        if (lane == 0) mbar_arrive(&ctl.v_empty[vst]);
        next_v();
      }
      const int kto = tile ? n : have ? base_n + g.t1 - g.t0 : base_n;
#pragma unroll 1
      while (ok && kpos < kto && (ok = wait_k())) {
        if (lane == 0) mbar_arrive(&ctl.k_empty[kst]);
        next_k();
      }
      if (!ok || (tile && !(ok = wait_k()))) break;
      if (pn >= 0) {
        if (!(ok = wait_v())) break;
        // V rows that no query sees (the tails of the last cached page and of the
        // window) become zeros: 0 * NaN would reach every row.  In pair mode both
        // issuers write the same zeros.
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          const int c = part ? pc1 : pc0;
          if (c <= 0 || c >= kSharedTile || !(c & 15)) continue;
          const int rows = 16 - (c & 15);
#pragma unroll 1
          for (int e = lane; e < 16 * (HD / 8); e += 32)
            if ((e & 15) < rows)
              *reinterpret_cast<uint4*>(v_ring + vst * C::kTileBytes +
                                        2 * ((c >> 4) * kPageBlock * HD +
                                             tile_off((c & 15) + (e & 15), (e >> 4) * 8, HD))) =
                  make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        if (!(ok = wait(&ctl.p_full[x], pph))) break;
        pph ^= 1u;
      }
      if (elect_one()) {
        tc_fence_after();
        if (pn >= 0) {
          const uint64_t dv = dv0 + (uint64_t)(vst * C::kTileBytes >> 4);
#pragma unroll
          for (int k = 0; k < kSharedTilePages; ++k)  // 16 keys: 8 columns of P
            if (k < pnp) mma_ts(dO, dS + k * 8, dv + k * (HD * 2), idPV, (k || !pfirst) ? 1u : 0u);
          if (plast) tc_commit(&ctl.o_done[x]);
          tc_commit(&ctl.v_empty[vst]);
        }
        if (tile) {
          const uint64_t dq = dq0 + (uint64_t)(buf * C::kQBytes >> 4);
          const uint64_t dk = dk0 + (uint64_t)(kst * C::kTileBytes >> 4);
          const uint32_t id = idesc_bf16_m128(np * kPageBlock);
#pragma unroll
          for (int k = 0; k < HD / 16; ++k)  // 16 dims: two 8-dim groups
            tc_mma_f16(dS, dq + (k / 4) * (128 * 128 / 16) + (k % 4) * 2, dk + k * 16, id,
                       k ? 1u : 0u);
          tc_commit(&ctl.s_full[x]);
          tc_commit(&ctl.k_empty[kst]);
          if (j + 1 == (x ? g.nB : g.n)) tc_commit(&ctl.q_empty[buf]);  // the last S from this Q
        }
      }
      __syncwarp();
      if (pn >= 0) next_v();
      if (tile) next_k();
      pn = tile ? n : -1;
      pnp = np;
      pfirst = j == 0;
      plast = j + 1 == (x ? g.nB : g.n);
      pc0 = g.b < 0 ? 0 : g.own_keys - t * kSharedTile;
      pc1 = g.b < 0 ? 0 : g.n_own * kPageBlock - t * kSharedTile + A.W;
    }
    // every MMA has completed before TMEM is freed
    if (elect_one()) tc_commit(&ctl.fin);
    mbar_wait(&ctl.fin, 0, A.err);
  } else {
    // ---------------- softmax ----------------
    // Warps q and q+4 hold query rows 32q .. 32q+31 of both streams (thread = row):
    // q the keys 0-63 of a tile and the first half of O's dims, q+4 the others.
    const int q = warp & 3, h = warp >> 2;
    const int r = 32 * q + lane;
    const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16);
    const float sc = A.scale_log2;
    uint32_t sph = 0, dph = 0, jph = 0;  // phases: bit x of s_full and o_done, of the pair's
    // The two warps of a row meet.  An mbarrier and not a named one, so that a wait
    // that expired elsewhere cannot leave one of them here for good.
    auto pair_sync = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.pair[q]);
      wait(&ctl.pair[q], jph);
      jph ^= 1u;
    };
    Seg g;
    int tiles = 0;  // tiles so far, for the raise flags
#pragma unroll 1
    while (get(g)) {
      float m2[2] = {-INFINITY, -INFINITY}, l2[2] = {0.f, 0.f};
#pragma unroll 1
      for (int i = 0; i < g.n + g.nB; ++i) {
        // A and B in turn (B's last tile may be missing)
        const int x = i & 1, j = i >> 1;
        const int t = seg_tile(g, x, j), np = tile_pages(g, t);
        const uint32_t tS = tl + kColS + (uint32_t)(x * 128);
        const uint32_t tO = tl + kColO + (uint32_t)(x * 128 + h * (HD / 2));
        float m = x ? m2[1] : m2[0];
        wait(&ctl.s_full[x], sph >> x & 1);
        sph ^= 1u << x;
        tc_fence_after();
        // what this row does not see becomes -inf, in TMEM and in a rolled loop:
        // only a unit's last tiles need it
        if (np < kSharedTilePages || (g.b >= 0 && (t + 1) * kSharedTile > g.own_keys)) {
          const int p_row = g.w0 + (g.pair ? x * TPB : 0) + r / G;  // window row
          const int c_own = g.b < 0 ? np * kPageBlock : g.own_keys - t * kSharedTile;
          const int c_win = g.n_own * kPageBlock - t * kSharedTile;
          const int c_end = g.b < 0 ? 0 : c_win + p_row + 1;  // window keys up to this row
#pragma unroll 1
          for (int c0 = h * 64; c0 < h * 64 + 64; c0 += 16) {
            if (c0 + 16 <= c_own) continue;  // the same for every row
            float e[16];
            uint32_t u[16];
            ld16(tS + c0, e);
            // bit i: column c0 + i is visible
            const uint32_t lo = c_own - c0 >= 16 ? ~0u : c_own <= c0 ? 0u : (1u << (c_own - c0)) - 1;
            const uint32_t up = c_end - c0 >= 16 ? ~0u : c_end <= c0 ? 0u : (1u << (c_end - c0)) - 1;
            const uint32_t dn = c_win - c0 >= 16 ? ~0u : c_win <= c0 ? 0u : (1u << (c_win - c0)) - 1;
            const uint32_t seen = lo | (up & ~dn);
#pragma unroll
            for (int k = 0; k < 16; ++k)
              u[k] = seen >> k & 1 ? __float_as_uint(e[k]) : 0xff800000u;
            st16(tS + c0, u);
          }
          wait_st();
        }
        float v[64];
        ld64(tS + h * 64, v);
        float mt = max64(v) * sc;
        // Does a row of either warp raise its maximum?  The meeting also keeps P
        // from S columns the other warp has not read yet.
        const int odd = ++tiles & 1;  // one of the two may be a tile ahead: two sets
        ctl.red[odd][h][r] = mt;
        if (__any_sync(0xffffffffu, mt > m + kRaise)) ctl.raise[odd][q] = tiles;
        pair_sync();
        if (ctl.raise[odd][q] == tiles) {
          mt = fmaxf(mt, ctl.red[odd][h ^ 1][r]);
          const bool raise = mt > m + kRaise;
          if (j > 0) {  // O holds the tiles before: S is committed behind their P V
            const float a = !raise ? 1.f : m == -INFINITY ? 0.f : ex2_approx(m - mt);
#pragma unroll 1
            for (int c = 0; c < HD / 2; c += 16) {
              float o[16];
              uint32_t u[16];
              ld16(tO + c, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(o[k] * a);
              st16(tO + c, u);
            }
            if (x) l2[1] *= a; else l2[0] *= a;
          }
          if (raise) m = mt;
          if (x) m2[1] = m; else m2[0] = m;
        }
        const float nm = m == -INFINITY ? 0.f : -m;
        const float ps = exp32(tS + h * 32, v, sc, nm) + exp32(tS + h * 32 + 16, v + 32, sc, nm);
        if (x) l2[1] += ps; else l2[0] += ps;
        wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.p_full[x]);
      }
      // The segment's partial: O once its last P V is done.  Pair: this warp's half
      // of the dims of both streams' rows.  Split: A and B joined.
      wait(&ctl.o_done[0], dph & 1);
      dph ^= 1u;
      if (g.nB > 0) {
        wait(&ctl.o_done[1], dph >> 1);
        dph ^= 2u;
      }
      tc_fence_after();
      pair_sync();  // the other warp is done with `red` too
      ctl.red[h][0][r] = l2[0];  // the row sums are in halves
      ctl.red[h][1][r] = l2[1];
      pair_sync();
      const int urows = g.b < 0 ? A.srows : A.prows;
      float4* po = (g.b < 0 ? A.part_s : A.part_p) +
                   ((size_t)g.slot * (HD / 4) + h * (HD / 8)) * urows;
      float2* ml = (g.b < 0 ? A.ml_s : A.ml_p) + (size_t)g.slot * urows;
      float f[2] = {1.f, 1.f};
      const float la = l2[0] + ctl.red[h ^ 1][0][r], lb = l2[1] + ctl.red[h ^ 1][1][r];
      if (!g.pair) {
        const float M = fmaxf(m2[0], m2[1]);
        f[0] = m2[0] == -INFINITY ? 0.f : ex2_approx(m2[0] - M);
        f[1] = m2[1] == -INFINITY ? 0.f : ex2_approx(m2[1] - M);
        if (h == 0 && r < g.ntok * G) ml[r] = make_float2(M, la * f[0] + lb * f[1]);
      }
#pragma unroll 1
      for (int x = 0; x < 1 + g.pair; ++x) {
        const int row = x * TPB * G + r;
        const bool valid = r < TPB * G && row < g.ntok * G;
        if (g.pair && h == 0 && valid) ml[row] = make_float2(x ? m2[1] : m2[0], x ? lb : la);
        const uint32_t tO = tl + kColO + (uint32_t)(x * 128 + h * (HD / 2));
        float4* dst = po + row;
#pragma unroll 1
        for (int c = 0; c < HD / 2; c += 16) {
          float o[16];
          ld16(tO + c, o);
          if (!g.pair) {
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] *= f[0];
            if (g.nB > 0) {  // else B's O holds nothing of this segment
              float ob[16];
              ld16(tO + 128 + c, ob);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = fmaf(ob[k], f[1], o[k]);
            }
          }
          if (valid) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              *dst = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
              dst += urows;
            }
          }
        }
      }
      tc_fence_before();
      pair_sync();  // `red` may be written again
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (ctl.abort && threadIdx.x == 256) {
    // a wait expired: let the copies still in flight land (bounded; a phase that
    // has passed answers at once)
#pragma unroll 1
    for (int i = max(0, ctl.issued[0] - C::kK); i < ctl.issued[0]; ++i)
      mbar_wait(&ctl.k_full[i % C::kK], (uint32_t)(i / C::kK) & 1u, A.err);
#pragma unroll 1
    for (int i = max(0, ctl.issued[1] - C::kV); i < ctl.issued[1]; ++i)
      mbar_wait(&ctl.v_full[i % C::kV], (uint32_t)(i / C::kV) & 1u, A.err);
#pragma unroll 1
    for (int x = 0; x < 2; ++x)
      if (ctl.issued[2 + x]) mbar_wait(&ctl.q_full[x], (uint32_t)(ctl.issued[2 + x] - 1) & 1u, A.err);
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static std::atomic<void*> cached{nullptr};
  void* p = cached.load(std::memory_order_acquire);
  if (!p) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    cached.store(p, std::memory_order_release);
  }
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
}

template <int HD>
cudaError_t launch(const SharedArgs& A, int TPB, cudaStream_t st) {
  const auto enc = encoder();
  if (!enc) return cudaErrorNotSupported;
  // q as {dim, head, token}: a box of 64 dims, G heads and TPB tokens is half (all) of
  // a row block, rows token * G + g of 128 bytes.  (Boxes of 8 dims, laid out like K,
  // are 16-byte pieces: a pair of row blocks took 5,000 cycles to arrive.)
  CUtensorMap mq;
  const cuuint64_t nq = (cuuint64_t)A.nkv * A.G;
  cuuint64_t dims[3] = {HD, nq, (cuuint64_t)A.B * A.W};
  cuuint64_t strides[2] = {HD * 2, nq * HD * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)A.G, (cuuint32_t)std::min(TPB, A.B * A.W)};
  cuuint32_t one[3] = {1, 1, 1};
  if (enc(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(A.q), dims, strides, box, one,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  constexpr size_t kSmem = Cfg<HD>::kData + sizeof(Ctl<HD>);
  static_assert(kSmem <= 227 * 1024, "shared memory of one SM");
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = raise_smem(done, (const void*)shared_attn_tc_kernel<HD>, (int)kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(shared_attn_tc_kernel<HD>, dim3(A.grid), dim3(kThreads), kSmem, st, mq,
                    A, TPB);
}

}  // namespace

cudaError_t launch_shared_attention_tc(const SharedArgs& A, int hd, int TPB, cudaStream_t st) {
  return hd == 128 ? launch<128>(A, TPB, st) : launch<64>(A, TPB, st);
}

}  // namespace wedlm
