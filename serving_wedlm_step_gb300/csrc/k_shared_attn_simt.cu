// Shared-prefix window attention on the CUDA cores (fp32), and the merge of the
// partials of either kernel.
//
// One pass over a segment's keys with the running maximum m and sum l of each
// row, in log2 units:
//   s = q k * log2(e)/sqrt(hd),  m' = max(m, max s),
//   l = l 2^(m-m') + sum 2^(s-m'),  O = O 2^(m-m') + 2^(s-m') V
// 64 rows x 128 keys per tile, 256 threads; a thread owns 4 rows x 8 keys of S
// and 4 rows x 8 (4) dims of O, so a step of 4 dims (keys) does 128 FMAs, in
// pairs, on 12 shared-memory vectors.  K, V and Q rows are padded by 4 floats: 8
// lanes that read 8 rows touch 32 different banks.  V comes during S, the next K
// during P V.  What bounds it is latency, with two warps a scheduler (an issue slot
// in three is used; the warps wait for shared memory and for the results of their own
// arithmetic): 40 sequences x 32 rows of 4 heads of 128 over 8192 shared positions and
// up to 700 of their own 604 us, 37 TFLOP/s of the 80 that FMAs alone could do; 16 x 32
// rows of 8 heads of 64, 2 kv heads, 289 us, 31 TFLOP/s.
//
// Units of at most 16 rows (a window's own keys, most often) take tiles of 16 rows,
// one a thread: 12 sequences x 8 rows of 4 heads of 64 over 2048 shared positions
// take 21 us so, 27 us with 64-row tiles for all; a single row over 32768 takes 35
// and 47 us.
#include "shared_attn.cuh"

namespace wedlm {
namespace {

constexpr int kSimtThreads = 256;
constexpr int kPRow = kSharedTile + 4;

__device__ __forceinline__ void cp_async16(float* dst, const float* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all groups but the newest are there
__device__ __forceinline__ void cp_wait_but_last() {
  asm volatile("cp.async.wait_group 1;" ::: "memory");
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}

template <int HD> constexpr int simt_smem_bytes() {
  return ((kSimtRows + 2 * kSharedTile) * (HD + 4) + kSimtRows * kPRow) * (int)sizeof(float);
}

// where a tile's pages lie (null: zeros), and the tokens of each that some row
// sees: of K, then of V
struct SimtPages {
  const float* src[2 * kSharedTilePages];
  int seen[2 * kSharedTilePages];
};

// One segment of a unit of up to 16 * RPT rows; thread (tx, ty) owns rows
// ty * RPT .. and keys tx + 16 j.
template <int HD, int RPT>
__device__ __forceinline__ void simt_segment(const SharedArgs& A, const SharedSeg& g, float* sm,
                                             SimtPages* s_pages) {
  constexpr int LD = HD + 4, ND = HD / 64;
  float* Qs = sm;                        // [64][LD], scaled
  float* Ks = Qs + kSimtRows * LD;       // [128][LD]
  float* Vs = Ks + kSharedTile * LD;     // [128][LD]
  float* Ps = Vs + kSharedTile * LD;     // [64][kPRow]
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int nq = A.nkv * A.G;
  const SeqSpan sp = g.sp;
  const int n_own = g.b < 0 ? 0 : own_pages(sp);
  const int own_keys = sp.len - sp.shared * kPageBlock;
  const int pages = g.b < 0 ? A.nsp : n_own + A.Wp / kPageBlock;
  const int urows = g.b < 0 ? A.srows : A.prows;
  const int all_rows = (g.b < 0 ? A.B : 1) * A.W * A.G;
  const int row0 = g.blk * urows, nrows = min(urows, all_rows - row0);
  const int tok0 = g.b < 0 ? 0 : g.b * A.W;
  // A tile's pages: their ids a phase ahead, then the addresses, which the copies of
  // the phase after find in shared memory
  auto id_of = [&](int t) -> int {
    const int j = t * kSharedTilePages + tid % kSharedTilePages;
    return tid < 2 * kSharedTilePages && t < g.t1 && j < (g.b < 0 ? pages : n_own)
               ? own_page_id(A, g.b, sp.shared, j)
               : -1;
  };
  auto put_pages = [&](int t, int id) {
    if (tid >= 2 * kSharedTilePages || t >= g.t1) return;
    const int kv = tid / kSharedTilePages, j = t * kSharedTilePages + tid % kSharedTilePages;
    const float* src = nullptr;
    int seen = kPageBlock;
    if (j >= pages) {
    } else if (g.b >= 0 && j >= n_own) {
      src = window_block<float>(A, g.b, j - n_own, kv, g.kvh, HD);
      seen = A.W - (j - n_own) * kPageBlock;
    } else {
      if (g.b >= 0) seen = own_keys - j * kPageBlock;
      if (id >= 0 && id < A.num_pages)
        src = cached_block<float>(A, id, kv, g.kvh, HD);
      else
        set_err(A.err, WEDLM_DEV_BAD_PAGE);
    }
    s_pages[t & 1].src[tid] = src;
    s_pages[t & 1].seen[tid] = seen;
  };
  // K or V of a tile, row-major; what no row sees becomes zeros
  auto copy = [&](int t, int kv) {
    constexpr int CH = kPageBlock * HD / 4;
    const SimtPages& pg = s_pages[t & 1];
#pragma unroll
    for (int i = 0; i < kSharedTilePages * CH / kSimtThreads; ++i) {
      const int e = tid + i * kSimtThreads, j = e / CH, el = e % CH * 4;
      const int tok = el / 64 / (HD / 8) * 8 + el % 64 / 8, d = el / 64 % (HD / 8) * 8 + el % 8;
      const float* src = pg.src[kv * kSharedTilePages + j];
      float* dst = (kv ? Vs : Ks) + (j * kPageBlock + tok) * LD + d;
      if (src && tok < pg.seen[kv * kSharedTilePages + j])
        cp_async16(dst, src + el);
      else
        *reinterpret_cast<float4*>(dst) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  const int first_id = id_of(g.t0);
  const float* q = static_cast<const float*>(A.q);
#pragma unroll
  for (int i = 0; i < 16 * RPT * HD / 4 / kSimtThreads; ++i) {
    const int e = tid + i * kSimtThreads, r = e / (HD / 4), d = e % (HD / 4) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < nrows) {
      const int row = row0 + r;
      v = *reinterpret_cast<const float4*>(
          q + ((size_t)(tok0 + row / A.G) * nq + g.kvh * A.G + row % A.G) * HD + d);
    }
    *reinterpret_cast<float4*>(Qs + r * LD + d) = make_float4(
        v.x * A.scale_log2, v.y * A.scale_log2, v.z * A.scale_log2, v.w * A.scale_log2);
  }
  float m[RPT], l[RPT];
  uint64_t o[RPT][2 * ND];  // pairs of dims
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < 2 * ND; ++j) o[i][j] = 0;
  }
  put_pages(g.t0, first_id);
  __syncthreads();
  copy(g.t0, 0);
  cp_commit();
  for (int t = g.t0; t < g.t1; ++t) {
    const int np = min(kSharedTilePages, pages - t * kSharedTilePages);
    const int k0 = t * kSharedTile, next_id = id_of(t + 1);
    copy(t, 1);  // on its way during S, as the next K is during P V
    cp_commit();
    cp_wait_but_last();
    __syncthreads();  // K (and Q) are there
    uint64_t s2[RPT][8];  // even and odd dims
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s2[i][j] = 0;
#pragma unroll 2
    for (int d = 0; d < HD; d += 4) {
      ulonglong2 qv[RPT], kv2[8];
#pragma unroll
      for (int i = 0; i < RPT; ++i)
        qv[i] = *reinterpret_cast<const ulonglong2*>(Qs + (ty * RPT + i) * LD + d);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        kv2[j] = *reinterpret_cast<const ulonglong2*>(Ks + (tx + 16 * j) * LD + d);
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s2[i][j] = fma2(qv[i].x, kv2[j].x, s2[i][j]);
          s2[i][j] = fma2(qv[i].y, kv2[j].y, s2[i][j]);
        }
    }
    float s[RPT][8];
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 e = unpack2(s2[i][j]);
        s[i][j] = e.x + e.y;
      }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int p_row = (row0 + ty * RPT + i) / A.G;
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int key = k0 + tx + 16 * j;
        bool ok = tx + 16 * j < np * kPageBlock;
        if (g.b >= 0) {
          const int w = key - n_own * kPageBlock;
          ok = ok && (w < 0 ? key < own_keys : w < A.W && w <= p_row);
        }
        if (!ok) s[i][j] = -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1)
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float mn = fmaxf(m[i], mx);
      const float base = mn == -INFINITY ? 0.f : mn;
      const float a = exp2f(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float p = exp2f(s[i][j] - base);
        sum += p;
        Ps[(ty * RPT + i) * kPRow + tx + 16 * j] = p;
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      l[i] = l[i] * a + sum;
      m[i] = mn;
#pragma unroll
      for (int j = 0; j < 2 * ND; ++j) o[i][j] = mul2(o[i][j], pack2(a, a));
    }
    put_pages(t + 1, next_id);
    __syncthreads();  // K has been read; P and the next tile's pages are there
    if (t + 1 < g.t1) copy(t + 1, 0);
    cp_commit();
    cp_wait_but_last();
    __syncthreads();  // V is there
#pragma unroll 2
    for (int k = 0; k < np * kPageBlock; k += 4) {
      float4 pv[RPT];
#pragma unroll
      for (int i = 0; i < RPT; ++i)
        pv[i] = *reinterpret_cast<const float4*>(Ps + (ty * RPT + i) * kPRow + k);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int j = 0; j < ND; ++j) {
          const ulonglong2 v =
              *reinterpret_cast<const ulonglong2*>(Vs + (k + kk) * LD + tx * 4 + 64 * j);
#pragma unroll
          for (int i = 0; i < RPT; ++i) {
            const float p = kk == 0 ? pv[i].x : kk == 1 ? pv[i].y : kk == 2 ? pv[i].z : pv[i].w;
            o[i][2 * j] = fma2(pack2(p, p), v.x, o[i][2 * j]);
            o[i][2 * j + 1] = fma2(pack2(p, p), v.y, o[i][2 * j + 1]);
          }
        }
    }
    __syncthreads();  // V and P have been read
  }
  if (tid == 0) record_unit(A, g);
  const size_t slot = seg_slot(A, g.unit, blockIdx.x);
  float4* po = (g.b < 0 ? A.part_s : A.part_p) + slot * urows * (HD / 4);
  float2* ml = (g.b < 0 ? A.ml_s : A.ml_p) + slot * urows;
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = ty * RPT + i;
    if (r >= nrows) continue;
#pragma unroll
    for (int j = 0; j < ND; ++j)
    {
      const float2 x = unpack2(o[i][2 * j]), y = unpack2(o[i][2 * j + 1]);
      po[(size_t)(tx + 16 * j) * urows + r] = make_float4(x.x, x.y, y.x, y.y);
    }
    if (tx == 0) ml[r] = make_float2(m[i], l[i]);
  }
}

template <int HD>
__global__ void __launch_bounds__(kSimtThreads)
shared_attn_simt_kernel(const __grid_constant__ SharedArgs A) {
  extern __shared__ __align__(16) float sm[];
  __shared__ SharedSeg s_seg;
  __shared__ bool s_more;
  __shared__ SimtPages s_pages[2];
  pdl_wait();
  pdl_trigger();
  SharedWalk walk;
  if (threadIdx.x < 32) walk.init(A);
  while (true) {
    if (threadIdx.x < 32) {
      SharedSeg next;
      const bool more = walk.next(A, next);
      if (threadIdx.x == 0) {
        s_seg = next;
        s_more = more;
      }
    }
    __syncthreads();  // also: the previous segment is done with shared memory
    if (!s_more) break;
    const SharedSeg g = s_seg;
    if ((g.b < 0 ? A.srows : A.prows) <= kSimtFewRows)
      simt_segment<HD, 1>(A, g, sm, s_pages);
    else
      simt_segment<HD, 4>(A, g, sm, s_pages);
  }
}

// The merge: row r of kv head kvh joins the partials of its shared unit (when
// its sequence takes part) and of its private unit, in slot order.  A block takes
// RPB rows; a warp 16 dims of them: 32 / RPB groups of lanes share a row's
// partials out among them and load four at a time with a running maximum, so that
// few rows with many partials do not wait for them one by one (one token of 8
// heads over 32768 shared positions, 150 partials a row: 23 us for the whole call
// with a load at a time, 16 so).  Where rows abound, two at a time leave registers
// for a third block per SM (3 us of 64 x 32 rows over 16384).  Partials lie
// dims-major, so that both the writer's warps (a lane per row) and these loads touch
// runs of rows.
template <typename T, int HD, int RPB>
__global__ void __launch_bounds__(2 * HD) shared_merge_kernel(const __grid_constant__ SharedArgs A) {
  constexpr int NG = 32 / RPB;           // lane groups of a row
  constexpr int PF = RPB == 8 ? 4 : 2;   // partials loaded together
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, d40 = threadIdx.x / 32 * 4;
  const int kvh = blockIdx.y, rows = A.B * A.W * A.G;
  const int grp = lane / RPB;
  const int r = blockIdx.x * RPB + lane % RPB;
  const bool row = r < rows;
  const int rr = row ? r : 0;
  const int tok = rr / A.G, b = tok / A.W, pr = rr - b * A.W * A.G;
  const int us = kvh * A.sblocks + rr / A.srows, is = rr % A.srows;
  const int up = A.nkv * A.sblocks + (b * A.nkv + kvh) * A.pblocks + pr / A.prows;
  const int ip = pr % A.prows;
  // clamped: after a wait that expired the records may be missing
  int2 bs = A.unit_blocks[us], bp = A.unit_blocks[up];
  bs.x = max(0, min(bs.x, A.grid - 1));
  bp.x = max(0, min(bp.x, A.grid - 1));
  const int ns = seq_span(A, b).shared ? max(0, min(bs.y, A.grid - 1) - bs.x + 1) : 0;
  const int n = row ? ns + max(0, min(bp.y, A.grid - 1) - bp.x + 1) : 0;
  const float2* ml_s = A.ml_s + (size_t)seg_slot(A, us, bs.x) * A.srows + is;
  const float2* ml_p = A.ml_p + (size_t)seg_slot(A, up, bp.x) * A.prows + ip;
  const float4* o_s = A.part_s + ((size_t)seg_slot(A, us, bs.x) * (HD / 4) + d40) * A.srows + is;
  const float4* o_p = A.part_p + ((size_t)seg_slot(A, up, bp.x) * (HD / 4) + d40) * A.prows + ip;
  // PF of this lane's partials from i0 on (none: a sum of 0)
  float2 ml[PF];
  float4 v[PF][4];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int c = 0; c < PF; ++c) {
      const int i = i0 + c * NG;
      ml[c] = make_float2(-INFINITY, 0.f);
      if (i >= n) continue;
      const bool sh = i < ns;
      const int st = sh ? A.srows : A.prows, q = sh ? i : i - ns;
      const float4* src = (sh ? o_s : o_p) + (size_t)q * (HD / 4) * st;
      ml[c] = (sh ? ml_s : ml_p)[(size_t)q * st];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[c][k] = src[(size_t)k * st];
    }
  };
  float M = -INFINITY, l = 0.f, acc[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) acc[k] = 0.f;
  // O and l from maximum M to another one
  auto raise = [&](float to) {
    const float f = M == -INFINITY ? 0.f : exp2f(M - to);
    l *= f;
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] *= f;
    M = to;
  };
#pragma unroll 1
  for (int i = grp; i < n; i += PF * NG) {
    fetch(i);
    float to = M;
#pragma unroll
    for (int c = 0; c < PF; ++c) to = fmaxf(to, ml[c].x);
    raise(to);
#pragma unroll
    for (int c = 0; c < PF; ++c) {
      if (ml[c].y == 0.f) continue;  // no key seen (keys that are all NaN leave l NaN)
      const float w = exp2f(ml[c].x - M);
      l = fmaf(ml[c].y, w, l);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        acc[4 * k] = fmaf(v[c][k].x, w, acc[4 * k]);
        acc[4 * k + 1] = fmaf(v[c][k].y, w, acc[4 * k + 1]);
        acc[4 * k + 2] = fmaf(v[c][k].z, w, acc[4 * k + 2]);
        acc[4 * k + 3] = fmaf(v[c][k].w, w, acc[4 * k + 3]);
      }
    }
  }
  if (NG > 1) {
    float all = M;
#pragma unroll
    for (int o = RPB; o < 32; o <<= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
    raise(all);
  }
#pragma unroll
  for (int o = RPB; o < 32; o <<= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] += __shfl_xor_sync(0xffffffffu, acc[k], o);
  }
  if (!row || grp) return;
  const float inv = 1.f / l;  // a window row sees itself: l > 0
  T* dst = static_cast<T*>(A.o) +
           ((size_t)tok * A.nkv * A.G + kvh * A.G + r % A.G) * HD + d40 * 4;
  constexpr int N = Vec16<T>::N;
#pragma unroll
  for (int k = 0; k < 16; k += N) {
    Vec16<T> v;
#pragma unroll
    for (int i = 0; i < N; ++i) v.set(i, acc[k + i] * inv);
    st16(dst + k, v);
  }
}

template <int HD>
cudaError_t launch_simt(const SharedArgs& A, cudaStream_t st) {
  constexpr int smem = simt_smem_bytes<HD>();
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = raise_smem(done, (const void*)shared_attn_simt_kernel<HD>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(shared_attn_simt_kernel<HD>, dim3(A.grid), dim3(kSimtThreads), smem, st, A);
}

template <typename T, int HD>
cudaError_t launch_merge(const SharedArgs& A, cudaStream_t st) {
  const int rows = A.B * A.W * A.G;
  // 8 rows a block while that leaves the GPU room, 32 (whole 512-byte runs) beyond.
  // Whole calls with 8 and with 32, by rows of all kv heads, us:
  //                                   2048       4096       6144       8192      16384
  //   heads of 128, 256 shared    13.8 15.7  16.0 15.6  17.8 16.0  19.6 16.3  32.6 23.5
  //   heads of 128, 8192 shared   22.0 31.1  29.4 32.8  36.9 36.7  45.5 43.3  76.2 68.0
  //   heads of 64, 256 shared     12.3 13.3  12.5 13.6  14.1 13.6  14.4 13.6  22.5 18.7
  //   heads of 64, 8192 shared    18.5 24.2  23.6 26.9  30.7 31.5  37.2 37.3  63.7 60.9
  if ((long long)rows * A.nkv <= 6 * 1024)
    return launch_pdl(shared_merge_kernel<T, HD, 8>, dim3((rows + 7) / 8, A.nkv), dim3(2 * HD), 0,
                      st, A);
  return launch_pdl(shared_merge_kernel<T, HD, 32>, dim3((rows + 31) / 32, A.nkv), dim3(2 * HD), 0,
                    st, A);
}

}  // namespace

cudaError_t launch_shared_attention_simt(const SharedArgs& A, int hd, cudaStream_t st) {
  return hd == 128 ? launch_simt<128>(A, st) : launch_simt<64>(A, st);
}

cudaError_t launch_shared_merge(const SharedArgs& A, int hd, bool is_bf16, cudaStream_t st) {
  if (is_bf16) return hd == 128 ? launch_merge<bf16, 128>(A, st) : launch_merge<bf16, 64>(A, st);
  return hd == 128 ? launch_merge<float, 128>(A, st) : launch_merge<float, 64>(A, st);
}

}  // namespace wedlm
