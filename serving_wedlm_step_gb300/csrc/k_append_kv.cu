// Appending keys and values to the paged cache, with the per-head RMSNorm
// and the rotate-half RoPE at logical positions (WeDLM summary page, Key
// claims §4.1) applied on the way.
//
//   x~ = x * rsqrt(mean(x^2) + eps) * gain                    (optional)
//   y[i] = x~[i] c - x~[i + hd/2] s,  y[i + hd/2] = x~[i + hd/2] c + x~[i] s
//   c, s = cos, sin(t * theta^(-2i/hd)),  0 <= i < hd/2, t the logical position
//
// The angle is kept in turns, as a 64-bit fraction: step[i] = theta^(-2i/hd)
// / 2 pi * 2^64, and t * step[i] modulo 2^64 is the fraction of a turn left
// after the whole ones, exact for any t (a phase accumulator).  Its top 32
// bits go through sincospif, so far positions lose nothing and no 64-bit
// floating point runs on the device.
//
// A thread holds 8 dims of the first half of a head and the 8 they rotate
// with, for one row; a warp covers 4 rows (head_dim 128) or 8 (64), so a row's
// head is read in whole 128-byte (64-byte) runs and 4 (8) neighbouring rows
// fill neighbouring 16-byte slots of the 8x8 tiles in the cache.  The thread
// computes its 8 angles once and walks over a run of heads with them.
#include <math.h>

#include <algorithm>

#include "internal.h"

namespace wedlm {
namespace {

constexpr int kAppendThreads = 128;

struct AppendArgs {
  int B, n, np;              // np: rows walked per sequence (n, or Wp with kv_win)
  int nq, nkv, heads;        // heads: nq (0 without q) + 2 nkv
  int heads_per_block;
  int max_pages, num_pages, Wp;
  float eps;
  wedlm_rows k, v, q;
  const void *q_norm, *k_norm;
  const int32_t *pos, *counts, *seq_len, *page_table;
  void *pool, *q_out, *kv_win;
  int32_t* new_seq_len;
  int* err;
  uint64_t step[64];         // angle per position, in 2^-64 turns
};

// 8 consecutive values
template <typename T> struct Vec8 {
  static constexpr int R = 8 * sizeof(T) / 16;
  uint4 raw[R];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < R; ++i) raw[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < R; ++i) reinterpret_cast<uint4*>(p)[i] = raw[i];
  }
  __device__ __forceinline__ float get(int i) const {
    return to_f(reinterpret_cast<const T*>(raw)[i]);
  }
  __device__ __forceinline__ void set(int i, float v) {
    reinterpret_cast<T*>(raw)[i] = from_f<T>(v);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < R; ++i) raw[i] = make_uint4(0, 0, 0, 0);
  }
};

template <typename T, int HD>
__global__ void __launch_bounds__(kAppendThreads)
append_kv_kernel(const __grid_constant__ AppendArgs A) {
  constexpr int DG = HD / 16;            // threads of one row
  constexpr int RW = 32 / DG;            // rows of a warp
  constexpr int RB = kAppendThreads / DG;
  __shared__ uint64_t s_step[HD / 2];
  if (threadIdx.x < HD / 2) s_step[threadIdx.x] = A.step[threadIdx.x];
  // The rows and lengths come from earlier kernels.  No pdl_trigger: nothing
  // starts before the pages and lengths written here are there.
  pdl_wait();
  __syncthreads();

  const int cap = A.max_pages * kPageBlock;  // bounded by the host check
  if (A.new_seq_len && blockIdx.x == 0 && blockIdx.y == 0) {
    for (int b = threadIdx.x; b < A.B; b += kAppendThreads) {
      const int L = A.seq_len[b];
      const int c = A.counts ? max(0, min(A.counts[b], A.n)) : A.n;
      A.new_seq_len[b] = L < 0 ? L : (int)max((long long)L, min((long long)L + c, (long long)cap));
    }
  }

  const int lane = threadIdx.x & 31, dg = lane % DG;
  const long long m = (long long)blockIdx.x * RB + threadIdx.x / 32 * RW + lane / DG;
  const bool live = m < (long long)A.B * A.np;  // no early exit: shuffles below
  const int b = live ? (int)(m / A.np) : 0, p = live ? (int)(m % A.np) : 0;
  const bool row = live && p < A.n;             // else a pad row of the window block
  int L = A.seq_len[b];
  int count = A.counts ? A.counts[b] : A.n;
  const bool tell = live && p == 0 && dg == 0 && blockIdx.y == 0;
  if (L < 0 || count < 0 || count > A.n) {
    if (tell) set_err(A.err, WEDLM_DEV_BAD_SEQLEN);
    if (L < 0) count = 0;
    count = max(0, min(count, A.n));
    L = max(0, L);
  }
  // the cache block of this row (its K of kv head 0), or null
  T* page = nullptr;
  const long long s = (long long)L + p;
  if (row && p < count) {
    if (s >= cap) {
      if (dg == 0 && blockIdx.y == 0) set_err(A.err, WEDLM_DEV_CAPACITY);
    } else {
      const int id = A.page_table[(size_t)b * A.max_pages + (int)s / kPageBlock];
      if (id < 0 || id >= A.num_pages) {
        if (dg == 0 && blockIdx.y == 0) set_err(A.err, WEDLM_DEV_BAD_PAGE);
      } else {
        page = static_cast<T*>(A.pool) + (size_t)id * 2 * A.nkv * kPageBlock * HD;
      }
    }
  }
  T* win = live && A.kv_win
               ? static_cast<T*>(A.kv_win) + (size_t)b * 2 * A.nkv * A.Wp * HD
               : nullptr;
  const bool kv_row = page || win;

  const int h0 = blockIdx.y * A.heads_per_block;
  const int h1 = min(A.heads, h0 + A.heads_per_block);
  float cs[8], sn[8];
  if (h0 < A.heads - A.nkv) {  // some head of the run rotates
    // 64 bits: a length of nearly 2^31 plus p passes 32
    const long long t = !row ? 0 : A.pos ? A.pos[(size_t)b * A.n + p] : s;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint64_t turn = (uint64_t)t * s_step[dg * 8 + j];
      // the top 32 bits as a signed fraction of a turn: 2 * it half turns
      sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn[j], &cs[j]);
    }
  }
  const int toff = tile_off((int)(s % kPageBlock), dg * 8, HD), thalf = HD / 2 * 8;
  const int woff = tile_off(p, dg * 8, HD);
  // 0: q, 1: k, 2: v, and the head's index within it
  auto kind_of = [&](int h, int& hh) {
    const int kind = h < A.nq ? 0 : h < A.nq + A.nkv ? 1 : 2;
    hh = kind == 0 ? h : kind == 1 ? h - A.nq : h - A.nq - A.nkv;
    return kind;
  };
  auto load = [&](int h, Vec8<T>& x1, Vec8<T>& x2) {
    int hh;
    const int kind = kind_of(h, hh);
    const wedlm_rows& R = kind == 0 ? A.q : kind == 1 ? A.k : A.v;
    if (row && (kind == 0 || kv_row)) {
      const T* src = static_cast<const T*>(R.ptr) + (int64_t)b * R.batch_stride +
                     (int64_t)p * R.row_stride + (int64_t)hh * R.head_stride + dg * 8;
      x1.load(src);
      x2.load(src + HD / 2);
    } else {
      x1.zero();
      x2.zero();
    }
  };
  Vec8<T> n1, n2;
  load(h0, n1, n2);
  for (int h = h0; h < h1; ++h) {
    int hh;
    const int kind = kind_of(h, hh);
    Vec8<T> x1 = n1, x2 = n2;
    if (h + 1 < h1) load(h + 1, n1, n2);  // in flight while this head is turned
    if (kind < 2) {
      float a[8], c[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[j] = x1.get(j);
        c[j] = x2.get(j);
      }
      const T* g = static_cast<const T*>(kind == 0 ? A.q_norm : A.k_norm);
      if (g) {  // the same for the block: every lane takes part in the shuffles
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(a[j], a[j], fmaf(c[j], c[j], ss));
#pragma unroll
        for (int o = DG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss * (1.f / HD) + A.eps);
        Vec8<T> g1, g2;
        g1.load(g + dg * 8);
        g2.load(g + HD / 2 + dg * 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          a[j] = a[j] * r * g1.get(j);
          c[j] = c[j] * r * g2.get(j);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x1.set(j, a[j] * cs[j] - c[j] * sn[j]);
        x2.set(j, c[j] * cs[j] + a[j] * sn[j]);
      }
      if (!row) {  // neither eps = 0 nor the gain makes a pad row NaN
        x1.zero();
        x2.zero();
      }
    }
    if (kind == 0) {
      if (row) {
        T* dst = static_cast<T*>(A.q_out) + (((size_t)b * A.n + p) * A.nq + hh) * HD + dg * 8;
        x1.store(dst);
        x2.store(dst + HD / 2);
      }
    } else {
      const size_t blk = (size_t)(kind - 1) * A.nkv + hh;
      if (win) {
        T* dst = win + blk * A.Wp * HD + woff;
        x1.store(dst);
        x2.store(dst + thalf);
      }
      if (page) {
        T* dst = page + blk * kPageBlock * HD + toff;
        x1.store(dst);
        x2.store(dst + thalf);
      }
    }
  }
}

bool bad_rows(const wedlm_rows& r, int es) {
  const int64_t a = 16 / es;
  return !r.ptr || (reinterpret_cast<uintptr_t>(r.ptr) & 15) || r.batch_stride < 0 ||
         r.row_stride < 0 || r.head_stride < 0 || r.batch_stride % a || r.row_stride % a ||
         r.head_stride % a;
}

}  // namespace
}  // namespace wedlm

using namespace wedlm;

extern "C" int wedlm_append_kv(const wedlm_append_args* a, void* stream) {
  if (!a) return WEDLM_ERR_INVALID_ARG;
  auto bad16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; };
  auto bad4 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) != 0; };
  if ((a->dtype != WEDLM_BF16 && a->dtype != WEDLM_FP32) ||
      (a->head_dim != 64 && a->head_dim != 128) || a->batch < 1 || a->rows < 1 ||
      (int64_t)a->batch * a->rows > INT32_MAX || a->n_kv_heads < 1 || a->n_kv_heads > 8192 ||
      a->max_pages_per_seq < 1 || a->max_pages_per_seq > INT32_MAX / kPageBlock ||
      a->num_pages < 1 || !(a->rope_theta >= 1.f) || !isfinite(a->rope_theta) ||
      !(a->rms_eps >= 0.f) || !isfinite(a->rms_eps) || !a->seq_len || !a->page_table ||
      !a->kv_pool || bad16(a->kv_pool) || bad16(a->kv_win) || bad16(a->q_out) ||
      bad16(a->q_norm) || bad16(a->k_norm) || bad4(a->pos) || bad4(a->counts) ||
      bad4(a->seq_len) || bad4(a->page_table) || bad4(a->new_seq_len) || bad4(a->error) ||
      (a->kv_win && a->rows > kMaxWindow))
    return WEDLM_ERR_INVALID_ARG;
  const int es = a->dtype == WEDLM_BF16 ? 2 : 4;
  const bool has_q = a->q.ptr != nullptr;
  if (bad_rows(a->k, es) || bad_rows(a->v, es) || has_q != (a->q_out != nullptr) ||
      (!has_q && a->q_norm) ||
      (has_q && (bad_rows(a->q, es) || a->n_q_heads < 1 || a->n_q_heads > 8192)))
    return WEDLM_ERR_INVALID_ARG;
  // one block writes new_seq_len while the others still read
  auto meets = [&](const int32_t* p, int64_t n) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a->new_seq_len), y = reinterpret_cast<uintptr_t>(p);
    return x && y && x < y + 4 * (uintptr_t)n && y < x + 4 * (uintptr_t)a->batch;
  };
  if (meets(a->seq_len, a->batch) || meets(a->counts, a->batch) ||
      meets(a->pos, (int64_t)a->batch * a->rows) ||
      meets(a->page_table, (int64_t)a->batch * a->max_pages_per_seq))
    return WEDLM_ERR_INVALID_ARG;
  AppendArgs A;
  A.B = a->batch;
  A.n = a->rows;
  A.Wp = (a->rows + kPageBlock - 1) / kPageBlock * kPageBlock;
  A.np = a->kv_win ? A.Wp : A.n;
  A.nq = has_q ? a->n_q_heads : 0;
  A.nkv = a->n_kv_heads;
  A.heads = A.nq + 2 * A.nkv;
  A.max_pages = a->max_pages_per_seq;
  A.num_pages = a->num_pages;
  A.eps = a->rms_eps;
  A.k = a->k;
  A.v = a->v;
  A.q = a->q;
  A.q_norm = a->q_norm;
  A.k_norm = a->k_norm;
  A.pos = a->pos;
  A.counts = a->counts;
  A.seq_len = a->seq_len;
  A.page_table = a->page_table;
  A.pool = a->kv_pool;
  A.q_out = a->q_out;
  A.kv_win = a->kv_win;
  A.new_seq_len = a->new_seq_len;
  A.err = a->error;
  const int half = a->head_dim / 2;
  for (int i = 0; i < half; ++i) {
    const double turns = pow((double)a->rope_theta, -2.0 * i / a->head_dim) / 6.283185307179586;
    A.step[i] = (uint64_t)(turns * 18446744073709551616.0);  // < 0.16 turns
  }
  const int rb = kAppendThreads * 16 / a->head_dim;
  const int64_t gx = ((int64_t)A.B * A.np + rb - 1) / rb;
  if (gx > INT32_MAX) return WEDLM_ERR_INVALID_ARG;
  // A block walks over a run of heads with one set of angles.  Long runs spare
  // angles; but while the row blocks alone leave the GPU idle the runs are cut, for
  // a block's time is its run's latency: one token of 32 + 8 + 8 heads took 23 us
  // in one run.  8 blocks an SM are about what is resident (7 in bf16 with 72
  // registers, 5 in fp32 with 91).
  const int sms = device_sms();
  if (sms < 1) return WEDLM_ERR_CUDA;
  const int64_t want = 8 * (int64_t)sms;
  A.heads_per_block = (int)std::max<int64_t>(1, std::min<int64_t>(A.heads, A.heads * gx / want));
  const int gy = (A.heads + A.heads_per_block - 1) / A.heads_per_block;
  if (gy > 65535) return WEDLM_ERR_INVALID_ARG;
  dim3 grid((unsigned)gx, (unsigned)gy);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a->dtype == WEDLM_BF16)
    e = a->head_dim == 128 ? launch_pdl(append_kv_kernel<bf16, 128>, grid, dim3(kAppendThreads), 0, st, A)
                           : launch_pdl(append_kv_kernel<bf16, 64>, grid, dim3(kAppendThreads), 0, st, A);
  else
    e = a->head_dim == 128 ? launch_pdl(append_kv_kernel<float, 128>, grid, dim3(kAppendThreads), 0, st, A)
                           : launch_pdl(append_kv_kernel<float, 64>, grid, dim3(kAppendThreads), 0, st, A);
  return e == cudaSuccess ? WEDLM_OK : WEDLM_ERR_CUDA;
}
