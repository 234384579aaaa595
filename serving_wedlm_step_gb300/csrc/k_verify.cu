// Verification of drafted tokens against a target's logits.
//
//   p_i = softmax(z_i / T);  draft i holds while u_i q_i(x_i) < p_i(x_i);
//   r the first that does not (or n): w = max(0, p_r - q_r), or p_n;
//   token = the lowest v with  w_0 + .. + w_v > u (w_0 + .. + w_{V-1})
//
// One kernel reads every row once and leaves, per span of it, the largest logit
// and the sum of exponentials.  A second one, a cluster of blocks per sequence,
// joins a sequence's spans, accepts or rejects its drafts and draws from one row.  Where a
// sequence has few spans the second kernel reads them itself.
//
// A draw by sums over the vocabulary has a border between any two tokens, and an
// error of the sums moves all of them: with 32-bit sums some draws would depend on
// the order of summation.  The weights are therefore
// whole multiples of 2^-42 of the largest, whose sums are exact in any order, and
// their exponential is good to 2^-29, 2^-32 on average: 2^(n + j/64) (1 + x), with
// 2^(j/64) from a table and x = 2^(G/64) - 1, |G| <= 1/2, by three terms of its
// series.  All of it in pairs of 32-bit floating point.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "internal.h"

namespace wedlm {
namespace {

constexpr int kMaxDrafts = 64;
constexpr int kMaxVocab = 1 << 20;
constexpr int kGroup = 8;                     // logits of a thread's load in the draw
constexpr int kStatWarps = 4;                 // of a block, a span each
constexpr int kStatVecs = 4;                  // 16-byte loads of a thread in flight
constexpr int kMaxRounds = 5;                 // of such loads, in a span
constexpr int kManyWarps = 152 * 32;          // a GB300 half full of them; fixed, so that the
                                              // workspace is the same for every device
// Spans of a sequence, one a warp, up to which one kernel does it all: 5 x 3 drafts over 1024
// tokens 6.1 us captured and 10.4 a call, not 6.8 and 12.1; with 32 spans and more the second
// round of them costs what the launch does
constexpr int kFewSpans = 16;
// Two blocks of the draw an SM.  Swept on GB300 (15 drafts over 151936 tokens, 32 x 7 with
// probabilities, 64 x 15, captured): 10.7, 39.5 and 66.8 us with these, 384 threads 12.1, 39.7
// and 68.4, 640 10.6, 41.5 and 68.1, four blocks of 256 11.8, 48.1 and 78.9, one of 512 10.9,
// 45.1 and 73.7, one of 1024 12.7, 50.0 and 73.4.
constexpr int kPickThreads = 512;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kMaxCluster = 8, kWideCluster = 16;  // the latter where the GPU has room for it
constexpr int kMaxGroups = 12288;             // of a block: their sums are 96 KB
constexpr float kMinTemp = 1e-30f, kMaxTemp = 1e18f;

// a span's largest logit, the sum of 2^(c z - c m), and for greedy draws the
// place of m
struct __align__(16) SpanStat {
  float m, s;
  int at, unused;
};

// 2^(j/64) as a float, and what that lacks of it, relative to it
static __device__ const float2 kPow[64] = {
    {1.f, 0.f}, {1.01088929f, -5.65007996e-09f}, {1.0218972f, -4.70845762e-08f},
    {1.03302491f, -2.71928524e-08f}, {1.04427373f, 4.62854715e-08f},
    {1.05564523f, -4.64850238e-08f}, {1.06714046f, -5.56042252e-08f},
    {1.07876074f, 5.06284152e-08f}, {1.09050775f, -1.19921575e-08f}, {1.10238254f, 3.86481283e-08f},
    {1.1143868f, -4.87760623e-08f}, {1.12652159f, 2.77282002e-08f}, {1.13878858f, 4.72978243e-08f},
    {1.15118921f, 1.90431617e-08f}, {1.1637249f, -3.48144269e-08f}, {1.17639697f, 2.18206537e-08f},
    {1.18920708f, 3.19341815e-08f}, {1.20215678f, -4.21721751e-08f},
    {1.21524739f, -2.68866653e-08f}, {1.22848058f, -3.36692345e-08f},
    {1.24185777f, 3.62105723e-08f}, {1.25538075f, 5.83268278e-09f}, {1.26905096f, 1.11842102e-09f},
    {1.28287005f, -2.97506499e-08f}, {1.29683959f, -3.09907193e-08f},
    {1.31096125f, -2.66718132e-08f}, {1.32523668f, -2.63830096e-08f},
    {1.33966756f, -2.58397996e-08f}, {1.35425556f, -7.47521334e-09f},
    {1.36900246f, -2.8092586e-08f}, {1.38390994f, -4.24563567e-08f}, {1.39897966f, 6.21126572e-09f},
    {1.41421354f, 1.71142709e-08f}, {1.42961335f, -9.39409883e-09f}, {1.44518077f, 2.30019666e-08f},
    {1.46091783f, -2.48382062e-08f}, {1.47682619f, -3.04768335e-08f},
    {1.49290776f, -2.29325625e-08f}, {1.50916445f, -1.65385377e-08f},
    {1.52559817f, -1.15551853e-08f}, {1.54221082f, 5.23333421e-09f},
    {1.55900443f, -1.65263589e-08f}, {1.5759809f, -3.5920646e-08f}, {1.59314215f, -3.07765174e-10f},
    {1.61049032f, 6.10759177e-09f}, {1.62802744f, -1.06018385e-08f},
    {1.64575553f, -3.11405444e-08f}, {1.66367662f, -2.3564068e-08f},
    {1.68179286f, -1.47196051e-08f}, {1.70010638f, -1.68527521e-08f},
    {1.71861935f, -2.82181016e-08f}, {1.73733389f, -3.36735688e-08f},
    {1.75625217f, -5.25879518e-09f}, {1.77537644f, 3.00961389e-08f},
    {1.79470909f, -6.36038733e-09f}, {1.81425214f, 2.05939301e-08f}, {1.8340081f, -6.12825968e-09f},
    {1.85397911f, 7.74852982e-09f}, {1.87416768f, -2.48804088e-08f}, {1.89457595f, 1.4833601e-08f},
    {1.91520655f, 5.14060927e-09f}, {1.93606174f, 2.76699463e-08f}, {1.95714414f, -8.69726691e-09f},
    {1.97845602f, 3.04920933e-09f},
};

// the same for Weigher: the float's bits less j << 17.  Apart, so that what two tokens need
// loads into neighbouring registers.
struct Pow {
  int hi[64];
  float lo[64];
};

struct VerifyArgs {
  int B, K, V, rounds, spans, cluster, groups_per_block, mask_id;
  const void* logits;
  int64_t batch_stride, row_stride;
  const int32_t* tokens;
  const float *draft_probs, *temperature, *accept_u, *sample_u;
  const int32_t* n_drafts;
  int32_t *n_accepted, *out_tokens;
  float *draft_p, *sampled_p;
  SpanStat* stats;  // [B * (K + 1)][spans]
  int* err;
};

// ---------------------------------------------------------------------------
// two floats at a time
// ---------------------------------------------------------------------------
__device__ __forceinline__ float2 two(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  return __fadd2_rn(a, make_float2(-b.x, -b.y));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// log2(e) / T, within one rounding of the quotient: __fdividef, then a step of Newton's
// iteration for the root of a / x - T, x + x (a - x T) / a (a division in its place costs
// 64 x 15 drafts over 151936 tokens 1.5 us of 65.5).  For a greedy draw T does not matter.
// NaN for a temperature out of range, which makes every statistic NaN.
__device__ __forceinline__ float log2_scale(float t, bool& greedy) {
  greedy = t == 0.f;
  const bool in_range = greedy | ((t >= kMinTemp) & (t <= kMaxTemp));
  const float x = __fdividef(1.44269502f, t);
  const float c = fmaf(fmaf(-x, t, 1.44269502f), x * 0.693147182f, x);
  return in_range ? (greedy ? 1.44269502f : c) : __int_as_float(0x7fc00000);
}

// What a sum's exponents are relative to: c m rounded.  The rounding is the same
// wherever it is used, so that it cancels (no fused multiply-add takes part in it).
__device__ __forceinline__ float ref_point(float m, float c) {
  return m == -INFINITY ? 0.f : __fmul_rn(m, c);
}

// elements of a row before its first 16-byte boundary, counted back from it: the
// first group starts at -lead
template <typename T>
__device__ __forceinline__ int lead_of(const T* row) {
  return (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
}

template <typename T>
__device__ __forceinline__ const T* row_of(const VerifyArgs& A, int b, int i) {
  return static_cast<const T*>(A.logits) + b * A.batch_stride + i * A.row_stride;
}

__device__ __forceinline__ int drafts_of(const VerifyArgs& A, int b) {
  return A.n_drafts ? max(0, min(A.n_drafts[b], A.K)) : A.K;
}

// ---------------------------------------------------------------------------
// a span of a row
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t word(const uint4& v, int k) {
  return k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w;
}
__device__ __forceinline__ uint32_t bits_of(float x) { return __float_as_uint(x); }
__device__ __forceinline__ uint32_t bits_of(bf16 x) { return __bfloat16_as_ushort(x); }

// 16 bytes of logits of a row from element e on (e may lie before the row or reach past
// it), -inf outside 0..V-1 and at tokens `mask` and `out`.  e is such that the address is a
// multiple of 16.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T* row, int e, int V, int mask, int out = -1) {
  constexpr int N = 16 / sizeof(T), kPer = 4 / sizeof(T);
  if (e >= 0 && e + N <= V && (unsigned)(mask - e) >= (unsigned)N && (unsigned)(out - e) >= (unsigned)N)
    return __ldg(reinterpret_cast<const uint4*>(row + e));
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    w[k] = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = e + k * kPer + i;
      const bool has = t >= 0 && t < V && t != mask && t != out;
      w[k] |= bits_of(has ? row[t] : from_f<T>(-INFINITY)) << (16 * i);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// two neighbouring logits of a vector: word k of 4 (bf16), words 2k and 2k + 1 (fp32)
__device__ __forceinline__ float2 pair_of(const uint4& v, int k, bf16) {
  const uint32_t w = word(v, k);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_of(const uint4& v, int k, float) {
  return make_float2(__uint_as_float(word(v, 2 * k)), __uint_as_float(word(v, 2 * k + 1)));
}

// the largest of kStatVecs vectors (a NaN counts for nothing)
__device__ __forceinline__ float max_of(const uint4* v, bf16) {
  uint32_t m = v[0].x;
#pragma unroll
  for (int k = 1; k < 4 * kStatVecs; ++k)
    asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(word(v[k / 4], k % 4)));
  return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}
__device__ __forceinline__ float max_of(const uint4* v, float) {
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < 4 * kStatVecs; ++k) m = fmaxf(m, __uint_as_float(word(v[k / 4], k % 4)));
  return m;
}

// A warp's: no barrier, and no exchange before the end.  Each thread's sum is relative to
// its own running maximum.
template <typename T>
__device__ __forceinline__ SpanStat span_stat(const VerifyArgs& A, const T* row, int span, float c,
                                              bool greedy) {
  constexpr int N = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  int e = span * A.rounds * kStatVecs * 32 * N + lane * N - lead_of(row);
  constexpr int kRound = kStatVecs * 32 * N;
  auto fetch = [&](uint4* v) {
    const int w = e - lane * N;  // the warp's first element; mostly all of its are in the row
    if (w >= 0 && w + kRound <= A.V && (unsigned)(A.mask_id - w) >= (unsigned)kRound) {
#pragma unroll
      for (int k = 0; k < kStatVecs; ++k)
        v[k] = __ldg(reinterpret_cast<const uint4*>(row + e) + k * 32);
    } else {
#pragma unroll
      for (int k = 0; k < kStatVecs; ++k) v[k] = load_vec(row, e + k * 32 * N, A.V, A.mask_id);
    }
  };
  float m = -INFINITY, s = 0.f, y0 = 0.f;
  int at = INT32_MAX;
  auto sum = [&](const uint4* v, int e_now) {
    float mr = max_of(v, T());
    // a lowest value as a mask: c mr is -inf, and so no reference point
    if (__fmul_rn(mr, c) == -INFINITY) mr = -INFINITY;
    if (greedy && mr > m) {
#pragma unroll
      for (int k = kStatVecs * N / 2 - 1; k >= 0; --k) {  // the lowest of equals last
        const float2 z = pair_of(v[k / (N / 2)], k % (N / 2), T());
        const int t = e_now + k / (N / 2) * 32 * N + k % (N / 2) * 2;
        at = z.x == mr ? t : z.y == mr ? t + 1 : at;
      }
    }
    // a sum of nothing (or of NaN) has no reference point yet
    const float m1 = fmaxf(m, mr), y1 = ref_point(m1, c);
    if (m != -INFINITY) s *= ex2(y0 - y1);
    m = m1;
    y0 = y1;
    const float2 cc = two(c), ny = two(-y1);
    float2 t = make_float2(s, 0.f), u = two(0.f);
#pragma unroll
    for (int k = 0; k < kStatVecs; ++k)
#pragma unroll
      for (int h = 0; h < N / 2; ++h) {
        const float2 y = fma2(pair_of(v[k], h, T()), cc, ny);
        const float2 ex = make_float2(ex2(y.x), ex2(y.y));
        if (h & 1) u = add2(u, ex);
        else t = add2(t, ex);
      }
    t = add2(t, u);
    s = t.x + t.y;
  };
  // one round in flight while the one before it is summed
  uint4 va[kStatVecs], vb[kStatVecs];
  fetch(va);
  for (int round = 0; round < A.rounds; round += 2) {
    const int e0 = e;
    e += kRound;
    if (round + 1 < A.rounds) fetch(vb);
    sum(va, e0);
    if (round + 1 == A.rounds) break;
    const int e1 = e;
    e += kRound;
    if (round + 2 < A.rounds) fetch(va);
    sum(vb, e1);
  }
  const float mw = warp_max(m);
  if (m != -INFINITY) s *= ex2(y0 - ref_point(mw, c));
  s = warp_sum(s);
  if (greedy) at = __reduce_min_sync(0xffffffffu, m == mw ? at : INT32_MAX);
  SpanStat o;
  o.m = mw;
  o.s = s;
  o.at = at;
  return o;
}

// A warp a span.  Bound by DRAM: 64 x 16 rows of 151936 bf16 logits
// (311 MB) take 50 us, 6.2 TB/s.  Spans of 4, 5 and 6 rounds: a call of them 67.4, 66.8 and
// 67.1 us, one of 32 x 8 rows with probabilities 39.6, 39.5 and 40.2.  Blocks an SM (and so
// registers): 6, 7, 8, 9 and 10 69.6, 68.0, 66.9, 66.8 and 68.3 us, the other 40.1, 39.0, 39.1,
// 39.5 and 40.8.
template <typename T>
__global__ void __launch_bounds__(32 * kStatWarps, 9)
verify_stats_kernel(const __grid_constant__ VerifyArgs A) {
  const int b = blockIdx.x, i = blockIdx.y;
  const int span = blockIdx.z * kStatWarps + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();  // the next kernel waits for all of this before it reads
  if (span >= A.spans || i > drafts_of(A, b)) return;
  bool greedy;
  const float c = log2_scale(A.temperature ? A.temperature[b] : 1.f, greedy);
  const SpanStat o = span_stat(A, row_of<T>(A, b, i), span, c, greedy);
  if ((threadIdx.x & 31) == 0) A.stats[((size_t)b * (A.K + 1) + i) * A.spans + span] = o;
}

// ---------------------------------------------------------------------------
// weights in fixed point
// ---------------------------------------------------------------------------
constexpr float kMagic = 12582912.f;            // 3 * 2^22: adding it rounds to whole numbers,
                                                // which are then the low bits
constexpr float kCoarse = 2.5f;                 // in [2, 4): rounds to multiples of 2^-22
constexpr float kFine = 2.86102295e-6f;         // 3 * 2^-20: to multiples of 2^-42

constexpr unsigned kCoarseBits = 0x40200000u, kFineBits = 0x36400000u;

// a sum of weights: multiples of 2^-22 and of 2^-42, with n times the constants that
// rounded them
struct Fixed {
  unsigned coarse = 0, fine = 0;
  __device__ __forceinline__ uint64_t value(unsigned n) const {
    return (uint64_t)(((long long)(int)(coarse - n * kCoarseBits) << 20) + (int)(fine - n * kFineBits));
  }
};

struct Weigher {
  float off, c, cl, per_c, k0, low;  // of 64ths of a power of two, see below
  const Pow* pow;  // in shared memory

  // For weights e^((z - m) / T).  The largest is not 1 but within 2^(1/128) of it: the
  // reference is c m rounded to a 64th, so that c z - reference needs no more bits
  // than c z itself.  Far from 0 it is m: where a weight counts, z - m is then exact.
  __device__ __forceinline__ Weigher(float scale, float temperature, const Pow* table) {
    c = 64.f * scale;
    // log2(e) = 1.44269502 + 1.92596299e-8; what scale * T lacks of it, over T
    cl = 64.f * __fdividef(fmaf(-scale, temperature, 1.44269502f) + 1.92596299e-8f, temperature);
    per_c = __frcp_rn(c);
    pow = table;
  }
  __device__ __forceinline__ void largest(float m) {
    const bool far = fabsf(c * m) > 64 * 128.f;
    off = far ? m : 0.f;
    const float ref = far ? 0.f : rintf(c * m);
    k0 = kMagic - ref;
    low = (ref - 2944.f) * per_c;  // 2^-46: rounds to a weight of 0, as -inf does
  }

  // weights of two logits as sums hi + lo
  __device__ __forceinline__ void operator()(float2 z, float2& hi, float2& lo) const {
    z = add2(z, two(-off));
    const float2 d = make_float2(fmaxf(z.x, low), fmaxf(z.y, low));
    const float2 cc = two(c);
    // c z - reference = k + G
    const float2 k = fma2(d, cc, two(k0));
    float2 g = fma2(d, cc, sub2(two(k0), k));
    g = fma2(d, two(cl), g);
    // 2^(G/64) - 1 = G (a + G (a^2/2 + G a^3/6)), a = ln 2 / 64
    float2 x = fma2(g, two(2.11731372e-7f), two(5.86490496e-5f));
    x = fma2(g, x, two(0.0108304247f));
    // k = 64 n + j: k << 17 is n in the exponent's place and j << 17
    const int b0 = __float_as_int(k.x), b1 = __float_as_int(k.y);
    const int j0 = b0 & 63, j1 = b1 & 63;
    const float2 t = make_float2(__int_as_float(pow->hi[j0] + (b0 << 17)),
                                 __int_as_float(pow->hi[j1] + (b1 << 17)));
    x = fma2(g, x, make_float2(pow->lo[j0], pow->lo[j1]));
    hi = fma2(t, x, t);
    lo = fma2(t, x, sub2(t, hi));
  }

  // adds two weights to a sum
  static __device__ __forceinline__ void add(float2 hi, float2 lo, Fixed& s) {
    const float2 a = add2(hi, two(kCoarse));
    const float2 rest = add2(sub2(hi, add2(a, two(-kCoarse))), lo);
    const float2 b = add2(rest, two(kFine));
    s.coarse += __float_as_uint(a.x) + __float_as_uint(a.y);
    s.fine += __float_as_uint(b.x) + __float_as_uint(b.y);
  }
};

// floor(u * w), 0 <= u <= 1
__device__ __forceinline__ uint64_t share_of(uint64_t w, float u) {
  const int bits = __float_as_int(u), ex = bits >> 23;
  const uint64_t mant = (bits & 0x7fffff) | (ex ? 0x800000 : 0);
  const int sh = 150 - max(ex, 1);  // u = mant * 2^-sh, sh >= 23
  const uint64_t lo = w * mant, up = __umul64hi(w, mant);
  if (sh >= 128) return 0;
  return sh >= 64 ? up >> (sh - 64) : (up << (64 - sh)) | (lo >> sh);
}

__device__ __forceinline__ float unit(float x) { return x > 0.f ? fminf(x, 1.f) : 0.f; }

// ---------------------------------------------------------------------------
// a sequence: its drafts accepted or not, its token drawn
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint64_t load_cluster(const uint64_t* p, int rank) {
  uint32_t a;
  uint64_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ uint64_t warp_incl64(uint64_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// What a row is drawn from: p, p without the rejected draft, or max(0, p - q).
enum { kAll = 0, kWithout = 1, kResidual = 2 };
template <int M> struct Mode {
  static constexpr int value = M;
};

// Bound by latency and by the weights' instructions (25 a token: 8 on pairs of floats, 10
// on integers and moves between pairs, most of both on one pipe).  From the end of the rows on,
// 64 sequences take 16 us: 2 until the drafts are decided, 8 (median of the blocks) on the
// weights, 1 on the number's place in the sums, the rest by blocks that share an SM.  32 with
// probabilities 21: the last cluster of eight finds its SMs only 5 us late, then 1, 5.4
// and 5.9 on the two passes of weights, 1 on the place.
//
// kAlone: the rows' spans too, where a sequence has few of them (kFewSpans); the kernel in
// front is then the caller's.
template <typename T, bool kAlone>
__global__ void __launch_bounds__(kPickThreads, 2)
verify_pick_kernel(const __grid_constant__ VerifyArgs A) {
  extern __shared__ uint64_t s_sums[];  // [groups_per_block] weights of each group
  __shared__ uint64_t s_part[kPickWarps];
  __shared__ uint64_t s_total[3];  // this block's sum, of one pass each: read by the cluster
  __shared__ Pow s_pow;
  __shared__ float s_m[kMaxDrafts + 1], s_s[kMaxDrafts + 1];
  __shared__ int s_at[kMaxDrafts + 1], s_x[kMaxDrafts], s_fall;
  const int rank = blockIdx.x % A.cluster, b = blockIdx.x / A.cluster;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < 64) {
    s_pow.hi[tid] = __float_as_int(kPow[tid].x) - (tid << 17);
    s_pow.lo[tid] = kPow[tid].y;
  }
  if (tid == 0) s_fall = kMaxDrafts + 1;
  if (kAlone) pdl_wait();
  // The inputs are read ahead of the wait: the kernel in front writes none of them, and
  // what came before it was complete when its blocks, all of them past their own wait, let
  // this one start.  This kernel's wait does not stand between, so that the loads are taken from
  // L2, where a finished kernel's writes are, and not from a line that L1 may still hold.
  const size_t mine = (size_t)b * A.K + tid;
  const int x = tid < A.K ? __ldcg(A.tokens + mine) : -1;  // a thread a draft
  const int n = A.n_drafts ? max(0, min(__ldcg(A.n_drafts + b), A.K)) : A.K;
  const float temp = A.temperature ? __ldcg(A.temperature + b) : 1.f;
  bool greedy;
  const float c = log2_scale(temp, greedy);
  const bool drafted = tid < n;
  const bool token = drafted && x >= 0 && x < A.V;
  const float zx = token ? to_f(__ldcg(row_of<T>(A, b, tid) + x)) : 0.f;
  const float qx = token && A.draft_probs ? unit(__ldcg(A.draft_probs + mine * A.V + x)) : 1.f;
  const float ux = drafted ? unit(__ldcg(A.accept_u + mine)) : 0.f;
  const float su = unit(__ldcg(A.sample_u + b));
  if (tid < A.K) s_x[tid] = x;
  Weigher weigh(c, temp, &s_pow);
  const SpanStat* stats = A.stats + (size_t)b * (A.K + 1) * A.spans;
  if (kAlone) {
    __shared__ SpanStat s_stats[kAlone ? kFewSpans : 1];
    for (int k = warp; k < (n + 1) * A.spans; k += kPickWarps) {
      const SpanStat o = span_stat(A, row_of<T>(A, b, k / A.spans), k % A.spans, c, greedy);
      if (lane == 0) s_stats[k] = o;
    }
    __syncthreads();
    stats = s_stats;
  } else {
    pdl_wait();
  }
  // rows from their spans, a warp a row; those beyond n are nobody's (and not waited for)
  for (int i = warp; i <= A.K; i += kPickWarps) {
    const SpanStat* st = stats + i * A.spans;
    float m = -INFINITY, s = 0.f;
    int at = INT32_MAX;
    for (int k = lane; k < A.spans; k += 32) {
      const uint4 raw = *reinterpret_cast<const uint4*>(st + k);
      const float om = __uint_as_float(raw.x), os = __uint_as_float(raw.y);
      // a span of -inf alone has a sum of 0 (or NaN) and no reference point
      const float m1 = fmaxf(m, om), y1 = ref_point(m1, c);
      s = (m == -INFINITY ? s : s * exp2f(ref_point(m, c) - y1)) +
          (om == -INFINITY ? os : os * exp2f(ref_point(om, c) - y1));
      if (om >= m1) at = om > m ? (int)raw.z : min(at, (int)raw.z);
      m = m1;
    }
    const float mw = warp_max(m);
    if (m != -INFINITY) s *= exp2f(ref_point(m, c) - ref_point(mw, c));
    s = warp_sum(s);
    at = __reduce_min_sync(0xffffffffu, m == mw ? at : INT32_MAX);
    if (lane == 0) {
      s_m[i] = mw;
      s_s[i] = mw == -INFINITY ? __int_as_float(0x7fc00000) : s;
      s_at[i] = at;
    }
  }
  __syncthreads();
  auto sound = [&](int i) { return s_s[i] > 0.f && s_s[i] < INFINITY; };
  if (drafted) {
    float p = 0.f;
    if (!sound(tid)) {
      p = __int_as_float(0x7fc00000);
    } else if (token && x != A.mask_id) {
      p = greedy ? (x == s_at[tid] ? 1.f : 0.f)
                 : exp2f(fmaf(zx, c, -ref_point(s_m[tid], c))) / s_s[tid];
    }
    if (!((greedy ? 0.f : ux * qx) < p)) atomicMin(&s_fall, tid);
    if (rank == 0) {
      if (!token) set_err(A.err, WEDLM_DEV_BAD_TOKEN);
      if (A.draft_p) A.draft_p[mine] = p;
    }
  } else if (tid < A.K && rank == 0 && A.draft_p) {
    A.draft_p[mine] = 0.f;
  }
  if (tid <= n && rank == 0 && !sound(tid)) set_err(A.err, WEDLM_DEV_NUMERIC);
  if (tid == 0 && rank == 0 && A.n_drafts && A.n_drafts[b] != n)
    set_err(A.err, WEDLM_DEV_BAD_SEQLEN);
  __syncthreads();
  const int r = min(s_fall, n);
  if (rank == 0 && tid <= A.K && tid != r)
    A.out_tokens[(size_t)b * (A.K + 1) + tid] = tid < r ? x : -1;
  if (rank == 0 && tid == 0) A.n_accepted[b] = r;
  const bool drawn = sound(r) && !greedy;
  if (!drawn) {  // the same for the whole cluster
    if (rank == 0 && tid == 0) {
      A.out_tokens[(size_t)b * (A.K + 1) + r] = sound(r) ? s_at[r] : -1;
      if (A.sampled_p) A.sampled_p[b] = sound(r) ? 1.f : __int_as_float(0x7fc00000);
    }
    return;
  }

  const T* row = row_of<T>(A, b, r);
  const int lead = lead_of(row);
  const int g0 = rank * A.groups_per_block;
  const int n_groups = max(0, min(A.groups_per_block, (A.V + lead + kGroup - 1) / kGroup - g0));
  const float* q = r < n && A.draft_probs ? A.draft_probs + ((size_t)b * A.K + r) * A.V : nullptr;
  const bool q_vec = ((uintptr_t)(q - lead) & 15) == 0;
  const int out = r < n && !A.draft_probs ? s_x[r] : -1;
  weigh.largest(s_m[r]);
  // a warp's groups are neighbours, so that its sum is a range of tokens
  const int per_warp = (A.groups_per_block + kPickWarps - 1) / kPickWarps;
  const int w0 = min(n_groups, warp * per_warp), w1 = min(n_groups, w0 + per_warp);
  float mass = 0.f, mass_lo = 0.f;  // the sum of p, in units of the reference

  constexpr int kVecs = kGroup * sizeof(T) / 16;
  struct Group {  // as loaded: logits, and the draft's probabilities
    uint4 z[kVecs];
    float q[kGroup];
  };
  // e: the lane's first token, w: the warp's, of `size` neighbouring ones
  auto load = [&](int e, int w, int size, auto mode, Group& g) {
    if (w >= 0 && w + size <= A.V && (unsigned)(A.mask_id - w) >= (unsigned)size &&
        (mode.value != kWithout || (unsigned)(out - w) >= (unsigned)size)) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) g.z[i] = __ldg(reinterpret_cast<const uint4*>(row + e) + i);
    } else {
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        g.z[i] = load_vec(row, e + i * (kGroup / kVecs), A.V, A.mask_id,
                          mode.value == kWithout ? out : -1);
    }
    if (mode.value == kResidual) {
      if (q_vec && e >= 0 && e + kGroup <= A.V) {
#pragma unroll
        for (int k = 0; k < kGroup; k += 4) {
          const float4 x = __ldg(reinterpret_cast<const float4*>(q + e + k));
          g.q[k] = x.x;
          g.q[k + 1] = x.y;
          g.q[k + 2] = x.z;
          g.q[k + 3] = x.w;
        }
      } else {
#pragma unroll
        for (int k = 0; k < kGroup; ++k) g.q[k] = e + k >= 0 && e + k < A.V ? __ldg(q + e + k) : 0.f;
      }
    }
  };
  auto logits = [&](const Group& g, int h) {  // tokens 2h and 2h + 1
    constexpr int kPairs = 4 / kVecs;
    return pair_of(g.z[h / kPairs], h % kPairs, T());
  };
  // weights of two tokens as sums hi + lo
  auto pair_weights = [&](auto mode, float2 z, float q0, float q1, float2& hi, float2& lo) {
    weigh(z, hi, lo);
    if (mode.value == kResidual) {
      // negative or NaN counts as 0; at 1 or above nothing is left of any p
      const float2 qq = make_float2(fmaxf(q0, 0.f), fmaxf(q1, 0.f));
      // hi + lo less q mass = a - off, and what the difference's rounding loses (exact where
      // hi is the larger, and hi = a up to a factor of two else)
      const float2 a = fma2(qq, two(mass), two(0.f)), off = fma2(qq, two(-mass), a);
      const float2 d = sub2(hi, a), lost = sub2(sub2(hi, d), a);
      lo = add2(add2(fma2(qq, two(-mass_lo), lo), off), lost);
      const bool left0 = d.x + lo.x > 0.f, left1 = d.y + lo.y > 0.f;
      hi = make_float2(left0 ? d.x : 0.f, left1 ? d.y : 0.f);
      lo = make_float2(left0 ? lo.x : 0.f, left1 ? lo.y : 0.f);
    }
  };
  // weights of all groups; returns the cluster's sum and the sum of the blocks before
  auto weigh_all = [&](auto mode, int slot, uint64_t* before) {
    uint64_t acc = 0;
    Group next;
    auto fetch = [&](int g, Group& x) {
      const int e = (g0 + g) * kGroup - lead;
      if (g < w1) load(e, e - lane * kGroup, 32 * kGroup, mode, x);
    };
    auto sum = [&](int g, const Group& x) {
      Fixed s;
#pragma unroll
      for (int h = 0; h < kGroup / 2; ++h) {
        float2 hi, lo;
        pair_weights(mode, logits(x, h), x.q[2 * h], x.q[2 * h + 1], hi, lo);
        Weigher::add(hi, lo, s);
      }
      const uint64_t t = s.value(kGroup);
      s_sums[g] = t;
      acc += t;
    };
    fetch(w0 + lane, next);
#pragma unroll 1  // two loads in flight, in twice the code, were 1 us slower
    for (int g = w0 + lane; g < w1; g += 32) {
      const Group now = next;
      fetch(g + 32, next);
      sum(g, now);
    }
    acc = warp_sum64(acc);
    __syncthreads();  // the sums of the pass before have been read
    if (lane == 0) s_part[warp] = acc;
    __syncthreads();
    const uint64_t here = warp_sum64(lane < kPickWarps ? s_part[lane] : 0);
    *before = 0;
    if (A.cluster == 1) return here;
    if (tid == 0) s_total[slot] = here;
    cluster_arrive();
    cluster_wait();
    const uint64_t t = lane < A.cluster ? load_cluster(&s_total[slot], lane) : 0;
    *before = warp_sum64(lane < rank ? t : 0);
    return warp_sum64(t);
  };
  uint64_t before, total;
  int mode = q ? kResidual : out >= 0 ? kWithout : kAll;
  if (mode == kResidual) {
    const uint64_t t = weigh_all(Mode<kAll>(), 0, &before);
    mass = __ull2float_rn(t);
    mass_lo = (float)(long long)(t - (uint64_t)mass) * 0x1p-42f;
    mass *= 0x1p-42f;
    total = weigh_all(Mode<kResidual>(), 1, &before);
  } else {
    total = mode == kWithout ? weigh_all(Mode<kWithout>(), 1, &before) : weigh_all(Mode<kAll>(), 1, &before);
  }
  if (total == 0) {  // nothing left of p: from p itself
    mode = kAll;
    total = weigh_all(Mode<kAll>(), 2, &before);
  }
  if (A.cluster > 1) cluster_arrive();  // this block has read the others' sums
  const uint64_t target = min(share_of(total, su), total - 1);
  const uint64_t at = before + warp_sum64(lane < warp ? s_part[lane] : 0);
  if (target >= at && target - at < s_part[warp]) {
    // this warp has it: the lane that does, with some neighbouring groups, then the group
    const int per = (per_warp + 31) / 32;
    const int a0 = min(w1, w0 + lane * per), a1 = min(w1, a0 + per);
    uint64_t t = 0;
    for (int g = a0; g < a1; ++g) t += s_sums[g];
    const uint64_t incl = warp_incl64(t);
    uint64_t rest = target - at - (incl - t);  // wraps in the lanes behind
    const bool has = target - at >= incl - t && rest < t;
    int g = a0;
    if (has)
      while (g + 1 < a1 && rest >= s_sums[g]) rest -= s_sums[g++];
    const int src = __ffs(__ballot_sync(0xffffffffu, has)) - 1;
    g = __shfl_sync(0xffffffffu, g, src & 31);
    rest = __shfl_sync(0xffffffffu, rest, src & 31);
    // a lane a token of the group
    const int e = (g0 + g) * kGroup - lead, k = lane & (kGroup - 1);
    Group x;
    float2 hi, lo;
    auto one = [&](auto m) {
      load(e, e, kGroup, m, x);
      float2 z = logits(x, 0), qq = make_float2(x.q[0], x.q[1]);
#pragma unroll
      for (int h = 1; h < kGroup / 2; ++h)
        if (h == k / 2) {
          z = logits(x, h);
          qq = make_float2(x.q[2 * h], x.q[2 * h + 1]);
        }
      pair_weights(m, z, qq.x, qq.y, hi, lo);
    };
    if (mode == kResidual) one(Mode<kResidual>());
    else if (mode == kWithout) one(Mode<kWithout>());
    else one(Mode<kAll>());
    Fixed s;  // this lane's of the two
    Weigher::add(make_float2(k & 1 ? hi.y : hi.x, 0.f), make_float2(k & 1 ? lo.y : lo.x, 0.f), s);
    const uint64_t w = warp_incl64(lane < kGroup ? s.value(2) : 0);
    const unsigned over = __ballot_sync(0xffffffffu, w > rest) | 1u << (kGroup - 1);
    if (lane == 0) {
      const int token = e + __ffs(over) - 1;
      A.out_tokens[(size_t)b * (A.K + 1) + r] = token;
      if (A.sampled_p)
        A.sampled_p[b] = exp2f(fmaf(to_f(row[token]), c, -ref_point(s_m[r], c))) / s_s[r];
    }
  }
  if (A.cluster > 1) cluster_wait();  // no block leaves while another may read its sums
}

// Whether clusters of kWideCluster blocks of the draw fit the current device (asked once).
template <typename T>
bool wide_clusters() {
  static std::atomic<int> known[64];  // 1: yes, 2: no
  int dev = 0, fit = 0, k;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if ((k = known[dev].load(std::memory_order_relaxed))) return k == 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kWideCluster);
  cfg.blockDim = dim3(kPickThreads);
  cfg.dynamicSmemBytes = 40 << 10;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kWideCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool ok =
      cudaFuncSetAttribute(reinterpret_cast<const void*>(verify_pick_kernel<T, false>),
                           cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
      cudaOccupancyMaxActiveClusters(&fit, verify_pick_kernel<T, false>, &cfg) == cudaSuccess && fit > 0;
  if (!ok) cudaGetLastError();
  known[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
  return ok;
}

template <typename T>
cudaError_t launch_verify(const VerifyArgs& A, cudaStream_t st) {
  const bool alone = A.cluster == 1 && (A.K + 1) * A.spans <= kFewSpans;
  cudaError_t e;
  if (!alone) {
    const dim3 grid(A.B, A.K + 1, (A.spans + kStatWarps - 1) / kStatWarps);
    e = launch_pdl(verify_stats_kernel<T>, grid, dim3(32 * kStatWarps), 0, st, A);
    if (e != cudaSuccess) return e;
  }
  void (*pick)(VerifyArgs) = alone ? verify_pick_kernel<T, true> : verify_pick_kernel<T, false>;
  const int smem = A.groups_per_block * (int)sizeof(uint64_t);
  if (smem > 40 << 10) {  // beyond what a kernel has without asking
    e = ensure_dyn_smem(reinterpret_cast<const void*>(pick),
                        (kMaxVocab / kGroup / kMaxCluster + 2) * (int)sizeof(uint64_t));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(A.B * A.cluster));
  cfg.blockDim = dim3(kPickThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = A.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = A.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, pick, A);
}

bool verify_sizes(const wedlm_verify_args& a) {
  return (a.dtype == WEDLM_BF16 || a.dtype == WEDLM_FP32) && a.batch >= 1 && a.drafts >= 0 &&
         a.drafts <= kMaxDrafts && (int64_t)a.batch * (a.drafts + 1) <= (1 << 20) && a.vocab >= 1 &&
         a.vocab <= kMaxVocab && a.mask_id >= -1 && a.mask_id < a.vocab;
}

// Rounds of loads of a span, and spans of a row.  Long spans spare records and keep
// loads in flight; a few rows are cut finer, so that there are warps for all SMs.
void verify_split(const wedlm_verify_args& a, int* rounds, int* spans) {
  const int n = a.dtype == WEDLM_BF16 ? 8 : 4, round = kStatVecs * 32 * n;
  const int64_t rows = (int64_t)a.batch * (a.drafts + 1), per_row = (a.vocab + round - 1) / round;
  *rounds = (int)std::max<int64_t>(1, std::min<int64_t>(kMaxRounds, rows * per_row / kManyWarps));
  const int span = *rounds * round;
  *spans = (a.vocab + n - 1 + span - 1) / span;  // a row may start within a vector
}

size_t verify_space(const wedlm_verify_args& a) {
  int rounds, spans;
  verify_split(a, &rounds, &spans);
  return ((size_t)a.batch * (a.drafts + 1) * spans * sizeof(SpanStat) + 255) / 256 * 256;
}

}  // namespace
}  // namespace wedlm

using namespace wedlm;

extern "C" size_t wedlm_verify_drafts_workspace(const wedlm_verify_args* a) {
  return a && verify_sizes(*a) ? verify_space(*a) : 0;
}

extern "C" int wedlm_verify_drafts(const wedlm_verify_args* a, void* stream) {
  if (!a || !verify_sizes(*a)) return WEDLM_ERR_INVALID_ARG;
  const int es = a->dtype == WEDLM_BF16 ? 2 : 4;
  auto odd = [](const void* p, int align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0; };
  auto bad4 = [&](const void* p) { return !p || odd(p, 4); };
  if (!a->logits || odd(a->logits, es) || a->batch_stride < 0 || a->row_stride < 0 ||
      bad4(a->sample_u) || bad4(a->n_accepted) || bad4(a->out_tokens) ||
      (a->drafts && (bad4(a->tokens) || bad4(a->accept_u))) || odd(a->draft_probs, 4) ||
      odd(a->n_drafts, 4) || odd(a->temperature, 4) || odd(a->draft_p, 4) || odd(a->sampled_p, 4) ||
      odd(a->error, 4) || !a->workspace || odd(a->workspace, 256))
    return WEDLM_ERR_INVALID_ARG;
  // outputs and workspace: over no input, over no other of them
  struct Span {
    const void* p;
    size_t n;
  };
  const size_t B = a->batch, K = a->drafts, V = a->vocab;
  const Span in[] = {
      {a->logits, ((B - 1) * a->batch_stride + K * a->row_stride + V) * es},
      {K ? a->tokens : nullptr, 4 * B * K},      {K ? a->draft_probs : nullptr, 4 * B * K * V},
      {a->n_drafts, 4 * B},                      {a->temperature, 4 * B},
      {K ? a->accept_u : nullptr, 4 * B * K},    {a->sample_u, 4 * B}};
  const Span out[] = {{a->n_accepted, 4 * B},
                      {a->out_tokens, 4 * B * (K + 1)},
                      {K ? a->draft_p : nullptr, 4 * B * K},
                      {a->sampled_p, 4 * B},
                      {a->workspace, verify_space(*a)}};
  auto meet = [](const Span& x, const Span& y) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(x.p), q = reinterpret_cast<uintptr_t>(y.p);
    return p && q && p < q + y.n && q < p + x.n;
  };
  for (const Span& o : out) {
    for (const Span& i : in)
      if (meet(o, i)) return WEDLM_ERR_INVALID_ARG;
    for (const Span& p : out)
      if (&o != &p && meet(o, p)) return WEDLM_ERR_INVALID_ARG;
  }
  if (a->workspace_bytes < verify_space(*a)) return WEDLM_ERR_CAPACITY;
  VerifyArgs A;
  A.B = a->batch;
  A.K = a->drafts;
  A.V = a->vocab;
  const int sms = device_sms();
  if (sms < 1) return WEDLM_ERR_CUDA;
  verify_split(*a, &A.rounds, &A.spans);
  const int groups = (a->vocab + 2 * (kGroup - 1)) / kGroup;
  // Blocks of a sequence: two of them fit an SM, and more of them than fit the GPU at
  // once would only wait.  64 x 15 drafts over 151936 tokens 66.8 us with these four, 71.7 with
  // eight, 76.6 with two; 32 x 7 with probabilities 39.5 with these eight, 51.3 with four.
  A.cluster = 1;
  while (A.cluster < kMaxCluster &&
         (groups > kMaxGroups * A.cluster ||
          (groups > 2 * kPickThreads * A.cluster && 2 * A.cluster * A.B <= 2 * sms)))
    A.cluster *= 2;
  // A few sequences: twice as many SMs for each.  8 x 3 drafts over 151936 tokens with
  // probabilities 16 us captured, not 25; one sequence's 15 drafts 10.6, not 11.3.
  if (A.cluster == kMaxCluster && kWideCluster * A.B <= sms &&
      (a->dtype == WEDLM_BF16 ? wide_clusters<bf16>() : wide_clusters<float>()))
    A.cluster = kWideCluster;
  A.groups_per_block = (groups + A.cluster - 1) / A.cluster;
  A.mask_id = a->mask_id;
  A.logits = a->logits;
  A.batch_stride = a->batch_stride;
  A.row_stride = a->row_stride;
  A.tokens = a->tokens;
  A.draft_probs = a->drafts ? a->draft_probs : nullptr;
  A.n_drafts = a->n_drafts;
  A.temperature = a->temperature;
  A.accept_u = a->accept_u;
  A.sample_u = a->sample_u;
  A.n_accepted = a->n_accepted;
  A.out_tokens = a->out_tokens;
  A.draft_p = a->draft_p;
  A.sampled_p = a->sampled_p;
  A.stats = static_cast<SpanStat*>(a->workspace);
  A.err = a->error;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->dtype == WEDLM_BF16 ? launch_verify<bf16>(A, st) : launch_verify<float>(A, st);
  return e == cudaSuccess ? WEDLM_OK : WEDLM_ERR_CUDA;
}
