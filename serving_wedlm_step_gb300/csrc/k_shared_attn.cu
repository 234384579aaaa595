// Shared-prefix window attention: argument checks, workspace and launches.
#include <math.h>

#include <algorithm>

#include "shared_attn.cuh"

namespace wedlm {
namespace {

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Sizes of a call: its split and the workspace's layout.  False for sizes the
// kernels do not take.
struct SharedPlan {
  SharedArgs A{};
  int TPB;  // tokens per row block of the tensor-core kernel
  size_t off_part_p, off_ml_s, off_ml_p, off_units, bytes;
};

bool shared_plan(const wedlm_shared_attn_args& a, SharedPlan* P) {
  if ((a.dtype != WEDLM_BF16 && a.dtype != WEDLM_FP32) ||
      (a.head_dim != 64 && a.head_dim != 128) || a.batch < 1 || a.batch > kSharedMaxBatch ||
      a.window < 1 || a.window > kMaxWindow || a.n_kv_heads < 1 || a.n_q_heads < a.n_kv_heads ||
      a.n_q_heads % a.n_kv_heads || a.n_q_heads / a.n_kv_heads > 128 || a.n_kv_heads > 1024 ||
      a.n_shared_pages < 0 || a.n_shared_pages > (1 << 26) || a.max_pages_per_seq < 1 ||
      a.max_pages_per_seq > (1 << 26) || a.num_pages < 1)
    return false;
  SharedArgs& A = P->A;
  A.B = a.batch;
  A.W = a.window;
  A.Wp = (a.window + kPageBlock - 1) / kPageBlock * kPageBlock;
  A.G = a.n_q_heads / a.n_kv_heads;
  A.nkv = a.n_kv_heads;
  A.nsp = a.n_shared_pages;
  A.max_pages = a.max_pages_per_seq;
  A.num_pages = a.num_pages;
  A.scale_log2 = (float)(1.4426950408889634 / sqrt((double)a.head_dim));
  const int rows = A.B * A.W * A.G, seq_rows = A.W * A.G;
  P->TPB = 128 / A.G;
  const int urows = a.dtype == WEDLM_BF16 ? 2 * P->TPB * A.G : kSimtRows;
  A.srows = std::min(urows, rows);
  A.prows = std::min(urows, seq_rows);
  A.sblocks = (rows + A.srows - 1) / A.srows;
  A.pblocks = (seq_rows + A.prows - 1) / A.prows;
  if (a.dtype == WEDLM_BF16) {
    // relative times, swept on GB300: a tile for 128 rows 16, for a pair of row
    // blocks 28; a unit's start and end 32, more with the rows whose partial it
    // writes.  64 x 32 rows over 16384 shared positions: 399 us with these, 397 to 404
    // with ends at 16 to 64, 411 with pairs at 20; heads of 64: 362, 359 to 367, 375.
    // 64 single tokens over 8192: 36.9 us, 41 to 43, 45.5; heads of 64: 33.6, 35 to
    // 39, 40.5.  Pairs at 32 are within 5 % on all of these.
    A.ucost = 32 + std::min(A.prows, 128) / 4;
    A.shared_cost = A.B * A.W > P->TPB ? 28 : 16;
    A.private_cost = A.W > P->TPB ? 28 : 16;
    A.min_share = 32;
  } else {
    // a tile of 64 rows 4, of 16 rows 2, a unit's ends 2, swept on GB300.  12 sequences
    // x 8 rows over 2048 shared positions, heads of 64: 20.8 us with these, 26.3 with
    // ends at 1, 20.9 at 4, 26.5 at 6; a 64-row tile at 3 20.9, at 6 26.1, at 8 28.8.
    // 16 x 32 rows over 8192: 289 us, 298, 283, 283; 284, 291, 303; heads of 128 within 3 %
    A.ucost = 2;
    A.shared_cost = A.srows > kSimtFewRows ? 4 : 2;
    A.private_cost = A.prows > kSimtFewRows ? 4 : 2;
    A.min_share = std::max(A.shared_cost, A.private_cost);
  }
  // the split counts in 31 bits: where full tables could pass that, a tile and a
  // unit's ends weigh 1, and beyond that the call is refused
  auto weight = [&]() {
    const long long st = (A.nsp + kSharedTilePages - 1) / kSharedTilePages;
    const long long pt = (A.max_pages + A.Wp / kPageBlock + kSharedTilePages - 1) / kSharedTilePages;
    return (long long)A.nkv * (A.sblocks * (A.ucost + st * A.shared_cost) +
                               (long long)A.B * A.pblocks * (A.ucost + pt * A.private_cost));
  };
  if (weight() > INT32_MAX) A.ucost = A.shared_cost = A.private_cost = A.min_share = 1;
  if (weight() > INT32_MAX) return false;
  const long long su = (long long)A.nkv * A.sblocks, pu = (long long)A.B * A.nkv * A.pblocks;
  if (su + pu > (1 << 24)) return false;
  const size_t ss = (size_t)su + kSharedMaxGrid, ps = (size_t)pu + kSharedMaxGrid;
  size_t at = align256(ss * A.srows * a.head_dim * sizeof(float));
  P->off_part_p = at;
  at += align256(ps * A.prows * a.head_dim * sizeof(float));
  P->off_ml_s = at;
  at += align256(ss * A.srows * sizeof(float2));
  P->off_ml_p = at;
  at += align256(ps * A.prows * sizeof(float2));
  P->off_units = at;
  at += align256((size_t)(su + pu) * sizeof(int2));
  P->bytes = at;
  return true;
}

}  // namespace
}  // namespace wedlm

using namespace wedlm;

extern "C" size_t wedlm_shared_attention_workspace(const wedlm_shared_attn_args* args) {
  SharedPlan P;
  return args && shared_plan(*args, &P) ? P.bytes : 0;
}

extern "C" int wedlm_shared_attention(const wedlm_shared_attn_args* a, void* stream) {
  if (!a) return WEDLM_ERR_INVALID_ARG;
  auto bad = [](const void* p, int align) {
    return !p || (reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0;
  };
  SharedPlan P;
  if (!shared_plan(*a, &P) || bad(a->q, 16) || bad(a->kv_pool, 16) || bad(a->kv_win, 16) ||
      bad(a->o, 16) || bad(a->page_table, 4) || bad(a->seq_len, 4) || bad(a->workspace, 256) ||
      (a->n_shared_pages && bad(a->shared_pages, 4)) || (a->error && bad(a->error, 4)))
    return WEDLM_ERR_INVALID_ARG;
  if (a->workspace_bytes < P.bytes) return WEDLM_ERR_CAPACITY;
  SharedArgs& A = P.A;
  const int sms = device_sms();
  if (sms < 1) return WEDLM_ERR_CUDA;
  A.grid = std::min(sms, kSharedMaxGrid);  // one block per SM
  A.q = a->q;
  A.pool = a->kv_pool;
  A.kv_win = a->kv_win;
  A.shared = a->shared_pages;
  A.page_table = a->page_table;
  A.seq_len = a->seq_len;
  A.o = a->o;
  A.err = a->error;
  char* ws = static_cast<char*>(a->workspace);
  A.part_s = reinterpret_cast<float4*>(ws);
  A.part_p = reinterpret_cast<float4*>(ws + P.off_part_p);
  A.ml_s = reinterpret_cast<float2*>(ws + P.off_ml_s);
  A.ml_p = reinterpret_cast<float2*>(ws + P.off_ml_p);
  A.unit_blocks = reinterpret_cast<int2*>(ws + P.off_units);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool is_bf16 = a->dtype == WEDLM_BF16;
  if ((is_bf16 ? launch_shared_attention_tc(A, a->head_dim, P.TPB, st)
               : launch_shared_attention_simt(A, a->head_dim, st)) != cudaSuccess ||
      launch_shared_merge(A, a->head_dim, is_bf16, st) != cudaSuccess)
    return WEDLM_ERR_CUDA;
  return WEDLM_OK;
}
