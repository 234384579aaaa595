// The pages of a cache: what fork, free, reserve and compact share.
#pragma once

#include <initializer_list>

#include "internal.h"

namespace wedlm {

constexpr int kPageMaxBatch = 4096;
constexpr int kReserveMaxBatch = 1024;
constexpr int kMaxColumns = 1 << 26;  // of a page table
constexpr int kMaxPages = 1 << 28;

// wedlm_page_state with the error word; the kernels read the old arrays and write
// the new ones, which may be the same
struct PageArrays {
  int B, cols, N;
  const int32_t *table, *seq_len, *refs;
  int32_t *new_table, *new_len, *new_refs;
  int* err;
};

struct PagePools {
  void* p[kMaxLayers];
  int n_layers;
  int64_t page_bytes;
};

// what a call writes beside the new state, and what it reads beside the old one
struct PageSpan {
  const void* p;
  int64_t n;  // int32 values
};

// The checks of a state. `uses_len`: seq_len is read; `new_len`: and its successor
// written. No output may meet an input (but new_x may be x) or another output.
bool page_state_ok(const wedlm_page_state& s, int max_batch, bool uses_len, bool new_len,
                   std::initializer_list<PageSpan> inputs, std::initializer_list<PageSpan> outputs);
bool page_pools_ok(const wedlm_page_pools& p, bool sizes_only);
// No array of the state and none of `others` lies in a pool (pools are read and written), and
// no pool over a part of another.
bool page_pools_apart(const wedlm_page_pools& p, const wedlm_page_state& s, bool uses_len,
                      std::initializer_list<PageSpan> others);
PageArrays page_arrays(const wedlm_page_state& s);
PagePools page_pools(const wedlm_page_pools& p);

// int32 values that launch_page_state_copy copies
int64_t page_state_ints(const PageArrays& S, bool table);
// new_refs (and new_table, `table` given) <- the old arrays, where they are others
cudaError_t launch_page_state_copy(const PageArrays& S, bool table, cudaStream_t st);

}  // namespace wedlm
