// Shared by the attention kernels: the argument block, the sequence of a token, and where a
// key of a sequence sits in the paged cache.
#pragma once

#include "rope_device.cuh"
#include "serving.h"

namespace rope {
namespace attend {

constexpr unsigned kSlotOutOfRange = 2u;

struct AttendArgs {
  int64_t T, B;
  int64_t q_stride;
  int64_t num_blocks;
  int64_t W;            // pages of a block table row
  int32_t nq, nk, G;    // G = nq / nk query heads share a key head
  int32_t D;
  int32_t block_size, bs_shift;  // bs_shift: log2(block_size), or -1
  int32_t P;            // keys of the shared prefix
  float scale_log2;     // scale * log2(e)
  Span q_span, k_span, v_span, bt_span, sl_span, qsl_span, pb_span, out_span, lse_span;
};

struct Pointers {
  const int64_t* block_table;
  const int64_t* seq_lens;
  const int64_t* qsl;
  const int64_t* prefix_blocks;
  unsigned int* err;
};

// Batch of token t: the largest b in [0, B) with query_start_loc[b] <= t.
__device__ __forceinline__ int64_t batch_of(int64_t t, const Pointers& g, const AttendArgs& a) {
  int64_t l = 0, h = a.B - 1;
  while (l < h) {
    const int64_t mid = (l + h + 1) >> 1;
    if (ldg(g.qsl + mid, a.qsl_span, g.err) <= t) l = mid; else h = mid - 1;
  }
  return l;
}

__device__ __forceinline__ int page_of(int j, const AttendArgs& a) {
  return a.bs_shift >= 0 ? j >> a.bs_shift : j / a.block_size;
}

// Cache row (page * Nk * BS + row of the page; the head's rows are head * BS further) of key
// j < P of the prefix, or of own key j - P of the sequence whose block table row is `table`.
// -1 when the page is outside the cache or the sequence has no such page.
__device__ __forceinline__ int64_t key_row(int j, const int64_t* table, const Pointers& g, const AttendArgs& a) {
  int64_t page;
  int i;
  if (j < a.P) {
    i = page_of(j, a);
    j -= i * a.block_size;
    page = ldg(g.prefix_blocks + i, a.pb_span, g.err);
  } else {
    j -= a.P;
    i = page_of(j, a);
    if (i >= a.W) return -1;
    j -= i * a.block_size;
    page = ldg(table + i, a.bt_span, g.err);
  }
  if (page < 0 || page >= a.num_blocks) return -1;
  return page * a.nk * a.block_size + j;
}

}  // namespace attend
}  // namespace rope
