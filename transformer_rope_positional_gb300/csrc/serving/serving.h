// Host-side interface between the C ABI (rope_api.cu) and the launchers of the serving
// operators: scaled rotary tables, append to a paged KV cache, attention over it.
// Arguments arrive here already validated.
#pragma once

#include "rope_launch.h"

namespace rope {

// Types beside those of rope_launch.h: 8-bit codes and scales of a cache, and whole numbers.
enum MoreTypes : int32_t { kE4M3 = 4, kE8M0 = 5, kI32 = 6, kU8 = 7 };

// cos/sin rows for given frequencies.
struct TableProblem {
  const double* inv_freq;  // host, F values
  int64_t F;
  double scale;
  const int64_t* positions;  // or NULL: row indices
  int64_t first;
  int64_t rows;
  void* cos;  // [rows, 2F]; the whole table (cos||sin rows) when sin is NULL
  void* sin;
  bool interleave;  // with sin: pairs of equal values, else equal halves
  int32_t dtype;
};

cudaError_t launch_table(const TableProblem& p, cudaStream_t stream);

// RoPE of query and key on the way to the query output and a paged KV cache.
struct AppendProblem {
  const int64_t* positions;
  const int64_t* slot_mapping;
  const void* query;  // or NULL
  const void* key;
  const void* value;
  const void* table;
  void* query_out;  // equal to query: in place
  void* k_cache;
  void* v_cache;
  int32_t dtype, table_dtype;
  int64_t T;
  int64_t hq, hk, hv;
  int64_t head_size, rotary_dim;
  int64_t max_seq;
  int64_t num_blocks, block_size;
  bool is_neox;
  int32_t mrope_rows;
  int32_t section_end[4];
  int32_t cache_mode;
  int64_t q_stride, k_stride, v_stride;
  // caches of codes only: E8M0 bytes [num_blocks, heads, scale_blocks]
  uint8_t* k_scale = nullptr;
  uint8_t* v_scale = nullptr;
  int64_t scale_blocks = 0;
};

cudaError_t launch_append(const AppendProblem& p, cudaStream_t stream);
cudaError_t launch_append_codes(const AppendProblem& p, cudaStream_t stream);

// Causal attention over a paged KV cache with a shared prefix.
struct AttendProblem {
  const void* query;
  int64_t q_stride;
  const void* k_cache;
  const void* v_cache;
  const int64_t* block_table;  // [B, W]
  const int64_t* seq_lens;
  const int64_t* query_start_loc;
  const int64_t* prefix_blocks;
  void* out;
  float* lse;  // or NULL
  void* workspace;
  int32_t dtype;
  int64_t T, B;
  int64_t nq, nk, D;
  int64_t num_blocks, block_size;
  int64_t W;
  int64_t prefix_len;
  float scale;
  // caches of codes only: E8M0 bytes [num_blocks, nk, scale_blocks]
  const uint8_t* k_scale = nullptr;
  const uint8_t* v_scale = nullptr;
  int64_t scale_blocks = 0;
};

cudaError_t launch_attend(const AttendProblem& p, cudaStream_t stream);
cudaError_t launch_attend_codes(const AttendProblem& p, cudaStream_t stream);
// (a part of it, by itself for the sake of the build's time)
namespace attend {
struct Pointers;
struct AttendArgs;
struct Cut;
cudaError_t launch_codes_tall(const AttendProblem& p, const Pointers& g, const AttendArgs& a, const Cut& c,
                              cudaStream_t stream);
}  // namespace attend
int64_t attend_codes_workspace(int64_t T, int64_t nq, int64_t nk, int64_t D, int32_t dtype, int64_t prefix_len);
int64_t attend_workspace(int64_t T, int64_t nq, int64_t nk, int64_t D, int32_t dtype, int64_t prefix_len);

// New sequences of old ones, and pages for them.
struct RearrangeProblem {
  const int64_t* table;   // [B, W]
  const int64_t* lens;    // [B]
  const int32_t* refs;    // [NB]
  const int64_t* parents;  // [rows]
  const int64_t* room;    // [rows], or NULL
  int64_t* new_table;     // [rows, new_W]
  int64_t* new_lens;      // [rows]
  int32_t* new_refs;      // [NB]; may be refs
  int64_t *src, *dst;     // [rows]
  int64_t* counts;        // [2]
  int64_t B, W, rows, new_W, NB, block_size, prefix_len;
};

cudaError_t launch_rearrange(const RearrangeProblem& p, cudaStream_t stream);
constexpr int64_t kMostRearranged = 8192;  // rows

// Live pages to the front.
struct CompactProblem {
  const int64_t* table;  // [B, W]
  const int64_t* lens;   // [B]
  const int32_t* refs;   // [NB]
  int64_t* new_table;    // [B, W]; may be table
  int32_t* new_refs;     // [NB]; may be refs
  const int64_t* prefix;  // [pages of the prefix], or NULL
  int64_t* new_prefix;    // may be prefix
  int64_t *src, *dst;     // [pairs]
  int64_t* counts;        // [2]
  int64_t B, W, NB, block_size, prefix_len, pairs;
};

cudaError_t launch_compact(const CompactProblem& p, cudaStream_t stream);

// Pages of several tensors, each tensor's pages `bytes` apart.
struct CopyTensor {
  char* data;
  int64_t bytes;
};
struct CopyProblem {
  const int64_t *src, *dst;  // [pairs]
  const int64_t* count;      // or NULL: all pairs
  int64_t pairs, NB;
  const CopyTensor* tensors;  // host
  int64_t num_tensors;
};

cudaError_t launch_copy_pages(const CopyProblem& p, cudaStream_t stream);

}  // namespace rope
