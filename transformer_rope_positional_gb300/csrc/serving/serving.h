// Host-side interface between the C ABI (rope_api.cu) and the launchers of the serving
// operators: scaled rotary tables, append to a paged KV cache, attention over it.
// Arguments arrive here already validated.
#pragma once

#include "rope_launch.h"

namespace rope {

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
};

cudaError_t launch_append(const AppendProblem& p, cudaStream_t stream);

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
};

cudaError_t launch_attend(const AttendProblem& p, cudaStream_t stream);
int64_t attend_workspace(int64_t T, int64_t nq, int64_t nk, int64_t D, int32_t dtype, int64_t prefix_len);

}  // namespace rope
