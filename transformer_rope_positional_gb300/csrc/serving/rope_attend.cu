// Causal attention of new tokens over a paged KV cache with a shared prefix.
//
// Per query row (token t at position p, head h) over the keys j <= p it sees:
//   s_j = scale <q, k_j>,  m = max s_j,  l = sum e^(s_j - m),  o = sum e^(s_j - m) v_j / l,
// in one pass over the keys with a running m, l and o (o and l are multiplied by
// e^(m_old - m_new) when the maximum grows).  Base-2 exponentials of scale * log2(e) * <q, k>.
// Partial results over key ranges are joined by
//   m = max m_s,  l = sum l_s e^(m_s - m),  o = sum o_s e^(m_s - m) / l.
//
// Heads of up to 256 take the unit kernels (16-bit data: rope_attend_mma.cuh for up to 16 rows
// a sequence and key head and for little work, rope_attend_tc.cuh beyond; binary32:
// rope_attend_f32.cuh), then, where units may be split, a kernel that joins partial results;
// larger heads a kernel with one warp per query row.
//
// A shared prefix has a launch of its own when a sequence's rows fill less than a unit: the
// rows of all sequences together fill the units of that launch, so the prefix is read once
// for the batch instead of once a sequence.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "rope_attend.cuh"
#include "rope_attend_f32.cuh"
#include "rope_attend_mma.cuh"
#include "rope_attend_tc.cuh"

namespace rope {
namespace {

using namespace attend;

constexpr int kWarps = 4;

// One warp per query row: heads over 256, and caches of 2^31 rows.  Every key is a round trip to
// memory and two sums over the lanes, and K and V are read again for each head of a group: 64 requests
// of up to 2048 tokens, 16 q and 4 k heads of 512, bf16: 11.5 ms where the bytes take 82 us, issue
// slots busy 3 % of the time.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
    attend_rows_kernel(const T* __restrict__ q, const T* __restrict__ kc, const T* __restrict__ vc, T* __restrict__ out,
                       float* __restrict__ lse, Pointers g, AttendArgs a) {
  wait_for_prior_grid();
  const int64_t rows = a.T * a.nq;
  const int64_t tokens = ldg(g.qsl + a.B, a.qsl_span, g.err);
  for (int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); row < rows; row += (int64_t)gridDim.x * kWarps) {
    const int64_t t = row / a.nq;
    if (t >= tokens) break;
    attend_row<T, 16>(t, (int)(row - t * a.nq), q, kc, vc, out, lse, g, a);
  }
}

// The joining kernels add the partial results of rows up, a warp to a row.  A row whose result
// is not finite, or of weights that are all 0, is computed again key by key (see mend_rows).

// Where partial result s of a row lies: (m, l) and O.
struct Source {
  const float* ml;
  const float* o;
};

__device__ __forceinline__ Source slot_source(const Cut& c, const AttendArgs& a, int cta, bool begins, int at) {
  return {slot_ml(c, a, cta, begins ? 1 : 0) + at * 2, slot_o(c, a, cta, begins ? 1 : 0) + (int64_t)at * a.D};
}

// Adds up n partial results of each of R rows, NS at a time, all loads before any arithmetic
// (fast_exp2 for binary32 too: one factor a part, of relative error 2^-22 as exp2f's):
// m, l, and this lane's columns 2 lane + 64 e of O.  source(r, s) is called for s < n only.
template <int E, int R, int NS, typename F>
__device__ __forceinline__ void add_up(int n, const AttendArgs& a, F&& source, float (&m)[R], float (&l)[R],
                                       float2 (&o)[R][E]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[r][e] = make_float2(0.f, 0.f);
  }
  for (int s0 = 0; s0 < n; s0 += NS) {
    float2 v[R][NS][E], ml[R][NS];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        ml[r][s] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < E; ++e) v[r][s][e] = make_float2(0.f, 0.f);
        if (s0 + s < n) {
          const Source x = source(r, s0 + s);
          ml[r][s] = *reinterpret_cast<const float2*>(x.ml);
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (lane * 2 + 64 * e < a.D) v[r][s][e] = *reinterpret_cast<const float2*>(x.o + lane * 2 + 64 * e);
        }
      }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float top = m[r];
#pragma unroll
      for (int s = 0; s < NS; ++s) top = fmaxf(top, ml[r][s].x);
      const float base = top == -INFINITY ? 0.f : top;
      const float keep = fast_exp2(m[r] - base);
      l[r] *= keep;
#pragma unroll
      for (int e = 0; e < E; ++e) o[r][e] = make_float2(o[r][e].x * keep, o[r][e].y * keep);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const float f = fast_exp2(ml[r][s].x - base);
        l[r] = fmaf(ml[r][s].y, f, l[r]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          o[r][e].x = fmaf(f, v[r][s][e].x, o[r][e].x);
          o[r][e].y = fmaf(f, v[r][s][e].y, o[r][e].y);
        }
      }
      m[r] = top;
    }
  }
}

// The row's result from m, l and O, if it is finite and some key had a weight (see inverse_sum; here rows
// without keys are left to attend_row too).
template <typename T, int E>
__device__ __forceinline__ bool write_row(int64_t row, float m, float l, float2 (&o)[E], T* __restrict__ out,
                                          float* __restrict__ lse, const Pointers& g, const AttendArgs& a) {
  const int lane = threadIdx.x & 31;
  const float inv = 1.f / l;
  bool fine = l > 0.f && l <= FLT_MAX;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    o[e] = make_float2(o[e].x * inv, o[e].y * inv);
    fine = fine && fabsf(o[e].x) <= FLT_MAX && fabsf(o[e].y) <= FLT_MAX;
  }
  if (!__all_sync(0xffffffffu, fine)) return false;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int d = lane * 2 + 64 * e;
    T* p = out + row * a.D + d;
    if (d < a.D && access_ok(p, 2 * sizeof(T), a.out_span, g.err)) narrow2(p, o[e]);
  }
  if (lse && lane == 0 && access_ok(lse + row, 4, a.lse_span, g.err))
    lse[row] = (m + log2f(l)) * 0.693147180559945309f;
  return true;
}

// With a launch for the prefix: every row has partial results of both, the prefix's first.
template <typename T, int E>
__global__ void __launch_bounds__(kWarps * 32)
    attend_join_both_kernel(const T* __restrict__ q, const T* __restrict__ kc, const T* __restrict__ vc,
                            T* __restrict__ out, float* __restrict__ lse, Pointers g, AttendArgs a, Cut own, Cut pre) {
  wait_for_prior_grid();
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= a.T * a.nq) return;
  const int64_t rows = min(ldg(g.qsl + a.B, a.qsl_span, g.err), a.T) * a.nq;
  const int2 x = own.rec[row], y = pre.rec[row];
  if (row >= rows) return;
  const int c0 = x.x & 0xffff, c1 = x.x >> 16, p0 = y.x & 0xffff, p1 = y.x >> 16;
  float m[1] = {-INFINITY}, l[1] = {NAN};
  float2 o[1][E] = {};
  // (a row that no unit covered, for starts out of order, has any record: key by key)
  if (c1 >= c0 && c1 < own.grid && (unsigned)x.y < (unsigned)own.slot_rows && p1 >= p0 && p1 < pre.grid &&
      (unsigned)y.y < (unsigned)pre.slot_rows) {
    const int n_pre = p1 - p0 + 1;
    add_up<E, 1, 8>(n_pre + c1 - c0 + 1, a, [&](int, int s) -> Source {
      const bool is_pre = s < n_pre;
      const Cut& c = is_pre ? pre : own;
      const int first = is_pre ? p0 : c0, last = is_pre ? p1 : c1;
      if (first == last) return {c.dense + a.T * a.nq * a.D + row * 2, c.dense + row * a.D};
      const int cta = first + (is_pre ? s : s - n_pre);
      return slot_source(c, a, cta, cta == first, is_pre ? y.y : x.y);
    }, m, l, o);
  }
  if (!write_row<T, E>(row, m[0], l[0], o[0], out, lse, g, a)) {
    const int64_t t = row / a.nq;
    attend_row<T, 2 * E>(t, (int)(row - t * a.nq), q, kc, vc, out, lse, g, a);
  }
}

// Without: the rows whose unit was split.  A warp looks at the records of per_warp consecutive
// rows with one load, and takes rows of two parts (most, where there are many rows) four at a time.
template <typename T, int E>
__global__ void __launch_bounds__(kWarps * 32)
    attend_join_kernel(const T* __restrict__ q, const T* __restrict__ kc, const T* __restrict__ vc, T* __restrict__ out,
                       float* __restrict__ lse, Pointers g, AttendArgs a, Cut own, int per_warp) {
  wait_for_prior_grid();
  const int lane = threadIdx.x & 31;
  const int64_t first = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * per_warp;
  const int64_t rows = min(ldg(g.qsl + a.B, a.qsl_span, g.err), a.T) * a.nq;
  int2 mine = make_int2(0, 0);
  if (lane < per_warp && first + lane < a.T * a.nq) mine = own.rec[first + lane];
  const int n_mine = (mine.x >> 16) - (mine.x & 0xffff) + 1;
  const bool todo = first + lane < rows && n_mine != 1;
  // (a row that no unit covered, for starts out of order, has any record)
  const bool known = mine.x >= 0 && n_mine > 1 && (mine.x >> 16) < own.grid && (unsigned)mine.y < (unsigned)own.slot_rows;
  uint32_t again = __ballot_sync(0xffffffffu, todo && !known), two = __ballot_sync(0xffffffffu, todo && known && n_mine == 2),
           more = __ballot_sync(0xffffffffu, todo && known && n_mine > 2);
  while (two) {
    int row[4], cta[4], at[4], count = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      row[r] = two ? __ffs(two) - 1 : row[r > 0 ? r - 1 : 0];
      count += two != 0;
      two &= two - 1;
      cta[r] = __shfl_sync(0xffffffffu, mine.x, row[r]) & 0xffff;
      at[r] = __shfl_sync(0xffffffffu, mine.y, row[r]);
    }
    float m[4], l[4];
    float2 o[4][E];
    add_up<E, 4, 2>(2, a, [&](int r, int s) { return slot_source(own, a, cta[r] + s, s == 0, at[r]); }, m, l, o);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r < count && !write_row<T, E>(first + row[r], m[r], l[r], o[r], out, lse, g, a)) again |= 1u << row[r];
  }
  while (more) {
    const int i = __ffs(more) - 1;
    more &= more - 1;
    const int x = __shfl_sync(0xffffffffu, mine.x, i), at = __shfl_sync(0xffffffffu, mine.y, i), cta = x & 0xffff;
    float m[1], l[1];
    float2 o[1][E];
    add_up<E, 1, 8>((x >> 16) - cta + 1, a, [&](int, int s) { return slot_source(own, a, cta + s, s == 0, at); }, m, l, o);
    if (!write_row<T, E>(first + i, m[0], l[0], o[0], out, lse, g, a)) again |= 1u << i;
  }
  while (again) {
    const int64_t row = first + __ffs(again) - 1, t = row / a.nq;
    again &= again - 1;
    attend_row<T, 2 * E>(t, (int)(row - t * a.nq), q, kc, vc, out, lse, g, a);
  }
}

template <typename T>
cudaError_t launch_rows(const AttendProblem& p, const Pointers& g, const AttendArgs& a, cudaStream_t stream) {
  auto kernel = attend_rows_kernel<T>;
  const int64_t resident = (int64_t)sm_count() * resident_blocks(reinterpret_cast<const void*>(kernel), kWarps * 32);
  const int64_t grid = std::max<int64_t>(1, std::min((p.T * p.nq + kWarps - 1) / kWarps, resident));
  return launch_overlapped(kernel, (unsigned)grid, kWarps * 32, stream, static_cast<const T*>(p.query),
                           static_cast<const T*>(p.k_cache), static_cast<const T*>(p.v_cache),
                           static_cast<T*>(p.out), p.lse, g, a);
}

// ---------------------------------------------------------------------------
// The cut path: sizes of its workspace, and its launches.
// ---------------------------------------------------------------------------
int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

int padded_columns(int64_t D) { return (int)round_up(D, 64); }

// A launch of units: its kernel, rows of a unit and grid.
struct Units {
  // 16-bit data: tall or not, M = 256 / 128 (rope_attend_tc.cuh) or 16 / 8 (rope_attend_mma.cuh);
  // binary32 (rope_attend_f32.cuh): 64 or 8 / 4
  bool tall;
  int64_t M, grid;
};

// The kernel of units of M rows.
Units units_of(int64_t M, int64_t D, int32_t dtype) {
  const int cols = padded_columns(D);
  Units u;
  u.tall = M > 16;
  u.M = M;
  int per_sm = 2;
  if (u.tall) per_sm = dtype != kF32 ? 1 : cols > 128 ? f32_ctas<256>() : 2;
  u.grid = (int64_t)sm_count() * per_sm;
  return u;
}

int64_t tall_rows(int64_t D, int32_t dtype) { return dtype == kF32 ? 64 : padded_columns(D) <= 128 ? 256 : 128; }

// The kernel for B sequences of `rows` rows a key head, on average, and up to `keys` keys: small
// units up to 16 rows (16 bits: 8 rows up to 8, else 16; binary32: 4 rows up to 4, else 8; 33 sequences of 16 rows: 10 us, with units of
// 64 rows 15 us).  Beyond, K and V are read again for every small unit, and tall ones take them once
// on the 5th-generation tensor cores, or in wider products; but a tall unit takes 12 us at the least,
// so where all the work is a few small tiles a CTA they stay (107 sequences of up to 8 tokens on 63,
// 4 heads of 64: 8.9 us, tall 12.3; 20 of up to 97 on 605: 12.3, 18.5; binary32, 5 of up to 26 on 61, 16
// heads of 160: 16.4, 25.3).  Four tiles of 128 columns a CTA, and two of 256 (four of those: 22
// sequences of up to 15 tokens on 188, 10 heads of 256: 19.1 us, tall 16.4); eight in binary32.
Units units_for(double rows, int64_t B, int64_t nk, int64_t keys, int64_t D, int32_t dtype) {
  const bool f32 = dtype == kF32;
  const int64_t few = !f32 ? (rows <= 8 ? 8 : kMmaRows) : rows > 4 ? 8 : 4;
  const Units u = units_of(few, D, dtype);
  if (rows <= 16) return u;
  const double tiles = (rows / (double)few + 1) * (double)(B * nk) * (double)(keys / (f32 ? kFewKeys : kMmaKeys) + 1);
  const double most = (double)u.grid * (f32 ? 8 : 512 / padded_columns(D));
  return tiles <= most ? u : units_of(tall_rows(D, dtype), D, dtype);
}

// One launch's part of the workspace: records, partial slots, and with `dense` the rows that
// one CTA finished.
struct Part {
  int64_t rec, slots, dense, bytes;  // offsets, and all of it
  int64_t slot_rows;
};

Part part_of(int64_t T, int64_t nq, int64_t nk, int64_t D, const Units& u, bool dense) {
  Part s;
  s.slot_rows = std::min(u.M, round_up(T * (nq / nk), 16));
  s.rec = 0;
  s.slots = round_up(T * nq * 8, 256);
  s.dense = s.slots + round_up(u.grid * 2 * s.slot_rows * (D + 2) * 4, 256);
  s.bytes = s.dense + (dense ? round_up(T * nq * (D + 2) * 4, 256) : 0);
  return s;
}

// The largest part of the kernels': which one runs depends on the batch as well.
int64_t part_bytes(int64_t T, int64_t nq, int64_t nk, int64_t D, int32_t dtype, bool dense) {
  int64_t most = 0;
  for (int64_t M : {(int64_t)4, (int64_t)8, (int64_t)kMmaRows, tall_rows(D, dtype)})
    most = std::max(most, part_of(T, nq, nk, D, units_of(M, D, dtype), dense).bytes);
  return most;
}

// The unit kernels keep cache rows in 32 bits: fewer than 2^31 rows of one head (137 GB a cache
// at the smallest 64-byte rows).
bool unit_path(int64_t D, int64_t cache_rows) { return D <= 256 && cache_rows < (int64_t(1) << 31); }

Cut cut_of(const Part& s, char* at, const Units& u, int32_t dtype) {
  Cut c;
  c.grid = (int32_t)u.grid;
  c.lo = 0;
  c.prefix = 0;
  c.shared = 0;
  c.slot_rows = (int32_t)s.slot_rows;
  c.whole = whole_tiles(u.M);
  c.cost = unit_cost(dtype);
  c.solo = 0;
  c.rec = reinterpret_cast<int2*>(at + s.rec);
  c.slots = reinterpret_cast<float*>(at + s.slots);
  c.dense = reinterpret_cast<float*>(at + s.dense);
  return c;
}

template <typename T, int DP, int MR>
cudaError_t launch_mma_rows(const AttendProblem& p, const Pointers& g, const AttendArgs& a, const Cut& c, int64_t grid,
                       cudaStream_t stream) {
  auto kernel = attend_mma_kernel<T, DP, MR>;
  const size_t smem = sizeof(MmaShared<DP>);
  const cudaError_t e = opt_in_shared(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  return launch_overlapped_smem(kernel, (unsigned)grid, kMmaThreads, smem, stream, static_cast<const T*>(p.query),
                                static_cast<const T*>(p.k_cache), static_cast<const T*>(p.v_cache),
                                static_cast<T*>(p.out), p.lse, g, a, c);
}

template <typename T, int DP>
cudaError_t launch_mma(const AttendProblem& p, const Pointers& g, const AttendArgs& a, const Cut& c, const Units& u,
                       cudaStream_t stream) {
  return u.M == 8 ? launch_mma_rows<T, DP, 8>(p, g, a, c, u.grid, stream)
                  : launch_mma_rows<T, DP, kMmaRows>(p, g, a, c, u.grid, stream);
}

template <typename T, int DP>
cudaError_t launch_tc(const AttendProblem& p, const Pointers& g, const AttendArgs& a, const Cut& c, int64_t grid,
                      cudaStream_t stream) {
  auto kernel = attend_tc_kernel<T, DP>;
  const size_t smem = sizeof(TcShared<DP>);
  const cudaError_t e = opt_in_shared(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  return launch_overlapped_smem(kernel, (unsigned)grid, TcShape<DP>::kThreads, smem, stream,
                                static_cast<const T*>(p.query), static_cast<const T*>(p.k_cache),
                                static_cast<const T*>(p.v_cache), static_cast<T*>(p.out), p.lse, g, a, c);
}

template <typename K>
cudaError_t launch_f32_kernel(K kernel, size_t smem, int threads, const AttendProblem& p, const Pointers& g,
                              const AttendArgs& a, const Cut& c, int64_t grid, cudaStream_t stream) {
  const cudaError_t e = opt_in_shared(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  return launch_overlapped_smem(kernel, (unsigned)grid, threads, smem, stream, static_cast<const float*>(p.query),
                                static_cast<const float*>(p.k_cache), static_cast<const float*>(p.v_cache),
                                static_cast<float*>(p.out), p.lse, g, a, c);
}

template <int DP>
cudaError_t launch_f32(const AttendProblem& p, const Pointers& g, const AttendArgs& a, const Cut& c, const Units& u,
                       cudaStream_t stream) {
  if (u.tall)
    return launch_f32_kernel(attend_f32_kernel<DP>, sizeof(F32Shared<DP>), kF32Threads, p, g, a, c, u.grid, stream);
  if (u.M == 8)
    return launch_f32_kernel(attend_f32_few_kernel<DP, 8>, sizeof(FewShared<DP>), kFewThreads, p, g, a, c, u.grid,
                             stream);
  return launch_f32_kernel(attend_f32_few_kernel<DP, 4>, sizeof(FewShared<DP>), kFewThreads, p, g, a, c, u.grid,
                           stream);
}

template <typename T>
cudaError_t launch_units(const AttendProblem& p, const Pointers& g, const AttendArgs& a, const Cut& c, const Units& u,
                         cudaStream_t stream) {
  const int cols = padded_columns(p.D);
  if constexpr (sizeof(T) == 4) {
    if (cols <= 64) return launch_f32<64>(p, g, a, c, u, stream);
    if (cols <= 128) return launch_f32<128>(p, g, a, c, u, stream);
    return launch_f32<256>(p, g, a, c, u, stream);
  } else {
    if (u.tall) {
      if (cols <= 64) return launch_tc<T, 64>(p, g, a, c, u.grid, stream);
      if (cols <= 128) return launch_tc<T, 128>(p, g, a, c, u.grid, stream);
      return launch_tc<T, 256>(p, g, a, c, u.grid, stream);
    }
    if (cols <= 64) return launch_mma<T, 64>(p, g, a, c, u, stream);
    if (cols <= 128) return launch_mma<T, 128>(p, g, a, c, u, stream);
    if (cols <= 192) return launch_mma<T, 192>(p, g, a, c, u, stream);
    return launch_mma<T, 256>(p, g, a, c, u, stream);
  }
}

template <typename T, int E>
cudaError_t launch_join(const AttendProblem& p, const Pointers& g, const AttendArgs& a, const Cut& own, const Cut& pre,
                        cudaStream_t stream) {
  const T *q = static_cast<const T*>(p.query), *kc = static_cast<const T*>(p.k_cache),
          *vc = static_cast<const T*>(p.v_cache);
  T* const out = static_cast<T*>(p.out);
  const int64_t rows = p.T * p.nq;
  if (own.shared)
    return launch_overlapped(attend_join_both_kernel<T, E>, (unsigned)((rows + kWarps - 1) / kWarps), kWarps * 32,
                             stream, q, kc, vc, out, p.lse, g, a, own, pre);
  // one row a warp while that leaves few warps to an SM, up to 32 where most rows are finished
  const int64_t warps = (int64_t)sm_count() * 32;
  const int per_warp = (int)std::min<int64_t>(32, (rows + warps - 1) / warps);
  const int64_t grid = (rows + (int64_t)per_warp * kWarps - 1) / ((int64_t)per_warp * kWarps);
  return launch_overlapped(attend_join_kernel<T, E>, (unsigned)grid, kWarps * 32, stream, q, kc, vc, out, p.lse, g, a,
                           own, per_warp);
}

// Where no sequence can have more keys than this, no unit is split and the joining launch is saved:
// 22 sequences of 1 or 2 tokens 8.2 -> 6.8 us; 12 of 14 tokens on 369, heads of 160 16.4 -> 15.6.  With more
// keys the tiles of a unit, one after the other, take longer than the launch (4 sequences of 300, units of 16
// rows: 8.9 -> 10.3 us; binary32, 6 of up to 40 tokens on 434: 14.4 -> 25.3).
int64_t solo_keys(const Units& u, int32_t dtype) {
  if (dtype == kF32) return u.tall ? kF32Keys : 4 * kFewKeys;
  return u.tall ? 512 : 4 * kMmaKeys;
}

template <typename T>
cudaError_t launch_cut(const AttendProblem& p, const Pointers& g, const AttendArgs& a, cudaStream_t stream) {
  // rows of a sequence and key head, on average: only the lengths' sum is known here
  const double rows = (double)p.T * a.G / (double)p.B;
  // the prefix has a launch of its own where that saves re-reads of it worth more than the launch
  // (8 MB are 1.2 us of the copy bandwidth) and a sequence's rows do not fill a tile by themselves
  const double saved = (double)(p.B - 1) * (double)p.prefix_len * (double)p.nk * (double)p.D * 4;
  const bool shared = saved > 8e6 && rows < 128;
  const Units u_own = units_for(rows, p.B, p.nk, p.W * p.block_size + (shared ? 0 : p.prefix_len), p.D, p.dtype),
              u_pre = units_for((double)p.T * a.G, 1, p.nk, p.prefix_len, p.D, p.dtype);
  const Part s_own = part_of(p.T, p.nq, p.nk, p.D, u_own, shared);
  char* const ws = static_cast<char*>(p.workspace);
  Cut own = cut_of(s_own, ws, u_own, p.dtype), pre = own;
  if (shared) {
    own.shared = 1;
    own.lo = a.P;
    pre = cut_of(part_of(p.T, p.nq, p.nk, p.D, u_pre, true), ws + s_own.bytes, u_pre, p.dtype);
    pre.shared = pre.prefix = 1;
    const cudaError_t e = launch_units<T>(p, g, a, pre, u_pre, stream);
    if (e != cudaSuccess) return e;
  } else if (p.prefix_len + p.W * p.block_size <= solo_keys(u_own, p.dtype)) {
    own.whole = INT32_MAX;
    own.solo = 1;
  }
  const cudaError_t e = launch_units<T>(p, g, a, own, u_own, stream);
  if (e != cudaSuccess || own.solo) return e;
  if (p.D <= 64) return launch_join<T, 1>(p, g, a, own, pre, stream);
  if (p.D <= 128) return launch_join<T, 2>(p, g, a, own, pre, stream);
  return launch_join<T, 4>(p, g, a, own, pre, stream);
}

template <typename T>
cudaError_t launch_typed(const AttendProblem& p, cudaStream_t stream) {
  AttendArgs a;
  a.T = p.T;
  a.B = p.B;
  a.q_stride = p.q_stride;
  a.num_blocks = p.num_blocks;
  a.W = p.W;
  a.nq = (int32_t)p.nq;
  a.nk = (int32_t)p.nk;
  a.G = (int32_t)(p.nq / p.nk);
  a.D = (int32_t)p.D;
  a.block_size = (int32_t)p.block_size;
  a.bs_shift = -1;
  for (int sh = 0; sh < 31; ++sh)
    if ((int64_t(1) << sh) == p.block_size) a.bs_shift = sh;
  a.P = (int32_t)p.prefix_len;
  a.scale_log2 = (float)((double)p.scale * 1.4426950408889634074);
  const int64_t e = sizeof(T), cache = p.num_blocks * p.nk * p.block_size * p.D * e;
  a.q_span = make_span(p.query, ((p.T - 1) * p.q_stride + p.nq * p.D) * e);
  a.k_span = make_span(p.k_cache, cache);
  a.v_span = make_span(p.v_cache, cache);
  a.bt_span = make_span(p.block_table, p.B * p.W * 8);
  a.sl_span = make_span(p.seq_lens, p.B * 8);
  a.qsl_span = make_span(p.query_start_loc, (p.B + 1) * 8);
  a.pb_span = make_span(p.prefix_blocks, (p.prefix_len + p.block_size - 1) / p.block_size * 8);
  a.out_span = make_span(p.out, p.T * p.nq * p.D * e);
  a.lse_span = make_span(p.lse, p.lse ? p.T * p.nq * 4 : 0);
  Pointers g;
  g.block_table = p.block_table;
  g.seq_lens = p.seq_lens;
  g.qsl = p.query_start_loc;
  g.prefix_blocks = p.prefix_blocks;
  const cudaError_t er = device_error_address(&g.err);
  if (er != cudaSuccess) return er;
  if (unit_path(p.D, p.num_blocks * p.nk * p.block_size)) return launch_cut<T>(p, g, a, stream);
  return launch_rows<T>(p, g, a, stream);
}

}  // namespace

int64_t attend_workspace(int64_t T, int64_t nq, int64_t nk, int64_t D, int32_t dtype, int64_t prefix_len) {
  if (!unit_path(D, 0)) return 256;
  const bool shared = prefix_len > 0;
  return std::max<int64_t>(256, part_bytes(T, nq, nk, D, dtype, shared) * (shared ? 2 : 1));
}

cudaError_t launch_attend(const AttendProblem& p, cudaStream_t stream) {
  switch (p.dtype) {
    case kF32:
      return launch_typed<float>(p, stream);
    case kF16:
      return launch_typed<__half>(p, stream);
    case kBF16:
      return launch_typed<__nv_bfloat16>(p, stream);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace rope
