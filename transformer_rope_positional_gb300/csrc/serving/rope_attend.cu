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
#include "rope_attend_join.cuh"
#include "rope_attend_mma.cuh"
#include "rope_attend_tc.cuh"

namespace rope {
namespace {

using namespace attend;

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

// The largest part of the kernels': which one runs depends on the batch as well.
int64_t part_bytes(int64_t T, int64_t nq, int64_t nk, int64_t D, int32_t dtype, bool dense) {
  int64_t most = 0;
  for (int64_t M : {(int64_t)4, (int64_t)8, (int64_t)kMmaRows, tall_rows(D, dtype)})
    most = std::max(most, part_of(T, nq, nk, D, units_of(M, D, dtype), dense).bytes);
  return most;
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
  auto kernel = attend_tc_kernel<T, DP, T>;
  const size_t smem = sizeof(TcShared<DP, false>);
  const cudaError_t e = opt_in_shared(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  return launch_overlapped_smem(kernel, (unsigned)grid, TcShape<DP, false>::kThreads, smem, stream,
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
  Pointers g;
  const cudaError_t er = arguments_of(p, sizeof(T), sizeof(T), a, g);
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
