// Causal attention of new tokens over a paged KV cache of 8-bit codes with a shared prefix: the formulas of
// rope_attend.cu with k and v being code * scale.
//
// Heads of up to 256 take unit kernels (rope_attend_codes_mma.cuh for up to 16 rows a sequence and key head, for
// little work and for binary32, rope_attend_tc.cuh beyond) over the cut of rope_attend.cuh, then, where
// units may be split, a kernel that joins partial results (rope_attend_join.cuh); larger heads a kernel with one
// warp per query row.
#include <algorithm>
#include <cmath>

#include "rope_attend_codes_mma.cuh"
#include "rope_attend_join.cuh"

namespace rope {
namespace {

using namespace attend;

constexpr int kMostShared = 228 * 1024;  // bytes of an SM, 1024 of them a CTA's own
constexpr int kSmallRows = 16;  // of the larger of the small units

Units units_of(int64_t M, int64_t D, int32_t dtype) {
  Units u;
  u.tall = M > kSmallRows;
  u.M = M;
  // (CodesShape's kCtas)
  const int ctas = u.tall ? 1 : M == 8 && padded_columns(D) <= 128 && dtype != kF32 ? CodesShape<__half, 128, 8>::kCtas : 2;
  u.grid = (int64_t)sm_count() * ctas;
  return u;
}

int64_t tall_rows(int64_t D) { return padded_columns(D) <= 128 ? 256 : 128; }

int64_t tile_keys(const Units& u, int64_t D) {
  const bool narrow = padded_columns(D) <= 128;
  return u.tall ? (narrow ? 128 : 64) : narrow ? CodesShape<float, 128, 8>::KT : CodesShape<float, 256, 8>::KT;
}

// The kernel for B sequences of `rows` rows a key head, on average, and up to `keys` keys.  A tall unit takes as long as
// four small ones of 16 rows, of more than 128 columns as 2.5, however few its rows are (32 sequences of up to 1000
// keys, 32 q and 8 k heads of 128: 32 rows 62 us by tall units, 35 by small ones; 64: 64, 61; 96: 67, 86; 16 heads of 256:
// 32 rows 148, 123; 48: 149, 178).  Where all small units' tiles are in one round, these are
// the shorter ones (one sequence of 64 tokens and up to 200 keys, 256 rows: 14 us, tall 20).
Units units_for(double rows, int64_t B, int64_t nk, int64_t keys, int64_t D, int32_t dtype) {
  const Units u = units_of(rows <= 8 ? 8 : kSmallRows, D, dtype);
  if (rows <= 16 || dtype == kF32) return u;
  const int64_t worth = padded_columns(D) <= 128 ? 4 : 2;
  if (std::ceil(rows / kSmallRows) <= (double)worth * std::ceil(rows / (double)tall_rows(D))) return u;
  const double tiles = (rows / (double)u.M + 1) * (double)(B * nk) * (double)(keys / tile_keys(u, D) + 1);
  const double most = (double)u.grid * (256 / padded_columns(D));
  return tiles <= most ? u : units_of(tall_rows(D), D, dtype);
}

// The largest part of the kernels': which one runs depends on the batch as well.
int64_t part_bytes(int64_t T, int64_t nq, int64_t nk, int64_t D, int32_t dtype, bool dense) {
  int64_t most = 0;
  for (int64_t M : {(int64_t)8, (int64_t)kSmallRows, tall_rows(D)})
    if (M <= kSmallRows || dtype != kF32) most = std::max(most, part_of(T, nq, nk, D, units_of(M, D, dtype), dense).bytes);
  return most;
}

template <typename T, int DP, int MR>
cudaError_t launch_small(const AttendProblem& p, const Pointers& g, const AttendArgs& a, const Cut& c, int64_t grid,
                         cudaStream_t stream) {
  auto kernel = attend_codes_kernel<T, DP, MR>;
  using Shape = CodesShape<T, DP, MR>;
  constexpr size_t smem = sizeof(CodesShared<T, DP, MR>);
  static_assert(smem <= (kMostShared - 1024 * Shape::kCtas) / Shape::kCtas, "so many CTAs share an SM");
  const cudaError_t e = opt_in_shared(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  return launch_overlapped_smem(kernel, (unsigned)grid, kCodesThreads, smem, stream, static_cast<const T*>(p.query),
                                static_cast<const Code*>(p.k_cache), static_cast<const Code*>(p.v_cache),
                                static_cast<T*>(p.out), p.lse, g, a, c);
}

template <typename T, int DP>
cudaError_t launch_as(const AttendProblem& p, const Pointers& g, const AttendArgs& a, const Cut& c, const Units& u,
                      cudaStream_t stream) {
  return u.M == 8 ? launch_small<T, DP, 8>(p, g, a, c, u.grid, stream)
                  : launch_small<T, DP, kSmallRows>(p, g, a, c, u.grid, stream);
}

template <typename T>
cudaError_t launch_units(const AttendProblem& p, const Pointers& g, const AttendArgs& a, const Cut& c, const Units& u,
                         cudaStream_t stream) {
  if (u.tall) return launch_codes_tall(p, g, a, c, stream);
  const int cols = padded_columns(p.D);
  if (cols <= 64) return launch_as<T, 64>(p, g, a, c, u, stream);
  if (cols <= 128) return launch_as<T, 128>(p, g, a, c, u, stream);
  if (cols <= 192) return launch_as<T, 192>(p, g, a, c, u, stream);
  return launch_as<T, 256>(p, g, a, c, u, stream);
}

// Where no sequence can have more keys than this, no unit is split and the joining launch is saved (4 sequences of up to
// 200 keys: 9.3 us, split 10.8; tall, 4 of 300 tokens and up to 500 keys: 35.9, 38.5).
int64_t solo_keys(const Units& u, int64_t D) { return u.tall ? 512 : 2 * tile_keys(u, D); }

template <typename T>
cudaError_t launch_cut(const AttendProblem& p, const Pointers& g, const AttendArgs& a, cudaStream_t stream) {
  // rows of a sequence and key head, on average: only the lengths' sum is known here
  const double rows = (double)p.T * a.G / (double)p.B;
  // the prefix has a launch of its own where that saves re-reads of it worth more than the launch
  // (8 MB are 1.2 us of the copy bandwidth) and a sequence's rows do not fill a tile by themselves
  const double saved = (double)(p.B - 1) * (double)p.prefix_len * (double)p.nk * (double)p.D * 2;
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
  } else if (p.prefix_len + p.W * p.block_size <= solo_keys(u_own, p.D)) {
    own.whole = INT32_MAX;
    own.solo = 1;
  }
  const cudaError_t e = launch_units<T>(p, g, a, own, u_own, stream);
  if (e != cudaSuccess || own.solo) return e;
  if (p.D <= 64) return launch_join<T, 1, Code>(p, g, a, own, pre, stream);
  if (p.D <= 128) return launch_join<T, 2, Code>(p, g, a, own, pre, stream);
  return launch_join<T, 4, Code>(p, g, a, own, pre, stream);
}

template <typename T>
cudaError_t launch_typed(const AttendProblem& p, cudaStream_t stream) {
  AttendArgs a;
  Pointers g;
  const cudaError_t er = arguments_of(p, sizeof(T), 1, a, g);
  if (er != cudaSuccess) return er;
  if (unit_path(p.D, p.num_blocks * p.nk * p.block_size)) return launch_cut<T>(p, g, a, stream);
  return launch_rows<T, Code>(p, g, a, stream);
}

}  // namespace

int64_t attend_codes_workspace(int64_t T, int64_t nq, int64_t nk, int64_t D, int32_t dtype, int64_t prefix_len) {
  if (!unit_path(D, 0)) return 256;
  const bool shared = prefix_len > 0;
  return std::max<int64_t>(256, part_bytes(T, nq, nk, D, dtype, shared) * (shared ? 2 : 1));
}

cudaError_t launch_attend_codes(const AttendProblem& p, cudaStream_t stream) {
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
