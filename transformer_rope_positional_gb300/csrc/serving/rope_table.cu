// cos/sin rows for given frequencies: the tables that the rotation kernels read.
//
// Row r stands for position p = first + (positions ? positions[r] : r); per frequency i
// the angle is p * f_i.
//
//  * The angle as a fraction of a turn.  The host turns f_i into w_i = f_i / 2pi mod 1 in
//    units of 2^-64, so p * w_i in wrapping 64-bit integers is the angle modulo whole turns,
//    exactly, for any p: there is no range reduction, and far positions lose nothing.  (The
//    same product in binary32 is off by a radian beyond 2^24.)  From row to row of one column
//    the angle grows by a constant: one 64-bit addition.
//  * sin and cos.  The two top bits (rounded) are the quadrant, the rest r in [-1/2, 1/2)
//    quadrants; sin(pi/2 r) = r S(r^2) and cos(pi/2 r) = C(r^2) with S and C fitted here at
//    Chebyshev nodes on [0, 1/4] (errors 6.8e-12 and 4.7e-11): 9 FMAs for both, two columns
//    in one packed instruction.
//  * One thread owns V consecutive frequencies (16 bytes of the output) and walks rows.
// About 25 instructions a value pair: the issue slots and the integer pipe are busy two thirds of the
// time, and that is twice the time of the stores: 131072 rows of 128 columns in bf16 take 10.2 us,
// 3.3 TB/s; 2048 x 64 binary32 for the in-place op 2.8 us.
#include <algorithm>
#include <cmath>

#include "rope_device.cuh"
#include "serving.h"

namespace rope {
namespace {

constexpr int kThreads = 128;
enum Layout : int { kCache = 0, kHalf = 1, kInterleave = 2 };

// Frequencies in turns of 2^-64 per position, by value in the launch (no device copy to
// keep alive, and a captured launch carries its own).
template <int N>
struct Turns {
  uint64_t w[N];
};

struct TableArgs {
  int64_t rows;
  int64_t first;
  int32_t F;
  int32_t cols;    // threads per row, ceil(F / V)
  int64_t stride;  // rows a thread steps by
  float scale;
  Span pos_span, cos_span, sin_span;
};

// What is left of the angle phase / 2^64 turns to the nearest quadrant, in quadrants: all 62
// bits count, for angles near a whole quadrant (the upper word converted, the top 23 bits of
// the lower one by an exponent put in front of them).
__device__ __forceinline__ float rest_of(uint64_t phase, uint32_t& quadrant) {
  const uint32_t hi = (uint32_t)(phase >> 32), lo = (uint32_t)phase;
  quadrant = (hi + 0x20000000u) >> 30;
  const int rest = (int)(hi - (quadrant << 30));  // [-2^29, 2^29)
  const float low = __uint_as_float(0x4b000000u | (lo >> 9)) - 8388608.0f;  // lo / 2^9
  return fmaf(low, 1.1102230246251565e-16f /* 2^-53 */, (float)rest * 9.31322574615478515625e-10f /* 2^-30 */);
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// sin and cos of two angles, scaled.
__device__ __forceinline__ void sin_cos_turn2(uint64_t p0, uint64_t p1, float scale, float2& sn, float2& cs) {
  uint32_t q0, q1;
  const float2 r = make_float2(rest_of(p0, q0), rest_of(p1, q1));
  const float2 z = __fmul2_rn(r, r);
  float2 s = __ffma2_rn(z, both(1.582063036e-4f), both(-4.681266257e-3f));
  s = __ffma2_rn(z, s, both(7.969258273e-2f));
  s = __ffma2_rn(z, s, both(-6.459640961e-1f));
  // pi/2 = 1.57079637 - 4.371139e-8: the leading term's own rounding is put back
  s = __ffma2_rn(z, s, both(-4.371139e-8f));
  s = __ffma2_rn(r, both(1.57079637050628662109375f), __fmul2_rn(r, s));
  float2 c = __ffma2_rn(z, both(9.036280664e-4f), both(-2.086006950e-2f));
  c = __ffma2_rn(z, c, both(2.536692037e-1f));
  c = __ffma2_rn(z, c, both(-1.233700541f));
  c = __ffma2_rn(z, c, both(1.0f));
  s = __fmul2_rn(s, both(scale));
  c = __fmul2_rn(c, both(scale));
  // quadrants 0..3: sin s, c, -s, -c; cos c, -s, -c, s
  auto sign = [](float v, uint32_t bit1) { return __uint_as_float(__float_as_uint(v) ^ ((bit1 << 30) & 0x80000000u)); };
  sn = make_float2(sign(q0 & 1 ? c.x : s.x, q0), sign(q1 & 1 ? c.y : s.y, q1));
  cs = make_float2(sign(q0 & 1 ? s.x : c.x, q0 + 1), sign(q1 & 1 ? s.y : c.y, q1 + 1));
}

// V frequencies per thread; VECTOR: F is a multiple of V and the outputs are 16-byte aligned.
template <typename T, int V, int LAYOUT, bool VECTOR, int N>
__global__ void __launch_bounds__(kThreads)
    table_kernel(const __grid_constant__ Turns<N> turns, const int64_t* __restrict__ positions, T* __restrict__ cos,
                 T* __restrict__ sin, unsigned int* __restrict__ err, TableArgs a) {
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  int64_t row = id / a.cols;
  if (row >= a.stride) return;  // the threads left over after whole rows
  const int i0 = (int)(id - row * a.cols) * V;
  uint64_t w[V];
#pragma unroll
  for (int e = 0; e < V; ++e) w[e] = i0 + e < a.F ? turns.w[i0 + e] : 0;
  wait_for_prior_grid();
  const int64_t width = 2 * (int64_t)a.F;
  // without positions: the angle of the first row, and what a step of rows adds to it
  uint64_t phase[V];
#pragma unroll
  for (int e = 0; e < V; ++e) phase[e] = (uint64_t)(a.first + row) * w[e];
  if (!positions) {
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] *= (uint64_t)a.stride;
  }
  for (; row < a.rows; row += a.stride) {
    if (positions) {
      const int64_t p = a.first + ldg(positions + row, a.pos_span, err);
#pragma unroll
      for (int e = 0; e < V; ++e) phase[e] = (uint64_t)p * w[e];
    }
    Vec<T, V> c, s;
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      float2 sn, cs;
      sin_cos_turn2(phase[e], phase[e + 1], a.scale, sn, cs);
      narrow2(&c.e[e], cs);
      narrow2(&s.e[e], sn);
    }
    if (!positions) {
#pragma unroll
      for (int e = 0; e < V; ++e) phase[e] += w[e];
    }
    T* const c0 = cos + row * width;
    T* const s0 = (LAYOUT == kCache ? cos : sin) + row * width;
    const Span& ss = LAYOUT == kCache ? a.cos_span : a.sin_span;
    if constexpr (VECTOR) {
      if constexpr (LAYOUT == kCache) {
        store_vec(c0 + i0, c, a.cos_span, err);
        store_vec(s0 + a.F + i0, s, ss, err);
      } else if constexpr (LAYOUT == kHalf) {
        store_vec(c0 + i0, c, a.cos_span, err);
        store_vec(c0 + a.F + i0, c, a.cos_span, err);
        store_vec(s0 + i0, s, ss, err);
        store_vec(s0 + a.F + i0, s, ss, err);
      } else {
        Vec<T, 2 * V> cc, sd;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          cc.e[2 * e] = cc.e[2 * e + 1] = c.e[e];
          sd.e[2 * e] = sd.e[2 * e + 1] = s.e[e];
        }
        store_vec(c0 + 2 * i0, cc, a.cos_span, err);
        store_vec(s0 + 2 * i0, sd, ss, err);
      }
    } else {
      auto put = [&](T* p_, T v, const Span& sp) {
        if (access_ok(p_, sizeof(T), sp, err)) *p_ = v;
      };
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int i = i0 + e;
        if (i >= a.F) break;
        if constexpr (LAYOUT == kCache) {
          put(c0 + i, c.e[e], a.cos_span);
          put(s0 + a.F + i, s.e[e], ss);
        } else {
          const int j0 = LAYOUT == kHalf ? i : 2 * i, j1 = LAYOUT == kHalf ? i + a.F : 2 * i + 1;
          put(c0 + j0, c.e[e], a.cos_span);
          put(c0 + j1, c.e[e], a.cos_span);
          put(s0 + j0, s.e[e], ss);
          put(s0 + j1, s.e[e], ss);
        }
      }
    }
  }
}

// f / 2pi modulo whole turns, in units of 2^-64: the product with 1/2pi as the sum of two
// doubles, hi exact by an FMA, so that the only rounding is the last one.  (Of |f|: the fraction
// of a small negative number is next to 1, where doubles are 2^-53 apart.)
uint64_t turns_of(double f) {
  if (f < 0) return -turns_of(-f);
  const double c1 = 0x1.45f306dc9c883p-3, c2 = -0x1.6b01ec5417056p-57;  // 1/2pi = c1 + c2
  const double hi = f * c1;
  const double lo = std::fma(f, c1, -hi) + f * c2;
  const double frac = hi - std::floor(hi);
  const double top = std::floor(frac * 0x1p32);
  const double rest = (frac * 0x1p32 - top) * 0x1p32 + lo * 0x1p64;
  return ((uint64_t)top << 32) + (uint64_t)(int64_t)std::llrint(rest);
}

template <typename T, int V, int LAYOUT, bool VECTOR, int N>
cudaError_t launch_n(const TableProblem& p, cudaStream_t stream) {
  Turns<N> t;
  for (int i = 0; i < N; ++i) t.w[i] = i < p.F ? turns_of(p.inv_freq[i]) : 0;
  TableArgs a;
  a.rows = p.rows;
  a.first = p.first;
  a.F = (int32_t)p.F;
  a.cols = (int32_t)((p.F + V - 1) / V);
  a.scale = (float)p.scale;
  a.pos_span = make_span(p.positions, p.rows * 8);
  a.cos_span = make_span(p.cos, p.rows * 2 * p.F * (int64_t)sizeof(T));
  a.sin_span = make_span(p.sin, p.rows * 2 * p.F * (int64_t)sizeof(T));
  auto kernel = table_kernel<T, V, LAYOUT, VECTOR, N>;
  // whole rows of threads: the threads of the grid are a multiple of cols, those past it idle
  const int64_t want = (p.rows * a.cols + kThreads - 1) / kThreads;
  const int64_t resident = (int64_t)sm_count() * resident_blocks(reinterpret_cast<const void*>(kernel), kThreads);
  int64_t grid = std::max<int64_t>(1, std::min(want, resident));
  grid = std::max(grid, (int64_t)(a.cols + kThreads - 1) / kThreads);
  a.stride = grid * kThreads / a.cols;
  unsigned int* err = nullptr;
  const cudaError_t e = device_error_address(&err);
  if (e != cudaSuccess) return e;
  return launch_overlapped(kernel, (unsigned)grid, kThreads, stream, t, p.positions, static_cast<T*>(p.cos),
                           static_cast<T*>(p.sin), err, a);
}

template <typename T, int LAYOUT>
cudaError_t launch_layout(const TableProblem& p, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  const bool vector = p.F % V == 0 && reinterpret_cast<uintptr_t>(p.cos) % 16 == 0 &&
                      reinterpret_cast<uintptr_t>(p.sin) % 16 == 0;
  // up to 128 frequencies (heads of 256) the launch carries 1 KB of them, else 8 KB; where the rows
  // allow no 16-byte stores a thread takes two columns, so that a warp's stores lie side by side
  // (85060 rows of 28 bf16 columns: 24.6 us with eight)
  if (p.F <= 128)
    return vector ? launch_n<T, V, LAYOUT, true, 128>(p, stream) : launch_n<T, 2, LAYOUT, false, 128>(p, stream);
  return vector ? launch_n<T, V, LAYOUT, true, 1024>(p, stream) : launch_n<T, 2, LAYOUT, false, 1024>(p, stream);
}

template <typename T>
cudaError_t launch_typed(const TableProblem& p, cudaStream_t stream) {
  if (!p.sin) return launch_layout<T, kCache>(p, stream);
  return p.interleave ? launch_layout<T, kInterleave>(p, stream) : launch_layout<T, kHalf>(p, stream);
}

}  // namespace

cudaError_t launch_table(const TableProblem& p, cudaStream_t stream) {
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
