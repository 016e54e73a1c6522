// cos/sin rows for given frequencies: the tables that the rotation kernels read.
//
// Row r stands for position p = first + (positions ? positions[r] : r); per frequency i
// the angle is p * f_i.
//
//  * The angle as a fraction of a turn.  The host turns f_i into w_i = f_i / 2pi mod 1 in
//    units of 2^-64, so p * w_i in wrapping 64-bit integers is the angle modulo whole turns,
//    exactly, for any p: there is no range reduction, and far positions lose nothing.  (The
//    same product in binary32 is off by a radian beyond 2^24; binary64 products and
//    reductions run at a sixtieth of the integer rate here.)
//  * sin and cos.  The two top bits (rounded) are the quadrant, the rest r in [-1/2, 1/2)
//    quadrants; sin(pi/2 r) = r S(r^2) and cos(pi/2 r) = C(r^2) with S and C fitted here at
//    Chebyshev nodes on [0, 1/4] (errors 6.8e-12 and 4.7e-11): 9 FMAs for both.
//  * One thread owns V consecutive frequencies (16 bytes of the output) and walks rows.
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

// sin and cos of 2 pi * phase / 2^64, scaled.
__device__ __forceinline__ void sin_cos_turn(uint64_t phase, float scale, float& sn, float& cs) {
  const uint64_t q = (phase + (uint64_t(1) << 61)) >> 62;  // nearest quadrant
  const int64_t rem = (int64_t)(phase - (q << 62));        // [-2^61, 2^61)
  const int hi = (int)(rem >> 32);
  float r = (float)hi;
  r *= 9.31322574615478515625e-10f;  // 2^-30
  // few bits left above the low word (angles near a whole quadrant): convert all 62
  if (abs(hi) < (1 << 25)) r = __ll2float_rn(rem) * 2.16840434497100886801e-19f;  // 2^-62
  const float z = r * r;
  float s = fmaf(z, 1.582063036e-4f, -4.681266257e-3f);
  s = fmaf(z, s, 7.969258273e-2f);
  s = fmaf(z, s, -6.459640961e-1f);
  // pi/2 = 1.57079637 - 4.371139e-8: the leading term's own rounding is put back
  s = fmaf(z, s, -4.371139e-8f);
  s = fmaf(r, 1.57079637050628662109375f, r * s);
  float c = fmaf(z, 9.036280664e-4f, -2.086006950e-2f);
  c = fmaf(z, c, 2.536692037e-1f);
  c = fmaf(z, c, -1.233700541f);
  c = fmaf(z, c, 1.0f);
  const bool odd = q & 1;
  const float a = odd ? c : s, b = odd ? s : c;
  // quadrants 0..3: sin s, c, -s, -c; cos c, -s, -c, s
  sn = (q & 2 ? -a : a) * scale;
  cs = ((q + 1) & 2 ? -b : b) * scale;
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
  for (; row < a.rows; row += a.stride) {
    const int64_t p = a.first + (positions ? ldg(positions + row, a.pos_span, err) : row);
    Vec<T, V> c, s;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float sn, cs;
      sin_cos_turn((uint64_t)p * w[e], a.scale, sn, cs);
      c.e[e] = narrow<T>(cs);
      s.e[e] = narrow<T>(sn);
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
// doubles, hi exact by an FMA, so that the only rounding is the last one.
uint64_t turns_of(double f) {
  const double c1 = 0x1.45f306dc9c883p-3, c2 = -0x1.6b01ec5417056p-57;  // 1/2pi = c1 + c2
  const double hi = f * c1;
  const double lo = std::fma(f, c1, -hi) + f * c2;
  const double frac = hi - std::floor(hi);
  const double top = std::floor(std::ldexp(frac, 32));
  const double rest = std::ldexp(std::ldexp(frac, 32) - top, 32) + std::ldexp(lo, 64);
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
  // up to 128 frequencies (heads of 256) the launch carries 1 KB of them, else 8 KB
  if (p.F <= 128)
    return vector ? launch_n<T, V, LAYOUT, true, 128>(p, stream) : launch_n<T, V, LAYOUT, false, 128>(p, stream);
  return vector ? launch_n<T, V, LAYOUT, true, 1024>(p, stream) : launch_n<T, V, LAYOUT, false, 1024>(p, stream);
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
