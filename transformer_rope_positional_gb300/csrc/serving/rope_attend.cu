// Causal attention of new tokens over a paged KV cache with a shared prefix.
//
// Per query row (token t at position p, head h) over the keys j <= p it sees:
//   s_j = scale <q, k_j>,  m = max s_j,  l = sum e^(s_j - m),  o = sum e^(s_j - m) v_j / l,
// in one pass over the keys with a running m, l and o (o and l are multiplied by
// e^(m_old - m_new) when the maximum grows).  Base-2 exponentials of scale * log2(e) * <q, k>.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "rope_attend.cuh"

namespace rope {
namespace {

using namespace attend;

constexpr int kWarps = 4;

// One warp per query row: lane i holds the row's elements i, i + 32, ..., and the warp walks
// the keys in groups of four.
template <typename T, int E>
__global__ void __launch_bounds__(kWarps * 32)
    attend_rows_kernel(const T* __restrict__ q, const T* __restrict__ kc, const T* __restrict__ vc, T* __restrict__ out,
                       float* __restrict__ lse, Pointers g, AttendArgs a) {
  constexpr int KU = 4;
  const int lane = threadIdx.x & 31;
  wait_for_prior_grid();
  const int64_t rows = a.T * a.nq;
  const int64_t tokens = ldg(g.qsl + a.B, a.qsl_span, g.err);
  for (int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); row < rows; row += (int64_t)gridDim.x * kWarps) {
    const int64_t t = row / a.nq;
    if (t >= tokens) break;
    const int h = (int)(row - t * a.nq);
    const int kh = h / a.G;
    const int64_t b = batch_of(t, g, a);
    const int64_t end = ldg(g.qsl + b + 1, a.qsl_span, g.err);
    const int64_t len = ldg(g.seq_lens + b, a.sl_span, g.err);
    const int64_t most = (int64_t)a.P + a.W * a.block_size;
    if (len > most && lane == 0) atomicOr(g.err, kSlotOutOfRange);
    const int64_t seen64 = len - (end - t) + 1;  // keys the row sees
    const int seen = (int)(seen64 < 0 ? 0 : seen64 > most ? most : seen64);
    const int64_t* table = g.block_table + b * a.W;
    float qv[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int d = lane + 32 * e;
      o[e] = 0.f;
      qv[e] = d < a.D ? widen(ldg(q + t * a.q_stride + (int64_t)h * a.D + d, a.q_span, g.err)) * a.scale_log2 : 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j0 = 0; j0 < seen; j0 += KU) {
      int64_t at[KU];
      float s[KU];
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        const int64_t r = j0 + u < seen ? key_row(j0 + u, table, g, a) : -1;
        if (r < 0 && j0 + u < seen && lane == 0) atomicOr(g.err, kSlotOutOfRange);
        at[u] = r < 0 ? -1 : (r + (int64_t)kh * a.block_size) * a.D;
        s[u] = 0.f;
      }
#pragma unroll
      for (int u = 0; u < KU; ++u)
        if (at[u] >= 0) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int d = lane + 32 * e;
            if (d < a.D) s[u] = fmaf(qv[e], widen(ldg(kc + at[u] + d, a.k_span, g.err)), s[u]);
          }
        }
#pragma unroll
      for (int sh = 16; sh > 0; sh /= 2)
#pragma unroll
        for (int u = 0; u < KU; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], sh);
      float top = m;
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        if (at[u] < 0) s[u] = -INFINITY;
        top = s[u] != s[u] ? s[u] : fmaxf(top, s[u]);
      }
      const float base = top == -INFINITY ? 0.f : top;  // no key seen yet: every weight is e^(-inf - 0) = 0
      const float keep = exp2f(m - base);
      l *= keep;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= keep;
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        if (at[u] < 0) continue;
        const float w = exp2f(s[u] - base);
        l += w;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int d = lane + 32 * e;
          if (d < a.D) o[e] = fmaf(w, widen(ldg(vc + at[u] + d, a.v_span, g.err)), o[e]);
        }
      }
      m = top;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int d = lane + 32 * e;
      T* p = out + row * a.D + d;
      if (d < a.D && access_ok(p, sizeof(T), a.out_span, g.err)) *p = narrow<T>(l == 0.f ? 0.f : o[e] * inv);
    }
    if (lse && lane == 0 && access_ok(lse + row, 4, a.lse_span, g.err))
      lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
  }
}

template <typename T, int E>
cudaError_t launch_rows(const AttendProblem& p, const Pointers& g, const AttendArgs& a, cudaStream_t stream) {
  auto kernel = attend_rows_kernel<T, E>;
  const int64_t resident = (int64_t)sm_count() * resident_blocks(reinterpret_cast<const void*>(kernel), kWarps * 32);
  const int64_t grid = std::max<int64_t>(1, std::min((p.T * p.nq + kWarps - 1) / kWarps, resident));
  return launch_overlapped(kernel, (unsigned)grid, kWarps * 32, stream, static_cast<const T*>(p.query),
                           static_cast<const T*>(p.k_cache), static_cast<const T*>(p.v_cache),
                           static_cast<T*>(p.out), p.lse, g, a);
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
  if (p.D <= 64) return launch_rows<T, 2>(p, g, a, stream);
  if (p.D <= 128) return launch_rows<T, 4>(p, g, a, stream);
  if (p.D <= 256) return launch_rows<T, 8>(p, g, a, stream);
  return launch_rows<T, 16>(p, g, a, stream);
}

}  // namespace

int64_t attend_workspace(int64_t T, int64_t nq, int64_t nk, int64_t D, int32_t dtype, int64_t prefix_len) {
  (void)T, (void)nq, (void)nk, (void)D, (void)dtype, (void)prefix_len;
  return 256;
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
