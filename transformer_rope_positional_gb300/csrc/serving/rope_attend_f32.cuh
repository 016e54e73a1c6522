// Attention units of binary32 data.
//
// The matrix units have no binary32 product (tf32 keeps 11 bits), so this is ordinary FMAs:
// bound by their rate once a unit has more than about 20 rows, by the cache's bytes below.
//  * A unit is 64 rows (or 16: decoding) with tiles of 64 keys, 256 threads as 16 x 16.  For
//    scores a thread has RPT rows x 4 keys, for outputs RPT rows x DP / 16 columns, so that
//    each 16-byte read from shared memory feeds 16 (4) FMAs; pairs of them in one packed
//    instruction.
//  * K and V have one buffer each, filled by cp.async in turn: V arrives while the scores are
//    computed, the next K while the outputs are.  Rows of Q and K are kept with their 16-byte
//    pieces rotated (piece ^ (row & 7)), which spreads the 16 keys of a read over the banks.
#pragma once

#include "rope_attend.cuh"
#include "rope_attend_mma.cuh"

namespace rope {
namespace attend {

constexpr int kF32Threads = 256;
constexpr int kF32Keys = 64;

template <int DP, int RPT>
struct F32Shared {
  static constexpr int M = 16 * RPT;
  alignas(16) float q[M * DP];
  alignas(16) float k[kF32Keys * DP];
  alignas(16) float v[kF32Keys * DP];
  alignas(16) float p[kF32Keys * M];  // weights, [key][row]
  int64_t rows[2][kF32Keys];          // cache rows of this and the next tile
};

template <int DP, int RPT>
__host__ __device__ constexpr int f32_ctas() {
  return RPT == 1 && sizeof(F32Shared<DP, RPT>) <= 75 * 1024 ? 3 : sizeof(F32Shared<DP, RPT>) <= 113 * 1024 ? 2 : 1;
}

__device__ __forceinline__ float2 lo2(const float4& v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 hi2(const float4& v) { return make_float2(v.z, v.w); }

template <int DP, int RPT>
__global__ void __launch_bounds__(kF32Threads, f32_ctas<DP, RPT>())
    attend_f32_kernel(const float* __restrict__ q, const float* __restrict__ kc, const float* __restrict__ vc,
                      float* __restrict__ out, float* __restrict__ lse, Pointers g, AttendArgs a, Cut c) {
  constexpr int M = 16 * RPT, KT = kF32Keys, CH = DP / 4, NC = DP / 64;
  extern __shared__ __align__(1024) unsigned char raw[];
  F32Shared<DP, RPT>& sm = *reinterpret_cast<F32Shared<DP, RPT>*>(raw);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  wait_for_prior_grid();
  Walk w = find_share<M, kF32Keys, kF32Threads>(g, a, c, reinterpret_cast<int64_t*>(sm.p));
  while (!w.done) {
    const int k1 = walk_k1(w);
    const int end = tile_end<M>(w.s, w.i, a, c);
    const UnitRows u = unit_rows<M>(w, a);
    const int64_t* table = g.block_table + w.b * a.W;
    // cache row of key tid (< 64) of tile k, into rows[k & 1]
    auto look_up = [&](int k) {
      if (tid < KT) {
        const int j = c.lo + k * KT + tid;
        int64_t r = -1;
        if (k < k1 && j < end) {
          r = key_row(j, table, g, a);
          if (r < 0) atomicOr(g.err, kSlotOutOfRange);
          else r = (r + (int64_t)w.h * a.block_size) * a.D;
        }
        sm.rows[k & 1][tid] = r;
      }
    };
    auto copy = [&](int k, float* dst, const float* __restrict__ src, const Span& span, bool rotate) {
      for (int idx = tid; idx < KT * CH; idx += kF32Threads) {
        const int key = idx / CH, ch = idx - key * CH;
        const int64_t at = sm.rows[k & 1][key];
        const bool there = at >= 0 && ch * 4 < a.D;
        const float* p = src + (there ? at + ch * 4 : 0);
        cp_async16_or_zero(smem_u32(dst + key * DP + ((rotate ? ch ^ (key & 7) : ch) << 2)), p,
                           there && access_ok(p, 16, span, g.err));
      }
      cp_async_commit();
    };
    look_up(w.k0);
    for (int idx = tid; idx < M * CH; idx += kF32Threads) {
      const int r = idx / CH, ch = idx - r * CH;
      const bool there = r < u.rows && ch * 4 < a.D;
      const RowAt at = row_at(u, r, w.h, a);
      const float* p = q + (there ? at.t * a.q_stride + (int64_t)at.h * a.D + ch * 4 : 0);
      cp_async16_or_zero(smem_u32(sm.q + r * DP + ((ch ^ (r & 7)) << 2)), p,
                         there && access_ok(p, 16, a.q_span, g.err));
    }
    __syncthreads();
    copy(w.k0, sm.k, kc, a.k_span, true);  // one group with Q
    int limit[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i)
      limit[i] = ty * RPT + i < u.rows ? row_limit(w, row_at(u, ty * RPT + i, w.h, a).t, g, a, c) : 0;
    float m[RPT], l[RPT];
    float2 o[RPT][NC * 2];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < NC * 2; ++j) o[i][j] = make_float2(0.f, 0.f);
    }
    for (int k = w.k0; k < k1; ++k) {
      look_up(k + 1);
      cp_async_wait<0>();
      __syncthreads();  // K (and Q) are there; the last outputs are done with V
      copy(k, sm.v, vc, a.v_span, false);
      // ---- scores of RPT rows x keys tx, tx + 16, tx + 32, tx + 48
      float2 s2[RPT][4];
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s2[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int ch = 0; ch < CH; ++ch) {
        float4 qv[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const int r = ty * RPT + i;
          qv[i] = *reinterpret_cast<const float4*>(sm.q + r * DP + ((ch ^ (r & 7)) << 2));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = tx + 16 * j;
          const float4 kv = *reinterpret_cast<const float4*>(sm.k + key * DP + ((ch ^ (key & 7)) << 2));
#pragma unroll
          for (int i = 0; i < RPT; ++i) {
            s2[i][j] = __ffma2_rn(lo2(qv[i]), lo2(kv), s2[i][j]);
            s2[i][j] = __ffma2_rn(hi2(qv[i]), hi2(kv), s2[i][j]);
          }
        }
      }
      // ---- unseen keys, maximum, weights
      bool there[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) there[j] = sm.rows[k & 1][tx + 16 * j] >= 0;
      const int j0 = c.lo + k * KT + tx;
      float w4[4][RPT];
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        float top = m[i];
        float s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[j] = there[j] && j0 + 16 * j < limit[i] ? (s2[i][j].x + s2[i][j].y) * a.scale_log2 : -INFINITY;
          top = fmaxf(top, s[j]);
        }
#pragma unroll
        for (int d = 1; d < 16; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float base = top == -INFINITY ? 0.f : top;
        if (top != m[i]) {  // the same for the row's 16 threads
          const float f = exp2f(m[i] - base);
          l[i] *= f;
#pragma unroll
          for (int j = 0; j < NC * 2; ++j) o[i][j] = make_float2(o[i][j].x * f, o[i][j].y * f);
          m[i] = top;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w4[j][i] = exp2f(s[j] - base);
          l[i] += w4[j][i];
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float* p = sm.p + (tx + 16 * j) * M + ty * RPT;
        if constexpr (RPT == 4) *reinterpret_cast<float4*>(p) = make_float4(w4[j][0], w4[j][1], w4[j][2], w4[j][3]);
        else
#pragma unroll
          for (int i = 0; i < RPT; ++i) p[i] = w4[j][i];
      }
      cp_async_wait<0>();
      __syncthreads();  // V and the weights are there; K is no longer read
      if (k + 1 < k1) copy(k + 1, sm.k, kc, a.k_span, true);
      // ---- outputs: RPT rows x columns 4 tx + 64 n
#pragma unroll 4
      for (int key = 0; key < KT; ++key) {
        float p[RPT];
        if constexpr (RPT == 4) {
          const float4 t = *reinterpret_cast<const float4*>(sm.p + key * M + ty * 4);
          p[0] = t.x;
          p[1] = t.y;
          p[2] = t.z;
          p[3] = t.w;
        } else {
#pragma unroll
          for (int i = 0; i < RPT; ++i) p[i] = sm.p[key * M + ty * RPT + i];
        }
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          const float4 v = *reinterpret_cast<const float4*>(sm.v + key * DP + 64 * n + 4 * tx);
#pragma unroll
          for (int i = 0; i < RPT; ++i) {
            const float2 pp = make_float2(p[i], p[i]);
            o[i][2 * n] = __ffma2_rn(pp, lo2(v), o[i][2 * n]);
            o[i][2 * n + 1] = __ffma2_rn(pp, hi2(v), o[i][2 * n + 1]);
          }
        }
      }
    }
    // ---- out
    const bool begins = w.k0 == 0, whole = begins && k1 == w.work, final = whole && !c.shared;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
#pragma unroll
      for (int d = 1; d < 16; d *= 2) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
      const int r = ty * RPT + i;
      const bool mine = r < u.rows;
      const RowAt at = row_at(u, mine ? r : 0, w.h, a);
      const int64_t row = at.t * a.nq + at.h;
      const float f = !final ? 1.f : l[i] == 0.f ? 0.f : 1.f / l[i];
      float* const to = final ? out + row * a.D
                        : whole ? c.dense + row * a.D
                                : slot_o(c, a, blockIdx.x, begins ? 1 : 0) + (int64_t)r * a.D;
      bool fine = l[i] <= FLT_MAX;
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        const float4 y = make_float4(o[i][2 * n].x * f, o[i][2 * n].y * f, o[i][2 * n + 1].x * f, o[i][2 * n + 1].y * f);
        fine = fine && fabsf(y.x) <= FLT_MAX && fabsf(y.y) <= FLT_MAX && fabsf(y.z) <= FLT_MAX && fabsf(y.w) <= FLT_MAX;
        const int d = 64 * n + 4 * tx;
        if (mine && d < a.D && (!final || access_ok(to + d, 16, a.out_span, g.err)))
          *reinterpret_cast<float4*>(to + d) = y;
      }
      const unsigned half = 0xffffu << (tid & 16);
      const bool all_fine = (__ballot_sync(0xffffffffu, fine) & half) == half;
      if (mine && tx == 0) {
        if (final) {
          if (lse && access_ok(lse + row, 4, a.lse_span, g.err))
            lse[row] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.693147180559945309f;
        } else {
          float* ml = whole ? c.dense + a.T * a.nq * a.D + row * 2
                            : slot_ml(c, a, blockIdx.x, begins ? 1 : 0) + r * 2;
          *reinterpret_cast<float2*>(ml) = make_float2(m[i], l[i]);
        }
        if (begins) c.rec[row] = final && !all_fine ? make_int2(-1, -1) : unit_record(w, r);
      }
    }
    __syncthreads();  // the buffers are free
    walk_next<M, kF32Keys>(w, g, a, c);
  }
}

}  // namespace attend
}  // namespace rope
