// Attention units of binary32 data.
//
// The matrix units have no binary32 product (tf32 keeps 11 bits), so this is ordinary FMAs: they
// take longer than the cache's bytes once a unit has more than about 20 rows.
//
// Many rows (attend_f32_kernel):
//  * A unit is 64 rows with tiles of 64 keys, 256 threads as 16 x 16.  For scores a thread has
//    4 rows x 4 keys, for outputs 4 rows x DP / 16 columns, so that each 16-byte read from
//    shared memory feeds 16 FMAs; pairs of them in one packed instruction.
//  * K and V have one buffer each, filled by cp.async in turn: V arrives while the scores are
//    computed, the next K while the outputs are.  Rows of Q and K are kept with their 16-byte
//    pieces rotated (piece ^ (row & 7)), which spreads the 16 keys of a read over the banks.
//  * A prompt of 4096 tokens, 8 q and 2 k heads of 128: 0.93 ms, 37 TFLOP/s.  Bound by the reads from
//    shared memory, whose data path is busy 79 % of the time, the FMA pipe 32 %.
//
// Few rows (attend_f32_few_kernel), decoding steps and short drafts: a unit is 4 or 8 rows.  As
// in rope_attend_mma.cuh each warp has its own ring of copies and its own m, l and O.  A lane
// owns DP / 32 columns of Q, K, V and O; the partial scores of 8 keys x 4 rows are summed over
// the lanes by halving: 31 shuffles for 32 sums, each lane ending with one of them.
//
// 64 requests of up to 335 tokens, 16 q and 4 k heads of 160: 24 us (8.5 us of bytes; units of 64
// rows took 78): issue slots and shared memory are busy a third of the time each, what is left is
// the latency of sums over the lanes between a tile's reads; 6 ragged sequences behind 101 tokens: 14
// us, latency.
#pragma once

#include "rope_attend.cuh"
#include "rope_attend_ring.cuh"

namespace rope {
namespace attend {

constexpr int kF32Threads = 256;
constexpr int kF32Keys = 64;

template <int DP>
struct F32Shared {
  static constexpr int M = 64;
  alignas(16) float q[M * DP];
  alignas(16) float k[kF32Keys * DP];
  alignas(16) float v[kF32Keys * DP];
  alignas(16) float p[kF32Keys * M];  // weights, [key][row]
  int32_t rows[2][kF32Keys];          // cache rows of this and the next tile
  int bad;                            // some finished row is not finite
};

template <int DP>
__host__ __device__ constexpr int f32_ctas() {
  return sizeof(F32Shared<DP>) <= 113 * 1024 ? 2 : 1;
}

__device__ __forceinline__ float2 lo2(const float4& v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 hi2(const float4& v) { return make_float2(v.z, v.w); }

template <int DP>
__global__ void __launch_bounds__(kF32Threads, f32_ctas<DP>())
    attend_f32_kernel(const float* __restrict__ q, const float* __restrict__ kc, const float* __restrict__ vc,
                      float* __restrict__ out, float* __restrict__ lse, Pointers g, AttendArgs a, Cut c) {
  constexpr int RPT = 4, M = 16 * RPT, KT = kF32Keys, CH = DP / 4, NC = DP / 64;
  extern __shared__ __align__(1024) unsigned char raw[];
  F32Shared<DP>& sm = *reinterpret_cast<F32Shared<DP>*>(raw);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  wait_for_prior_grid();
  Walk w = find_share<M, kF32Keys, kF32Threads>(g, a, c, reinterpret_cast<int64_t*>(sm.p));
  if (w.done) return;
  if (tid == 0) sm.bad = 0;
  while (!w.done) {
    const int k1 = walk_k1(w, c);
    const int end = tile_end<M>(w.s, w.i, a, c);
    const UnitRows u = unit_rows<M>(w, a);
    const int64_t* table = g.block_table + w.b * a.W;
    // page of key tid (< 64) of tile k, and a tile later its cache row, into rows[k & 1]
    PageRow page = {-2, 0};
    auto look_up = [&](int k) {
      page = {-2, 0};
      const int j = c.lo + k * KT + tid;
      if (tid < KT && k < k1 && j < end) page = page_row(j, table, g, a);
    };
    auto keep_row = [&](int k) {
      if (tid < KT) {
        int r = -1;
        if (page.page >= 0 && page.page < a.num_blocks)
          r = ((int)page.page * a.nk + w.h) * a.block_size + page.row;
        else if (page.page != -2)
          atomicOr(g.err, kSlotOutOfRange);
        sm.rows[k & 1][tid] = r;
      }
    };
    auto copy = [&](int k, float* dst, const float* __restrict__ src, const Span& span, bool rotate) {
      for (int idx = tid; idx < KT * CH; idx += kF32Threads) {
        const int key = idx / CH, ch = idx - key * CH;
        const int r = sm.rows[k & 1][key];
        const bool there = r >= 0 && ch * 4 < a.D;
        const float* p = src + (there ? (int64_t)r * a.D + ch * 4 : 0);
        cp_async16_or_zero(smem_u32(dst + key * DP + ((rotate ? ch ^ (key & 7) : ch) << 2)), p,
                           there && access_ok(p, 16, span, g.err));
      }
      cp_async_commit();
    };
    look_up(w.k0);
    keep_row(w.k0);
    look_up(w.k0 + 1);
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
      keep_row(k + 1);
      look_up(k + 2);
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
        *reinterpret_cast<float4*>(p) = make_float4(w4[j][0], w4[j][1], w4[j][2], w4[j][3]);
      }
      cp_async_wait<0>();
      __syncthreads();  // V and the weights are there; K is no longer read
      if (k + 1 < k1) copy(k + 1, sm.k, kc, a.k_span, true);
      // ---- outputs: RPT rows x columns 4 tx + 64 n
#pragma unroll 4
      for (int key = 0; key < KT; ++key) {
        const float4 p4 = *reinterpret_cast<const float4*>(sm.p + key * M + ty * 4);
        const float p[RPT] = {p4.x, p4.y, p4.z, p4.w};
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
      const float f = !final ? 1.f : mine ? inverse_sum(l[i], w, at.t) : 0.f;
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
        if (final && !all_fine) sm.bad = 1;
        if (begins && !c.solo) c.rec[row] = unit_record(w, r, c);
      }
    }
    __syncthreads();  // the buffers are free
    walk_next<M, kF32Keys>(w, g, a, c);
  }
  if (sm.bad)
    mend_rows<float, DP, M, kF32Keys, kF32Threads>(q, kc, vc, out, lse, g, a, c, reinterpret_cast<int64_t*>(sm.p));
}

// ---------------------------------------------------------------------------
// Few rows.
// ---------------------------------------------------------------------------
constexpr int kFewThreads = 128;
constexpr int kFewKeys = 32;  // of a tile: 8 a warp

template <int DP>
struct FewShape {
  static constexpr int kStages = DP <= 64 ? 11 : DP <= 128 ? 6 : 3;
  static constexpr int kJoin = DP <= 128 ? 4 : 2;  // rows of the four warps put together at a time
};

template <int DP>
struct FewShared {
  alignas(16) float ring[4][FewShape<DP>::kStages][8 * DP];
  alignas(16) float o[4][FewShape<DP>::kJoin][DP];
  float ml[4][8][2];
  int bad;  // some finished row is not finite
  int64_t tmp[kFewThreads / 32 + 2];
};

// Sums of v[0 .. 31] over the lanes: lane i gets the one of v[i].
__device__ __forceinline__ float lane_sums(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 16; n > 0; n /= 2) {
    const bool up = lane & n;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = up ? v[i + n] : v[i], give = up ? v[i] : v[i + n];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, n);
    }
  }
  return v[0];
}

// E = DP / 32 columns of this lane: pairs 2 lane + 64 n, or for E a multiple of 4, fours 4 lane + 128 n.
template <int E>
struct LaneColumns {
  float2 v[E / 2];
  static __device__ __forceinline__ int column(int n) {  // of the pair v[n]
    const int lane = threadIdx.x & 31;
    return E % 4 ? 2 * lane + 64 * n : 4 * lane + 128 * (n >> 1) + 2 * (n & 1);
  }
  __device__ __forceinline__ void read(const float* row) {
    if constexpr (E % 4) {
#pragma unroll
      for (int n = 0; n < E / 2; ++n) v[n] = *reinterpret_cast<const float2*>(row + column(n));
    } else {
#pragma unroll
      for (int n = 0; n < E / 2; n += 2) {
        const float4 x = *reinterpret_cast<const float4*>(row + column(n));
        v[n] = lo2(x);
        v[n + 1] = hi2(x);
      }
    }
  }
};

// R: rows of a unit, 4 or 8.
template <int DP, int R>
__global__ void __launch_bounds__(kFewThreads, 2)
    attend_f32_few_kernel(const float* __restrict__ q, const float* __restrict__ kc, const float* __restrict__ vc,
                          float* __restrict__ out, float* __restrict__ lse, Pointers g, AttendArgs a, Cut c) {
  constexpr int S = FewShape<DP>::kStages, E = DP / 32, RG = R / 4, RJ = FewShape<DP>::kJoin;
  extern __shared__ __align__(1024) unsigned char raw[];
  FewShared<DP>& sm = *reinterpret_cast<FewShared<DP>*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int my_row = lane >> 3, my_key = lane & 7;  // of each group of 4 rows x 8 keys
  wait_for_prior_grid();
  Walk w = find_share<R, kFewKeys, kFewThreads>(g, a, c, sm.tmp);
  if (w.done) return;
  if (threadIdx.x == 0) sm.bad = 0;
  Ring<float, 8, DP, S, R, kFewKeys, false> ring;
  ring.start(w, reinterpret_cast<unsigned char*>(sm.ring[warp][0]), g, a, c);
#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) ring.copy(kc, vc, g, a, c);

  while (!w.done) {
    const UnitRows u = unit_rows<R>(w, a);
    LaneColumns<E> qv[R], o[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int n = 0; n < E / 2; ++n) {
        o[r].v[n] = make_float2(0.f, 0.f);
        qv[r].v[n] = make_float2(0.f, 0.f);
        const int d = LaneColumns<E>::column(n);
        if (r < u.rows && d < a.D) {
          const RowAt at = row_at(u, r, w.h, a);
          const float* p = q + at.t * a.q_stride + (int64_t)at.h * a.D + d;
          if (access_ok(p, 8, a.q_span, g.err)) qv[r].v[n] = __ldg(reinterpret_cast<const float2*>(p));
        }
      }
    }
    int limit[RG];
    float m[RG], l[RG];  // of row 4 i + my_row; l of this lane's keys
#pragma unroll
    for (int i = 0; i < RG; ++i) {
      const int r = 4 * i + my_row;
      limit[i] = r < u.rows ? row_limit(w, row_at(u, r, w.h, a).t, g, a, c) : 0;
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
    const int k1 = walk_k1(w, c);
    for (int k = w.k0; k < k1; ++k) {
      cp_async_wait<S - 2>();
      __syncwarp();
      const uint32_t there = ring.seen();
      const float* kt = reinterpret_cast<const float*>(ring.take(kc, vc, g, a, c));
      const int j = c.lo + k * kFewKeys + warp * 8 + my_key;
      float p[RG];
#pragma unroll
      for (int i = 0; i < RG; ++i) {
        float s[32];  // [row][key]
#pragma unroll
        for (int key = 0; key < 8; ++key) {
          LaneColumns<E> kv;
          kv.read(kt + key * DP);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float2 x = make_float2(0.f, 0.f);
#pragma unroll
            for (int n = 0; n < E / 2; ++n) x = __ffma2_rn(qv[4 * i + r].v[n], kv.v[n], x);
            s[r * 8 + key] = x.x + x.y;
          }
        }
        const float dot = lane_sums(s);
        const float x = ((there >> my_key) & 1) && j < limit[i] ? dot * a.scale_log2 : -INFINITY;
        float top = fmaxf(m[i], x);
#pragma unroll
        for (int d = 1; d < 8; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float base = top == -INFINITY ? 0.f : top;
        if (__any_sync(0xffffffffu, top != m[i])) {  // some row's maximum grew
          const float f = exp2f(m[i] - base);
          l[i] *= f;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float fr = __shfl_sync(0xffffffffu, f, r * 8);
#pragma unroll
            for (int n = 0; n < E / 2; ++n) o[4 * i + r].v[n] = __fmul2_rn(o[4 * i + r].v[n], make_float2(fr, fr));
          }
          m[i] = top;
        }
        p[i] = exp2f(x - base);
        l[i] += p[i];
      }
      cp_async_wait<S - 2>();
      __syncwarp();
      const float* vt = reinterpret_cast<const float*>(ring.take(kc, vc, g, a, c));
#pragma unroll
      for (int key = 0; key < 8; ++key) {
        LaneColumns<E> vv;
        vv.read(vt + key * DP);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float pr = __shfl_sync(0xffffffffu, p[r / 4], (r % 4) * 8 + key);
#pragma unroll
          for (int n = 0; n < E / 2; ++n) o[r].v[n] = __ffma2_rn(make_float2(pr, pr), vv.v[n], o[r].v[n]);
        }
      }
      __syncwarp();
    }

    // ---- the four warps' rows together, a few rows at a time, to the output or a partial result
#pragma unroll
    for (int i = 0; i < RG; ++i) {
#pragma unroll
      for (int d = 1; d < 8; d *= 2) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
      if (my_key == 0) {
        sm.ml[warp][4 * i + my_row][0] = m[i];
        sm.ml[warp][4 * i + my_row][1] = l[i];
      }
    }
    const bool begins = w.k0 == 0, whole = begins && k1 == w.work, final = whole && !c.shared;
    float* const po = slot_o(c, a, blockIdx.x, begins ? 1 : 0);
    float* const pml = slot_ml(c, a, blockIdx.x, begins ? 1 : 0);
#pragma unroll
    for (int p0 = 0; p0 < R; p0 += RJ) {
      if (p0 >= u.rows) break;
#pragma unroll
      for (int r = 0; r < RJ; ++r)
#pragma unroll
        for (int n = 0; n < E / 2; ++n)
          *reinterpret_cast<float2*>(&sm.o[warp][r][LaneColumns<E>::column(n)]) = o[p0 + r].v[n];
      __syncthreads();
      for (int idx = threadIdx.x; idx < RJ * (DP / 4); idx += kFewThreads) {
        const int r = idx / (DP / 4), d = (idx - r * (DP / 4)) * 4;
        const int rr = p0 + r;
        if (rr >= u.rows || d >= a.D) continue;
        const float top = fmaxf(fmaxf(sm.ml[0][rr][0], sm.ml[1][rr][0]), fmaxf(sm.ml[2][rr][0], sm.ml[3][rr][0]));
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f = exp2f(sm.ml[e][rr][0] - base);
          const float4 x = *reinterpret_cast<const float4*>(&sm.o[e][r][d]);
          sum = fmaf(sm.ml[e][rr][1], f, sum);
          v.x = fmaf(x.x, f, v.x);
          v.y = fmaf(x.y, f, v.y);
          v.z = fmaf(x.z, f, v.z);
          v.w = fmaf(x.w, f, v.w);
        }
        const RowAt at = row_at(u, rr, w.h, a);
        const int64_t row = at.t * a.nq + at.h;
        if (final) {
          const float inv = inverse_sum(sum, w, at.t);
          v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
          if (!(fabsf(v.x) <= FLT_MAX && fabsf(v.y) <= FLT_MAX && fabsf(v.z) <= FLT_MAX && fabsf(v.w) <= FLT_MAX &&
                sum <= FLT_MAX))
            sm.bad = 1;
          float* to = out + row * a.D + d;
          if (access_ok(to, 16, a.out_span, g.err)) *reinterpret_cast<float4*>(to) = v;
          if (d == 0 && lse && access_ok(lse + row, 4, a.lse_span, g.err))
            lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.693147180559945309f;
        } else {
          *reinterpret_cast<float4*>(whole ? c.dense + row * a.D + d : po + rr * a.D + d) = v;
          if (d == 0) {
            float* ml = whole ? c.dense + a.T * a.nq * a.D + row * 2 : pml + rr * 2;
            *reinterpret_cast<float2*>(ml) = make_float2(top, sum);
          }
        }
      }
      __syncthreads();
    }
    if (begins && !c.solo && threadIdx.x < u.rows) {
      const RowAt at = row_at(u, threadIdx.x, w.h, a);
      c.rec[at.t * a.nq + at.h] = unit_record(w, threadIdx.x, c);
    }
    walk_next<R, kFewKeys>(w, g, a, c);
  }
  cp_async_wait<0>();
  __syncthreads();
  if (sm.bad) mend_rows<float, DP, R, kFewKeys, kFewThreads>(q, kc, vc, out, lse, g, a, c, sm.tmp);
}

}  // namespace attend
}  // namespace rope
