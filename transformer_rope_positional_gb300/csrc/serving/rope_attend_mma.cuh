// Attention units of up to 16 query rows: decoding steps, short drafts.
//
// Bound by the cache's bytes: a unit of 16 rows does 32 operations per byte of K and V, far
// below the matrix units' 280, so the kernel is built to keep loads in flight.
//  * A CTA's four warps each take 16 keys of every 64-key tile and run on their own, each with
//    its own ring of copies (rope_attend_ring.cuh) and its own running m, l and O; there is no
//    barrier until the unit ends, and the copies of the next unit are already on their way
//    then.  Two CTAs an SM, so that one copies while the other ends a unit (heads of 256 with
//    one CTA: 105 us for the own keys of 32 drafts, with two 58).
//  * Scores and outputs by mma.sync m16n8k16: the tensor core's newer instruction wants 64 or 128
//    rows a tile, and these units have 1 to 16.  Units of 16 rows take them as the 16 of the
//    instruction; units of 8 as its 8, keys (then columns of V) being the 16: half the products
//    and half the registers for O (32 of up to 5 drafted tokens, heads of 256: 62.2 us with 16
//    rows, 59.0 with 8).
//  * The weights of a score tile are, register for register, the A operand of the product
//    with V (8 rows: transposed, its B operand).  They are rounded to the data's type there (half
//    a step relative each, the sums l taken before); m, l and O stay in binary32.  binary16's
//    exponents end at 2^-14 (2^-24 in its subnormals), so its weights are taken 2^15 times as large
//    (see weight_lift): from 2^-29 of the largest on the half step is relative, and what is below is
//    off by 2^-40 of the largest at most.  (Without, 20000 keys 17.6 nats below one vanished from O
//    but not from l.)
//
// 64 requests of up to 8192 tokens, 32 q and 8 k heads of 128, bf16: 174 us, 6.4 TB/s, 0.94 of
// the measured copy bandwidth.  4 requests of 300 tokens: 8.0 us with the joining kernel, all of
// it latency (lengths, pages, rows, two launches).
#pragma once

#include <type_traits>

#include "rope_attend_ring.cuh"

namespace rope {
namespace attend {

constexpr int kMmaThreads = 128;
constexpr int kMmaRows = 16;
constexpr int kMmaKeys = 64;

// Stages of 16 rows of K or of V in a warp's ring, and rows of the four warps that are put
// together at a time: as many as let two CTAs share an SM.
template <int DP>
struct MmaShape {
  static constexpr int kStages = DP <= 64 ? 11 : DP <= 128 ? 6 : DP <= 192 ? 4 : 3;
  static constexpr int kJoin = DP <= 128 ? 4 : 2;
  static constexpr int kStage = 16 * DP * 2;  // bytes
};

template <int DP>
struct MmaShared {
  using S = MmaShape<DP>;
  alignas(1024) unsigned char ring[4][S::kStages][S::kStage];
  alignas(16) unsigned char q[16 * DP * 2];
  float o[4][S::kJoin][DP + 8];
  float ml[4][16][2];
  int bad;  // some finished row is not finite
  int64_t tmp[kMmaThreads / 32 + 2];
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], unsigned at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], unsigned at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit values, two of a row a lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack2(const __half*, float x, float y) {
  const __half2 v = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(const __nv_bfloat16*, float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Weights of up to 2^over are taken 2^lift times as large: up to 2^15 in binary16, whose largest
// value is just below 2^16; as they are in bfloat16, whose exponents are binary32's.  l and O are of
// the same weights, so the m that leaves with them is smaller by lift.
template <typename T>
__host__ __device__ constexpr int weight_lift(int over) {
  return std::is_same<T, __half>::value ? 15 - over : 0;
}

// DP: D rounded up to a multiple of 64; columns past D are zeros in shared memory.
// MR: rows of a unit, 16 or 8.
template <typename T, int DP, int MR>
__global__ void __launch_bounds__(kMmaThreads, 2)
    attend_mma_kernel(const T* __restrict__ q, const T* __restrict__ kc, const T* __restrict__ vc, T* __restrict__ out,
                      float* __restrict__ lse, Pointers g, AttendArgs a, Cut c) {
  using Shape = MmaShape<DP>;
  constexpr int S = Shape::kStages;
  constexpr int CH = DP / 8;   // 16-byte chunks of a row
  constexpr int KS = DP / 16;  // k steps of the score product
  constexpr bool kEight = MR == 8;
  constexpr bool kHoldQ = DP <= 128;  // the row tile's A operands stay in registers
  constexpr float kLift = (float)weight_lift<T>(0);
  extern __shared__ __align__(1024) unsigned char raw[];
  MmaShared<DP>& sm = *reinterpret_cast<MmaShared<DP>*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_for_prior_grid();
  Walk w = find_share<MR, kMmaKeys, kMmaThreads>(g, a, c, sm.tmp);
  if (w.done) return;
  if (threadIdx.x == 0) sm.bad = 0;

  Ring<T, 16, DP, S, MR, kMmaKeys, true> ring;
  ring.start(w, sm.ring[warp][0], g, a, c);
  // a unit's query rows, in 16-byte pieces of this thread: read while the unit before ends
  constexpr int NQ = (MR * CH + kMmaThreads - 1) / kMmaThreads;
  uint4 qv[NQ];
  auto read_q = [&](const Walk& x) {
    const UnitRows u = unit_rows<MR>(x, a);
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int idx = threadIdx.x + kMmaThreads * i;
      const int r = idx / CH, ch = idx - r * CH;
      qv[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < u.rows && ch * 8 < a.D) {
        const RowAt at = row_at(u, r, x.h, a);
        const T* p = q + at.t * a.q_stride + (int64_t)at.h * a.D + ch * 8;
        if (access_ok(p, 16, a.q_span, g.err)) qv[i] = __ldg(reinterpret_cast<const uint4*>(p));
      }
    }
  };

  read_q(w);
#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) ring.copy(kc, vc, g, a, c);

  const int r0 = lane >> 2, cq = (lane & 3) * 2;
  const unsigned q_at = smem_u32(sm.q);
  // ldmatrix rows: K (and Q) by (key, chunk), V transposed
  const int k_row = ((lane >> 4) << 3) + (lane & 7), k_ch = (lane >> 3) & 1;
  const int v_row = (((lane >> 3) & 1) << 3) + (lane & 7), v_ch = lane >> 4;

  while (!w.done) {
    const UnitRows u = unit_rows<MR>(w, a);
    // ---- the unit's query rows, as A operands
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int idx = threadIdx.x + kMmaThreads * i;
      const int r = idx / CH, ch = idx - r * CH;
      if (idx < MR * CH) *reinterpret_cast<uint4*>(sm.q + r * (DP * 2) + ((ch ^ (r & 7)) << 4)) = qv[i];
    }
    __syncthreads();
    uint32_t qa[kEight ? KS / 2 : kHoldQ ? KS : 1][4];  // kEight: two steps' B operands each
    auto load_q = [&](uint32_t (&f)[4], int ks) {
      const int r = (lane & 7) + (((lane >> 3) & 1) << 3), ch = ks * 2 + (lane >> 4);
      ldmatrix4(f, q_at + r * (DP * 2) + ((ch ^ (r & 7)) << 4));
    };
    if constexpr (kEight) {
#pragma unroll
      for (int i = 0; i < KS / 2; ++i)
        ldmatrix4(qa[i], q_at + (lane & 7) * (DP * 2) + (((i * 4 + (lane >> 3)) ^ (lane & 7)) << 4));
    } else if constexpr (kHoldQ) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) load_q(qa[ks], ks);
    }
    // this lane's two rows and their limits
    const int ra = kEight ? cq : r0, rb = kEight ? cq + 1 : r0 + 8;
    int lim0 = lane < u.rows ? row_limit(w, row_at(u, lane, w.h, a).t, g, a, c) : 0;
    const int lim1 = __shfl_sync(0xffffffffu, lim0, rb);
    lim0 = __shfl_sync(0xffffffffu, lim0, ra);
    const int k1 = walk_k1(w, c);

    constexpr int NO = kEight ? DP / 16 : DP / 8;
    float o[NO][4];  // kEight: columns by rows
#pragma unroll
    for (int n = 0; n < NO; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    for (int k = w.k0; k < k1; ++k) {
      cp_async_wait<S - 2>();
      __syncwarp();
      const uint32_t there = ring.seen();
      const unsigned kt = smem_u32(ring.take(kc, vc, g, a, c));
      const int j0 = c.lo + k * kMmaKeys + warp * 16;
      if constexpr (kEight) {
        // ---- scores, keys by rows: two chains of products
        float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < KS; ks += 2) {
          uint32_t f[4];
          ldmatrix4(f, kt + v_row * (DP * 2) + (((ks * 2 + v_ch) ^ (v_row & 7)) << 4));
          mma16816<T>(s, f, qa[ks / 2][0], qa[ks / 2][1]);
          ldmatrix4(f, kt + v_row * (DP * 2) + (((ks * 2 + 2 + v_ch) ^ (v_row & 7)) << 4));
          mma16816<T>(s2, f, qa[ks / 2][2], qa[ks / 2][3]);
        }
        // ---- unseen keys, maximum, weights
        float t0 = m0, t1 = m1;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = r0 + e * 8;
          const bool in = (there >> i) & 1;
          s[2 * e] = in && j0 + i < lim0 ? (s[2 * e] + s2[2 * e]) * a.scale_log2 : -INFINITY;
          s[2 * e + 1] = in && j0 + i < lim1 ? (s[2 * e + 1] + s2[2 * e + 1]) * a.scale_log2 : -INFINITY;
          t0 = fmaxf(t0, s[2 * e]);
          t1 = fmaxf(t1, s[2 * e + 1]);
        }
#pragma unroll
        for (int d = 4; d < 32; d *= 2) {
          t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, d));
          t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, d));
        }
        const float b0 = t0 == -INFINITY ? 0.f : t0 - kLift, b1 = t1 == -INFINITY ? 0.f : t1 - kLift;
        if (__any_sync(0xffffffffu, t0 != m0 || t1 != m1)) {  // some row's maximum grew
          const float f0 = fast_exp2(m0 - kLift - b0), f1 = fast_exp2(m1 - kLift - b1);
          l0 *= f0;
          l1 *= f1;
#pragma unroll
          for (int n = 0; n < NO; ++n) {
            o[n][0] *= f0;
            o[n][1] *= f1;
            o[n][2] *= f0;
            o[n][3] *= f1;
          }
          m0 = t0;
          m1 = t1;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[2 * e] = fast_exp2(s[2 * e] - b0);
          s[2 * e + 1] = fast_exp2(s[2 * e + 1] - b1);
          l0 += s[2 * e];
          l1 += s[2 * e + 1];
        }
        // (rows, keys) from (keys, rows): the B operand
        const uint32_t p0 = transposed(pack2((const T*)nullptr, s[0], s[1]));
        const uint32_t p1 = transposed(pack2((const T*)nullptr, s[2], s[3]));
        // ---- outputs
        cp_async_wait<S - 2>();
        __syncwarp();
        const unsigned vt = smem_u32(ring.take(kc, vc, g, a, c));
#pragma unroll
        for (int n = 0; n < NO; ++n) {
          uint32_t f[4];
          ldmatrix4_trans(f, vt + k_row * (DP * 2) + (((n * 2 + k_ch) ^ (k_row & 7)) << 4));
          mma16816<T>(o[n], f, p0, p1);
        }
        __syncwarp();
      } else {
      // ---- scores
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t b[4], f[4];
        ldmatrix4(b, kt + k_row * (DP * 2) + (((ks * 2 + k_ch) ^ (k_row & 7)) << 4));
        if constexpr (!kHoldQ) load_q(f, ks);
        mma16816<T>(s[0], kHoldQ ? qa[kHoldQ ? ks : 0] : f, b[0], b[1]);
        mma16816<T>(s[1], kHoldQ ? qa[kHoldQ ? ks : 0] : f, b[2], b[3]);
      }
      // ---- unseen keys, maximum, weights
      float t0 = m0, t1 = m1;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = n * 8 + cq + e;
          const bool in = (there >> i) & 1;
          s[n][e] = in && j0 + i < lim0 ? s[n][e] * a.scale_log2 : -INFINITY;
          s[n][2 + e] = in && j0 + i < lim1 ? s[n][2 + e] * a.scale_log2 : -INFINITY;
          t0 = fmaxf(t0, s[n][e]);
          t1 = fmaxf(t1, s[n][2 + e]);
        }
#pragma unroll
      for (int d = 1; d < 4; d *= 2) {
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, d));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, d));
      }
      const float b0 = t0 == -INFINITY ? 0.f : t0 - kLift, b1 = t1 == -INFINITY ? 0.f : t1 - kLift;
      if (__any_sync(0xffffffffu, t0 != m0 || t1 != m1)) {  // some row's maximum grew
        const float f0 = fast_exp2(m0 - kLift - b0), f1 = fast_exp2(m1 - kLift - b1);
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int n = 0; n < DP / 8; ++n) {
          o[n][0] *= f0;
          o[n][1] *= f0;
          o[n][2] *= f1;
          o[n][3] *= f1;
        }
        m0 = t0;
        m1 = t1;
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[n][e] = fast_exp2(s[n][e] - b0);
          s[n][2 + e] = fast_exp2(s[n][2 + e] - b1);
          l0 += s[n][e];
          l1 += s[n][2 + e];
        }
      const uint32_t p[4] = {pack2((const T*)nullptr, s[0][0], s[0][1]), pack2((const T*)nullptr, s[0][2], s[0][3]),
                             pack2((const T*)nullptr, s[1][0], s[1][1]), pack2((const T*)nullptr, s[1][2], s[1][3])};
      // ---- outputs
      cp_async_wait<S - 2>();
      __syncwarp();
      const unsigned vt = smem_u32(ring.take(kc, vc, g, a, c));
#pragma unroll
      for (int n = 0; n < DP / 16; ++n) {
        uint32_t b[4];
        ldmatrix4_trans(b, vt + v_row * (DP * 2) + (((n * 2 + v_ch) ^ (v_row & 7)) << 4));
        mma16816<T>(o[2 * n], p, b[0], b[1]);
        mma16816<T>(o[2 * n + 1], p, b[2], b[3]);
      }
      __syncwarp();
      }
    }

    // ---- the four warps' rows together, a few rows at a time, to the output or a partial result
#pragma unroll
    for (int d = kEight ? 4 : 1; d < (kEight ? 32 : 4); d *= 2) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    if (kEight ? r0 == 0 : cq == 0) {
      sm.ml[warp][ra][0] = m0 - kLift;
      sm.ml[warp][ra][1] = l0;
      sm.ml[warp][rb][0] = m1 - kLift;
      sm.ml[warp][rb][1] = l1;
    }
    Walk nw = w;
    walk_next<MR, kMmaKeys>(nw, g, a, c);
    if (!nw.done) read_q(nw);
    const bool begins = w.k0 == 0, whole = begins && k1 == w.work, final = whole && !c.shared;
    float* const po = slot_o(c, a, blockIdx.x, begins ? 1 : 0);
    float* const pml = slot_ml(c, a, blockIdx.x, begins ? 1 : 0);
    constexpr int RJ = Shape::kJoin;
    for (int p0 = 0; p0 < u.rows; p0 += RJ) {
      if constexpr (kEight) {
        if (cq >= p0 && cq < p0 + RJ) {  // both of this lane's rows
          float* to = &sm.o[warp][cq - p0][r0];
#pragma unroll
          for (int n = 0; n < NO; ++n) {
            to[n * 16] = o[n][0];
            to[n * 16 + DP + 8] = o[n][1];
            to[n * 16 + 8] = o[n][2];
            to[n * 16 + 8 + DP + 8] = o[n][3];
          }
        }
      } else if ((r0 & (8 - RJ)) == (p0 & (8 - RJ))) {  // this lane has row r0 % RJ of them: r0, or r0 + 8
        float* to = &sm.o[warp][r0 & (RJ - 1)][cq];
#pragma unroll
        for (int n = 0; n < DP / 8; ++n)
          *reinterpret_cast<float2*>(to + n * 8) = p0 < 8 ? make_float2(o[n][0], o[n][1]) : make_float2(o[n][2], o[n][3]);
      }
      __syncthreads();
#pragma unroll
      for (int idx = threadIdx.x; idx < RJ * (DP / 4); idx += kMmaThreads) {  // RJ rows x DP / 4 pieces
        const int r = idx / (DP / 4), d = (idx - r * (DP / 4)) * 4;
        const int rr = p0 + r;
        if (rr >= u.rows || d >= a.D) continue;
        const float m = fmaxf(fmaxf(sm.ml[0][rr][0], sm.ml[1][rr][0]), fmaxf(sm.ml[2][rr][0], sm.ml[3][rr][0]));
        const float base = m == -INFINITY ? 0.f : m;
        float l = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float f = fast_exp2(sm.ml[j][rr][0] - base);
          const float4 x = *reinterpret_cast<const float4*>(&sm.o[j][r][d]);
          l = fmaf(sm.ml[j][rr][1], f, l);
          v.x = fmaf(x.x, f, v.x);
          v.y = fmaf(x.y, f, v.y);
          v.z = fmaf(x.z, f, v.z);
          v.w = fmaf(x.w, f, v.w);
        }
        const RowAt at = row_at(u, rr, w.h, a);
        const int64_t row = at.t * a.nq + at.h;
        if (final) {
          const float inv = inverse_sum(l, w, at.t);
          v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
          if (!(fabsf(v.x) <= FLT_MAX && fabsf(v.y) <= FLT_MAX && fabsf(v.z) <= FLT_MAX && fabsf(v.w) <= FLT_MAX &&
                l <= FLT_MAX))
            sm.bad = 1;
          Vec<T, 4> y;
          narrow2(&y.e[0], make_float2(v.x, v.y));
          narrow2(&y.e[2], make_float2(v.z, v.w));
          store_vec(out + row * a.D + d, y, a.out_span, g.err);
          if (d == 0 && lse && access_ok(lse + row, 4, a.lse_span, g.err))
            lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
        } else {
          *reinterpret_cast<float4*>(whole ? c.dense + row * a.D + d : po + rr * a.D + d) = v;
          if (d == 0) {
            float* ml = whole ? c.dense + a.T * a.nq * a.D + row * 2 : pml + rr * 2;
            *reinterpret_cast<float2*>(ml) = make_float2(m, l);
          }
        }
      }
      __syncthreads();
    }
    if (begins && !c.solo && threadIdx.x < u.rows) {
      const RowAt at = row_at(u, threadIdx.x, w.h, a);
      c.rec[at.t * a.nq + at.h] = unit_record(w, threadIdx.x, c);
    }
    w = nw;
  }
  cp_async_wait<0>();
  __syncthreads();
  if (sm.bad) mend_rows<T, DP, MR, kMmaKeys, kMmaThreads>(q, kc, vc, out, lse, g, a, c, sm.tmp);
}

}  // namespace attend
}  // namespace rope
