// Attention units of up to 16 query rows over a cache of 8-bit codes: decoding steps, short drafts, and binary32
// queries of any number.
//
// Bound by the cache's bytes, half as many as rope_attend_mma.cuh's, so what a byte costs in instructions counts:
//  * As there, a CTA's four warps each take KW keys of every tile and run on their own, each with its own ring of
//    copies and its own running m, l and O, until the unit ends.
//  * The codes become binary16, exactly, on the way from shared memory to the operands of mma.sync m16n8k16, two an
//    instruction; no product sees a scale.  A score is multiplied by its key's, a power of two, in binary32.  V's
//    scale goes into the weight: with V_j = c_j 2^(b_j), O holds sum p_j 2^(b_j - B) c_j for the largest b_j so far, B
//    (one a warp), and is multiplied by 2^(B_old - B) where that grows; l is the sum of p_j.  Where that would take what
//    O holds out of binary32 (beyond 2^90 of the unit it began in) it becomes NaN, for mend_rows to find, and what is 0
//    stays 0: each lane looks at its elements of O, which are sums over all keys, not at its l, which is one over some.
//  * Which column of q and K a product's place along k stands for is free, as long as both agree, and so is which key
//    and which column of V an operand's row stands for.  A lane's places are chosen so that it reads 16 bytes of a key
//    (8 of a value) at once and has the operands of four products (of two keys and 8 columns) in its registers: no
//    ldmatrix, which knows no 8-bit elements, and no shuffles; V's bytes of two keys are put side by side by a byte
//    permutation.
//  * Queries are binary16 too.  bfloat16 and binary32 rows are multiplied by the power of two that brings their largest
//    element to [2^8, 2^9): bfloat16 stays exact down to 2^-22 of it and is off by 2^-33 of it below.  binary32 is taken as
//    the sum of two binary16 parts (off by 2^-23 of an element, or 2^-33 of the largest), with two products each.
//  * Weights are rounded to binary16 times 2^15 (see weight_lift), V's scale among them: with 2^-n of the largest scale,
//    half a step relative from 2^(n - 29) of the largest weight on, and 2^(n - 40) of it below; n is 15 at most (kNoWeight).
//    With binary32 they are two parts as well.
#pragma once

#include <climits>

#include "rope_attend_mma.cuh"

namespace rope {
namespace attend {

constexpr int kCodesThreads = 128;

// KW: keys that a warp takes of a tile.  Three CTAs an SM where registers and shared memory allow it (64 requests of up
// to 8192 tokens, 8 rows: two 101 us, issue slots half used and hardly a wait for data), else two; as many stages of a
// warp's ring as fit then.
template <typename T, int DP, int MR>
struct CodesShape {
  static constexpr int KW = DP <= 128 ? 32 : 16;
  static constexpr int KT = 4 * KW;
  static constexpr int kCtas = MR == 8 && DP <= 128 && sizeof(T) == 2 ? 3 : 2;
  static constexpr int kStages = kCtas == 3  ? (DP <= 64 ? 7 : 4)
                                 : DP <= 64  ? 10
                                 : DP <= 128 ? 5
                                 : DP <= 192 ? 6
                                             : (sizeof(T) == 4 ? 4 : 5);
  static constexpr int kStage = KW * DP;  // bytes
  static constexpr int kJoin = DP <= 128 && kCtas == 2 ? 4 : 2;
  static constexpr int kRecent = kStages <= 5 ? 4 : 8;  // tiles whose keys' scales are kept
  static constexpr int kParts = sizeof(T) == 4 ? 2 : 1;  // binary16 parts of a query
  static_assert(kStages >= 4 && kStages / 2 + 2 <= kRecent, "a tile's scales are there before it is used");
};

template <typename T, int DP, int MR>
struct CodesShared {
  using S = CodesShape<T, DP, MR>;
  alignas(1024) unsigned char ring[4][S::kStages][S::kStage];
  union {
    float o[4][S::kJoin][DP + 8];
    alignas(16) unsigned char q[MR * DP * sizeof(T)];
  };
  // query operands: of k step ks for lane l, MR = 16: four registers, 8: two
  alignas(16) uint32_t operand[S::kParts][DP / 16][32][MR / 4];
  float2 scales[4][S::kRecent][32];  // of a tile's keys: K's and V's
  uint2 there[4][S::kRecent];        // which keys are there, and the largest of V's bytes
  float ml[4][MR][2];
  int power[MR];                     // rows are times 2^power
  int first[4];                      // a warp's unit in which O was first not 0 (after NaN, again)
  int bad;                           // some finished row is not finite
  int64_t tmp[kCodesThreads / 32 + 2];
};

// Place of 16-byte piece `ch` of row `r` of a stage: chosen so that the reads below meet every bank once (V with rows of
// 192 bytes: twice).
template <int DP, bool IS_V>
__device__ __forceinline__ int piece_at(int r, int ch) {
  if constexpr (DP == 64) return ((r ^ ((r >> 1) & 1)) * 4 + (ch ^ (((r >> 2) & 1) << 1))) * 16;
  if constexpr (DP == 192) return r * DP + (IS_V ? ch ^ (((r >> 1) & 1) << 1) : ch) * 16;
  return r * DP + (IS_V ? ch ^ (((r >> 1) & 3) << 1) : ch ^ ((r & 1) << 2)) * 16;
}

// A warp's own pipeline of K and V codes (see rope_attend_ring.cuh), and of their scales.
template <typename T, int DP, int MR>
struct CodesRing {
  using S = CodesShape<T, DP, MR>;
  static constexpr int CH = DP / 16;

  Walk pw;            // unit of the next copy
  int pk, pk1, pend;  // its tile, the end of the unit's tiles here, and where its keys end
  int slot;           // stage of the next copy
  PageRow page;       // of this lane's key of the next tile
  int row;            // cache row of the key of the tile whose K was copied last
  int made;           // tiles whose K was copied
  uint32_t kb, vb;    // scale bytes of the key of that tile (0 of none: its weight is 0 times what is finite)
  int cur, tile;      // stage and tile of the next product
  unsigned char* ring;
  float2 (*scales)[32];
  uint2* there;

  __device__ __forceinline__ void look_up(const Pointers& g, const AttendArgs& a, const Cut& c) {
    page = {-2, 0};  // no such key
    if (pw.done) return;
    const int lane = threadIdx.x & 31;
    const int j = c.lo + pk * S::KT + (threadIdx.x >> 5) * S::KW + lane;
    if (lane < S::KW && j < pend) page = page_row(j, g.block_table + (int64_t)pw.b * a.W, g, a);
  }

  __device__ __forceinline__ void start(const Walk& w, unsigned char* at, float2 (*z)[32], uint2* t, const Pointers& g,
                                        const AttendArgs& a, const Cut& c) {
    pw = w;
    pk = pw.k0;
    pk1 = walk_k1(pw, c);
    pend = tile_end<MR>(pw.s, pw.i, a, c);
    slot = cur = tile = made = 0;
    row = -1;
    kb = vb = 0;
    ring = at;
    scales = z;
    there = t;
    look_up(g, a, c);
  }

  // IS_V: of V, else of the next tile's K: they take turns, and the caller knows whose it is.
  template <bool IS_V>
  __device__ __forceinline__ void copy(const Code* __restrict__ kc, const Code* __restrict__ vc, const Pointers& g,
                                       const AttendArgs& a, const Cut& c) {
    const int lane = threadIdx.x & 31;
    if constexpr (!IS_V) {
      // the scales of the tile before have arrived
      if (made > 0) {
        const int at = (made - 1) & (S::kRecent - 1);
        const uint32_t which = __ballot_sync(0xffffffffu, row >= 0);
        const uint32_t most = __reduce_max_sync(0xffffffffu, vb != 255 ? vb : 0);
        // (a V that is NaN makes its key's scores NaN, so that it counts where its weight would not)
        scales[at][lane] = make_float2(power_of(vb != 255 ? kb : 255), power_of(vb));
        if (lane == 0) there[at] = make_uint2(which, most);
      }
      ++made;
      row = -1;
      kb = vb = 0;
      if (page.page >= 0 && page.page < a.num_blocks) {
        row = ((int)page.page * a.nk + pw.h) * a.block_size + page.row;
        const uint32_t z = a.per_shift >= 0 ? (uint32_t)row >> a.per_shift : (uint32_t)row / (uint32_t)a.per;
        kb = ldg(g.k_scale + z, a.ks_span, g.err);
        vb = ldg(g.v_scale + z, a.vs_span, g.err);
      } else if (page.page != -2) {
        atomicOr(g.err, kSlotOutOfRange);
      }
      if (!pw.done) {
        if (++pk == pk1) {
          walk_next<MR, S::KT>(pw, g, a, c);
          pk = pw.k0;
          if (!pw.done) {
            pk1 = walk_k1(pw, c);
            pend = tile_end<MR>(pw.s, pw.i, a, c);
          }
        }
      }
      look_up(g, a, c);
    }
    const Code* const src = IS_V ? vc : kc;
    const Span& span = IS_V ? a.v_span : a.k_span;
    unsigned char* const to = ring + slot * S::kStage;
    const uint32_t which = __ballot_sync(0xffffffffu, row >= 0);
    const unsigned dst = smem_u32(to);
    // (heads that do not fill their columns in the loop that is unrolled, too: 96, 107 -> 90 us for 64 requests of up to 8192;
    // wider ones, with more pieces a row, lose by it: 192, 160 -> 175; by three in the other loop 160 takes 187, by one 215)
    constexpr bool kWhole = DP > 128;
    if (which == (uint32_t)((1ull << S::KW) - 1) && (!kWhole || a.D == DP)) {  // rows of all keys
#pragma unroll
      for (int i = 0; i < S::KW * CH / 32; ++i) {
        const int idx = lane + 32 * i;
        const int key = idx / CH, ch = idx - key * CH;
        const int r = __shfl_sync(0xffffffffu, row, key);
        const bool inside = kWhole || ch * 16 < a.D;
        const Code* p = src + (inside ? ch * 16 : 0) + (uint64_t)(uint32_t)r * (uint32_t)(kWhole ? DP : a.D);
        cp_async16_or_zero(dst + piece_at<DP, IS_V>(key, ch), p, inside && access_ok(p, 16, span, g.err));
      }
    } else if (which) {
#pragma unroll 3
      for (int i = 0; i < S::KW * CH / 32; ++i) {
        const int idx = lane + 32 * i;
        const int key = idx / CH, ch = idx - key * CH;
        const int r = __shfl_sync(0xffffffffu, row, key);
        const bool ok = r >= 0 && ch * 16 < a.D;
        const Code* p = src + ((uint64_t)(uint32_t)max(r, 0) * (uint32_t)a.D + (ok ? ch * 16 : 0));
        cp_async16_or_zero(dst + piece_at<DP, IS_V>(key, ch), p,
                           ok && access_ok(p, 16, span, g.err));
      }
    } else if (IS_V) {  // no key of the tile: its weights are 0, and V must not be NaN
#pragma unroll
      for (int i = 0; i < S::KW * CH / 32; ++i)
        *reinterpret_cast<uint4*>(to + (lane + 32 * i) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    cp_async_commit();
    slot = slot + 1 == S::kStages ? 0 : slot + 1;
  }

  // The next stage, once its copies are there (and its last readers done: the caller has
  // converged the warp after them); another copy, IS_V or not, is issued into the stage before it.
  template <bool IS_V>
  __device__ __forceinline__ const unsigned char* take(const Code* __restrict__ kc, const Code* __restrict__ vc,
                                                       const Pointers& g, const AttendArgs& a, const Cut& c) {
    copy<IS_V>(kc, vc, g, a, c);
    const unsigned char* at = ring + cur * S::kStage;
    cur = cur + 1 == S::kStages ? 0 : cur + 1;
    return at;
  }
};

// Where some key's V is in units of less than 2^-15 of the largest, binary16 has too few exponents for its weight: it is
// made NaN, and mend_rows finds the row, unless it is as small as this, which is taken as 0 (not in l).
constexpr float kNoWeight = 0x1p-30f;

// DP: D rounded up to a multiple of 64; columns past D are zeros in shared memory.
// MR: rows of a unit, 16 or 8.
template <typename T, int DP, int MR>
__global__ void __launch_bounds__(kCodesThreads, CodesShape<T, DP, MR>::kCtas)
    attend_codes_kernel(const T* __restrict__ q, const Code* __restrict__ kc, const Code* __restrict__ vc,
                        T* __restrict__ out, float* __restrict__ lse, Pointers g, AttendArgs a, Cut c) {
  using Shape = CodesShape<T, DP, MR>;
  using Shared = CodesShared<T, DP, MR>;
  constexpr int S = Shape::kStages, KW = Shape::KW, KT = Shape::KT;
  constexpr int KS = DP / 16;        // k steps of the score product
  constexpr int MT = KW / 16;        // products of 16 keys
  constexpr int QP = Shape::kParts;
  constexpr bool kEight = MR == 8;
  constexpr int NO = kEight ? DP / 16 : DP / 8;
  constexpr bool kHoldQ = KS * QP * (MR / 4) + NO * 4 <= 160;  // the queries' operands stay in registers
  constexpr int VEC = 16 / sizeof(T), CHT = DP / VEC;  // 16-byte pieces of a query row
  extern __shared__ __align__(1024) unsigned char raw[];
  Shared& sm = *reinterpret_cast<Shared*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_for_prior_grid();
  Walk w = find_share<MR, KT, kCodesThreads>(g, a, c, sm.tmp);
  if (w.done) return;
  if (threadIdx.x == 0) sm.bad = 0;

  CodesRing<T, DP, MR> ring;
  ring.start(w, sm.ring[warp][0], sm.scales[warp], sm.there[warp], g, a, c);
  // a unit's query rows, in 16-byte pieces of this thread: read while the unit before ends
  constexpr int NQ = (MR * CHT + kCodesThreads - 1) / kCodesThreads;
  uint4 qv[NQ];
  auto read_q = [&](const Walk& x) {
    const UnitRows u = unit_rows<MR>(x, a);
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int idx = threadIdx.x + kCodesThreads * i;
      const int r = idx / CHT, ch = idx - r * CHT;
      qv[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < u.rows && ch * VEC < a.D) {
        const RowAt at = row_at(u, r, x.h, a);
        const T* p = q + at.t * a.q_stride + (int64_t)at.h * a.D + ch * VEC;
        if (access_ok(p, 16, a.q_span, g.err)) qv[i] = __ldg(reinterpret_cast<const uint4*>(p));
      }
    }
  };

  read_q(w);
#pragma unroll 1
  for (int i = 0; i < S - 1; i += 2) {
    ring.template copy<false>(kc, vc, g, a, c);
    if (i + 1 < S - 1) ring.template copy<true>(kc, vc, g, a, c);
  }
  // (S - 1 copies are ahead: with S even the one that is issued when a K is taken is a V's)

  const int r0 = lane >> 2, cl = lane & 3, cq = cl * 2;
  // where this lane reads in a stage: key r0 (and r0 + 8, ...) of K; keys cq (and cq + 1, cq + 8, ...) of V
  unsigned k_at[DP / 64], v_at[DP / 64];
#pragma unroll
  for (int i = 0; i < DP / 64; ++i) {
    k_at[i] = piece_at<DP, false>(r0, 4 * i + cl);
    v_at[i] = piece_at<DP, true>(cq, 4 * i + (r0 >> 1)) + (r0 & 1) * 8;
  }
  // (8 keys further the same place of a row 8 rows down; the next key, where it is even, too: for rows of 64 bytes the
  // other half of the pair)
  const int next_key = DP == 64 ? piece_at<DP, true>(cq + 1, 0) - piece_at<DP, true>(cq, 0) : DP;

  while (!w.done) {
    const UnitRows u = unit_rows<MR>(w, a);
    // ---- the unit's query rows, as operands: lane (r0, cl) has columns 16 cl + 64 i + 4 ks .. + 3 of step 4 i + ks
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int idx = threadIdx.x + kCodesThreads * i;
      if (idx < MR * CHT) *reinterpret_cast<uint4*>(sm.q + idx * 16) = qv[i];
    }
    __syncthreads();
    const T* const qs = reinterpret_cast<const T*>(sm.q);
    if constexpr (!std::is_same<T, __half>::value) {
      const int r = threadIdx.x >> 3;  // 8 threads a row
      if (r < MR) {                    // (whole warps)
        float most = 0.f;
        for (int d = threadIdx.x & 7; d < DP; d += 8) most = fmaxf(most, fabsf(widen(qs[r * DP + d])));
#pragma unroll
        for (int d = 1; d < 8; d *= 2) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
        if ((threadIdx.x & 7) == 0) sm.power[r] = row_power(most);
      }
      __syncthreads();
    }
#pragma unroll
    for (int ks = warp; ks < KS; ks += 4) {
      const int d = 64 * (ks >> 2) + 16 * cl + 4 * (ks & 3);
#pragma unroll
      for (int half = 0; half < MR / 8; ++half) {
        const int r = r0 + 8 * half;
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = widen(qs[r * DP + d + e]);
        if constexpr (!std::is_same<T, __half>::value) {
          // (exact: an element that leaves binary32 downwards is below 2^-33 of the largest)
          const float up = power(sm.power[r]);
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] *= up;
        }
#pragma unroll
        for (int part = 0; part < QP; ++part) {
          sm.operand[part][ks][lane][half] = pack2((const __half*)nullptr, f[0], f[1]);
          sm.operand[part][ks][lane][half + MR / 8] = pack2((const __half*)nullptr, f[2], f[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] -= __half2float(__float2half_rn(f[e]));
        }
      }
    }
    __syncthreads();
    uint32_t qa[kHoldQ ? QP : 1][kHoldQ ? KS : 1][MR / 4];
    auto load_q = [&](uint32_t (&f)[MR / 4], int part, int ks) {
      if constexpr (kEight) {
        const uint2 v = *reinterpret_cast<const uint2*>(sm.operand[part][ks][lane]);
        f[0] = v.x, f[1] = v.y;
      } else {
        const uint4 v = *reinterpret_cast<const uint4*>(sm.operand[part][ks][lane]);
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
      }
    };
    if constexpr (kHoldQ) {
#pragma unroll
      for (int part = 0; part < QP; ++part)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) load_q(qa[part][ks], part, ks);
    }
    // this lane's two rows, their limits and their factors
    const int ra = kEight ? cq : r0, rb = kEight ? cq + 1 : r0 + 8;
    int lim0 = lane < u.rows ? row_limit(w, row_at(u, lane, w.h, a).t, g, a, c) : INT_MAX;  // (no such row: any result)
    const int lim1 = __shfl_sync(0xffffffffu, lim0, rb);
    lim0 = __shfl_sync(0xffffffffu, lim0, ra);
    float fac0 = a.scale_log2, fac1 = a.scale_log2;
    if constexpr (!std::is_same<T, __half>::value) {
      fac0 *= power(-sm.power[ra]);
      fac1 *= power(-sm.power[rb]);
    }
    const int k1 = walk_k1(w, c);

    float o[NO][4];  // kEight: columns by rows
#pragma unroll
    for (int n = 0; n < NO; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    int unit = 15;  // O is in units of 2^(unit - 142): V's largest byte so far, at least 15
    sm.first[warp] = 15;

    for (int k = w.k0; k < k1; ++k) {
      cp_async_wait<S - 2>();
      __syncwarp();
      const unsigned char* const kt = ring.template take<S % 2 == 0>(kc, vc, g, a, c);
      const int at = ring.tile++ & (Shape::kRecent - 1);
      const uint2 about = sm.there[warp][at];
      const int j0 = c.lo + k * KT + warp * KW;
      // ---- scores.  kEight: keys by rows, else rows by keys; s[mt][e][0], [1]: key or row r0 of e = 0, r0 + 8 of e = 1
      float s[MT][2][4];  // kEight: [mt][0] only
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < (kEight ? 1 : 2); ++e) s[mt][e][0] = s[mt][e][1] = s[mt][e][2] = s[mt][e][3] = 0.f;
#pragma unroll
      for (int i = 0; i < DP / 64; ++i) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint4 x = *reinterpret_cast<const uint4*>(kt + k_at[i] + mt * 16 * DP);
          const uint4 y = *reinterpret_cast<const uint4*>(kt + k_at[i] + (mt * 16 + 8) * DP);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            uint32_t f[4];  // keys r0: 0 and 2, r0 + 8: 1 and 3
            halves(ks == 0 ? x.x : ks == 1 ? x.y : ks == 2 ? x.z : x.w, f[0], f[2]);
            halves(ks == 0 ? y.x : ks == 1 ? y.y : ks == 2 ? y.z : y.w, f[1], f[3]);
#pragma unroll
            for (int part = 0; part < QP; ++part) {
              uint32_t b[MR / 4];
              if constexpr (kHoldQ) {
#pragma unroll
                for (int e = 0; e < MR / 4; ++e) b[e] = qa[part][i * 4 + ks][e];
              } else {
                load_q(b, part, i * 4 + ks);
              }
              if constexpr (kEight) {
                mma16816<__half>(s[mt][0], f, b[0], b[1]);
              } else {
                mma16816<__half>(s[mt][0], b, f[0], f[2]);
                mma16816<__half>(s[mt][1], b, f[1], f[3]);
              }
            }
          }
        }
      }
      // ---- K's scales, unseen keys, maximum
      constexpr int NK = kEight ? 2 : 4;  // keys of this lane in each 16
      auto score = [&](int mt, int e, int row) -> float& {
        return kEight ? s[mt][0][2 * e + row] : s[mt][e >> 1][2 * row + (e & 1)];
      };
      auto key_of = [&](int mt, int e) { return mt * 16 + (kEight ? r0 + e * 8 : (e >> 1) * 8 + cq + (e & 1)); };
      float vf[MT][NK];  // V's scales of this lane's keys
      float t0 = -INFINITY, t1 = -INFINITY;
      const bool open = __all_sync(0xffffffffu, about.x == (uint32_t)((1ull << KW) - 1) && j0 + KW <= min(lim0, lim1));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < NK; ++e) {
          const float2 z = sm.scales[warp][at][key_of(mt, e)];
          vf[mt][e] = z.y;
          score(mt, e, 0) *= z.x;
          score(mt, e, 1) *= z.x;
        }
      if (!open)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < NK; ++e) {
            const int i = key_of(mt, e);
            const bool in = (about.x >> i) & 1;
            if (!in || j0 + i >= lim0) score(mt, e, 0) = -INFINITY;
            if (!in || j0 + i >= lim1) score(mt, e, 1) = -INFINITY;
          }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < NK; ++e) {
          t0 = fmaxf(t0, score(mt, e, 0));
          t1 = fmaxf(t1, score(mt, e, 1));
        }
#pragma unroll
      for (int d = kEight ? 4 : 1; d < (kEight ? 32 : 4); d *= 2) {
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, d));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, d));
      }
      t0 = fmaxf(m0, t0 * fac0);  // (-infinity stays: the factors are > 0)
      t1 = fmaxf(m1, t1 * fac1);
      const float b0 = t0 == -INFINITY ? 0.f : t0, b1 = t1 == -INFINITY ? 0.f : t1;
      const bool bigger = (int)about.y > unit;  // V's unit grows
      if (__any_sync(0xffffffffu, t0 != m0 || t1 != m1 || bigger)) {  // some row's maximum grew
        float f0 = fast_exp2(m0 - b0), f1 = fast_exp2(m1 - b1);
        l0 *= f0;
        l1 *= f1;
        m0 = t0;
        m1 = t1;
        bool far = false;
        if (bigger) {
          if (k == w.k0) {  // O is 0
            sm.first[warp] = (int)about.y;
          } else if ((int)about.y - sm.first[warp] <= 90) {
            f0 *= power(unit - (int)about.y);
            f1 *= power(unit - (int)about.y);
          } else {
            bool some = false;
#pragma unroll
            for (int n = 0; n < NO; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) some = some || o[n][e] != 0.f;
            far = __any_sync(0xffffffffu, some);
            sm.first[warp] = (int)about.y;  // (the vote: all have read it)
          }
          unit = (int)about.y;
        }
#pragma unroll
        for (int n = 0; n < NO; ++n) {
          o[n][0] *= f0;
          o[n][1] *= kEight ? f1 : f0;
          o[n][2] *= kEight ? f0 : f1;
          o[n][3] *= f1;
        }
        if (far)
#pragma unroll
          for (int n = 0; n < NO; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = o[n][e] == 0.f ? 0.f : NAN;
      }
      // ---- weights: the operands of the product with V
      const float to_unit = power(142 - unit);
      bool lost = false;  // V's scale is too small for the weight's exponents (or NaN, as the weight then is)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < NK; ++e) {
          const float f = vf[mt][e] * to_unit;
          vf[mt][e] = f >= 1.f || vf[mt][e] == 0.f ? f : NAN;
          lost = lost || vf[mt][e] != vf[mt][e];
        }
      lost = __any_sync(0xffffffffu, lost);
      uint32_t p[QP][MT][kEight ? 2 : 4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float e0[NK], e1[NK];
#pragma unroll
        for (int e = 0; e < NK; ++e) {
          e0[e] = fast_exp2(fmaf(score(mt, e, 0), fac0, -b0));
          e1[e] = fast_exp2(fmaf(score(mt, e, 1), fac1, -b1));
          l0 += e0[e];
          l1 += e1[e];
        }
        if (lost)
#pragma unroll
          for (int e = 0; e < NK; ++e) {
            e0[e] = e0[e] <= kNoWeight ? 0.f : e0[e] * vf[mt][e];
            e1[e] = e1[e] <= kNoWeight ? 0.f : e1[e] * vf[mt][e];
          }
        else
#pragma unroll
          for (int e = 0; e < NK; ++e) {
            e0[e] *= vf[mt][e];
            e1[e] *= vf[mt][e];
          }
#pragma unroll
        for (int part = 0; part < QP; ++part) {
          if constexpr (kEight) {  // (rows, keys) from (keys, rows)
            p[part][mt][0] = transposed(pack2((const __half*)nullptr, e0[0], e1[0]));
            p[part][mt][1] = transposed(pack2((const __half*)nullptr, e0[1], e1[1]));
          } else {
            p[part][mt][0] = pack2((const __half*)nullptr, e0[0], e0[1]);
            p[part][mt][1] = pack2((const __half*)nullptr, e1[0], e1[1]);
            p[part][mt][2] = pack2((const __half*)nullptr, e0[2], e0[3]);
            p[part][mt][3] = pack2((const __half*)nullptr, e1[2], e1[3]);
          }
          if constexpr (QP > 1) {
#pragma unroll
            for (int e = 0; e < (kEight ? 2 : 4); ++e) {
              e0[e] -= __half2float(__float2half_rn(e0[e]));
              e1[e] -= __half2float(__float2half_rn(e1[e]));
            }
          }
        }
      }
      // ---- outputs: this lane has keys cq, cq + 1, cq + 8, cq + 9 of every 16, and columns 8 r0 + 64 i .. + 7
      cp_async_wait<S - 2>();
      __syncwarp();
      const unsigned char* const vt = ring.template take<S % 2 != 0>(kc, vc, g, a, c);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < DP / 64; ++i) {
          uint2 v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = *reinterpret_cast<const uint2*>(vt + v_at[i] + (mt * 16 + (e >> 1) * 8) * DP + (e & 1 ? next_key : 0));
#pragma unroll
          for (int t = 0; t < 4; ++t) {  // two columns
            const uint32_t x0 = t < 2 ? v[0].x : v[0].y, x1 = t < 2 ? v[1].x : v[1].y;
            const uint32_t x2 = t < 2 ? v[2].x : v[2].y, x3 = t < 2 ? v[3].x : v[3].y;
            const uint32_t order = t & 1 ? 0x7362 : 0x5140;
            uint32_t f[4];
            halves(__byte_perm(x0, x1, order), f[0], f[1]);  // keys cq, cq + 1: even column, odd column
            halves(__byte_perm(x2, x3, order), f[2], f[3]);  // cq + 8, cq + 9
#pragma unroll
            for (int part = 0; part < QP; ++part) {
              if constexpr (kEight) {
                mma16816<__half>(o[i * 4 + t], f, p[part][mt][0], p[part][mt][1]);
              } else {
                mma16816<__half>(o[i * 8 + 2 * t], p[part][mt], f[0], f[2]);
                mma16816<__half>(o[i * 8 + 2 * t + 1], p[part][mt], f[1], f[3]);
              }
            }
          }
        }
      __syncwarp();
    }

    // ---- the four warps' rows together, a few rows at a time, to the output or a partial result
#pragma unroll
    for (int d = kEight ? 4 : 1; d < (kEight ? 32 : 4); d *= 2) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    if (kEight ? r0 == 0 : cl == 0) {
      sm.ml[warp][ra][0] = m0;
      sm.ml[warp][ra][1] = l0;
      sm.ml[warp][rb][0] = m1;
      sm.ml[warp][rb][1] = l1;
    }
    const float scale = power_of(unit), lift = power(-15);
    Walk nw = w;
    walk_next<MR, KT>(nw, g, a, c);
    if (!nw.done) read_q(nw);
    const bool begins = w.k0 == 0, whole = begins && k1 == w.work, final = whole && !c.shared;
    float* const po = slot_o(c, a, blockIdx.x, begins ? 1 : 0);
    float* const pml = slot_ml(c, a, blockIdx.x, begins ? 1 : 0);
    constexpr int RJ = Shape::kJoin;
    for (int p0 = 0; p0 < u.rows; p0 += RJ) {
      if constexpr (kEight) {
        if (cq >= p0 && cq < p0 + RJ) {  // both of this lane's rows: pairs of columns
          float* to = &sm.o[warp][cq - p0][8 * r0];
#pragma unroll
          for (int n = 0; n < NO; ++n) {
            const int d = 64 * (n >> 2) + 2 * (n & 3);
            *reinterpret_cast<float2*>(to + d) = make_float2(o[n][0] * scale * lift, o[n][2] * scale * lift);
            *reinterpret_cast<float2*>(to + DP + 8 + d) = make_float2(o[n][1] * scale * lift, o[n][3] * scale * lift);
          }
        }
      } else if ((r0 & (8 - RJ)) == (p0 & (8 - RJ))) {  // this lane has row r0 % RJ of them: r0, or r0 + 8
        float* to = &sm.o[warp][r0 & (RJ - 1)][16 * cl];
#pragma unroll
        for (int n = 0; n < NO; ++n) {
          const int d = 64 * (n >> 3) + (n & 7);
          to[d] = (p0 < 8 ? o[n][0] : o[n][2]) * scale * lift;
          to[d + 8] = (p0 < 8 ? o[n][1] : o[n][3]) * scale * lift;
        }
      }
      __syncthreads();
#pragma unroll
      for (int idx = threadIdx.x; idx < RJ * (DP / 4); idx += kCodesThreads) {  // RJ rows x DP / 4 pieces
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
  if (sm.bad) mend_rows<T, DP, MR, KT, kCodesThreads>(q, kc, vc, out, lse, g, a, c, sm.tmp);
}

}  // namespace attend
}  // namespace rope
