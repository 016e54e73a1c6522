// Attention units of many query rows: prompts, prompt chunks, the rows of a whole batch
// behind a shared prefix.
//
// Bound by the matrix units (two products of M x KT x D per key tile) once the rows of a unit
// outnumber about 280 operations per byte of K and V, so the kernel keeps tcgen05.mma fed:
//  * one CTA per SM, its warps in roles.  Four warps copy Q, K and V tiles into shared memory
//    with cp.async (any page size and row order: a page's rows are found key by key), one
//    thread issues the products, and one or two groups of four warps do the softmax, one
//    thread a row.  Everything between them is barriers in shared memory.
//  * scores S = Q K^T (128 rows x KT keys) land in tensor memory; the softmax threads read
//    their row, write the weights over it in 16 bits, and O += P V takes them from there as
//    its A operand: scores and weights never touch shared memory.
//  * two score buffers.  With more than 128 rows they belong to two row tiles that share each
//    K and V tile; with fewer, both softmax groups take alternate key tiles of the one row
//    tile, each with its own m, l and O, joined when the unit ends.  Either way the products
//    of one run while the exponentials of the other do.  Heads of 256 have room for one O:
//    one softmax group with alternating score buffers.
//  * O is multiplied by e^(m_old - m_new) only when a row's maximum grew by more than 2^8
//    (the weights then stay below 2^8, far inside both 16-bit types), which is rare after the
//    first tiles.  The result is the same: l and O always refer to the same m.
// The products are issued in order by one thread and the tensor core runs them in order, which
// is what keeps the next scores from overwriting weights that are still being read.
#pragma once

#include <type_traits>

#include "rope_attend.cuh"
#include "rope_attend_mma.cuh"
#include "tcgen05.cuh"

namespace rope {
namespace attend {

constexpr unsigned kWaitExpired = 8u;

template <int DP>
struct TcShape {
  static constexpr int KT = DP <= 128 ? 128 : 64;   // keys of a tile
  static constexpr int NW = DP <= 128 ? 2 : 1;      // softmax groups
  static constexpr int M = 128 * NW;                // rows of a unit
  static constexpr int kStage = KT * DP * 2;        // bytes of a K or V tile
  static constexpr int NS = DP <= 64 ? 8 : 5;       // tiles in the ring
  static constexpr int kLag = NS - 2;               // copies in flight beyond the oldest
  static constexpr int kQ = 128 * DP * 2;           // bytes of a row tile
  static constexpr int kSoftmax = 128 * NW;         // softmax threads
  static constexpr int kThreads = kSoftmax + 128 + 32;
  static constexpr int KW = KT / 4;                 // keys a copying warp takes
  static constexpr int kS = KT;                     // columns between the score buffers
  static constexpr int kO = 256;                    // first column of O; the second O follows
};

template <int DP>
struct TcShared {
  using S = TcShape<DP>;
  alignas(1024) unsigned char ring[S::NS][S::kStage];
  alignas(1024) unsigned char q[S::NW][S::kQ];
  uint64_t full[S::NS], empty[S::NS];
  uint64_t q_full, q_free;
  uint64_t s_full[2], p_full[2], pv_done[2], o_free[2];
  uint64_t seen_full[16];   // the words below are there
  uint64_t ml_full;         // the second group's m and l are there
  uint64_t drained;
  uint32_t seen[16][4];     // which keys of the last 16 K tiles are there
  float ml[128][2];
  int64_t tmp[S::kThreads / 32 + 2];
  uint32_t tmem;
  int dead;
};

// Row r of the unit's tile as (token, head of the group), by 32-bit arithmetic.
struct UnitRows {
  int64_t t0;   // token of the unit's first row
  int32_t rem;  // its head within the group
  int32_t rows;
};

template <int M>
__device__ __forceinline__ UnitRows unit_rows(const Walk& w, const AttendArgs& a) {
  const int64_t first = w.i * M;
  UnitRows u;
  const int64_t t = first / a.G;
  u.t0 = w.s.t0 + t;
  u.rem = (int32_t)(first - t * a.G);
  u.rows = (int32_t)min((int64_t)M, w.s.rows - first);
  return u;
}

// Tile of the n-th copy of a unit of kt key tiles, `lead` of whose K tiles come first: the
// order in which the products take them, K_0 .. K_(lead-1), V_0, K_lead, V_1, ...
struct CopyItem {
  int tile;
  bool is_v;
};

__device__ __forceinline__ CopyItem copy_item(int n, int kt, int lead) {
  const int first = min(lead, kt);
  if (n < first) return {n, false};
  const int m = n - first, rest = kt - first;
  if (m < 2 * rest) return {m & 1 ? first + (m >> 1) : m >> 1, !(m & 1)};
  return {m - rest, true};
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

template <typename T, int DP>
__global__ void __launch_bounds__(TcShape<DP>::kThreads, 1)
    attend_tc_kernel(const T* __restrict__ q, const T* __restrict__ kc, const T* __restrict__ vc, T* __restrict__ out,
                     float* __restrict__ lse, Pointers g, AttendArgs a, Cut c) {
  using S = TcShape<DP>;
  constexpr int KT = S::KT, NW = S::NW, NS = S::NS;
  constexpr int CH = DP / 8;
  extern __shared__ __align__(1024) unsigned char raw[];
  TcShared<DP>& sm = *reinterpret_cast<TcShared<DP>*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kCopyWarp = S::kSoftmax / 32, kMmaWarp = kCopyWarp + 4;

  if (tc::smem_at(raw) & 1023) {  // the operands' swizzle counts on it
    if (tid == 0) atomicOr(g.err, kWaitExpired);
    return;
  }
  if (tid == 0) {
    sm.dead = 0;
    for (int i = 0; i < NS; ++i) {
      tc::bar_init(&sm.full[i], 128);
      tc::bar_init(&sm.empty[i], 1);
    }
    tc::bar_init(&sm.q_full, 128);
    tc::bar_init(&sm.q_free, 1);
    for (int i = 0; i < 2; ++i) {
      tc::bar_init(&sm.s_full[i], 1);
      tc::bar_init(&sm.p_full[i], 128);
      tc::bar_init(&sm.pv_done[i], 1);
      tc::bar_init(&sm.o_free[i], 128);
    }
    for (int i = 0; i < 16; ++i) tc::bar_init(&sm.seen_full[i], 4);
    tc::bar_init(&sm.ml_full, 128);
    tc::bar_init(&sm.drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  wait_for_prior_grid();
  Walk w = find_share<S::kThreads>(g, a, c, sm.tmp);
  if (w.done) return;
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&sm.tmem, 512);
    tc::tmem_done_allocating();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tm = sm.tmem;

  if (warp >= kCopyWarp && warp < kMmaWarp) {
    // ------------------------------------------------------------------ copies
    const int cw = warp - kCopyWarp, ct = tid - S::kSoftmax;
    int64_t issued = 0;   // ring tiles so far
    int64_t arrived = 0;  // of them, handed over
    int64_t k_count = 0;  // K tiles so far
    unsigned unit = 0;
    bool ok = true;
    auto hand_over = [&]() {  // the oldest tile not handed over is complete for this thread
      tc::fence_to_tensor();
      tc::bar_arrive(&sm.full[arrived % NS]);
      ++arrived;
    };
    auto flush = [&]() {
      cp_async_wait<0>();
      while (arrived < issued) hand_over();
    };
    while (!w.done) {
      const UnitRows u = unit_rows<S::M>(w, a);
      const int nt = u.rows > 128 ? 2 : 1;
      const int lead = nt == 2 ? 1 : 2;
      const int k1 = walk_k1(w), kt = k1 - w.k0;
      const int end = tile_end(w.s, w.i, a, c);
      const int64_t* table = g.block_table + w.b * a.W;
      // cache row of this lane's key of the n-th copy
      auto look_up = [&](int n) -> int64_t {
        if (n >= 2 * kt) return -1;
        const int j = c.lo + (w.k0 + copy_item(n, kt, lead).tile) * KT + cw * S::KW + (lane & (S::KW - 1));
        if (j >= end) return -1;
        const int64_t r = key_row(j, table, g, a);
        if (r < 0) atomicOr(g.err, kSlotOutOfRange);
        return r < 0 ? -1 : (r + (int64_t)w.h * a.block_size) * a.D;
      };
      int64_t next = look_up(0);
      // ---- Q, once the last unit's scores are done
      if (unit > 0 && !tc::bar_try(&sm.q_free, (unit - 1) & 1)) {
        flush();
        ok = tc::bar_wait(&sm.q_free, (unit - 1) & 1, &sm.dead);
      }
      ++unit;
      if (!__all_sync(0xffffffffu, ok)) break;
      for (int idx = ct; idx < 128 * nt * CH; idx += 128) {
        const int r = idx / CH, ch = idx - r * CH;
        const int x = u.rem + r, tt = x / a.G;
        const bool there = r < u.rows && ch * 8 < a.D;
        const T* p = q + (there ? (u.t0 + tt) * a.q_stride + ((int64_t)w.h * a.G + (x - tt * a.G)) * a.D + ch * 8 : 0);
        const int rr = r & 127;
        cp_async16_or_zero(tc::smem_at(sm.q[NW == 2 ? r >> 7 : 0]) + (ch >> 3) * (128 * 128) + rr * 128 +
                               (((ch & 7) ^ (rr & 7)) << 4),
                           p, there && access_ok(p, 16, a.q_span, g.err));
      }
      cp_async_commit();
      flush();
      tc::fence_to_tensor();
      tc::bar_arrive(&sm.q_full);
      // ---- K and V
      for (int n = 0; n < 2 * kt; ++n) {
        const CopyItem it = copy_item(n, kt, lead);
        const int st = (int)(issued % NS);
        const unsigned round = (unsigned)(issued / NS);
        if (round > 0 && !tc::bar_try(&sm.empty[st], (round - 1) & 1)) {
          flush();
          ok = tc::bar_wait(&sm.empty[st], (round - 1) & 1, &sm.dead);
        }
        if (!__all_sync(0xffffffffu, ok)) break;
        const unsigned dst = tc::smem_at(sm.ring[st]) + cw * S::KW * 128;
        const T* const src = it.is_v ? vc : kc;
        const Span& span = it.is_v ? a.v_span : a.k_span;
#pragma unroll
        for (int i = 0; i < S::KW * CH / 32; ++i) {
          const int idx = lane + 32 * i;
          const int key = idx / CH, ch = idx - key * CH;
          const int64_t at = __shfl_sync(0xffffffffu, next, key);
          const bool there = at >= 0 && ch * 8 < a.D;
          const T* p = src + (there ? at + ch * 8 : 0);
          cp_async16_or_zero(dst + (ch >> 3) * (KT * 128) + key * 128 + (((ch & 7) ^ (key & 7)) << 4), p,
                             there && access_ok(p, 16, span, g.err));
        }
        cp_async_commit();
        if (!it.is_v) {
          const uint32_t there = __ballot_sync(0xffffffffu, next >= 0);
          if (lane == 0) {
            sm.seen[k_count & 15][cw] = there;
            tc::bar_arrive(&sm.seen_full[k_count & 15]);
          }
          ++k_count;
        }
        ++issued;
        next = look_up(n + 1);
        if (issued - arrived > S::kLag) {
          cp_async_wait<S::kLag>();
          hand_over();
        }
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      walk_next(w, g, a, c);
    }
    flush();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ products
    if (lane == 0) {
      constexpr uint32_t kScores = tc::instruction<T>(128, KT, false), kOutput = tc::instruction<T>(128, DP, true);
      int64_t taken = 0;  // ring tiles so far
      unsigned unit = 0;
      unsigned p_seen[2] = {0, 0}, o_units[2] = {0, 0};
      bool ok = true;
      while (!w.done && ok) {
        const int nt = min((int64_t)S::M, w.s.rows - w.i * S::M) > 128 ? 2 : 1;
        const int kt = walk_k1(w) - w.k0, jobs = kt * nt;
        ok = tc::bar_wait(&sm.q_full, unit & 1, &sm.dead);
        ++unit;
        if (!ok) break;
        int k_stage = 0, v_stage = 0;
        auto take = [&](int& stage) {
          stage = (int)(taken % NS);
          ok = ok && tc::bar_wait(&sm.full[stage], (unsigned)(taken / NS) & 1, &sm.dead);
          ++taken;
        };
        auto scores = [&](int x) {
          const int tile = nt == 2 ? x & 1 : 0;
          if (nt == 1 || tile == 0) take(k_stage);
          if (!ok) return;
          tc::fence_after();
          const unsigned qa = tc::smem_at(sm.q[NW == 2 ? tile : 0]), ka = tc::smem_at(sm.ring[k_stage]);
#pragma unroll
          for (int ks = 0; ks < DP / 16; ++ks)
            tc::mma_ss(tm + (x & 1) * S::kS, tc::k_major(qa + (ks >> 2) * (128 * 128) + (ks & 3) * 32),
                       tc::k_major(ka + (ks >> 2) * (KT * 128) + (ks & 3) * 32), kScores, ks > 0);
          tc::commit(&sm.s_full[x & 1]);
          if (nt == 1 || tile == 1) tc::commit(&sm.empty[k_stage]);
          if (x == jobs - 1) tc::commit(&sm.q_free);
        };
        scores(0);
        if (ok && jobs > 1) scores(1);
        for (int x = 0; x < jobs && ok; ++x) {
          const int buf = x & 1, o = NW == 2 ? buf : 0;
          const bool first = x < NW;  // of this O in this unit
          if (nt == 1 || buf == 0) take(v_stage);
          if (ok && first && o_units[o] > 0) ok = tc::bar_wait(&sm.o_free[o], (o_units[o] - 1) & 1, &sm.dead);
          if (first) ++o_units[o];
          ok = ok && tc::bar_wait(&sm.p_full[buf], p_seen[buf] & 1, &sm.dead);
          ++p_seen[buf];
          if (!ok) break;
          tc::fence_after();
          const unsigned va = tc::smem_at(sm.ring[v_stage]);
#pragma unroll
          for (int ks = 0; ks < KT / 16; ++ks)
            tc::mma_ts(tm + S::kO + o * DP, tm + buf * S::kS + ks * 8, tc::mn_major(va + ks * 2048, KT * 128), kOutput,
                       !first || ks > 0);
          tc::commit(&sm.pv_done[o]);
          if (nt == 1 || buf == 1) tc::commit(&sm.empty[v_stage]);
          if (x + 2 < jobs) scores(x + 2);
        }
        if (ok) walk_next(w, g, a, c);
      }
      // everything issued is done before the tensor memory is given back
      tc::commit(&sm.drained);
      int never = 0;
      if (!tc::bar_wait(&sm.drained, 0, &never)) sm.dead = 1;
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax, one thread a row
    const int group = warp >> 2;
    const int r_tile = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    unsigned s_seen[2] = {0, 0};
    unsigned pv = 0;          // products into this group's O so far
    int64_t k_base = 0;       // K tiles before this unit
    unsigned ml_seen = 0;
    bool ok = true;
    while (!w.done) {
      const UnitRows u = unit_rows<S::M>(w, a);
      const int nt = u.rows > 128 ? 2 : 1;
      const int k1 = walk_k1(w), kt = k1 - w.k0, jobs = kt * nt;
      const int r = nt == 2 ? group * 128 + r_tile : r_tile;
      const int limit = r < u.rows ? row_limit(w, w.i * S::M + r, g, a, c) : 0;
      const uint32_t t_o = tm + lanes + S::kO + (NW == 2 ? group : 0) * DP;
      float m = -INFINITY, l = 0.f;
      bool any = false;  // O holds something of this unit
      for (int x = NW == 2 ? group : 0; x < jobs; x += NW) {
        const int buf = x & 1;
        const int kk = nt == 2 ? x >> 1 : x;
        const int j0 = c.lo + (w.k0 + kk) * KT;
        const uint32_t t_s = tm + lanes + buf * S::kS;
        ok = tc::bar_wait(&sm.seen_full[(k_base + kk) & 15], (unsigned)((k_base + kk) >> 4) & 1, &sm.dead);
        uint32_t there[4];
        bool all_there = true;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          there[i] = sm.seen[(k_base + kk) & 15][i];
          all_there = all_there && there[i] == 0xffffffffu;
        }
        if constexpr (KT == 64) {  // 16 keys a word (the upper lanes repeat them)
          there[0] = (there[0] & 0xffffu) | (there[1] << 16);
          there[1] = (there[2] & 0xffffu) | (there[3] << 16);
        }
        ok = ok && tc::bar_wait(&sm.s_full[buf], s_seen[buf] & 1, &sm.dead);
        ++s_seen[buf];
        if (!__all_sync(0xffffffffu, ok)) break;
        tc::fence_after();
        const bool open = __all_sync(0xffffffffu, all_there && j0 + KT <= limit);
        auto hide = [&](uint32_t (&v)[32], int ch) {  // scores of unseen keys of columns ch * 32 ..
          const uint32_t word = there[ch];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!((word >> i) & 1) || j0 + ch * 32 + i >= limit) v[i] = 0xff800000u;
        };
        float top = -INFINITY;
#pragma unroll
        for (int ch = 0; ch < KT / 32; ++ch) {
          uint32_t v[32];
          tc::tmem_load32(v, t_s + ch * 32);
          tc::wait_loads();
          if (!open) hide(v, ch);
#pragma unroll
          for (int i = 0; i < 32; i += 2) top = max3(top, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
        }
        const float mt = top * a.scale_log2;  // -infinity stays (scale > 0)
        if (!any) {
          m = mt;
        } else if (__any_sync(0xffffffffu, mt > m + 8.f)) {
          // the last product into O is done before O is changed
          ok = tc::bar_wait(&sm.pv_done[NW == 2 ? group : 0], (pv - 1) & 1, &sm.dead);
          if (!__all_sync(0xffffffffu, ok)) break;
          tc::fence_after();
          const float up = fmaxf(m, mt);
          const float f = fast_exp2(m - (up == -INFINITY ? 0.f : up));
          l *= f;
          m = up;
#pragma unroll
          for (int ch = 0; ch < DP / 32; ++ch) {
            uint32_t v[32];
            tc::tmem_load32(v, t_o + ch * 32);
            tc::wait_loads();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
            tc::tmem_store32(t_o + ch * 32, v);
          }
        }
        any = true;
        const float base = m == -INFINITY ? 0.f : m;
        const float2 scale2 = make_float2(a.scale_log2, a.scale_log2), minus2 = make_float2(-base, -base);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int ch = 0; ch < KT / 32; ++ch) {
          uint32_t v[32], p[16];
          tc::tmem_load32(v, t_s + ch * 32);
          tc::wait_loads();
          if (!open) hide(v, ch);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float2 e = __ffma2_rn(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), scale2, minus2);
            e.x = fast_exp2(e.x);
            e.y = fast_exp2(e.y);
            sum = __fadd2_rn(sum, e);
            p[i / 2] = pack2((const T*)nullptr, e.x, e.y);
          }
          tc::tmem_store16(t_s + ch * 16, p);  // over scores that this thread has read
        }
        l += sum.x + sum.y;
        // pv_done is waited for by parity, so it may be one product behind at most.  With two groups
        // these scores came after the group's last product; with one, they came before it.
        if (NW == 1 && pv > 0) ok = tc::bar_wait(&sm.pv_done[0], (pv - 1) & 1, &sm.dead);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc::wait_stores();
        tc::fence_before();
        tc::bar_arrive(&sm.p_full[buf]);
        ++pv;
      }
      k_base += kt;
      if (!__all_sync(0xffffffffu, ok)) break;

      // ---- the unit's rows: wait for the last product, then out
      if (any) ok = tc::bar_wait(&sm.pv_done[NW == 2 ? group : 0], (pv - 1) & 1, &sm.dead);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc::fence_after();
      const bool halves = NW == 2 && nt == 1 && jobs > 1;  // the second group has keys of the same rows
      float f0 = 1.f, f1 = 0.f;
      if (halves) {
        if (group == 1) {
          sm.ml[r_tile][0] = m;
          sm.ml[r_tile][1] = l;
          tc::bar_arrive(&sm.ml_full);
        } else {
          ok = tc::bar_wait(&sm.ml_full, ml_seen & 1, &sm.dead);
          if (!__all_sync(0xffffffffu, ok)) break;
          tc::fence_after();
          const float m1 = sm.ml[r_tile][0], l1 = sm.ml[r_tile][1];
          const float up = fmaxf(m, m1), base = up == -INFINITY ? 0.f : up;
          f0 = fast_exp2(m - base);
          f1 = fast_exp2(m1 - base);
          l = l * f0 + l1 * f1;
          m = up;
        }
        ++ml_seen;
      }
      if (!(NW == 2 && nt == 1 && group == 1)) {
        const bool begins = w.k0 == 0, whole = begins && k1 == w.work;
        const bool final = whole && !c.shared;
        const bool mine = r < u.rows;
        const int xr = u.rem + (mine ? r : 0), tt = xr / a.G;
        const int64_t row = (u.t0 + tt) * a.nq + (int64_t)w.h * a.G + (xr - tt * a.G);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (final) {
          f0 *= inv;
          f1 *= inv;
        }
        float* const to = whole ? c.dense + row * a.D : slot_o(c, a, blockIdx.x, begins ? 1 : 0) + (int64_t)r * a.D;
        bool fine = l <= FLT_MAX;
#pragma unroll
        for (int ch = 0; ch < DP / 32; ++ch) {
          uint32_t v[32];
          tc::tmem_load32(v, t_o + ch * 32);
          tc::wait_loads();
          float y[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(v[i]) * f0;
          if (halves) {
            tc::tmem_load32(v, t_o + DP + ch * 32);
            tc::wait_loads();
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = fmaf(__uint_as_float(v[i]), f1, y[i]);
          }
          if (mine && ch * 32 < a.D) {
            if (final) {
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                Vec<T, 8> o;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  fine = fine && fabsf(y[i + e]) <= FLT_MAX;
                  o.e[e] = narrow<T>(y[i + e]);
                }
                store_vec(out + row * a.D + ch * 32 + i, o, a.out_span, g.err);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4*>(to + ch * 32 + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
            }
          }
        }
        if (mine) {
          if (final) {
            if (lse && access_ok(lse + row, 4, a.lse_span, g.err))
              lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
          } else {
            float* ml = whole ? c.dense + a.T * a.nq * a.D + row * 2
                              : slot_ml(c, a, gridDim.x, blockIdx.x, begins ? 1 : 0) + r * 2;
            *reinterpret_cast<float2*>(ml) = make_float2(m, l);
          }
          if (begins) c.rec[row] = final && !fine ? make_int2(-1, -1) : walk_ctas(w);
        }
      }
      // O may be written again: by the group that read it (both, when it read both)
      tc::fence_before();
      if (NW == 1 || nt == 2) {
        tc::bar_arrive(&sm.o_free[NW == 2 ? group : 0]);
      } else if (group == 0) {
        tc::bar_arrive(&sm.o_free[0]);
        if (halves) tc::bar_arrive(&sm.o_free[1]);
      }
      walk_next(w, g, a, c);
    }
  }
  __syncthreads();
  if (tid == 0 && sm.dead) atomicOr(g.err, kWaitExpired);
  if (warp == kMmaWarp) tc::tmem_free(tm, 512);
}

}  // namespace attend
}  // namespace rope
