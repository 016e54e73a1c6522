// Attention units of many query rows: prompts, prompt chunks, the rows of a whole batch
// behind a shared prefix.
//
// Bound by the matrix units (two products of M x KT x D per key tile) once the rows of a unit
// outnumber about 280 operations per byte of K and V, so the kernel keeps tcgen05.mma fed:
//  * one CTA per SM, its warps in roles.  Four warps (two for heads of 256) copy Q, K and V
//    tiles into shared memory with cp.async (any page size and row order: a page's rows are
//    found key by key; two warps were not enough for heads of 128: 582 us against 548 for the
//    example below as the kernel was then), one thread relays the finished copies to the tensor core, one issues the
//    products, and one or two groups of four warps do the softmax, one thread a row.
//    Everything between them is barriers in shared memory.
//  * scores S = Q K^T (128 rows x KT keys) land in tensor memory; the softmax threads read
//    their row, write the weights over it in 16 bits, and O += P V takes them from there as
//    its A operand: scores and weights never touch shared memory.
//  * heads of up to 128: two softmax groups.  With more than 128 rows they have a row tile each
//    and share every K and V tile; with fewer, they take alternate key tiles of the one row
//    tile, each with its own m, l and O, joined when the unit ends.  The products of one run
//    while the other works.  A group hands the weights over 64 keys at a time, so that the
//    first half's product runs while it works on the second.  (Scores of 128 keys are one
//    product of full rate; products of 64 keys read the queries from shared memory twice as
//    often and run at two thirds of it.)
//  * heads of 256 have room for one O: one softmax group with two score buffers of 64 keys.
//  * O is multiplied by e^(m_old - m_new) only when a row's maximum grew by more than 2^kLag, which
//    is rare after the first tiles.  The result is the same: l and O always refer to the same m.
//    bfloat16: by 2^8, and the weights are up to 2^8.  binary16, whose exponents are few: by 2^4, and
//    the weights are taken 2^11 times as large, up to 2^15 (see weight_lift): from 2^-25 of the
//    largest on their rounding is half a step relative, below it 2^-36 of the largest at most.
// The products are issued in order by one thread and the tensor core runs them in order, which
// is what keeps the next scores from overwriting weights that are still being read.
//
// 4 chunks of 1984 tokens behind 4096 shared ones, 32 q and 8 k heads of 128, bf16: 0.50 to 0.53
// ms, 1.3 PFLOP/s, 0.67 of the measured matrix rate.  The tensor pipe is active 58 % of the time,
// issue slots 54, the pipe of the exponentials 29: none of them is the bound.  What is left is the
// softmax's latency between a tile's two products, and the ends of units, where 256 rows of results
// leave lane by lane.
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
  static constexpr int kParts = KT / 64;            // parts of 64 keys in which its weights are handed over
  static constexpr int M = 128 * NW;                // rows of a unit
  static constexpr int kStage = KT * DP * 2;        // bytes of a K or V tile
  static constexpr int NS = DP <= 64 ? 8 : 5;       // tiles in the ring
  static constexpr int kQ = 128 * DP * 2;           // bytes of a row tile
  static constexpr int kSoftmax = 128 * NW;         // softmax threads
  static constexpr int kCopy = DP <= 128 ? 128 : 64;  // copying threads
  static constexpr int kThreads = kSoftmax + kCopy + 64;
  static constexpr int KW = KT / (kCopy / 32);      // keys a copying warp takes, one a lane
  static constexpr int kAhead = 2;                  // scores ahead of the outputs
  static constexpr int kO = 256;                    // first column of O; the second O follows
};

template <int DP>
struct TcShared {
  using S = TcShape<DP>;
  alignas(1024) unsigned char ring[S::NS][S::kStage];
  alignas(1024) unsigned char q[S::NW][S::kQ];
  uint64_t copied[S::NS], full[S::NS], empty[S::NS];  // a tile is there, visible to the tensor core, read
  uint64_t q_copied, q_full, q_free;
  uint64_t s_full[2];             // of a score buffer (of a group, or alternate ones of the one group)
  uint64_t p_full[4];             // [2 * group + part or buffer]
  uint64_t pv_done[4];            // [2 * group + parity of the product]
  uint64_t o_free[2];
  uint64_t seen_full[16];   // the words below are there
  uint64_t ml_full;         // the second group's m and l are there
  uint64_t drained;
  uint32_t seen[16][4];     // which keys of the last 16 K tiles are there
  float ml[128][2];
  int64_t tmp[S::kThreads / 32 + 2];
  uint32_t tmem;
  int dead;
  int bad;  // some finished row is not finite
};

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

// 32 bytes at once: whole sectors, where each lane writes a row of its own.
__device__ __forceinline__ void store8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
               "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
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
  const int tid = threadIdx.x, warp = (int)tc::uniform(tid >> 5), lane = tid & 31;
  constexpr int kCopyWarp = S::kSoftmax / 32, kMmaWarp = kCopyWarp + S::kCopy / 32,
                kRelayWarp = kMmaWarp + 1;

  if (tc::smem_at(raw) & 1023) {  // the operands' swizzle counts on it
    if (tid == 0) atomicOr(g.err, kWaitExpired);
    return;
  }
  if (tid == 0) {
    sm.dead = 0;
    sm.bad = 0;
    for (int i = 0; i < NS; ++i) {
      tc::bar_init(&sm.copied[i], S::kCopy);
      tc::bar_init(&sm.full[i], 1);
      tc::bar_init(&sm.empty[i], 1);
    }
    tc::bar_init(&sm.q_copied, S::kCopy);
    tc::bar_init(&sm.q_full, 1);
    tc::bar_init(&sm.q_free, 1);
    for (int i = 0; i < 4; ++i) {
      tc::bar_init(&sm.p_full[i], 128);
      tc::bar_init(&sm.pv_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::bar_init(&sm.s_full[i], 1);
      tc::bar_init(&sm.o_free[i], 128);
    }
    for (int i = 0; i < 16; ++i) tc::bar_init(&sm.seen_full[i], S::kCopy / 32);
    tc::bar_init(&sm.ml_full, 128);
    tc::bar_init(&sm.drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  wait_for_prior_grid();
  Walk w = find_share<S::M, KT, S::kThreads>(g, a, c, sm.tmp);
  if (w.done) return;
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&sm.tmem, 512);
    tc::tmem_done_allocating();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tm = tc::uniform(sm.tmem);

  if (warp >= kCopyWarp && warp < kMmaWarp) {
    // ------------------------------------------------------------------ copies
    // Copies never wait for their data: the barrier of a tile gets an arrival of each copying
    // thread when its part is there.  Pages are looked up one K tile ahead; the rows of a tile
    // are kept until its V follows.
    static_assert(S::KW == 32, "a lane looks up one key");
    const int cw = warp - kCopyWarp, ct = tid - S::kSoftmax;
    int stage = 0;
    unsigned round = 0;   // of the ring
    int k_count = 0;      // K tiles so far
    unsigned unit = 0;
    bool ok = true;
    while (!w.done) {
      const UnitRows u = unit_rows<S::M>(w, a);
      const int nt = u.rows > 128 ? 2 : 1;
      const int lead = S::kAhead / nt;
      const int k1 = walk_k1(w, c), kt = k1 - w.k0;
      const int end = tile_end<S::M>(w.s, w.i, a, c);
      const int64_t* table = g.block_table + w.b * a.W;
      PageRow page;                    // of this lane's key of the next K tile
      int rows[S::kAhead];             // cache rows of its keys of the K tiles whose V has not followed
      int waiting = 0;                 // so many
      auto look_up = [&](int tile) {
        const int j = c.lo + (w.k0 + tile) * KT + cw * S::KW + lane;
        page = {-2, 0};  // no such key
        if (tile < kt && j < end) page = page_row(j, table, g, a);
      };
      look_up(0);
      // ---- Q, once the last unit's scores are done
      if (unit > 0) ok = tc::bar_wait(&sm.q_free, (unit - 1) & 1, &sm.dead);
      ++unit;
      if (!__all_sync(0xffffffffu, ok)) break;
      {
        // this thread's piece of rows ct / CH, + kStep, ...: (token, head) stepped without division
        constexpr int kStep = S::kCopy / (CH < S::kCopy ? CH : S::kCopy);
        const int ch = ct % CH;
        const RowAt at = row_at(u, ct / CH, w.h, a);
        int head = at.h - w.h * a.G;
        const T* p = q + at.t * a.q_stride + (int64_t)at.h * a.D + ch * 8;
        const int64_t next_token = a.q_stride - (int64_t)a.G * a.D;
        unsigned dst = tc::smem_at(sm.q[0]) + (ch >> 3) * (128 * 128);
#pragma unroll 4
        for (int r = ct / CH; r < 128 * nt; r += kStep) {
          const bool there = r < u.rows && ch * 8 < a.D;
          const int rr = r & 127;
          cp_async16_or_zero(dst + (NW == 2 ? r >> 7 : 0) * S::kQ + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4),
                             there ? p : q, there && access_ok(p, 16, a.q_span, g.err));
          p += kStep * a.D;
          head += kStep;
          while (head >= a.G) head -= a.G, p += next_token;
        }
        tc::bar_arrive_after_copies(&sm.q_copied);
      }
      for (int n = 0; n < 2 * kt; ++n) {
        // ---- K and V
        const CopyItem it = copy_item(n, kt, lead);
        if (round > 0) ok = tc::bar_wait(&sm.empty[stage], (round - 1) & 1, &sm.dead);
        if (!__all_sync(0xffffffffu, ok)) break;
        int now = rows[0];
        if (!it.is_v) {
          now = -1;
          if (page.page >= 0 && page.page < a.num_blocks)
            now = ((int)page.page * a.nk + w.h) * a.block_size + page.row;
          else if (page.page != -2)
            atomicOr(g.err, kSlotOutOfRange);
#pragma unroll
          for (int e = 0; e < S::kAhead; ++e)
            if (e == waiting) rows[e] = now;
          ++waiting;
          const uint32_t there = __ballot_sync(0xffffffffu, now >= 0);
          if (lane == 0) {
            sm.seen[k_count & 15][cw] = there;
            tc::bar_arrive(&sm.seen_full[k_count & 15]);
          }
          ++k_count;
          look_up(it.tile + 1);
        } else {
#pragma unroll
          for (int e = 0; e + 1 < S::kAhead; ++e) rows[e] = rows[e + 1];
          --waiting;
        }
        const unsigned dst = tc::smem_at(sm.ring[stage]) + cw * S::KW * 128;
        const T* const src = it.is_v ? vc : kc;
        const Span& span = it.is_v ? a.v_span : a.k_span;
#pragma unroll
        for (int i = 0; i < S::KW * CH / 32; ++i) {
          const int idx = lane + 32 * i;
          const int key = idx / CH, ch = idx - key * CH;
          const int r = __shfl_sync(0xffffffffu, now, key);
          const bool there = r >= 0 && ch * 8 < a.D;
          const T* p = src + ((uint64_t)(uint32_t)max(r, 0) * (uint32_t)a.D + (there ? ch * 8 : 0));
          cp_async16_or_zero(dst + (ch >> 3) * (KT * 128) + key * 128 + (((ch & 7) ^ (key & 7)) << 4), p,
                             there && access_ok(p, 16, span, g.err));
        }
        tc::bar_arrive_after_copies(&sm.copied[stage]);
        if (++stage == NS) stage = 0, ++round;
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      walk_next<S::M, KT>(w, g, a, c);
    }
    cp_async_commit();
    cp_async_wait<0>();
  } else if (warp == kRelayWarp) {
    // ------------------------------------------------------------------ relay
    // What cp.async wrote becomes visible to the tensor core by a fence that takes about 600
    // cycles: one thread does nothing else, ahead of the products.
    if (lane == 0) {
      int stage = 0;
      unsigned round = 0, unit = 0;
      bool ok = true;
      while (!w.done && ok) {
        const int kt = walk_k1(w, c) - w.k0;
        ok = tc::bar_wait(&sm.q_copied, unit & 1, &sm.dead);
        tc::fence_to_tensor();
        if (ok) tc::bar_arrive(&sm.q_full);
        for (int n = 0; n < 2 * kt && ok; ++n) {
          ok = ok && tc::bar_wait(&sm.copied[stage], round & 1, &sm.dead);
          tc::fence_to_tensor();
          if (ok) tc::bar_arrive(&sm.full[stage]);
          if (++stage == NS) stage = 0, ++round;
        }
        ++unit;
        if (ok) walk_next<S::M, KT>(w, g, a, c);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ products
    constexpr uint32_t kScores = tc::instruction<T>(128, KT, false), kOutput = tc::instruction<T>(128, DP, true);
    const uint32_t q0 = tc::uniform(tc::k_major(tc::smem_at(sm.q[0])));
    const uint32_t k0 = tc::uniform(tc::k_major(tc::smem_at(sm.ring[0])));
    const uint32_t v0 = tc::uniform(tc::mn_major(tc::smem_at(sm.ring[0]), KT * 128));
    int next_stage = 0;
    unsigned round = 0;  // of the ring
    unsigned unit = 0;
    // the one group's score buffer that is next, for scores and for outputs; a bit a group: whether
    // its O was used, and its parity; a bit a buffer: parity of its weights
    unsigned s_next = 0, o_next = 0, o_used = 0, o_parity = 0, p_parity = 0;
    bool ok = true;
    while (__any_sync(0xffffffffu, !w.done && ok)) {
      const int nt = (int)tc::uniform(w.s.rows - w.i * S::M > 128 && S::M > 128 ? 2 : 1);
      const int jobs = (int)tc::uniform((walk_k1(w, c) - w.k0) * nt);  // job x is of group x % NW
      ok = __all_sync(0xffffffffu, tc::bar_wait(&sm.q_full, unit & 1, &sm.dead));
      ++unit;
      if (!ok) break;
      int k_stage = 0, v_stage = 0;
      auto take = [&]() {
        const int stage = next_stage;
        ok = __all_sync(0xffffffffu, tc::bar_wait(&sm.full[stage], round & 1, &sm.dead));
        if (++next_stage == NS) next_stage = 0, ++round;
        return stage;
      };
      auto scores = [&](int x) {
        const int group = NW == 2 ? x & 1 : 0;
        const bool second = nt == 2 && group == 1;  // the other row tile, on the K tile of the first
        if (!second) k_stage = take();
        if (!ok) return;
        tc::fence_after();
        const int buf = NW == 2 ? group : s_next;
        s_next ^= 1u;
        const uint32_t qa = q0 + (second ? S::kQ / 16 : 0), ka = k0 + k_stage * (S::kStage / 16);
        const uint32_t to = tm + buf * KT;
        if (tc::elect()) {
#pragma unroll
          for (int ks = 0; ks < DP / 16; ++ks)
            tc::mma_ss(to, tc::operand(qa + ((ks >> 2) * (128 * 128) + (ks & 3) * 32) / 16),
                       tc::operand(ka + ((ks >> 2) * (KT * 128) + (ks & 3) * 32) / 16), kScores, ks > 0);
          tc::commit(&sm.s_full[buf]);
          if (nt == 1 || second) tc::commit(&sm.empty[k_stage]);
          if (x == jobs - 1) tc::commit(&sm.q_free);
        }
        __syncwarp();
      };
      for (int x = 0; x < S::kAhead && x < jobs && ok; ++x) scores(x);
      for (int x = 0; x < jobs && ok; ++x) {
        const int group = NW == 2 ? x & 1 : 0;
        const bool first = x < NW;  // of this O in this unit
        const bool second = nt == 2 && group == 1;
        if (!second) v_stage = take();
        if (first) {
          if (ok && ((o_used >> group) & 1)) {
            ok = __all_sync(0xffffffffu, tc::bar_wait(&sm.o_free[group], (o_parity >> group) & 1, &sm.dead));
            o_parity ^= 1u << group;
          }
          o_used |= 1u << group;
        }
        const uint32_t va = v0 + v_stage * (S::kStage / 16);
        const uint32_t to = tm + S::kO + group * DP, from = tm + (NW == 2 ? group : o_next) * KT;
#pragma unroll
        for (int part = 0; part < S::kParts; ++part) {
          const int bar = NW == 2 ? group * 2 + part : o_next;
          ok = __all_sync(0xffffffffu, ok && tc::bar_wait(&sm.p_full[bar], (p_parity >> bar) & 1, &sm.dead));
          p_parity ^= 1u << bar;
          if (!ok) break;
          tc::fence_after();
          if (tc::elect()) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc::mma_ts(to, from + part * 64 + ks * 8, tc::operand(va + (part * 4 + ks) * 2048 / 16), kOutput,
                         !first || part > 0 || ks > 0);
            tc::commit(&sm.pv_done[bar]);
            if (part == S::kParts - 1 && (nt == 1 || second)) tc::commit(&sm.empty[v_stage]);
          }
          __syncwarp();
        }
        o_next ^= 1u;
        if (!ok) break;
        if (x + S::kAhead < jobs) scores(x + S::kAhead);
      }
      if (ok) walk_next<S::M, KT>(w, g, a, c);
    }
    // everything issued is done before the tensor memory is given back
    if (tc::elect()) tc::commit(&sm.drained);
    __syncwarp();
    int never = 0;
    if (!tc::bar_wait(&sm.drained, 0, &never)) sm.dead = 1;
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax, one thread a row
    const int group = warp >> 2;
    const int r_tile = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    unsigned pv = 0;          // parts of scores, and products into this group's O, so far
    int k_base = 0;           // K tiles before this unit
    unsigned ml_seen = 0;
    const bool wide = reinterpret_cast<uintptr_t>(out) % 32 == 0;  // a row of out is a multiple of 64 bytes
    bool ok = true;
    constexpr int kLag = std::is_same<T, __half>::value ? 4 : 8;
    constexpr float kLift = (float)weight_lift<T>(kLag);
    // The last product into this group's O.  Even and odd ones have a barrier each: by the time
    // that one is waited for, the one before it on the same barrier was done (two groups: before
    // these scores; one group: before the last but one), so its parity is not taken for it.
    auto product_done = [&]() -> bool {
      return __all_sync(0xffffffffu, tc::bar_wait(&sm.pv_done[(NW == 2 ? group * 2 : 0) + ((pv - 1) & 1)],
                                                  ((pv - 1) >> 1) & 1, &sm.dead));
    };
    while (!w.done) {
      const UnitRows u = unit_rows<S::M>(w, a);
      const int nt = u.rows > 128 ? 2 : 1;
      const int k1 = walk_k1(w, c), kt = k1 - w.k0, jobs = kt * nt;
      const int r = nt == 2 ? group * 128 + r_tile : r_tile;
      const bool mine = r < u.rows;
      const RowAt at = row_at(u, mine ? r : 0, w.h, a);
      const int limit = mine ? row_limit(w, at.t, g, a, c) : 0;
      const uint32_t t_o = tm + lanes + S::kO + (NW == 2 ? group : 0) * DP;
      float m = -INFINITY, l = 0.f;
      bool any = false;  // O holds something of this unit
      // parts of 64 keys: part y & 1 of job x, or one a job
      const int parts = NW == 2 ? nt == 2 ? 2 * kt : ((jobs + 1 - group) >> 1) * 2 : jobs;
      uint32_t there[2 * S::kParts];  // which keys of the job are there
      // The second group has no part of a unit of one row tile and one key tile, waits for nothing there
      // and may come out many tiles ahead of the copies.  The barriers of `seen` come round every 16
      // tiles, so that a parity tells the wanted tile from those 16 before and after it only while the
      // group is less than that away: its first scores of a unit bring it there.
      if (NW == 2 && parts > 0) {
        ok = tc::bar_wait(&sm.s_full[group], (pv >> 1) & 1, &sm.dead);
        if (!__all_sync(0xffffffffu, ok)) break;
      }
      for (int y = 0; y < parts; ++y) {
        const int x = NW == 2 ? (y >> 1) * 2 + group : y;
        const int part = NW == 2 ? y & 1 : 0;
        const int buf = (NW == 2 ? group * 2 : 0) + (pv & 1);  // of the weights
        const int kk = nt == 2 ? x >> 1 : x;
        const int j0 = c.lo + (w.k0 + kk) * KT + part * 64;
        const uint32_t t_s = tm + lanes + buf * 64;  // scores of 128 keys are two parts side by side
        if (part == 0) {
          ok = tc::bar_wait(&sm.seen_full[(k_base + kk) & 15], (unsigned)((k_base + kk) >> 4) & 1, &sm.dead);
#pragma unroll
          for (int i = 0; i < 2 * S::kParts; ++i) there[i] = sm.seen[(k_base + kk) & 15][i];
          ok = ok && tc::bar_wait(&sm.s_full[NW == 2 ? group : buf], (pv >> 1) & 1, &sm.dead);
          if (!__all_sync(0xffffffffu, ok)) break;
          tc::fence_after();
        } else {
          there[0] = there[2 * S::kParts - 2];
          there[1] = there[2 * S::kParts - 1];
        }
        const bool open = __all_sync(0xffffffffu, (there[0] & there[1]) == 0xffffffffu && j0 + 64 <= limit);
        uint32_t v[2][32];
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) tc::tmem_load32(v[ch], t_s + ch * 32);
        tc::wait_loads();
        if (!open) {  // scores of unseen keys
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            const uint32_t word = there[ch];
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((word >> i) & 1) || j0 + ch * 32 + i >= limit) v[ch][i] = 0xff800000u;
          }
        }
        float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            top4[(i >> 1) & 3] = max3(top4[(i >> 1) & 3], __uint_as_float(v[ch][i]), __uint_as_float(v[ch][i + 1]));
        const float top = fmaxf(max3(top4[0], top4[1], top4[2]), top4[3]);
        const float mt = top * a.scale_log2 - kLift;  // -infinity stays (scale > 0)
        if (!any) {
          m = mt;
        } else if (__any_sync(0xffffffffu, mt > m + (float)kLag)) {
          // the last product into O is done before O is changed
          ok = product_done();
          if (!ok) break;
          tc::fence_after();
          const float up = fmaxf(m, mt);
          const float f = fast_exp2(m - (up == -INFINITY ? 0.f : up));
          l *= f;
          m = up;
#pragma unroll 1
          for (int ch = 0; ch < DP / 16; ++ch) {  // rare: few registers rather than few waits
            uint32_t x[16];
            tc::tmem_load16(x, t_o + ch * 16);
            tc::wait_loads();
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
            tc::tmem_store16(t_o + ch * 16, x);
          }
        }
        any = true;
        const float base = m == -INFINITY ? 0.f : m;
        const float2 scale2 = make_float2(a.scale_log2, a.scale_log2), minus2 = make_float2(-base, -base);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float2 e =
                __ffma2_rn(make_float2(__uint_as_float(v[ch][i]), __uint_as_float(v[ch][i + 1])), scale2, minus2);
            e.x = fast_exp2(e.x);
            e.y = fast_exp2(e.y);
            sum = __fadd2_rn(sum, e);
            p[i / 2] = pack2((const T*)nullptr, e.x, e.y);
          }
          tc::tmem_store16(t_s + ch * 16, p);  // over the scores
        }
        l += sum.x + sum.y;
        tc::wait_stores();
        tc::fence_before();
        tc::bar_arrive(&sm.p_full[buf]);
        ++pv;
      }
      k_base += kt;
      if (!__all_sync(0xffffffffu, ok)) break;

      // ---- the unit's rows: wait for the last product, then out
      if (any) ok = product_done();
      if (!ok) break;
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
        const int64_t row = at.t * a.nq + at.h;
        if (final) {
          const float inv = inverse_sum(l, w, at.t);
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
              for (int i = 0; i < 32; i += 16) {
                alignas(16) T o[16];
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                  fine = fine && fabsf(y[i + e]) <= FLT_MAX && fabsf(y[i + e + 1]) <= FLT_MAX;
                  narrow2(&o[e], make_float2(y[i + e], y[i + e + 1]));
                }
                T* const p = out + row * a.D + ch * 32 + i;
                if (access_ok(p, 32, a.out_span, g.err)) {
                  if (wide) {
                    store8(reinterpret_cast<float*>(p), reinterpret_cast<const float*>(o));
                  } else {
                    reinterpret_cast<uint4*>(p)[0] = reinterpret_cast<const uint4*>(o)[0];
                    reinterpret_cast<uint4*>(p)[1] = reinterpret_cast<const uint4*>(o)[1];
                  }
                }
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 8) store8(to + ch * 32 + i, &y[i]);
            }
          }
        }
        if (mine) {
          if (final) {
            if (lse && access_ok(lse + row, 4, a.lse_span, g.err))
              lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
          } else {
            float* ml = whole ? c.dense + a.T * a.nq * a.D + row * 2
                              : slot_ml(c, a, blockIdx.x, begins ? 1 : 0) + r * 2;
            *reinterpret_cast<float2*>(ml) = make_float2(m, l);
          }
          if (final && !fine) sm.bad = 1;
          if (begins && !c.solo) c.rec[row] = unit_record(w, r, c);
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
      walk_next<S::M, KT>(w, g, a, c);
    }
  }
  __syncthreads();
  if (tid == 0 && sm.dead) atomicOr(g.err, kWaitExpired);
  if (warp == kMmaWarp) tc::tmem_free(tm, 512);
  __syncwarp();
  if (sm.bad && !sm.dead) mend_rows<T, DP, S::M, KT, S::kThreads>(q, kc, vc, out, lse, g, a, c, sm.tmp);
}

}  // namespace attend
}  // namespace rope
