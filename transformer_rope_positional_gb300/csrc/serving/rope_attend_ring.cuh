// A warp's own pipeline of K and V rows: shared by the kernels whose units have few rows.
//
// The warp takes KEYS keys of every KT-key tile and copies their K and V rows into its ring of
// S stages with cp.async (16-byte pieces), K and V of a tile one stage each, in the order of
// use, over the units of the CTA's share.  Pages are looked up a tile ahead of their use.  The
// warp waits for its own copies only.
#pragma once

#include "rope_attend.cuh"

namespace rope {
namespace attend {

__device__ __forceinline__ unsigned smem_u32(const void* p) { return (unsigned)__cvta_generic_to_shared(p); }

// 16 bytes, or zeros where !ok.
__device__ __forceinline__ void cp_async16_or_zero(unsigned dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}

// 2^x, relative error 2^-22 (0 for -infinity).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// DP: columns of a row in shared memory (those past D are zeros).  SWIZZLE: piece i of row r at
// place i ^ (r & 7).  At most 6 tiles are under way (S <= 11).
template <typename T, int KEYS, int DP, int S, int M, int KT, bool SWIZZLE>
struct Ring {
  static constexpr int kRow = DP * (int)sizeof(T);
  static constexpr int kStage = KEYS * kRow;
  static constexpr int VEC = 16 / (int)sizeof(T);
  static constexpr int CH = DP / VEC;  // pieces of a row
  static_assert(S <= 11 && KEYS <= 16 && KEYS * CH % 32 == 0, "ring shape");

  Walk pw;             // unit of the next copy
  int pk, pend;        // its tile, and where the unit's keys end
  int slot;            // stage of the next copy
  int next_tile;       // its tile, modulo 6
  bool next_v;         // it is V
  PageRow page;        // of this lane's key (lane % KEYS) of the next tile
  int row;             // cache row of the key of the tile whose K was copied last
  uint32_t valid[3];   // 16 bits a tile: which of its keys are there, for the last 6 tiles
  int cur, tile;       // stage and tile of the next product
  unsigned char* ring;

  __device__ __forceinline__ void look_up(const Pointers& g, const AttendArgs& a, const Cut& c) {
    page = {-2, 0};  // no such key
    if (pw.done) return;
    const int lane = threadIdx.x & 31;
    const int j = c.lo + pk * KT + (threadIdx.x >> 5) * KEYS + lane % KEYS;
    if (j < pend) page = page_row(j, g.block_table + (int64_t)pw.b * a.W, g, a);
  }

  __device__ __forceinline__ void start(const Walk& w, unsigned char* at, const Pointers& g, const AttendArgs& a,
                                        const Cut& c) {
    pw = w;
    pk = pw.k0;
    pend = tile_end<M>(pw.s, pw.i, a, c);
    slot = next_tile = cur = tile = 0;
    next_v = false;
    row = -1;
    valid[0] = valid[1] = valid[2] = 0;
    ring = at;
    look_up(g, a, c);
  }

  __device__ __forceinline__ void copy(const T* __restrict__ kc, const T* __restrict__ vc, const Pointers& g,
                                       const AttendArgs& a, const Cut& c) {
    const int lane = threadIdx.x & 31;
    if (!next_v) {
      row = -1;
      if (page.page >= 0 && page.page < a.num_blocks)
        row = ((int)page.page * a.nk + pw.h) * a.block_size + page.row;
      else if (page.page != -2)
        atomicOr(g.err, kSlotOutOfRange);
      const uint32_t there = __ballot_sync(0xffffffffu, row >= 0) & ((1u << KEYS) - 1u);
      uint32_t& word = next_tile < 2 ? valid[0] : next_tile < 4 ? valid[1] : valid[2];
      word = next_tile & 1 ? (word & 0x0000ffffu) | (there << 16) : (word & 0xffff0000u) | there;
      next_tile = next_tile == 5 ? 0 : next_tile + 1;
      if (!pw.done) {
        if (++pk == walk_k1(pw, c)) {
          walk_next<M, KT>(pw, g, a, c);
          pk = pw.k0;
          if (!pw.done) pend = tile_end<M>(pw.s, pw.i, a, c);
        }
      }
      look_up(g, a, c);
    }
    const T* const src = next_v ? vc : kc;
    const Span& span = next_v ? a.v_span : a.k_span;
    unsigned char* const to = ring + slot * kStage;
    if (__any_sync(0xffffffffu, row >= 0)) {
      const unsigned dst = smem_u32(to);
#pragma unroll
      for (int i = 0; i < KEYS * CH / 32; ++i) {
        const int idx = lane + 32 * i;
        const int key = idx / CH, ch = idx - key * CH;
        const int r = __shfl_sync(0xffffffffu, row, key);
        const bool ok = r >= 0 && ch * VEC < a.D;
        const T* p = src + ((uint64_t)(uint32_t)max(r, 0) * (uint32_t)a.D + (ok ? ch * VEC : 0));
        cp_async16_or_zero(dst + key * kRow + ((SWIZZLE ? ch ^ (key & 7) : ch) << 4), p,
                           ok && access_ok(p, 16, span, g.err));
      }
    } else if (next_v) {  // no key of the tile: its weights are 0, and V must not be NaN
#pragma unroll
      for (int i = 0; i < KEYS * CH / 32; ++i)
        *reinterpret_cast<uint4*>(to + (lane + 32 * i) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    next_v = !next_v;
    cp_async_commit();
    slot = slot + 1 == S ? 0 : slot + 1;
  }

  // Which keys of the next tile are there.
  __device__ __forceinline__ uint32_t seen() {
    const uint32_t word = tile < 2 ? valid[0] : tile < 4 ? valid[1] : valid[2];
    const uint32_t there = (tile & 1 ? word >> 16 : word) & 0xffffu;
    tile = tile == 5 ? 0 : tile + 1;
    return there;
  }

  // The next stage, once its copies are there (and its last readers done: the caller has
  // converged the warp after them); another copy is issued into the stage before it.
  __device__ __forceinline__ const unsigned char* take(const T* __restrict__ kc, const T* __restrict__ vc,
                                                       const Pointers& g, const AttendArgs& a, const Cut& c) {
    copy(kc, vc, g, a, c);
    const unsigned char* at = ring + cur * kStage;
    cur = cur + 1 == S ? 0 : cur + 1;
    return at;
  }
};

}  // namespace attend
}  // namespace rope
