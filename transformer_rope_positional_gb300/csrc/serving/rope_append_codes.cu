// RoPE of query and key on the way to the query output and to a paged KV cache of 8-bit codes.
//
// The rotation is rope_append.cu's.  What goes to the cache is, for every scale block (one head's `per`
// tokens of a page) that the call writes,
//   most = max |x| of its values that are finite,  e = the least integer with most <= 448 * 2^e
// kept as the byte e + 127 (1 to 254; 0 where all values are 0), and the codes rn(x * 2^-e), E4M3's largest
// value being 448.  Rows of the block that stand before the first one written stay: the byte is then no less
// than it was, and where it grew their codes are rn(c * 2^(old - new)).  A power of two scales exactly, so a
// value is rounded once, and kept rows lose nothing but subnormals' last bits.
//
// The tokens of a scale block stand one after the other in the batch: a run.  A group of D / 16 threads has a row.  A
// short run is one group's, the groups of a warp having a head each; a longer one is a warp's, for one head, its groups
// taking the rows in turn.  Runs of one row go kRows at a time.  A thread has slots of its own in shared memory for its
// pieces of kRows rows and of their table rows, which it copies with cp.async, all at once: an item is a few round
// trips to memory.  Up to kRows rows a group are read once, longer runs again (from L2) once their largest value is known.  Queries go by heads of a token.
#include <cuda_fp8.h>

#include <algorithm>

#include "rope_device.cuh"
#include "serving.h"

namespace rope {
namespace {

constexpr int kThreads = 256;
// Heads of a token that a thread takes pieces of, for queries.
template <typename T, bool MROPE>
__host__ __device__ constexpr int query_heads() {
  return MROPE || sizeof(T) == 4 ? 2 : 4;
}
constexpr unsigned kPositionOutOfRange = 1u;
constexpr unsigned kSlotOutOfRange = 2u;

struct CodesArgs {
  int64_t T, max_seq, num_slots;
  int64_t q_items, items;  // warps' work: first those of keys and values, then of queries
  int64_t q_stride, k_stride, v_stride;
  int32_t hq, hk, hv;
  int32_t kv_sets, q_sets;  // sets of heads that a warp takes at a time
  int32_t D, R;
  int32_t group, per_warp;  // C threads to a head, heads of a warp
  int32_t block_size, per, S;
  int32_t window;  // tokens in which a warp looks for the beginnings of runs
  int32_t subs;    // warps that share a set's heads
  int32_t mrope_rows;
  int32_t section_end[4];
  int32_t interleave_end;  // > 0: the interleaved splice below this index
  bool copy_tail;          // q is written to another place, so its columns [R, D) too
  bool items32;
  Span pos_span, slot_span, q_span, k_span, v_span, tab_span, qo_span, kc_span, vc_span, ks_span, vs_span;
};

__device__ __forceinline__ int row_of(int i, const CodesArgs& a) {
  if (a.interleave_end > 0) return i < a.interleave_end ? i % 3 : 0;
  return (i >= a.section_end[0]) + (i >= a.section_end[1]) + (i >= a.section_end[2]);
}

template <bool EXACT>
__device__ __forceinline__ float rotate_one(float a, float b, float c, float d) {
  if constexpr (EXACT) return __fmaf_rn(a, b, -__fmul_rn(c, d));
  return diff_of_products(a, b, c, d);
}

// 2^(e - 127), e from 0 to 254.
__device__ __forceinline__ float power_of(int e) { return __uint_as_float(e == 0 ? 0x00400000u : (uint32_t)e << 23); }

// The byte of the least power of two e with most <= 448 * 2^e (448 = 1.75 * 2^8), at least 1; 0 for 0.
__device__ __forceinline__ int byte_for(float most) {
  const uint32_t u = __float_as_uint(most);
  if (u == 0) return 0;
  return max(1, (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u));
}

// Codes of two values times f; what is not finite is NaN, the format holding no infinity (ANY: there may be some).
template <bool ANY>
__device__ __forceinline__ uint32_t codes_of(float2 v, float2 f) {
  float2 x = __fmul2_rn(v, f);
  if (ANY) x = make_float2(fabsf(v.x) <= FLT_MAX ? x.x : NAN, fabsf(v.y) <= FLT_MAX ? x.y : NAN);
  return __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// Each thread's own slots: what it copies there it reads back, with no barrier.
template <typename T, typename TT>
struct Staged {
  static constexpr int kPieces = 8 * sizeof(T) / 16;   // 16-byte pieces of a chunk
  static constexpr int kTurns = 16 * sizeof(TT) / 16;  // of the cos and sin of a row's two chunks
  static constexpr int kRows = 4 / kPieces;            // rows that a thread has under way
  uint4 data[kRows][2 * kPieces][kThreads];
  uint4 turns[kRows][kTurns][kThreads];
};

// 16 or 8 bytes of a table row, which other warps read too.
__device__ __forceinline__ void copy16(void* smem, const void* p, const Span& s, unsigned* err) {
  const unsigned to = (unsigned)__cvta_generic_to_shared(smem);
  if (access_ok(p, 16, s, err)) asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p) : "memory");
}

// Four cos and four sin of a chunk: binary32 to two slots, 16 bits to the halves of one.
template <typename TT>
__device__ __forceinline__ void copy_turns(uint4* a, uint4* b, const TT* cos, const TT* sin, const Span& s, unsigned* err) {
  if constexpr (sizeof(TT) == 4) {
    copy16(a, cos, s, err);
    copy16(b, sin, s, err);
  } else {
    const unsigned to = (unsigned)__cvta_generic_to_shared(a);
    if (access_ok(cos, 8, s, err)) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(cos) : "memory");
    if (access_ok(sin, 8, s, err)) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to + 8), "l"(sin) : "memory");
  }
}

// T: data; TT: table (T or float).
template <typename T, typename TT, bool NEOX, bool MROPE>
__global__ void __launch_bounds__(kThreads, 2)
    append_codes_kernel(const int64_t* __restrict__ pos, const int64_t* __restrict__ slots, const T* q,
                        const T* __restrict__ k, const T* __restrict__ v, const TT* __restrict__ table, T* qo,
                        uint8_t* __restrict__ kc, uint8_t* __restrict__ vc, uint8_t* __restrict__ ks,
                        uint8_t* __restrict__ vs, unsigned int* __restrict__ err, CodesArgs a) {
  constexpr int VEC = 8;                   // columns of a chunk; a thread owns two chunks of a head
  constexpr int NC = NEOX ? VEC : VEC / 2;  // cos (and sin) values of one chunk
  constexpr bool kExact = sizeof(T) == 2 && sizeof(TT) == 2;
  constexpr int kPieces = Staged<T, TT>::kPieces, kTurns = Staged<T, TT>::kTurns, kRows = Staged<T, TT>::kRows;
  extern __shared__ __align__(16) unsigned char raw[];
  Staged<T, TT>& sm = *reinterpret_cast<Staged<T, TT>*>(raw);
  constexpr int kQueryHeads = query_heads<T, MROPE>();
  const int lane = threadIdx.x & 31;
  const int C = a.group;
  const int g = lane / C, c = lane - g * C;
  const int half = a.R / 2;
  // this thread's two chunks of a head, as first columns, and which of them rotate
  int ca, cb;
  bool ra, rb;  // NEOX: the pair (ca, cb) rotates when ra; else each by itself
  if (NEOX) {
    const int pairs = half / VEC;
    ra = rb = c < pairs;
    ca = ra ? c * VEC : a.R + 2 * (c - pairs) * VEC;
    cb = ra ? ca + half : ca + VEC;
  } else {
    ca = c * VEC;
    cb = (c + C) * VEC;
    ra = ca < a.R;
    rb = cb < a.R;
  }
  const uint64_t policy = l2_evict_first_policy();
  const int ia = NEOX ? ca : ca / 2, ib = cb / 2;  // first cos index of each (NEOX: of the pair)
  wait_for_prior_grid();

  struct Place {
    int64_t p[4];
    bool ok;
  };
  auto place_of = [&](int64_t t) {
    Place x = {{0, 0, 0, 0}, true};
    x.p[0] = ldg(pos + t, a.pos_span, err);
    if constexpr (MROPE) {
      x.p[1] = ldg(pos + a.T + t, a.pos_span, err);
      x.p[2] = ldg(pos + 2 * a.T + t, a.pos_span, err);
      if (a.mrope_rows > 3) x.p[3] = ldg(pos + 3 * a.T + t, a.pos_span, err);
    }
#pragma unroll
    for (int j = 0; j < (MROPE ? 4 : 1); ++j) x.ok = x.ok && x.p[j] >= 0 && x.p[j] < a.max_seq;
    return x;
  };
  auto gather = [&](const Place& x, int i0, float (&cf)[NC], float (&sf)[NC]) {
    const int k0 = MROPE ? row_of(i0, a) : 0;
    bool one = true;
    if constexpr (MROPE) one = a.interleave_end > 0 ? i0 >= a.interleave_end : k0 == row_of(i0 + NC - 1, a);
    auto row = [&](int s) { return table + (s == 0 ? x.p[0] : s == 1 ? x.p[1] : s == 2 ? x.p[2] : x.p[3]) * a.R; };
    if (one) {
      load_f32<TT, NC>(cf, row(k0) + i0, a.tab_span, err);
      load_f32<TT, NC>(sf, row(k0) + half + i0, a.tab_span, err);
    } else {
#pragma unroll
      for (int e = 0; e < NC; ++e) {
        const TT* w = row(row_of(i0 + e, a));
        cf[e] = widen(ldg(w + i0 + e, a.tab_span, err));
        sf[e] = widen(ldg(w + half + i0 + e, a.tab_span, err));
      }
    }
  };
  // cos and sin of both chunks (NEOX: of the pair, in the first two)
  auto turns = [&](const Place& where, float (&cf)[NC], float (&sf)[NC], float (&cg)[NC], float (&sg)[NC]) {
    if (ra) gather(where, ia, cf, sf);
    if (!NEOX && rb) gather(where, ib, cg, sg);
  };
  // both chunks of a head, rotated, in binary32
  auto turn = [&](const Vec<T, VEC>& x, const Vec<T, VEC>& y, const float (&cf)[NC], const float (&sf)[NC],
                  const float (&cg)[NC], const float (&sg)[NC], float (&xf)[VEC], float (&yf)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      xf[e] = widen(x.e[e]);
      yf[e] = widen(y.e[e]);
    }
    if constexpr (NEOX) {
      if (ra) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float a1 = xf[e], a2 = yf[e];
          xf[e] = rotate_one<kExact>(a1, cf[e], a2, sf[e]);
          yf[e] = rotate_one<kExact>(a2, cf[e], -a1, sf[e]);
        }
      }
    } else {
      auto one = [&](float (&z)[VEC], const float (&co)[NC], const float (&si)[NC]) {
#pragma unroll
        for (int e = 0; e < NC; ++e) {
          const float a1 = z[2 * e], a2 = z[2 * e + 1];
          z[2 * e] = rotate_one<kExact>(a1, co[e], a2, si[e]);
          z[2 * e + 1] = rotate_one<kExact>(a2, co[e], -a1, si[e]);
        }
      };
      if (ra) one(xf, cf, sf);
      if (rb) one(yf, cg, sg);
    }
  };

  const int64_t kv_items = a.items - a.q_items;
  for (int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); item < a.items;
       item += (int64_t)gridDim.x * (kThreads / 32)) {
    if (item >= kv_items) {
      // ---- queries: some heads of one token
      const int64_t t = div_index(item - kv_items, a.q_sets, a.items32);
      const int set = (int)(item - kv_items - t * a.q_sets);
      const int64_t slot = set == 0 ? ldg(slots + t, a.slot_span, err) : 0;
      const Place where = place_of(t);
      const bool ta = ra || a.copy_tail, tb = rb || a.copy_tail;
      Vec<T, VEC> x[kQueryHeads] = {}, y[kQueryHeads] = {};
      bool mine[kQueryHeads];
#pragma unroll
      for (int e = 0; e < kQueryHeads; ++e) {
        const int h = (set * kQueryHeads + e) * a.per_warp + g;
        mine[e] = g < a.per_warp && h < a.hq && where.ok;
        const T* src = q + t * a.q_stride + (int64_t)h * a.D;
        if (mine[e] && ta) load_vec<true>(x[e], src + ca, a.q_span, err);
        if (mine[e] && tb) load_vec<true>(y[e], src + cb, a.q_span, err);
      }
      if (set == 0 && lane == 0) {  // reported once a token
        if (!where.ok) atomicOr(err, kPositionOutOfRange);
        else if (slot >= a.num_slots) atomicOr(err, kSlotOutOfRange);
      }
      if (!mine[0]) continue;  // (then none is)
      float cf[NC], sf[NC], cg[NC], sg[NC];
      turns(where, cf, sf, cg, sg);
#pragma unroll
      for (int e = 0; e < kQueryHeads; ++e) {
        if (!mine[e]) continue;
        float xf[VEC], yf[VEC];
        turn(x[e], y[e], cf, sf, cg, sg, xf, yf);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          x[e].e[i] = narrow<T>(xf[i]);
          y[e].e[i] = narrow<T>(yf[i]);
        }
        const int h = (set * kQueryHeads + e) * a.per_warp + g;
        T* dst = qo + (a.copy_tail ? t * (int64_t)a.hq * a.D : t * a.q_stride) + (int64_t)h * a.D;
        if (ta) store_vec(dst + ca, x[e], a.qo_span, err);
        if (tb) store_vec(dst + cb, y[e], a.qo_span, err);
      }
      continue;
    }
    // ---- keys and values: the runs that begin in a window of tokens, a set of heads
    const int64_t w = div_index(item, a.kv_sets * a.subs, a.items32);
    const int rest = (int)(item - w * (a.kv_sets * a.subs)), set = rest / a.subs, sub = rest - set * a.subs;
    const int u0 = set * a.per_warp, all = a.hk + a.hv;
    // lane i looks at token t0 + i: those of the window, and those behind it that their runs go on to
    const int64_t t0 = w * a.window;
    const bool token = t0 + lane < a.T;
    const int64_t slot = token ? ldg(slots + t0 + lane, a.slot_span, err) : -1;
    const int64_t at0 = !MROPE && token ? ldg(pos + t0 + lane, a.pos_span, err) : 0;
    int64_t prev = __shfl_up_sync(0xffffffffu, slot, 1);
    if (lane == 0) prev = t0 > 0 ? ldg(slots + t0 - 1, a.slot_span, err) : -1;
    const bool there = slot >= 0 && slot < a.num_slots;
    const int64_t block = there ? div_index(slot, a.per, a.items32) : 0;
    const int first = (int)(slot - block * a.per);
    const bool goes_on = there && prev >= 0 && prev + 1 == slot && first > 0;  // the run of the token before
    if (a.hq == 0 && rest == 0 && token && lane < a.window) {  // reported once a token: here without queries
      if (!place_of(t0 + lane).ok) atomicOr(err, kPositionOutOfRange);
      else if (slot >= a.num_slots) atomicOr(err, kSlotOutOfRange);
    }
    const uint32_t on_mask = __ballot_sync(0xffffffffu, goes_on);
    uint32_t begins = __ballot_sync(0xffffffffu, there && !goes_on) & (uint32_t)((1ull << a.window) - 1);
    // position(s) of the token `t0 + i`, i different in every lane; all lanes call it
    auto place_at = [&](int i, bool wanted) {
      if constexpr (MROPE) {
        return wanted ? place_of(t0 + i) : Place{{0, 0, 0, 0}, false};
      } else {
        Place x = {{__shfl_sync(0xffffffffu, at0, i & 31), 0, 0, 0}, false};
        if (wanted && i >= 32) x.p[0] = ldg(pos + t0 + i, a.pos_span, err);
        x.ok = wanted && x.p[0] >= 0 && x.p[0] < a.max_seq;
        return x;
      }
    };
    int singles = 0;
    while (begins) {
      // ---- what is done at a time: a run of several rows, head by head; or up to kRows runs of one, their heads side by side
      int i0 = __ffs(begins) - 1;
      int n = 1;
      {
        const uint32_t after = i0 == 31 ? 0u : ~(on_mask >> (i0 + 1));  // the first 1: where the run has ended
        n += after ? __ffs(after) - 1 : 31;
        n = min(n, 32 - i0);
        const int64_t s0 = __shfl_sync(0xffffffffu, slot, i0);
        const int f0 = __shfl_sync(0xffffffffu, first, i0);
        while (i0 + n >= 32) {  // beyond what the lanes look at
          const int j = n + lane;
          const bool on = f0 + j < a.per && t0 + i0 + j < a.T && ldg(slots + t0 + i0 + j, a.slot_span, err) == s0 + j;
          const uint32_t off = ~__ballot_sync(0xffffffffu, on);
          n += off ? __ffs(off) - 1 : 32;
          if (off) break;
        }
      }
      const bool single = n == 1;
      uint32_t run_of = 0x01010101u * i0;  // the tokens that begin the runs, relative to t0: 8 bits each
      int count = 1;
      begins &= begins - 1;
      while (single && count < kRows && begins) {
        const int j = __ffs(begins) - 1;
        if (on_mask >> (j + 1) & 1) break;  // (j is below 16)
        run_of = (run_of & ~(0xffu << 8 * count)) | (uint32_t)j << 8 * count;
        ++count;
        begins &= begins - 1;
      }
      if (single && singles++ % a.subs != sub) continue;  // the warps that share the set take them in turn
      const int head0 = single ? 0 : sub, heads_here = single ? 1 : min(a.per_warp, all - u0);
      const int by = single ? 1 : a.subs;
      for (int j = head0; j < heads_here; j += by) {
        const int u = u0 + (single ? g : j);
        const bool mine = g < a.per_warp && u < all;
        const bool is_v = u >= a.hk;
        const int h = is_v ? u - a.hk : u, heads = is_v ? a.hv : a.hk;
        const T* const src = (is_v ? v : k) + (int64_t)h * a.D;
        const int64_t stride = is_v ? a.v_stride : a.k_stride;
        const Span& sspan = is_v ? a.v_span : a.k_span;
        const Span& cspan = is_v ? a.vc_span : a.kc_span;
        const Span& zspan = is_v ? a.vs_span : a.ks_span;
        const int step = single ? 1 : a.per_warp, g0 = single ? 0 : g;
        // the scale byte and the rows of the block of token t0 + i, and the row of that token in it; all lanes call it
        auto block_at = [&](int i, uint8_t*& at, uint8_t*& rows, int& f) {
          const int64_t b = __shfl_sync(0xffffffffu, block, i);
          f = __shfl_sync(0xffffffffu, first, i);
          const int64_t page = div_index(b, a.S, a.items32);
          const int part = (int)(b - page * a.S);
          at = (is_v ? vs : ks) + (page * heads + h) * a.S + part;
          rows = (is_v ? vc : kc) + ((page * heads + h) * a.block_size + (int64_t)part * a.per) * a.D;
        };
        // Rows under way, in slot e: of the one run the row base + e * step, or of run e its only one; with their table rows.
        auto token_of = [&](int base, int e) { return single ? (int)(run_of >> 8 * e & 0xffu) : i0 + base + e * step; };
        uint32_t on = 0;  // which of them are written, a bit a slot
        auto read = [&](int base) {
          on = 0;
#pragma unroll 1
          for (int e = 0; e < kRows; ++e) {
            const bool is_row = mine && (single ? e < count : base + e * step < n);
            const int i = token_of(base, e);
            const Place where = place_at(i, is_row);
            if (where.ok) {
              on |= 1u << e;
              const T* const p = src + (t0 + i) * stride;
#pragma unroll
              for (int z = 0; z < kPieces; ++z) {
                cp_async16(&sm.data[e][z][threadIdx.x], p + ca + z * (16 / sizeof(T)), policy, sspan, err);
                cp_async16(&sm.data[e][kPieces + z][threadIdx.x], p + cb + z * (16 / sizeof(T)), policy, sspan, err);
              }
              if (!MROPE && !is_v) {
                const TT* const row = table + where.p[0] * a.R;
                if constexpr (NEOX) {
                  if (ra)
#pragma unroll
                    for (int z = 0; z < kTurns / 2; ++z) {
                      copy16(&sm.turns[e][z][threadIdx.x], row + ia + z * (16 / sizeof(TT)), a.tab_span, err);
                      copy16(&sm.turns[e][kTurns / 2 + z][threadIdx.x], row + half + ia + z * (16 / sizeof(TT)), a.tab_span, err);
                    }
                } else {
                  if (ra) copy_turns<TT>(&sm.turns[e][0][threadIdx.x], &sm.turns[e][kTurns / 4][threadIdx.x], row + ia, row + half + ia, a.tab_span, err);
                  if (rb) copy_turns<TT>(&sm.turns[e][kTurns / 2][threadIdx.x], &sm.turns[e][kTurns * 3 / 4][threadIdx.x], row + ib, row + half + ib, a.tab_span, err);
                }
              }
            }
            __syncwarp();
          }
          cp_async_commit();
          cp_async_wait<0>();
        };
        // Slot e in binary32: rotated twice, for the largest value and for the codes, rather than held.  Two roundings an
        // element, 2^-24 of the two terms each: a code's step is 2^-4 of it.
        float2 xf[VEC / 2], yf[VEC / 2];
        auto values = [&](int base, int e) {
          Vec<T, VEC> x, y;
#pragma unroll
          for (int z = 0; z < kPieces; ++z) {
            reinterpret_cast<uint4*>(x.e)[z] = sm.data[e][z][threadIdx.x];
            reinterpret_cast<uint4*>(y.e)[z] = sm.data[e][kPieces + z][threadIdx.x];
          }
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i) {
            xf[i] = widen2(&x.e[2 * i]);
            yf[i] = widen2(&y.e[2 * i]);
          }
          if (is_v) return;
          float cf[NC], sf[NC], cg[NC], sg[NC];
          if constexpr (MROPE) {
            turns(place_of(t0 + token_of(base, e)), cf, sf, cg, sg);
          } else {
            Vec<TT, 2 * VEC> z;  // as they were copied: NEOX cos, sin; else cos, sin of the first chunk, of the second
#pragma unroll
            for (int i = 0; i < kTurns; ++i) reinterpret_cast<uint4*>(z.e)[i] = sm.turns[e][i][threadIdx.x];
#pragma unroll
            for (int i = 0; i < NC; ++i) {
              cf[i] = widen(z.e[i]);
              sf[i] = widen(z.e[NC + i]);
              if constexpr (!NEOX) {
                cg[i] = widen(z.e[2 * NC + i]);
                sg[i] = widen(z.e[3 * NC + i]);
              }
            }
          }
          if constexpr (NEOX) {
            if (ra)
#pragma unroll
              for (int i = 0; i < VEC / 2; ++i) {
                const float2 co = make_float2(cf[2 * i], cf[2 * i + 1]), si = make_float2(sf[2 * i], sf[2 * i + 1]);
                const float2 t = __fmul2_rn(yf[i], si), s = __fmul2_rn(xf[i], si);
                xf[i] = __ffma2_rn(xf[i], co, make_float2(-t.x, -t.y));
                yf[i] = __ffma2_rn(yf[i], co, s);
              }
          } else {
            auto one = [&](float2 (&z)[VEC / 2], const float (&co)[NC], const float (&si)[NC]) {
#pragma unroll
              for (int i = 0; i < NC; ++i)
                z[i] = make_float2(fmaf(z[i].x, co[i], -(z[i].y * si[i])), fmaf(z[i].y, co[i], z[i].x * si[i]));
            };
            if (ra) one(xf, cf, sf);
            if (rb) one(yf, cg, sg);
          }
        };
        auto largest = [&]() {  // (NaN is passed over, an infinity is not)
          float m = 0.f;
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i) {
            m = max3(m, fabsf(xf[i].x), fabsf(xf[i].y));
            m = max3(m, fabsf(yf[i].x), fabsf(yf[i].y));
          }
          return m;
        };
        auto largest_finite = [&]() {
          float m = 0.f;
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i)
            for (float v : {xf[i].x, xf[i].y, yf[i].x, yf[i].y})
              if (fabsf(v) <= FLT_MAX) m = fmaxf(m, fabsf(v));
          return m;
        };
        // the block's byte; rows before the first one written again where it grew
        auto byte_of = [&](float most, int old, int f, uint8_t* rows) {
          const int byte = byte_for(most);
          if (f > 0 && old >= byte) return old;
          const float scale = old == 0 ? 0.f : power_of(max(127 + old - byte, 0));
#pragma unroll 1
          for (int i = g0; i < f; i += step)
#pragma unroll 1
            for (int z = 0; z < 2; ++z) {
              uint8_t* const p = rows + (int64_t)i * a.D + (z ? cb : ca);
              if (!access_ok(p, VEC, cspan, err)) continue;
              uint2 was = *reinterpret_cast<const uint2*>(p);
              uint32_t now[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __half2_raw r =
                    __nv_cvt_fp8x2_to_halfraw2((e < 2 ? was.x : was.y) >> (e & 1) * 16 & 0xffffu, __NV_E4M3);
                const float2 d = __half22float2(__half2(r));
                now[e] = codes_of<false>(d, make_float2(scale, scale));
              }
              *reinterpret_cast<uint2*>(p) = make_uint2(now[0] | now[1] << 16, now[2] | now[3] << 16);
            }
          return byte;
        };
        uint8_t *at, *rows;
        int f;
        uint32_t old = 0;  // bytes of the blocks (singles: 8 bits each) that hold rows before
        for (int e = single ? count - 1 : 0; e >= 0; --e) {
          block_at(token_of(0, e), at, rows, f);
          old = old << 8 | (mine && f > 0 && access_ok(at, 1, zspan, err) ? (uint32_t)*at : 0u);
        }
        __syncwarp();  // (read by all before they are written)
        const int passes = single ? 1 : (n + kRows * step - 1) / (kRows * step);
        float most = 0.f;
        bool any = false;     // some token of the run is written
        uint32_t bytes = 0;   // of the blocks now, singles: 8 bits each
        for (int pass = 0; pass < passes; ++pass) {
          const int base = pass * kRows * step + g0;
          read(base);
#pragma unroll 1
          for (int e = 0; e < kRows; ++e) {
            float m = 0.f;
            if (on >> e & 1) {
              values(base, e);
              m = largest();
              if (m > FLT_MAX) m = largest_finite();
            }
            if (!single) {
              most = fmaxf(most, m);
              any = any || on != 0;
              continue;
            }
            if (e >= count) break;
            // over the group: the windows of lanes that a value has seen double, round the group
            for (int d = 1; d < C; d *= 2) {
              int from = c + d;
              if (from >= C) from -= C;
              m = fmaxf(m, __shfl_sync(0xffffffffu, m, min(g * C + from, 31)));
            }
            block_at(token_of(0, e), at, rows, f);
            if (on >> e & 1) {
              const int byte = byte_of(m, old >> 8 * e & 0xffu, f, rows);
              bytes |= (uint32_t)byte << 8 * e;
              if (c == 0 && access_ok(at, 1, zspan, err)) *at = (uint8_t)byte;
            }
            __syncwarp();
          }
        }
        if (!single) {
          most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
          if (!__any_sync(0xffffffffu, any)) continue;
          bytes = mine ? byte_of(most, old, f, rows) : 0;
          if (lane == 0 && access_ok(at, 1, zspan, err)) *at = (uint8_t)bytes;
          __syncwarp();
        }
        for (int pass = passes - 1; pass >= 0; --pass) {
          const int base = pass * kRows * step + g0;
          if (pass != passes - 1) read(base);  // (the last one's rows are still there)
#pragma unroll 1
          for (int e = 0; e < kRows; ++e) {
            if (single) {
              if (e >= count) break;
              block_at(token_of(0, e), at, rows, f);
            }
            if (on >> e & 1) {
              values(base, e);
              const uint32_t byte = single ? bytes >> 8 * e & 0xffu : bytes;
              const float f1 = byte == 255 ? NAN : power_of(254 - byte);
              const float2 scale = make_float2(f1, f1);
              uint32_t z[8];
              if (largest() > FLT_MAX) {
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = codes_of<true>(xf[i], scale), z[4 + i] = codes_of<true>(yf[i], scale);
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = codes_of<false>(xf[i], scale), z[4 + i] = codes_of<false>(yf[i], scale);
              }
              uint8_t* const p = rows + (int64_t)(single ? f : f + base + e * step) * a.D;
              if (access_ok(p + ca, VEC, cspan, err))
                *reinterpret_cast<uint2*>(p + ca) = make_uint2(z[0] | z[1] << 16, z[2] | z[3] << 16);
              if (access_ok(p + cb, VEC, cspan, err))
                *reinterpret_cast<uint2*>(p + cb) = make_uint2(z[4] | z[5] << 16, z[6] | z[7] << 16);
            }
            __syncwarp();
          }
        }
      }
    }
  }
}

template <typename T, typename TT, bool NEOX, bool MROPE>
cudaError_t launch_as(const AppendProblem& p, cudaStream_t stream) {
  CodesArgs a;
  a.T = p.T;
  a.max_seq = p.max_seq;
  a.num_slots = p.num_blocks * p.block_size;
  a.q_stride = p.q_stride;
  a.k_stride = p.k_stride;
  a.v_stride = p.v_stride;
  a.hq = p.query ? (int32_t)p.hq : 0;
  a.hk = (int32_t)p.hk;
  a.hv = (int32_t)p.hv;
  a.D = (int32_t)p.head_size;
  a.R = (int32_t)p.rotary_dim;
  a.group = a.D / 16;
  a.per_warp = 32 / a.group;
  a.kv_sets = (a.hk + a.hv + a.per_warp - 1) / a.per_warp;
  constexpr int kQueryHeads = query_heads<T, MROPE>();
  a.q_sets = (a.hq + kQueryHeads * a.per_warp - 1) / (kQueryHeads * a.per_warp);
  a.block_size = (int32_t)p.block_size;
  a.S = (int32_t)p.scale_blocks;
  a.per = a.block_size / a.S;
  // Few tokens: one to a window, so that all SMs are busy.  Many: up to 16.
  a.window = 1;
  a.subs = a.per_warp;
  const int64_t enough = (int64_t)sm_count() * 16;
  while (a.window < 16 && p.T / (2 * a.window) * a.kv_sets * a.subs >= enough) a.window *= 2;
  a.q_items = p.T * a.q_sets;
  a.items = a.q_items + (p.T + a.window - 1) / a.window * a.kv_sets * a.subs;
  a.mrope_rows = p.mrope_rows;
  for (int i = 0; i < 4; ++i) a.section_end[i] = i < p.mrope_rows ? p.section_end[i] : a.R / 2;
  a.interleave_end = p.cache_mode == 1 ? 3 * (p.section_end[1] - p.section_end[0]) : 0;
  a.copy_tail = p.query_out != p.query;
  a.items32 = a.items <= 0xffffffffLL && a.num_slots <= 0xffffffffLL;
  const int64_t e = sizeof(T), D = p.head_size;
  a.pos_span = make_span(p.positions, (p.mrope_rows ? p.mrope_rows : 1) * p.T * 8);
  a.slot_span = make_span(p.slot_mapping, p.T * 8);
  a.q_span = make_span(p.query, ((p.T - 1) * p.q_stride + a.hq * D) * e);
  a.k_span = make_span(p.key, ((p.T - 1) * p.k_stride + p.hk * D) * e);
  a.v_span = make_span(p.value, ((p.T - 1) * p.v_stride + p.hv * D) * e);
  a.tab_span = make_span(p.table, p.max_seq * p.rotary_dim * (int64_t)sizeof(TT));
  a.qo_span = make_span(p.query_out, (a.copy_tail ? p.T * a.hq * D : (p.T - 1) * p.q_stride + a.hq * D) * e);
  a.kc_span = make_span(p.k_cache, a.num_slots * p.hk * D);
  a.vc_span = make_span(p.v_cache, a.num_slots * p.hv * D);
  a.ks_span = make_span(p.k_scale, p.num_blocks * p.hk * p.scale_blocks);
  a.vs_span = make_span(p.v_scale, p.num_blocks * p.hv * p.scale_blocks);
  auto kernel = append_codes_kernel<T, TT, NEOX, MROPE>;
  const int64_t warps = kThreads / 32;
  const size_t smem = sizeof(Staged<T, TT>);
  unsigned int* err = nullptr;
  cudaError_t er = device_error_address(&err);
  if (er == cudaSuccess) er = opt_in_shared(reinterpret_cast<const void*>(kernel), smem);
  if (er != cudaSuccess) return er;
  const int64_t resident = (int64_t)sm_count() * resident_blocks(reinterpret_cast<const void*>(kernel), kThreads, smem);
  const int64_t grid = std::max<int64_t>(1, std::min((a.items + warps - 1) / warps, resident));
  return launch_overlapped_smem(kernel, (unsigned)grid, kThreads, smem, stream, p.positions, p.slot_mapping,
                           static_cast<const T*>(p.query), static_cast<const T*>(p.key),
                           static_cast<const T*>(p.value), static_cast<const TT*>(p.table),
                           static_cast<T*>(p.query_out), static_cast<uint8_t*>(p.k_cache),
                           static_cast<uint8_t*>(p.v_cache), p.k_scale, p.v_scale, err, a);
}

template <typename T, typename TT>
cudaError_t launch_typed(const AppendProblem& p, cudaStream_t stream) {
  if (p.is_neox)
    return p.mrope_rows ? launch_as<T, TT, true, true>(p, stream) : launch_as<T, TT, true, false>(p, stream);
  return p.mrope_rows ? launch_as<T, TT, false, true>(p, stream) : launch_as<T, TT, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_append_codes(const AppendProblem& p, cudaStream_t stream) {
  const bool wide = p.table_dtype == kF32;
  switch (p.dtype) {
    case kF32:
      return launch_typed<float, float>(p, stream);
    case kF16:
      return wide ? launch_typed<__half, float>(p, stream) : launch_typed<__half, __half>(p, stream);
    case kBF16:
      return wide ? launch_typed<__nv_bfloat16, float>(p, stream)
                  : launch_typed<__nv_bfloat16, __nv_bfloat16>(p, stream);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace rope
