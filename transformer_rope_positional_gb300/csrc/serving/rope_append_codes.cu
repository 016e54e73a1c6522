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
// The tokens of a scale block stand one after the other in the batch: a run.  A group of D / 16 threads has a row of a
// head, a thread two chunks of 8 columns of it: for NeoX a rotated pair (or two of the tail), else D / 2 columns apart.
//
// Few tokens: latency counts.  A warp has a token and a set of heads, a group a head; the first warps of a longer run
// share its heads instead, the groups of a warp taking a head's rows in turn.  (32 q, 8 k and 8 v heads of 128, bf16: 64
// requests' tokens 3.5 us, the kernel for many 4.7; a prompt of 512 9.4, 13.7; 1024 requests 11.5, 12.4; 2048 21.3, 20.7.)
//
// Many: what an item costs in round trips and instructions counts as much as its bytes.  A warp has the runs that begin in a window of
// tokens, for a set of heads: a run of up to kRows rows is one group's, the groups having a head each, kRows rows at a
// time (the example below in scale blocks of 2 tokens: 111 us, 218 as longer runs go); a longer one is the warp's, head by
// head, its groups taking the rows in turn.  A thread has slots of its own in
// shared memory for its pieces of kRows rows and of their table rows, which it copies with cp.async, all at once: an item
// is a few round trips to memory.  Up to kRows rows a group are read once, longer runs again (from L2) once their largest
// value is known.  Queries go by heads of a token.  (16384 tokens 84 us, 67% of the copy rate; without the codes, or
// without the queries, 40 and 53.  Nothing is full: DRAM 44 %, issue slots 52 %, and 22 % of the warps; an item's copies are
// waited for before its arithmetic, two rotations and a conversion an element, so it is latency that bounds it.)
#include <cuda_fp8.h>

#include <algorithm>

#include "rope_device.cuh"
#include "serving.h"

namespace rope {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int64_t kFewTokens = 1024;
// Heads of a token that a thread takes pieces of, for queries.
template <typename T, bool MROPE>
__host__ __device__ constexpr int query_heads() {
  return MROPE || sizeof(T) == 4 ? 2 : 4;
}
constexpr unsigned kPositionOutOfRange = 1u;
constexpr unsigned kSlotOutOfRange = 2u;

struct CodesArgs {
  int64_t T, max_seq, num_slots;
  int64_t q_items, items;  // warps' work; many tokens: first those of keys and values, then of queries
  int64_t q_stride, k_stride, v_stride;
  int32_t hq, hk, hv;
  int32_t kv_sets, q_sets;  // sets of heads that a warp takes at a time; few tokens: of keys and values first
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

// 2^(e - 127), e from 0 to 254 (of 0, too, unlike the scale that the byte 0 stands for).
__device__ __forceinline__ float two_to(int e) { return __uint_as_float(e == 0 ? 0x00400000u : (uint32_t)e << 23); }

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

template <typename T, typename TT>
struct Data {
  const int64_t* pos;
  const int64_t* slots;
  const T *q, *k, *v;
  const TT* table;
  T* qo;
  uint8_t *kc, *vc, *ks, *vs;
  unsigned int* err;
};

struct Place {
  int64_t p[4];
  bool ok;
};

// What a thread has to do with a row of a head, and the arithmetic of it.
template <typename T, typename TT, bool NEOX, bool MROPE>
struct Lane {
  static constexpr int VEC = 8;                     // columns of a chunk
  static constexpr int NC = NEOX ? VEC : VEC / 2;   // cos (and sin) values of one chunk
  static constexpr bool kExact = sizeof(T) == 2 && sizeof(TT) == 2;
  int g, c;       // group (row of the warp's), place in it
  int ca, cb;     // first columns of the two chunks
  bool ra, rb;    // which of them rotate (NEOX: the pair does when ra)
  int ia, ib;     // first cos index of each (NEOX: of the pair)

  __device__ __forceinline__ explicit Lane(const CodesArgs& a) {
    const int lane = threadIdx.x & 31, half = a.R / 2;
    g = lane / a.group;
    c = lane - g * a.group;
    if (NEOX) {
      const int pairs = half / VEC;
      ra = rb = c < pairs;
      ca = ra ? c * VEC : a.R + 2 * (c - pairs) * VEC;
      cb = ra ? ca + half : ca + VEC;
    } else {
      ca = c * VEC;
      cb = (c + a.group) * VEC;
      ra = ca < a.R;
      rb = cb < a.R;
    }
    ia = NEOX ? ca : ca / 2;
    ib = cb / 2;
  }

  static __device__ __forceinline__ Place place_of(int64_t t, const Data<T, TT>& d, const CodesArgs& a) {
    Place x = {{0, 0, 0, 0}, true};
    x.p[0] = ldg(d.pos + t, a.pos_span, d.err);
    if constexpr (MROPE) {
      x.p[1] = ldg(d.pos + a.T + t, a.pos_span, d.err);
      x.p[2] = ldg(d.pos + 2 * a.T + t, a.pos_span, d.err);
      if (a.mrope_rows > 3) x.p[3] = ldg(d.pos + 3 * a.T + t, a.pos_span, d.err);
    }
#pragma unroll
    for (int j = 0; j < (MROPE ? 4 : 1); ++j) x.ok = x.ok && x.p[j] >= 0 && x.p[j] < a.max_seq;
    return x;
  }

  // N cos and N sin values from index i0 on, of the token at x.
  template <int N>
  static __device__ __forceinline__ void gather(const Place& x, int i0, float (&cf)[N], float (&sf)[N],
                                                const Data<T, TT>& d, const CodesArgs& a) {
    const int half = a.R / 2, k0 = MROPE ? row_of(i0, a) : 0;
    bool one = true;
    if constexpr (MROPE) one = a.interleave_end > 0 ? i0 >= a.interleave_end : k0 == row_of(i0 + N - 1, a);
    auto row = [&](int s) { return d.table + (s == 0 ? x.p[0] : s == 1 ? x.p[1] : s == 2 ? x.p[2] : x.p[3]) * a.R; };
    if (one) {
      load_f32<TT, N>(cf, row(k0) + i0, a.tab_span, d.err);
      load_f32<TT, N>(sf, row(k0) + half + i0, a.tab_span, d.err);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const TT* w = row(row_of(i0 + e, a));
        cf[e] = widen(ldg(w + i0 + e, a.tab_span, d.err));
        sf[e] = widen(ldg(w + half + i0 + e, a.tab_span, d.err));
      }
    }
  }

  // The chunks x and y rotated; cf, sf of the first (NEOX: of the pair), cg, sg of the second.
  __device__ __forceinline__ void turn(Vec<T, VEC>& x, Vec<T, VEC>& y, const float (&cf)[NC], const float (&sf)[NC],
                                       const float (&cg)[NC], const float (&sg)[NC]) const {
    if constexpr (NEOX) {
      if (ra)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float a1 = widen(x.e[e]), a2 = widen(y.e[e]);
          x.e[e] = narrow<T>(rotate_one<kExact>(a1, cf[e], a2, sf[e]));
          y.e[e] = narrow<T>(rotate_one<kExact>(a2, cf[e], -a1, sf[e]));
        }
    } else {
      auto one = [&](Vec<T, VEC>& z, const float (&co)[NC], const float (&si)[NC]) {
#pragma unroll
        for (int e = 0; e < NC; ++e) {
          const float a1 = widen(z.e[2 * e]), a2 = widen(z.e[2 * e + 1]);
          z.e[2 * e] = narrow<T>(rotate_one<kExact>(a1, co[e], a2, si[e]));
          z.e[2 * e + 1] = narrow<T>(rotate_one<kExact>(a2, co[e], -a1, si[e]));
        }
      };
      if (ra) one(x, cf, sf);
      if (rb) one(y, cg, sg);
    }
  }

  // The chunks in binary32, rotated where `is_key`.  Two roundings an element, 2^-24 of the two terms each: a code's
  // step is 2^-4 of it.
  __device__ __forceinline__ void values(const Vec<T, VEC>& x, const Vec<T, VEC>& y, bool is_key, const float (&cf)[NC],
                                         const float (&sf)[NC], const float (&cg)[NC], const float (&sg)[NC],
                                         float2 (&xf)[VEC / 2], float2 (&yf)[VEC / 2]) const {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      xf[i] = widen2(&x.e[2 * i]);
      yf[i] = widen2(&y.e[2 * i]);
    }
    if (!is_key) return;
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
  }

  // The largest magnitude that is finite.
  static __device__ __forceinline__ float largest(const float2 (&xf)[VEC / 2], const float2 (&yf)[VEC / 2]) {
    float m = 0.f;  // (NaN is passed over, an infinity is not)
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      m = max3(m, fabsf(xf[i].x), fabsf(xf[i].y));
      m = max3(m, fabsf(yf[i].x), fabsf(yf[i].y));
    }
    if (m <= FLT_MAX) return m;
    m = 0.f;
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i)
      for (float v : {xf[i].x, xf[i].y, yf[i].x, yf[i].y})
        if (fabsf(v) <= FLT_MAX) m = fmaxf(m, fabsf(v));
    return m;
  }

  // The largest over the group's threads: the windows of lanes that a value has seen double, round the group.
  __device__ __forceinline__ float over_group(float m, int C) const {
    for (int d = 1; d < C; d *= 2) {
      int from = c + d;
      if (from >= C) from -= C;
      m = fmaxf(m, __shfl_sync(0xffffffffu, m, min(g * C + from, 31)));
    }
    return m;
  }

  // The codes of a row at p, in units of 2^(byte - 127).
  __device__ __forceinline__ void write(uint8_t* p, int byte, const float2 (&xf)[VEC / 2], const float2 (&yf)[VEC / 2],
                                        const Span& span, unsigned* err) const {
    const float f1 = byte == 255 ? NAN : two_to(254 - byte);
    const float2 f = make_float2(f1, f1);
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) m = max3(max3(m, fabsf(xf[i].x), fabsf(xf[i].y)), fabsf(yf[i].x), fabsf(yf[i].y));
    uint32_t z[8];
    if (m > FLT_MAX) {
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = codes_of<true>(xf[i], f), z[4 + i] = codes_of<true>(yf[i], f);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = codes_of<false>(xf[i], f), z[4 + i] = codes_of<false>(yf[i], f);
    }
    if (access_ok(p + ca, VEC, span, err))
      *reinterpret_cast<uint2*>(p + ca) = make_uint2(z[0] | z[1] << 16, z[2] | z[3] << 16);
    if (access_ok(p + cb, VEC, span, err))
      *reinterpret_cast<uint2*>(p + cb) = make_uint2(z[4] | z[5] << 16, z[6] | z[7] << 16);
  }

  // The block's byte, given the largest of what is written and (rows stand before) the byte that was there.
  static __device__ __forceinline__ int byte_of(float most, int before, int old) {
    const int byte = byte_for(most);
    return before > 0 ? max(byte, old) : byte;
  }

  // The first `before` rows of a block, each `step`-th from i0 on, in units of its new byte.
  __device__ __forceinline__ void again(uint8_t* rows, int i0, int step, int before, int old, int byte,
                                        const Span& span, unsigned* err, const CodesArgs& a) const {
    if (before == 0 || old == byte) return;
    const float s = old == 0 ? 0.f : two_to(max(127 + old - byte, 0));
    const float2 scale = make_float2(s, s);
#pragma unroll 1
    for (int i = i0; i < before; i += step)
#pragma unroll 1
      for (int z = 0; z < 2; ++z) {
        uint8_t* const p = rows + (int64_t)i * a.D + (z ? cb : ca);
        if (!access_ok(p, VEC, span, err)) continue;
        const uint2 was = *reinterpret_cast<const uint2*>(p);
        uint32_t now[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t two = (e < 2 ? was.x : was.y) >> (e & 1) * 16 & 0xffffu;
          const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3);
          now[e] = codes_of<false>(__half22float2(__half2(r)), scale);
        }
        *reinterpret_cast<uint2*>(p) = make_uint2(now[0] | now[1] << 16, now[2] | now[3] << 16);
      }
  }
};

// ---------------------------------------------------------------------------
// Few tokens
// ---------------------------------------------------------------------------
template <typename T, typename TT, bool NEOX, bool MROPE>
__global__ void __launch_bounds__(kThreads, 2) append_few_kernel(Data<T, TT> d, CodesArgs a) {
  using L = Lane<T, TT, NEOX, MROPE>;
  constexpr int VEC = L::VEC, NC = L::NC;
  const L me(a);
  const int lane = threadIdx.x & 31;
  unsigned* const err = d.err;
  const int sets = a.kv_sets + a.q_sets;
  wait_for_prior_grid();
  for (int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); item < a.items;
       item += (int64_t)gridDim.x * kWarps) {
    const int64_t t = div_index(item, sets, a.items32);
    const int set = (int)(item - t * sets);
    const bool is_query = set >= a.kv_sets;
    const int64_t slot = ldg(d.slots + t, a.slot_span, err);
    if (set == 0 && lane == 0) {  // reported once a token
      if (!L::place_of(t, d, a).ok) atomicOr(err, kPositionOutOfRange);
      else if (slot >= a.num_slots) atomicOr(err, kSlotOutOfRange);
    }
    if (is_query) {
      const Place where = L::place_of(t, d, a);
      const int h = (set - a.kv_sets) * a.per_warp + me.g;
      if (me.g >= a.per_warp || h >= a.hq) continue;
      const T* const src = d.q + t * a.q_stride + (int64_t)h * a.D;
      const bool ta = me.ra || a.copy_tail, tb = me.rb || a.copy_tail;
      Vec<T, VEC> x = {}, y = {};
      if (ta) load_vec<true>(x, src + me.ca, a.q_span, err);
      if (tb) load_vec<true>(y, src + me.cb, a.q_span, err);
      if (!where.ok) continue;
      float cf[NC], sf[NC], cg[NC], sg[NC];
      if (me.ra) L::gather(where, me.ia, cf, sf, d, a);
      if (!NEOX && me.rb) L::gather(where, me.ib, cg, sg, d, a);
      me.turn(x, y, cf, sf, cg, sg);
      T* const dst = d.qo + (a.copy_tail ? t * (int64_t)a.hq * a.D : t * a.q_stride) + (int64_t)h * a.D;
      if (ta) store_vec(dst + me.ca, x, a.qo_span, err);
      if (tb) store_vec(dst + me.cb, y, a.qo_span, err);
      continue;
    }
    Vec<T, VEC> x = {}, y = {};
    Place where;
    const int P = a.per_warp, all = a.hk + a.hv;
    auto read = [&](int u, int64_t row) {
      const bool is_v = u >= a.hk;
      const T* const src = is_v ? d.v + row * a.v_stride + (int64_t)(u - a.hk) * a.D
                                : d.k + row * a.k_stride + (int64_t)u * a.D;
      where = L::place_of(row, d, a);
      load_vec<false>(x, src + me.ca, is_v ? a.v_span : a.k_span, err);
      load_vec<false>(y, src + me.cb, is_v ? a.v_span : a.k_span, err);
    };
    where.ok = false;
    if (me.g < P && set * P + me.g < all) read(set * P + me.g, t);  // while the run is looked for
    if (slot < 0 || slot >= a.num_slots) continue;
    const int64_t block = div_index(slot, a.per, a.items32);
    const int first = (int)(slot - block * a.per);
    // the run's tokens before this one and from it on
    const bool joins =
        lane < first && t - 1 - lane >= 0 && ldg(d.slots + t - 1 - lane, a.slot_span, err) == slot - 1 - lane;
    int n = 1;
    for (;;) {
      const int i = n + lane;
      const bool on = first + i < a.per && t + i < a.T && ldg(d.slots + t + i, a.slot_span, err) == slot + i;
      const uint32_t off = ~__ballot_sync(0xffffffffu, on);
      n += off ? __ffs(off) - 1 : 32;
      if (off) break;
    }
    const uint32_t apart = ~__ballot_sync(0xffffffffu, joins);
    const int mine_of = apart ? __ffs(apart) - 1 : 32;  // this token's place in its run
    n += mine_of;
    // A run of one row: the groups have a head each.  A longer one: its first warps share the set's heads, and a warp's
    // groups take a head's rows in turn.
    const bool single = n == 1;
    const int parts = min(n, P), step = single ? 1 : P, g0 = single ? 0 : me.g;
    const int f = first - mine_of;  // rows of the block before the run
    const int64_t t0 = t - mine_of;
    const int64_t page = div_index(block, a.S, a.items32);
    const int part = (int)(block - page * a.S);
    for (int j = mine_of; j < P && set * P + j < all; j += single ? P : parts) {
      const int u = set * P + (single ? me.g : j);
      const bool mine = me.g < P && u < all;
      const bool is_v = u >= a.hk;
      const int h = is_v ? u - a.hk : u, heads = is_v ? a.hv : a.hk;
      uint8_t* const at = (is_v ? d.vs : d.ks) + (page * heads + h) * a.S + part;
      uint8_t* const rows = (is_v ? d.vc : d.kc) + ((page * heads + h) * a.block_size + (int64_t)part * a.per) * a.D;
      const Span& cspan = is_v ? a.vc_span : a.kc_span;
      const Span& zspan = is_v ? a.vs_span : a.ks_span;
      const int old = mine && f > 0 && access_ok(at, 1, zspan, err) ? *at : 0;
      float2 xf[VEC / 2], yf[VEC / 2];
      auto values = [&] {
        float cf[NC], sf[NC], cg[NC], sg[NC];
        if (!is_v && me.ra) L::gather(where, me.ia, cf, sf, d, a);
        if (!NEOX && !is_v && me.rb) L::gather(where, me.ib, cg, sg, d, a);
        me.values(x, y, !is_v, cf, sf, cg, sg, xf, yf);
      };
      float most = 0.f;
      bool any = false;
      for (int i = g0; mine && i < n; i += step) {
        if (!single) read(u, t0 + i);
        if (!where.ok) continue;
        any = true;
        values();
        most = fmaxf(most, L::largest(xf, yf));
      }
      __syncwarp();  // (the byte is read by all before it is written)
      if (single) {
        most = me.over_group(most, a.group);
      } else {
        most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
        any = __any_sync(0xffffffffu, any);
      }
      if (!mine || !any) continue;
      const int byte = L::byte_of(most, f, old);
      me.again(rows, g0, step, f, old, byte, cspan, err, a);
      for (int i = g0; i < n; i += step) {
        if (n > step) read(u, t0 + i), values();  // (else it is there)
        if (where.ok) me.write(rows + (int64_t)(f + i) * a.D, byte, xf, yf, cspan, err);
      }
      if ((single ? me.c : lane) == 0 && access_ok(at, 1, zspan, err)) *at = (uint8_t)byte;
    }
  }
}

// ---------------------------------------------------------------------------
// Many tokens
// ---------------------------------------------------------------------------
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
__device__ __forceinline__ void copy_turns(uint4* a, uint4* b, const TT* cos, const TT* sin, const Span& s,
                                           unsigned* err) {
  if constexpr (sizeof(TT) == 4) {
    copy16(a, cos, s, err);
    copy16(b, sin, s, err);
  } else {
    const unsigned to = (unsigned)__cvta_generic_to_shared(a);
    if (access_ok(cos, 8, s, err))
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(cos) : "memory");
    if (access_ok(sin, 8, s, err))
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to + 8), "l"(sin) : "memory");
  }
}

// T: data; TT: table (T or float).
template <typename T, typename TT, bool NEOX, bool MROPE>
__global__ void __launch_bounds__(kThreads, 2)
    append_many_kernel(Data<T, TT> d, CodesArgs a) {
  using L = Lane<T, TT, NEOX, MROPE>;
  constexpr int VEC = L::VEC, NC = L::NC;
  constexpr int kPieces = Staged<T, TT>::kPieces, kTurns = Staged<T, TT>::kTurns, kRows = Staged<T, TT>::kRows;
  extern __shared__ __align__(16) unsigned char raw[];
  Staged<T, TT>& sm = *reinterpret_cast<Staged<T, TT>*>(raw);
  constexpr int kQueryHeads = query_heads<T, MROPE>();
  const int lane = threadIdx.x & 31;
  const L me(a);
  const int g = me.g, C = a.group, half = a.R / 2;
  const int ca = me.ca, cb = me.cb, ia = me.ia, ib = me.ib;
  const bool ra = me.ra, rb = me.rb;
  const TT* const table = d.table;
  unsigned* const err = d.err;
  const uint64_t policy = l2_evict_first_policy();
  wait_for_prior_grid();

  const int64_t kv_items = a.items - a.q_items;
  // Runs begin at even distances, and windows with none are no work: an odd number of CTAs, neighbours in different ones.
  for (int64_t item = blockIdx.x + (int64_t)gridDim.x * (threadIdx.x >> 5); item < a.items;
       item += (int64_t)gridDim.x * kWarps) {
    if (item >= kv_items) {
      // ---- queries: some heads of one token
      const int64_t t = div_index(item - kv_items, a.q_sets, a.items32);
      const int set = (int)(item - kv_items - t * a.q_sets);
      const int64_t slot = set == 0 ? ldg(d.slots + t, a.slot_span, err) : 0;
      const Place where = L::place_of(t, d, a);
      const bool ta = ra || a.copy_tail, tb = rb || a.copy_tail;
      Vec<T, VEC> x[kQueryHeads] = {}, y[kQueryHeads] = {};
      bool mine[kQueryHeads];
#pragma unroll
      for (int e = 0; e < kQueryHeads; ++e) {
        const int h = (set * kQueryHeads + e) * a.per_warp + g;
        mine[e] = g < a.per_warp && h < a.hq && where.ok;
        const T* src = d.q + t * a.q_stride + (int64_t)h * a.D;
        if (mine[e] && ta) load_vec<true>(x[e], src + ca, a.q_span, err);
        if (mine[e] && tb) load_vec<true>(y[e], src + cb, a.q_span, err);
      }
      if (set == 0 && lane == 0) {  // reported once a token
        if (!where.ok) atomicOr(err, kPositionOutOfRange);
        else if (slot >= a.num_slots) atomicOr(err, kSlotOutOfRange);
      }
      if (!mine[0]) continue;  // (then none is)
      float cf[NC], sf[NC], cg[NC], sg[NC];
      if (ra) L::gather(where, ia, cf, sf, d, a);
      if (!NEOX && rb) L::gather(where, ib, cg, sg, d, a);
#pragma unroll
      for (int e = 0; e < kQueryHeads; ++e) {
        if (!mine[e]) continue;
        me.turn(x[e], y[e], cf, sf, cg, sg);
        const int h = (set * kQueryHeads + e) * a.per_warp + g;
        T* dst = d.qo + (a.copy_tail ? t * (int64_t)a.hq * a.D : t * a.q_stride) + (int64_t)h * a.D;
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
    const int64_t slot = token ? ldg(d.slots + t0 + lane, a.slot_span, err) : -1;
    const int64_t at0 = !MROPE && token ? ldg(d.pos + t0 + lane, a.pos_span, err) : 0;
    int64_t prev = __shfl_up_sync(0xffffffffu, slot, 1);
    if (lane == 0) prev = t0 > 0 ? ldg(d.slots + t0 - 1, a.slot_span, err) : -1;
    const bool there = slot >= 0 && slot < a.num_slots;
    const int64_t block = there ? div_index(slot, a.per, a.items32) : 0;
    const int first = (int)(slot - block * a.per);
    const bool goes_on = there && prev >= 0 && prev + 1 == slot && first > 0;  // the run of the token before
    if (a.hq == 0 && rest == 0 && token && lane < a.window) {  // reported once a token: here without queries
      if (!L::place_of(t0 + lane, d, a).ok) atomicOr(err, kPositionOutOfRange);
      else if (slot >= a.num_slots) atomicOr(err, kSlotOutOfRange);
    }
    const uint32_t on_mask = __ballot_sync(0xffffffffu, goes_on);
    uint32_t begins = __ballot_sync(0xffffffffu, there && !goes_on) & (uint32_t)((1ull << a.window) - 1);
    // position(s) of the token `t0 + i`, i different in every lane; all lanes call it
    auto place_at = [&](int i, bool wanted) {
      if constexpr (MROPE) {
        return wanted ? L::place_of(t0 + i, d, a) : Place{{0, 0, 0, 0}, false};
      } else {
        Place x = {{__shfl_sync(0xffffffffu, at0, i & 31), 0, 0, 0}, false};
        if (wanted && i >= 32) x.p[0] = ldg(d.pos + t0 + i, a.pos_span, err);
        x.ok = wanted && x.p[0] >= 0 && x.p[0] < a.max_seq;
        return x;
      }
    };
    int singles = 0;
    while (begins) {
      // ---- what is done at a time: a run of more than kRows rows, head by head; or up to kRows rows of shorter runs,
      // the heads side by side
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
          const bool on = f0 + j < a.per && t0 + i0 + j < a.T && ldg(d.slots + t0 + i0 + j, a.slot_span, err) == s0 + j;
          const uint32_t off = ~__ballot_sync(0xffffffffu, on);
          n += off ? __ffs(off) - 1 : 32;
          if (off) break;
        }
      }
      const bool single = n <= kRows;
      uint32_t run_of = 0, starts = 0;  // single: the slots' tokens, relative to t0, 8 bits each, and which begin runs
      int count = 0;
      if (single) {
        for (;;) {
          starts |= 1u << count;
          run_of |= (0x03020100u + 0x01010101u * i0) << 8 * count;
          count += n;
          if (count < 4) run_of &= (1u << 8 * count) - 1u;
          begins &= begins - 1;
          if (!begins) break;
          i0 = __ffs(begins) - 1;  // (below 16)
          n = __ffs(~(on_mask >> (i0 + 1)));
          if (count + n > kRows) break;
        }
      } else {
        begins &= begins - 1;
      }
      if (single && singles++ % a.subs != sub) continue;  // the warps that share the set take them in turn
      const int head0 = single ? 0 : sub, heads_here = single ? 1 : min(a.per_warp, all - u0);
      const int by = single ? 1 : a.subs;
      bool turned = false;  // the slots hold the table rows of all the run's rows
      for (int j = head0; j < heads_here; j += by) {
        const int u = u0 + (single ? g : j);
        const bool mine = g < a.per_warp && u < all;
        const bool is_v = u >= a.hk;
        const int h = is_v ? u - a.hk : u, heads = is_v ? a.hv : a.hk;
        const T* const src = (is_v ? d.v : d.k) + (int64_t)h * a.D;
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
          at = (is_v ? d.vs : d.ks) + (page * heads + h) * a.S + part;
          rows = (is_v ? d.vc : d.kc) + ((page * heads + h) * a.block_size + (int64_t)part * a.per) * a.D;
        };
        // Rows under way, in slot e: of the one run the row base + e * step, or token e of the short runs'; with their
        // table rows.
        auto token_of = [&](int base, int e) { return single ? (int)(run_of >> 8 * e & 0xffu) : i0 + base + e * step; };
        uint32_t on = 0;  // which of them are written, a bit a slot
        auto read = [&](int base) {
          on = 0;
#pragma unroll
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
              if (!MROPE && !is_v && !turned) {
                const TT* const row = table + where.p[0] * a.R;
                if constexpr (NEOX) {
                  if (ra)
#pragma unroll
                    for (int z = 0; z < kTurns / 2; ++z) {
                      copy16(&sm.turns[e][z][threadIdx.x], row + ia + z * (16 / sizeof(TT)), a.tab_span, err);
                      copy16(&sm.turns[e][kTurns / 2 + z][threadIdx.x], row + half + ia + z * (16 / sizeof(TT)),
                             a.tab_span, err);
                    }
                } else {
                  auto turn_at = [&](int i) { return &sm.turns[e][i][threadIdx.x]; };
                  if (ra) copy_turns<TT>(turn_at(0), turn_at(kTurns / 4), row + ia, row + half + ia, a.tab_span, err);
                  if (rb)
                    copy_turns<TT>(turn_at(kTurns / 2), turn_at(kTurns * 3 / 4), row + ib, row + half + ib, a.tab_span, err);
                }
              }
            }
            __syncwarp();
          }
          cp_async_commit();
          cp_async_wait<0>();
          turned = turned || (!single && !is_v && n <= kRows * step);
        };
        // Slot e in binary32: rotated twice, for the largest value and for the codes, rather than held.
        float2 xf[VEC / 2], yf[VEC / 2];
        auto values = [&](int base, int e) {
          Vec<T, VEC> x, y;
#pragma unroll
          for (int z = 0; z < kPieces; ++z) {
            reinterpret_cast<uint4*>(x.e)[z] = sm.data[e][z][threadIdx.x];
            reinterpret_cast<uint4*>(y.e)[z] = sm.data[e][kPieces + z][threadIdx.x];
          }
          float cf[NC], sf[NC], cg[NC], sg[NC];
          if (is_v) {
          } else if constexpr (MROPE) {
            const Place where = L::place_of(t0 + token_of(base, e), d, a);
            if (ra) L::gather(where, ia, cf, sf, d, a);
            if (!NEOX && rb) L::gather(where, ib, cg, sg, d, a);
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
          me.values(x, y, !is_v, cf, sf, cg, sg, xf, yf);
        };
        uint8_t *at, *rows;
        int f;
        uint32_t old = 0;  // bytes of the blocks (short runs: of each slot's, 8 bits each) that hold rows before
        for (int e = single ? count - 1 : 0; e >= 0; --e) {
          block_at(token_of(0, e), at, rows, f);
          old = old << 8 | (mine && f > 0 && access_ok(at, 1, zspan, err) ? (uint32_t)*at : 0u);
        }
        __syncwarp();  // (read by all before they are written)
        const int passes = single ? 1 : (n + kRows * step - 1) / (kRows * step);
        float most = 0.f;
        bool any = false;     // some token of the run is written
        uint32_t bytes = 0;   // of the blocks now, short runs: 8 bits a slot
        for (int pass = 0; pass < passes; ++pass) {
          const int base = pass * kRows * step + g0;
          read(base);
          int e0 = 0;  // (short runs: the first slot of this one)
#pragma unroll 1
          for (int e = 0; e < kRows; ++e) {
            if (on >> e & 1) {
              values(base, e);
              most = fmaxf(most, L::largest(xf, yf));
            }
            if (!single) {
              any = any || on != 0;
              continue;
            }
            if (e >= count) break;
            if (e + 1 < count && !(starts >> (e + 1) & 1)) continue;
            most = me.over_group(most, C);
            block_at(token_of(0, e0), at, rows, f);
            if (on >> e0 & ((2u << (e - e0)) - 1u)) {
              const int was = (int)(old >> 8 * e0 & 0xffu), byte = L::byte_of(most, f, was);
              me.again(rows, 0, 1, f, was, byte, cspan, err, a);
              bytes |= (0x01010101u >> 8 * (3 - (e - e0))) * (uint32_t)byte << 8 * e0;
              if (me.c == 0 && access_ok(at, 1, zspan, err)) *at = (uint8_t)byte;
            }
            most = 0.f;
            e0 = e + 1;
            __syncwarp();
          }
        }
        if (!single) {
          most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
          if (!__any_sync(0xffffffffu, any)) continue;
          bytes = (uint32_t)L::byte_of(most, f, (int)old);
          if (mine) me.again(rows, g0, step, f, (int)old, (int)bytes, cspan, err, a);
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
              me.write(rows + (int64_t)(single ? f : f + base + e * step) * a.D, (int)byte, xf, yf, cspan, err);
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
  a.block_size = (int32_t)p.block_size;
  a.S = (int32_t)p.scale_blocks;
  a.per = a.block_size / a.S;
  a.mrope_rows = p.mrope_rows;
  for (int i = 0; i < 4; ++i) a.section_end[i] = i < p.mrope_rows ? p.section_end[i] : a.R / 2;
  a.interleave_end = p.cache_mode == 1 ? 3 * (p.section_end[1] - p.section_end[0]) : 0;
  a.copy_tail = p.query_out != p.query;
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
  Data<T, TT> d;
  d.pos = p.positions;
  d.slots = p.slot_mapping;
  d.q = static_cast<const T*>(p.query);
  d.k = static_cast<const T*>(p.key);
  d.v = static_cast<const T*>(p.value);
  d.table = static_cast<const TT*>(p.table);
  d.qo = static_cast<T*>(p.query_out);
  d.kc = static_cast<uint8_t*>(p.k_cache);
  d.vc = static_cast<uint8_t*>(p.v_cache);
  d.ks = p.k_scale;
  d.vs = p.v_scale;
  cudaError_t er = device_error_address(&d.err);
  if (er != cudaSuccess) return er;
  if (p.T <= kFewTokens) {
    a.q_sets = (a.hq + a.per_warp - 1) / a.per_warp;
    a.items = p.T * (a.kv_sets + a.q_sets);
    a.items32 = a.items <= 0xffffffffLL && a.num_slots <= 0xffffffffLL;
    const int64_t grid = (a.items + kWarps - 1) / kWarps;
    return launch_overlapped(append_few_kernel<T, TT, NEOX, MROPE>, (unsigned)grid, kThreads, stream, d, a);
  }
  constexpr int kQueryHeads = query_heads<T, MROPE>();
  a.q_sets = (a.hq + kQueryHeads * a.per_warp - 1) / (kQueryHeads * a.per_warp);
  // One token to a window, so that all SMs are busy, up to 16 where there are many.  Two warps share a set's heads (16384
  // tokens, 32 q, 8 k and 8 v heads of 128: 83 us; one 87, four 89), four where a block's rows do not fit their slots (scale
  // blocks of 64: 120 us, 136 by two).
  constexpr int kRows = Staged<T, TT>::kRows;
  a.window = 1;
  a.subs = std::min(a.per_warp, a.per > kRows * a.per_warp ? 4 : 2);
  const int64_t enough = (int64_t)sm_count() * 16;
  while (a.window < 16 && p.T / (2 * a.window) * a.kv_sets * a.subs >= enough) a.window *= 2;
  a.q_items = p.T * a.q_sets;
  a.items = a.q_items + (p.T + a.window - 1) / a.window * a.kv_sets * a.subs;
  a.items32 = a.items <= 0xffffffffLL && a.num_slots <= 0xffffffffLL;
  auto kernel = append_many_kernel<T, TT, NEOX, MROPE>;
  const size_t smem = sizeof(Staged<T, TT>);
  er = opt_in_shared(reinterpret_cast<const void*>(kernel), smem);
  if (er != cudaSuccess) return er;
  const int64_t resident = (int64_t)sm_count() * resident_blocks(reinterpret_cast<const void*>(kernel), kThreads, smem);
  const int64_t grid = std::min((a.items + kWarps - 1) / kWarps, resident);
  return launch_overlapped_smem(kernel, (unsigned)(grid - (grid > 1 && grid % 2 == 0)), kThreads, smem, stream, d, a);
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
