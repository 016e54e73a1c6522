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
// The tokens of a scale block stand one after the other in the batch: a run.  A group of D / 16 threads takes
// a run of one head: it looks through the run's values for the largest, then reads them again (from L1 or L2)
// and writes their codes.  Queries go by groups of heads of a token.
#include <cuda_fp8.h>

#include <algorithm>

#include "rope_device.cuh"
#include "serving.h"

namespace rope {
namespace {

constexpr int kThreads = 256;
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

// Codes of two values in units of 2^(byte - 127); what is not finite is NaN, the format holding no infinity.
__device__ __forceinline__ uint32_t codes_of(float x, float y, float f) {
  x = fabsf(x) <= FLT_MAX ? x * f : NAN;
  y = fabsf(y) <= FLT_MAX ? y * f : NAN;
  return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}

// T: data; TT: table (T or float).
template <typename T, typename TT, bool NEOX, bool MROPE>
__global__ void __launch_bounds__(kThreads)
    append_codes_kernel(const int64_t* __restrict__ pos, const int64_t* __restrict__ slots, const T* q,
                        const T* __restrict__ k, const T* __restrict__ v, const TT* __restrict__ table, T* qo,
                        uint8_t* __restrict__ kc, uint8_t* __restrict__ vc, uint8_t* __restrict__ ks,
                        uint8_t* __restrict__ vs, unsigned int* __restrict__ err, CodesArgs a) {
  constexpr int VEC = 8;                   // columns of a chunk; a thread owns two chunks of a head
  constexpr int NC = NEOX ? VEC : VEC / 2;  // cos (and sin) values of one chunk
  constexpr bool kExact = sizeof(T) == 2 && sizeof(TT) == 2;
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
  // both chunks of a head, rotated, in binary32
  auto turn = [&](const Place& where, const Vec<T, VEC>& x, const Vec<T, VEC>& y, float (&xf)[VEC], float (&yf)[VEC]) {
    float cf[NC], sf[NC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      xf[e] = widen(x.e[e]);
      yf[e] = widen(y.e[e]);
    }
    if constexpr (NEOX) {
      if (ra) {
        gather(where, ia, cf, sf);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float a1 = xf[e], a2 = yf[e];
          xf[e] = rotate_one<kExact>(a1, cf[e], a2, sf[e]);
          yf[e] = rotate_one<kExact>(a2, cf[e], -a1, sf[e]);
        }
      }
    } else {
      auto one = [&](float (&z)[VEC]) {
#pragma unroll
        for (int e = 0; e < NC; ++e) {
          const float a1 = z[2 * e], a2 = z[2 * e + 1];
          z[2 * e] = rotate_one<kExact>(a1, cf[e], a2, sf[e]);
          z[2 * e + 1] = rotate_one<kExact>(a2, cf[e], -a1, sf[e]);
        }
      };
      if (ra) {
        gather(where, ia, cf, sf);
        one(xf);
      }
      if (rb) {
        gather(where, ib, cf, sf);
        one(yf);
      }
    }
  };

  const int64_t kv_items = a.items - a.q_items;
  for (int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); item < a.items;
       item += (int64_t)gridDim.x * (kThreads / 32)) {
    if (item >= kv_items) {
      // ---- queries: a set of heads of one token
      const int64_t t = div_index(item - kv_items, a.q_sets, a.items32);
      const int set = (int)(item - kv_items - t * a.q_sets);
      const int h = set * a.per_warp + g;
      const Place where = place_of(t);
      if (set == 0 && lane == 0) {  // reported once a token
        const int64_t slot = ldg(slots + t, a.slot_span, err);
        if (!where.ok) atomicOr(err, kPositionOutOfRange);
        else if (slot >= a.num_slots) atomicOr(err, kSlotOutOfRange);
      }
      if (g >= a.per_warp || h >= a.hq || !where.ok) continue;
      const T* src = q + t * a.q_stride + (int64_t)h * a.D;
      T* dst = qo + (a.copy_tail ? t * (int64_t)a.hq * a.D : t * a.q_stride) + (int64_t)h * a.D;
      const bool ta = ra || a.copy_tail, tb = rb || a.copy_tail;
      Vec<T, VEC> x = {}, y = {};
      if (ta) load_vec<true>(x, src + ca, a.q_span, err);
      if (tb) load_vec<true>(y, src + cb, a.q_span, err);
      float xf[VEC], yf[VEC];
      turn(where, x, y, xf, yf);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        x.e[e] = narrow<T>(xf[e]);
        y.e[e] = narrow<T>(yf[e]);
      }
      if (ta) store_vec(dst + ca, x, a.qo_span, err);
      if (tb) store_vec(dst + cb, y, a.qo_span, err);
      continue;
    }
    // ---- keys and values: the runs that begin in a window of tokens, a set of heads
    const int64_t w = div_index(item, a.kv_sets, a.items32);
    const int set = (int)(item - w * a.kv_sets);
    const int u = set * a.per_warp + g;
    const bool mine = g < a.per_warp && u < a.hk + a.hv;
    const bool is_v = u >= a.hk;
    const int h = is_v ? u - a.hk : u, heads = is_v ? a.hv : a.hk;
    const T* const src0 = is_v ? v : k;
    const int64_t stride = is_v ? a.v_stride : a.k_stride;
    const Span& sspan = is_v ? a.v_span : a.k_span;
    uint8_t* const codes = is_v ? vc : kc;
    uint8_t* const scales = is_v ? vs : ks;
    const Span& cspan = is_v ? a.vc_span : a.kc_span;
    const Span& zspan = is_v ? a.vs_span : a.ks_span;
    const int64_t end = min(w * a.window + a.window, a.T);
    int64_t before = w * a.window > 0 ? ldg(slots + w * a.window - 1, a.slot_span, err) : -1;
    for (int64_t t = w * a.window; t < end; ++t) {
      const int64_t slot = ldg(slots + t, a.slot_span, err);
      const bool there = slot >= 0 && slot < a.num_slots;
      if (a.hq == 0 && set == 0 && lane == 0) {  // reported once a token: here without queries
        if (!place_of(t).ok) atomicOr(err, kPositionOutOfRange);
        else if (slot >= a.num_slots) atomicOr(err, kSlotOutOfRange);
      }
      const int64_t block = there ? div_index(slot, a.per, a.items32) : 0;
      const int first = there ? (int)(slot - block * a.per) : 0;
      const bool begins = there && !(before >= 0 && before + 1 == slot && first > 0);
      before = slot;
      if (!begins) continue;
      // the run: tokens t, t + 1, ... in the rows first, first + 1, ... of the block
      int n = 1;
      while (first + n < a.per && t + n < a.T && ldg(slots + t + n, a.slot_span, err) == slot + n) ++n;
      const int64_t page = div_index(block, a.S, a.items32);
      const int part = (int)(block - page * a.S);
      uint8_t* const at = scales + (page * heads + h) * a.S + part;
      uint8_t* const rows = codes + ((page * heads + h) * a.block_size + (int64_t)part * a.per) * a.D;
      Vec<T, VEC> x = {}, y = {};
      float xf[VEC], yf[VEC];
      auto read = [&](int i) {
        const Place where = place_of(t + i);
        if (!where.ok) return false;
        const T* const src = src0 + (t + i) * stride + (int64_t)h * a.D;
        load_vec<false>(x, src + ca, sspan, err);
        load_vec<false>(y, src + cb, sspan, err);
        if (is_v) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            xf[e] = widen(x.e[e]);
            yf[e] = widen(y.e[e]);
          }
        } else {
          turn(where, x, y, xf, yf);
        }
        return true;
      };
      const int old = mine && first > 0 && access_ok(at, 1, zspan, err) ? *at : 0;
      __syncwarp();  // read by all before it is written
      float most = 0.f;
      bool any = false;  // some token of the run is written
      if (mine)
        for (int i = 0; i < n; ++i)
          if (read(i)) {
            any = true;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              if (fabsf(xf[e]) <= FLT_MAX) most = fmaxf(most, fabsf(xf[e]));
              if (fabsf(yf[e]) <= FLT_MAX) most = fmaxf(most, fabsf(yf[e]));
            }
          }
      // over the group: the windows of lanes that a value has seen double, round the group
      for (int d = 1; d < C; d *= 2) {
        int from = c + d;
        if (from >= C) from -= C;
        most = fmaxf(most, __shfl_sync(0xffffffffu, most, min(g * C + from, 31)));
      }
      if (!mine || !any) continue;
      int byte = byte_for(most);
      if (first > 0) {
        if (old < byte) {
          const float f = old == 0 ? 0.f : power_of(max(127 + old - byte, 0));
          for (int i = 0; i < first; ++i)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              uint8_t* const p = rows + (int64_t)i * a.D + (z ? cb : ca);
              if (!access_ok(p, VEC, cspan, err)) continue;
              uint2 was = *reinterpret_cast<const uint2*>(p);
              uint32_t now[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((e < 2 ? was.x : was.y) >> (e & 1) * 16 & 0xffffu, __NV_E4M3);
                const float2 d = __half22float2(__half2(r));
                now[e] = codes_of(d.x, d.y, f);
              }
              *reinterpret_cast<uint2*>(p) = make_uint2(now[0] | now[1] << 16, now[2] | now[3] << 16);
            }
        } else {
          byte = old;
        }
      }
      const float f = byte == 255 ? NAN : power_of(254 - byte);
      for (int i = 0; i < n; ++i) {
        if (!read(i)) continue;
        uint8_t* const p = rows + (int64_t)(first + i) * a.D;
        uint32_t z[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          z[e] = codes_of(xf[2 * e], xf[2 * e + 1], f);
          z[4 + e] = codes_of(yf[2 * e], yf[2 * e + 1], f);
        }
        if (access_ok(p + ca, VEC, cspan, err))
          *reinterpret_cast<uint2*>(p + ca) = make_uint2(z[0] | z[1] << 16, z[2] | z[3] << 16);
        if (access_ok(p + cb, VEC, cspan, err))
          *reinterpret_cast<uint2*>(p + cb) = make_uint2(z[4] | z[5] << 16, z[6] | z[7] << 16);
      }
      if (c == 0 && access_ok(at, 1, zspan, err)) *at = (uint8_t)byte;
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
  a.q_sets = (a.hq + a.per_warp - 1) / a.per_warp;
  a.block_size = (int32_t)p.block_size;
  a.S = (int32_t)p.scale_blocks;
  a.per = a.block_size / a.S;
  a.window = 1;
  a.q_items = p.T * a.q_sets;
  a.items = a.q_items + (p.T + a.window - 1) / a.window * a.kv_sets;
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
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>((a.items + warps - 1) / warps, 1 << 30));
  unsigned int* err = nullptr;
  const cudaError_t er = device_error_address(&err);
  if (er != cudaSuccess) return er;
  return launch_overlapped(kernel, (unsigned)grid, kThreads, stream, p.positions, p.slot_mapping,
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
