// RoPE of query and key on the way to the query output and to a paged KV cache.
//
// Per token t: cos and sin from the table row of its position(s); query heads rotated to
// query_out, key heads rotated to k_cache[slot/BS, h, slot%BS, :], value heads copied to
// v_cache[slot/BS, h, slot%BS, :].  NeoX pairs column i with i + R/2, GPT-J 2i with 2i + 1,
// i < R/2; columns [R, D) pass through.
//
// Bound by memory: every head row is read and written once and a token's table row is
// shared by its heads, about 0.15 floating operations a byte.  So the kernel is a copy with
// arithmetic on the way:
//  * an item is U heads of one kind (q, k or v) of one token, a row group of C = D / (2 VEC)
//    threads works on it, each owning two 16-byte chunks of every head.  For NeoX the two
//    are a rotated pair (or two chunks of the tail), otherwise chunks c and c + C.
//  * all loads of an item leave before its arithmetic; items are handed out in token order
//    to a persistent grid.  U = 2 and 256 threads: more row groups under way than with U = 4
//    at the same bytes (67 us and 66 us below), fewer look-ups a byte than with U = 1 (76, 67).
//
// 16384 tokens of 32 q, 8 k and 8 v heads of 128, bf16 with a binary32 table: 64.5 us, 6.4 TB/s,
// 0.94 of the measured copy bandwidth; 8192 tokens of 16 heads of 256, 64 columns interleaved,
// f16: 62.7 us, 0.95; 64 tokens: 2.8 us.
#include <algorithm>

#include "rope_device.cuh"
#include "serving.h"

namespace rope {
namespace {

constexpr int kThreads = 256;
constexpr unsigned kPositionOutOfRange = 1u;
constexpr unsigned kSlotOutOfRange = 2u;

struct AppendArgs {
  int64_t T, max_seq, num_slots, items;
  int64_t q_stride, k_stride, v_stride;
  int32_t hq, hk, hv;
  int32_t iq, ik, per_token;  // q items, k items and all items of a token
  int32_t D, R;
  int32_t group;  // C, threads per row group
  int32_t block_size;
  int32_t mrope_rows;
  int32_t section_end[4];
  int32_t interleave_end;  // > 0: the interleaved splice below this index
  bool copy_tail;          // q is written to another place, so its columns [R, D) too
  bool items32;
  Span pos_span, slot_span, q_span, k_span, v_span, tab_span, qo_span, kc_span, vc_span;
};

// Row (of the position rows) that cos/sin index i is taken from.
__device__ __forceinline__ int row_of(int i, const AppendArgs& a) {
  if (a.interleave_end > 0) return i < a.interleave_end ? i % 3 : 0;
  return (i >= a.section_end[0]) + (i >= a.section_end[1]) + (i >= a.section_end[2]);
}

// a*b - c*d rounded so that the result is within one rounding of exact: a single FMA where
// the product c*d is exact in binary32 (16-bit factors), else the compensated form.
template <bool EXACT>
__device__ __forceinline__ float rotate_one(float a, float b, float c, float d) {
  if constexpr (EXACT) return __fmaf_rn(a, b, -__fmul_rn(c, d));
  return diff_of_products(a, b, c, d);
}

// T: data; TT: table (T or float); U: heads per item.
template <typename T, typename TT, bool NEOX, bool MROPE, int U>
__global__ void __launch_bounds__(kThreads)
    append_kernel(const int64_t* __restrict__ pos, const int64_t* __restrict__ slots, const T* q,
                  const T* __restrict__ k, const T* __restrict__ v, const TT* __restrict__ table, T* qo,
                  T* __restrict__ kc, T* __restrict__ vc, unsigned int* __restrict__ err, AppendArgs a) {
  constexpr int VEC = 16 / sizeof(T);
  constexpr int NC = NEOX ? VEC : VEC / 2;  // cos (and sin) values of one chunk
  constexpr bool kExact = sizeof(T) == 2 && sizeof(TT) == 2;
  const int C = a.group;
  const int P = kThreads / C;
  const int g = threadIdx.x / C;
  if (g >= P) return;
  const int c = threadIdx.x - g * C;
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

  for (int64_t item = (int64_t)blockIdx.x * P + g; item < a.items; item += (int64_t)gridDim.x * P) {
    const int64_t t = div_index(item, a.per_token, a.items32);
    const int r = (int)(item - t * a.per_token);
    const int kind = r < a.iq ? 0 : r < a.iq + a.ik ? 1 : 2;
    const int h0 = (kind == 0 ? r : kind == 1 ? r - a.iq : r - a.iq - a.ik) * U;
    const int heads = kind == 0 ? a.hq : kind == 1 ? a.hk : a.hv;
    const int n = min(U, heads - h0);
    const T* src = (kind == 0   ? q + t * a.q_stride
                    : kind == 1 ? k + t * a.k_stride
                                : v + t * a.v_stride) +
                   (int64_t)h0 * a.D;
    const Span& sspan = kind == 0 ? a.q_span : kind == 1 ? a.k_span : a.v_span;
    const bool tail = kind != 0 || a.copy_tail;  // columns that do not rotate are written too
    const bool ta = ra || tail, tb = rb || tail;
    const int64_t slot = ldg(slots + t, a.slot_span, err);
    int64_t p[4] = {0, 0, 0, 0};
    p[0] = ldg(pos + t, a.pos_span, err);
    if constexpr (MROPE) {
      p[1] = ldg(pos + a.T + t, a.pos_span, err);
      p[2] = ldg(pos + 2 * a.T + t, a.pos_span, err);
      if (a.mrope_rows > 3) p[3] = ldg(pos + 3 * a.T + t, a.pos_span, err);
    }
    Vec<T, VEC> x[U], y[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < n) {
        if (ta) load_vec<true>(x[u], src + (int64_t)u * a.D + ca, sspan, err);
        if (tb) load_vec<true>(y[u], src + (int64_t)u * a.D + cb, sspan, err);
      }
    bool ok = true;
#pragma unroll
    for (int j = 0; j < (MROPE ? 4 : 1); ++j) ok = ok && p[j] >= 0 && p[j] < a.max_seq;
    const bool in_cache = slot >= 0 && slot < a.num_slots;
    if (c == 0 && r == 0) {  // reported once per token
      if (!ok) atomicOr(err, kPositionOutOfRange);
      else if (slot >= a.num_slots) atomicOr(err, kSlotOutOfRange);
    }
    if (!ok || (kind != 0 && !in_cache)) continue;
    T* dst;
    int64_t step = a.D;
    if (kind == 0) {
      dst = qo + ((a.copy_tail ? t * (int64_t)a.hq * a.D : t * a.q_stride) + (int64_t)h0 * a.D);
    } else {
      const int64_t blk = div_index(slot, a.block_size, a.items32), at = slot - blk * a.block_size;
      dst = (kind == 1 ? kc : vc) + ((blk * heads + h0) * a.block_size + at) * a.D;
      step = (int64_t)a.block_size * a.D;
    }
    const Span& dspan = kind == 0 ? a.qo_span : kind == 1 ? a.kc_span : a.vc_span;
    if (kind != 2) {
      auto gather = [&](int i0, float (&cf)[NC], float (&sf)[NC]) {
        const int k0 = MROPE ? row_of(i0, a) : 0;
        bool one = true;
        if constexpr (MROPE) one = a.interleave_end > 0 ? i0 >= a.interleave_end : k0 == row_of(i0 + NC - 1, a);
        auto row = [&](int s) { return table + (s == 0 ? p[0] : s == 1 ? p[1] : s == 2 ? p[2] : p[3]) * a.R; };
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
      float cf[NC], sf[NC];
      if constexpr (NEOX) {
        if (ra) {
          gather(ia, cf, sf);
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (u < n) {
#pragma unroll
              for (int e = 0; e < VEC; ++e) {
                const float a1 = widen(x[u].e[e]), a2 = widen(y[u].e[e]);
                x[u].e[e] = narrow<T>(rotate_one<kExact>(a1, cf[e], a2, sf[e]));
                y[u].e[e] = narrow<T>(rotate_one<kExact>(a2, cf[e], -a1, sf[e]));
              }
            }
        }
      } else {
        auto turn = [&](Vec<T, VEC>(&z)[U]) {
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (u < n) {
#pragma unroll
              for (int e = 0; e < NC; ++e) {
                const float a1 = widen(z[u].e[2 * e]), a2 = widen(z[u].e[2 * e + 1]);
                z[u].e[2 * e] = narrow<T>(rotate_one<kExact>(a1, cf[e], a2, sf[e]));
                z[u].e[2 * e + 1] = narrow<T>(rotate_one<kExact>(a2, cf[e], -a1, sf[e]));
              }
            }
        };
        if (ra) {
          gather(ia, cf, sf);
          turn(x);
        }
        if (rb) {
          gather(ib, cf, sf);
          turn(y);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < n) {
        if (ta) store_vec(dst + u * step + ca, x[u], dspan, err);
        if (tb) store_vec(dst + u * step + cb, y[u], dspan, err);
      }
  }
}

template <typename T, typename TT, bool NEOX, bool MROPE, int U>
cudaError_t launch_u(const AppendProblem& p, cudaStream_t stream) {
  constexpr int VEC = 16 / sizeof(T);
  AppendArgs a;
  a.T = p.T;
  a.max_seq = p.max_seq;
  a.num_slots = p.num_blocks * p.block_size;
  a.q_stride = p.q_stride;
  a.k_stride = p.k_stride;
  a.v_stride = p.v_stride;
  a.hq = p.query ? (int32_t)p.hq : 0;
  a.hk = (int32_t)p.hk;
  a.hv = (int32_t)p.hv;
  a.iq = (a.hq + U - 1) / U;
  a.ik = (a.hk + U - 1) / U;
  a.per_token = a.iq + a.ik + (a.hv + U - 1) / U;
  a.items = p.T * a.per_token;
  a.D = (int32_t)p.head_size;
  a.R = (int32_t)p.rotary_dim;
  a.group = a.D / (2 * VEC);
  a.block_size = (int32_t)p.block_size;
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
  a.kc_span = make_span(p.k_cache, a.num_slots * p.hk * D * e);
  a.vc_span = make_span(p.v_cache, a.num_slots * p.hv * D * e);
  auto kernel = append_kernel<T, TT, NEOX, MROPE, U>;
  const int64_t groups = kThreads / a.group;
  const int64_t resident = (int64_t)sm_count() * resident_blocks(reinterpret_cast<const void*>(kernel), kThreads);
  const int64_t grid = std::max<int64_t>(1, std::min((a.items + groups - 1) / groups, resident));
  unsigned int* err = nullptr;
  const cudaError_t er = device_error_address(&err);
  if (er != cudaSuccess) return er;
  return launch_overlapped(kernel, (unsigned)grid, kThreads, stream, p.positions, p.slot_mapping,
                           static_cast<const T*>(p.query), static_cast<const T*>(p.key),
                           static_cast<const T*>(p.value), static_cast<const TT*>(p.table),
                           static_cast<T*>(p.query_out), static_cast<T*>(p.k_cache), static_cast<T*>(p.v_cache), err,
                           a);
}

template <typename T, typename TT>
cudaError_t launch_typed(const AppendProblem& p, cudaStream_t stream) {
  constexpr int U = 2;
  if (p.is_neox)
    return p.mrope_rows ? launch_u<T, TT, true, true, U>(p, stream) : launch_u<T, TT, true, false, U>(p, stream);
  return p.mrope_rows ? launch_u<T, TT, false, true, U>(p, stream) : launch_u<T, TT, false, false, U>(p, stream);
}

}  // namespace

cudaError_t launch_append(const AppendProblem& p, cudaStream_t stream) {
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
