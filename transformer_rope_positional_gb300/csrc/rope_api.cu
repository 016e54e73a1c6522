// C ABI of the RoPE library: argument checks, dispatch, status strings, and the host
// arithmetic of scaled frequencies.
//
// The checks follow the constraint and error-code lists of the two operator
// pages ("CANN ops-transformer 的 aclnnInplacePartialRotaryMul 算子…", sections
// 返回值与错误码 and 约束说明; "CANN ops-transformer 旋转位置编码算子
// RopeWithSinCosCache 深度解析…", sections 约束说明 and 入参校验逻辑).  Every check
// runs on the host before anything is enqueued, and no check touches the GPU,
// so a rejected call has no side effect at all.
#include <cmath>
#include <initializer_list>

#include "rope_gb300.h"
#include "rope_launch.h"
#include "serving/serving.h"


namespace {

using rope::kBF16;
using rope::kF16;
using rope::kF32;
using rope::kI64;

bool is_float(int32_t dt) { return dt == kF32 || dt == kF16 || dt == kBF16; }

// Largest element count accepted: the byte size of any tensor (8 bytes per
// element at most) and every element offset the kernels form stay in int64.
constexpr int64_t kMaxElements = INT64_MAX / 8;

// Product of the dims of a tensor that passed shape_ok().
int64_t numel(const rope_tensor_t* t) {
  int64_t n = 1;
  for (int i = 0; i < t->ndim; ++i) n *= t->shape[i];
  return n;
}

// 1 to 4 non-negative dims whose product (taken in order) stays within
// kMaxElements; a shape whose product overflows is rejected, not wrapped.
bool shape_ok(const rope_tensor_t* t) {
  if (t->ndim < 1 || t->ndim > 4) return false;
  int64_t n = 1;
  for (int i = 0; i < t->ndim; ++i) {
    if (t->shape[i] < 0) return false;
    if (__builtin_mul_overflow(n, t->shape[i], &n) || n > kMaxElements) return false;
  }
  return true;
}

// Elements spanned by `rows` rows of `width` elements, `stride` apart:
// (rows - 1) * stride + width, or -1 when that leaves kMaxElements.
int64_t strided_extent(int64_t rows, int64_t stride, int64_t width) {
  int64_t n = 0;
  if (rows <= 0) return 0;
  if (__builtin_mul_overflow(rows - 1, stride, &n) || __builtin_add_overflow(n, width, &n) || n > kMaxElements)
    return -1;
  return n;
}

bool aligned(const void* p, uintptr_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

int64_t elem_size(int32_t dt) { return dt == kF32 ? 4 : dt == kI64 ? 8 : 2; }

// Whether two sets of `rows` rows share a byte: set a starts at byte address
// a, its rows are aw bytes wide and as bytes apart (likewise b).  Sets whose
// byte ranges meet are treated as overlapping unless both have one stride s
// and their columns are disjoint modulo s (e.g. the q and k column ranges of
// one fused QKV buffer).  Empty sets overlap nothing.
bool rows_overlap(uintptr_t a, int64_t as, int64_t aw, uintptr_t b, int64_t bs, int64_t bw, int64_t rows) {
  if (rows <= 0 || aw <= 0 || bw <= 0) return false;
  const uintptr_t a_end = a + (uintptr_t)((rows - 1) * as + aw), b_end = b + (uintptr_t)((rows - 1) * bs + bw);
  if (a_end <= b || b_end <= a) return false;
  if (rows == 1 || as != bs || aw > as || bw > bs) return true;
  // a covers [0, aw) of every period of as bytes, b covers [r, r + bw)
  const int64_t d = (int64_t)(b - a);
  const int64_t r = ((d % as) + as) % as;
  return r < aw || r + bw > as;
}

// Whether the byte ranges [a, a + an) and [b, b + bn) share a byte.
bool ranges_overlap(uintptr_t a, int64_t an, uintptr_t b, int64_t bn) {
  return an > 0 && bn > 0 && a < b + (uintptr_t)bn && b < a + (uintptr_t)an;
}

// Whether two contiguous tensors (the byte ranges of their elements) overlap.
bool tensors_overlap(const rope_tensor_t* x, const rope_tensor_t* y) {
  return ranges_overlap(reinterpret_cast<uintptr_t>(x->data), numel(x) * elem_size(x->dtype),
                        reinterpret_cast<uintptr_t>(y->data), numel(y) * elem_size(y->dtype));
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? ROPE_OK : ROPE_ERR_CUDA; }

// Checks shared by the forward and backward in-place calls, then the launch.
int inplace_call(const rope_tensor_t* x, const rope_tensor_t* cos, const rope_tensor_t* sin, int64_t rotary_mode,
                 int64_t start, int64_t end, bool backward, void* stream) {
  if (!x || !cos || !sin) return ROPE_ERR_PARAM_NULLPTR;
  // dtypes: x in {F32, F16, BF16}; cos == sin; cos == x, or F32 with a half x
  if (!is_float(x->dtype) || !is_float(cos->dtype) || cos->dtype != sin->dtype) return ROPE_ERR_PARAM_INVALID;
  if (cos->dtype != x->dtype && !(cos->dtype == kF32 && x->dtype != kF32)) return ROPE_ERR_PARAM_INVALID;
  // modes: 1 interleave, 0 half; the other enum values have no formula
  if (rotary_mode != 1 && rotary_mode != 0) return ROPE_ERR_PARAM_INVALID;
  if (x->ndim != 4 || cos->ndim != 4 || sin->ndim != 4) return ROPE_ERR_PARAM_INVALID;
  if (!shape_ok(x) || !shape_ok(cos) || !shape_ok(sin)) return ROPE_ERR_PARAM_INVALID;
  for (int i = 0; i < 4; ++i)
    if (cos->shape[i] != sin->shape[i]) return ROPE_ERR_PARAM_INVALID;
  const int64_t D = x->shape[3];
  if (D > 1024 || D % 2) return ROPE_ERR_PARAM_INVALID;
  if (start < 0 || end < 0 || end > D || start > end) return ROPE_ERR_PARAM_INVALID;
  if (start == 0 && end == 0) end = D;  // no slice: the whole D axis
  const int64_t L = end - start;
  if (L % 2) return ROPE_ERR_PARAM_INVALID;
  if (L == 0) return ROPE_OK;  // empty slice: no-op, nothing enqueued
  if (cos->shape[3] != L) return ROPE_ERR_PARAM_INVALID;
  for (int i = 0; i < 3; ++i)
    if (cos->shape[i] != 1 && cos->shape[i] != x->shape[i]) return ROPE_ERR_PARAM_INVALID;
  if (numel(x) == 0) return ROPE_OK;
  if (!x->data || !cos->data || !sin->data) return ROPE_ERR_PARAM_NULLPTR;
  const uintptr_t xe = x->dtype == kF32 ? 4 : 2, ce = cos->dtype == kF32 ? 4 : 2;
  if (!aligned(x->data, xe) || !aligned(cos->data, ce) || !aligned(sin->data, ce)) return ROPE_ERR_PARAM_INVALID;
  // x is rewritten while cos/sin are read: they must not share memory
  if (tensors_overlap(x, cos) || tensors_overlap(x, sin)) return ROPE_ERR_PARAM_INVALID;

  rope::InplaceProblem p;
  p.mode = (int32_t)rotary_mode;
  p.backward = backward;
  p.x = x->data;
  p.cos = cos->data;
  p.sin = sin->data;
  p.x_dtype = x->dtype;
  p.cs_dtype = cos->dtype;
  p.B = x->shape[0];
  p.S = x->shape[1];
  p.N = x->shape[2];
  p.D = D;
  p.start = start;
  p.L = L;
  const int64_t cB = cos->shape[0], cS = cos->shape[1], cN = cos->shape[2];
  p.cs_n = cN == 1 ? 0 : 1;
  p.cs_s = cS == 1 ? 0 : cN;
  p.cs_b = cB == 1 ? 0 : cS * cN;
  p.cs_rows = cB * cS * cN;
  return cuda_status(rope::launch_inplace(p, static_cast<cudaStream_t>(stream)));
}

// Checks shared by the V1 and V2 cache calls, then the launch.
int cache_call(const rope_tensor_t* positions, const rope_tensor_t* query, const rope_tensor_t* key,
               const rope_tensor_t* cos_sin_cache, int64_t head_size, int64_t rotary_dim, int32_t is_neox,
               const int64_t* mrope_section, int64_t mrope_section_len, int32_t cache_mode, int64_t q_row_stride,
               int64_t k_row_stride, const rope_tensor_t* query_out, const rope_tensor_t* key_out, void* stream) {
  if (!positions || !query || !key || !cos_sin_cache) return ROPE_ERR_PARAM_NULLPTR;
  // dtypes: positions int64; query, key and cache the same floating type
  if (positions->dtype != kI64 || !is_float(query->dtype)) return ROPE_ERR_PARAM_INVALID;
  if (key->dtype != query->dtype || cos_sin_cache->dtype != query->dtype) return ROPE_ERR_PARAM_INVALID;
  // shapes: query, key, cache 2-D and non-empty; same token count
  if (query->ndim != 2 || key->ndim != 2 || cos_sin_cache->ndim != 2) return ROPE_ERR_PARAM_INVALID;
  if (!shape_ok(query) || !shape_ok(key) || !shape_ok(cos_sin_cache) || !shape_ok(positions))
    return ROPE_ERR_PARAM_INVALID;
  if (numel(query) == 0 || numel(key) == 0 || numel(cos_sin_cache) == 0) return ROPE_ERR_PARAM_INVALID;
  const int64_t T = query->shape[0];
  if (key->shape[0] != T) return ROPE_ERR_PARAM_INVALID;
  // head size and rotary dim: 64-byte multiples; R == cache width <= head size
  const int64_t mult = query->dtype == kF32 ? 16 : 32;
  if (head_size <= 0 || head_size % mult) return ROPE_ERR_PARAM_INVALID;
  if (query->shape[1] % head_size || key->shape[1] % head_size) return ROPE_ERR_PARAM_INVALID;
  if (rotary_dim != cos_sin_cache->shape[1]) return ROPE_ERR_PARAM_INVALID;
  if (rotary_dim <= 0 || rotary_dim % mult || rotary_dim > head_size) return ROPE_ERR_PARAM_INVALID;
  // mode and positions shape
  const bool mrope = mrope_section != nullptr && mrope_section_len > 0 && mrope_section[0] > 0;
  if (mrope_section != nullptr && mrope_section_len != 3 && mrope_section_len != 4) return ROPE_ERR_PARAM_INVALID;
  int32_t section_end[4] = {0, 0, 0, 0};
  if (mrope_section != nullptr) {
    int64_t sum = 0;
    for (int64_t i = 0; i < mrope_section_len; ++i) {
      if (mrope_section[i] < 0) return ROPE_ERR_PARAM_INVALID;
      sum += mrope_section[i];
      section_end[i] = (int32_t)sum;
    }
    if (mrope && 2 * sum != rotary_dim) return ROPE_ERR_PARAM_INVALID;
  }
  if (mrope) {
    if (positions->ndim != 2 || positions->shape[0] != mrope_section_len || positions->shape[1] != T)
      return ROPE_ERR_PARAM_INVALID;
  } else {
    if (positions->ndim != 1 || positions->shape[0] != T) return ROPE_ERR_PARAM_INVALID;
  }
  // V2: interleaved splice only for three-section mrope
  if (cache_mode != 0 && cache_mode != 1) return ROPE_ERR_PARAM_INVALID;
  if (cache_mode == 1 && !(mrope && mrope_section_len == 3)) return ROPE_ERR_PARAM_INVALID;
  // row strides (elements): 0 means contiguous rows
  const int64_t qw = query->shape[1], kw = key->shape[1];
  const int64_t qs = q_row_stride ? q_row_stride : qw, ks = k_row_stride ? k_row_stride : kw;
  const int64_t esz = query->dtype == kF32 ? 4 : 2;
  if (qs < qw || ks < kw || qs % (16 / esz) || ks % (16 / esz)) return ROPE_ERR_PARAM_INVALID;
  if (strided_extent(T, qs, qw) < 0 || strided_extent(T, ks, kw) < 0) return ROPE_ERR_PARAM_INVALID;
  // outputs: both or neither; contiguous, same shape and dtype as the inputs
  if ((query_out == nullptr) != (key_out == nullptr)) return ROPE_ERR_PARAM_NULLPTR;
  if (query_out) {
    if (query_out->dtype != query->dtype || key_out->dtype != key->dtype) return ROPE_ERR_PARAM_INVALID;
    if (query_out->ndim != 2 || key_out->ndim != 2 || query_out->shape[0] != T || query_out->shape[1] != qw ||
        key_out->shape[0] != T || key_out->shape[1] != kw)
      return ROPE_ERR_PARAM_INVALID;
    if (!query_out->data || !key_out->data) return ROPE_ERR_PARAM_NULLPTR;
    if (!aligned(query_out->data, 16) || !aligned(key_out->data, 16)) return ROPE_ERR_PARAM_INVALID;
  }
  if (!positions->data || !query->data || !key->data || !cos_sin_cache->data) return ROPE_ERR_PARAM_NULLPTR;
  if (!aligned(positions->data, 8) || !aligned(query->data, 16) || !aligned(key->data, 16) ||
      !aligned(cos_sin_cache->data, 16))
    return ROPE_ERR_PARAM_INVALID;
  // an output that is its input (same pointer, contiguous rows) means in place;
  // any other overlap between the outputs and the inputs is rejected
  bool in_place = query_out == nullptr;
  if (!in_place && query_out->data == query->data && key_out->data == key->data && qs == qw && ks == kw)
    in_place = true;
  {
    // rewritten rows must not share memory with each other or with the tables
    const uintptr_t qa = reinterpret_cast<uintptr_t>(query->data), ka = reinterpret_cast<uintptr_t>(key->data);
    const int64_t pb = numel(positions) * 8, cb = numel(cos_sin_cache) * esz;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(positions->data),
                    ca = reinterpret_cast<uintptr_t>(cos_sin_cache->data);
    const int64_t qn = ((T - 1) * qs + qw) * esz, kn = ((T - 1) * ks + kw) * esz;
    if (in_place && (rows_overlap(qa, qs * esz, qw * esz, ka, ks * esz, kw * esz, T) ||
                     ranges_overlap(qa, qn, pa, pb) || ranges_overlap(qa, qn, ca, cb) ||
                     ranges_overlap(ka, kn, pa, pb) || ranges_overlap(ka, kn, ca, cb)))
      return ROPE_ERR_PARAM_INVALID;
  }
  if (!in_place) {
    const char* spans[4][2] = {
        {static_cast<const char*>(query->data), static_cast<const char*>(query->data) + ((T - 1) * qs + qw) * esz},
        {static_cast<const char*>(key->data), static_cast<const char*>(key->data) + ((T - 1) * ks + kw) * esz},
        {static_cast<const char*>(query_out->data), static_cast<const char*>(query_out->data) + T * qw * esz},
        {static_cast<const char*>(key_out->data), static_cast<const char*>(key_out->data) + T * kw * esz}};
    for (int o = 2; o < 4; ++o)
      for (int i = 0; i < 4; ++i)
        if (i != o && spans[o][0] < spans[i][1] && spans[i][0] < spans[o][1]) return ROPE_ERR_PARAM_INVALID;
  }

  rope::CacheProblem p;
  p.positions = static_cast<const int64_t*>(positions->data);
  p.query = query->data;
  p.key = key->data;
  p.cache = cos_sin_cache->data;
  p.dtype = query->dtype;
  p.T = T;
  p.hq = query->shape[1] / head_size;
  p.hk = key->shape[1] / head_size;
  p.head_size = head_size;
  p.rotary_dim = rotary_dim;
  p.max_seq = cos_sin_cache->shape[0];
  p.is_neox = is_neox != 0;
  p.mrope_rows = mrope ? (int32_t)mrope_section_len : 0;
  for (int i = 0; i < 4; ++i) p.section_end[i] = section_end[i];
  p.cache_mode = cache_mode;
  p.q_stride = qs;
  p.k_stride = ks;
  p.query_out = in_place ? nullptr : query_out->data;
  p.key_out = in_place ? nullptr : key_out->data;
  // one team of threads must fit one block of the cache kernel
  if (rope::cache_team_threads(p) > rope::cache_max_team_threads()) return ROPE_ERR_PARAM_INVALID;
  if (p.hq + p.hk > (int64_t)1 << 30 || head_size > (int64_t)1 << 30) return ROPE_ERR_PARAM_INVALID;
  return cuda_status(rope::launch_cache(p, static_cast<cudaStream_t>(stream)));
}

// Checks of the fused QKV call, then the launch.
int qkv_call(const rope_tensor_t* qkv, int64_t nq, int64_t nk, int64_t nv, const rope_tensor_t* q_gamma,
             const rope_tensor_t* k_gamma, float eps, const rope_tensor_t* cache, const rope_tensor_t* seq_lens,
             const rope_tensor_t* qsl, const rope_tensor_t* slot_mapping, const rope_tensor_t* q_out,
             const rope_tensor_t* k_cache, const rope_tensor_t* v_cache, void* stream) {
  const rope_tensor_t* all[] = {qkv, q_gamma, k_gamma, cache, seq_lens, qsl, slot_mapping, q_out, k_cache, v_cache};
  for (const rope_tensor_t* t : all)
    if (!t) return ROPE_ERR_PARAM_NULLPTR;
  for (const rope_tensor_t* t : all)
    if (!shape_ok(t)) return ROPE_ERR_PARAM_INVALID;
  // dtypes: one floating type for the data, int64 for the metadata
  const int32_t dt = qkv->dtype;
  if (!is_float(dt)) return ROPE_ERR_PARAM_INVALID;
  for (const rope_tensor_t* t : {q_gamma, k_gamma, cache, q_out, k_cache, v_cache})
    if (t->dtype != dt) return ROPE_ERR_PARAM_INVALID;
  for (const rope_tensor_t* t : {seq_lens, qsl, slot_mapping})
    if (t->dtype != kI64 || t->ndim != 1) return ROPE_ERR_PARAM_INVALID;
  // shapes
  if (nq < 0 || nk < 0 || nv < 0 || nq + nk + nv < 1) return ROPE_ERR_PARAM_INVALID;
  if (qkv->ndim != 2 || qkv->shape[0] < 1 || qkv->shape[1] % (nq + nk + nv)) return ROPE_ERR_PARAM_INVALID;
  const int64_t T = qkv->shape[0], D = qkv->shape[1] / (nq + nk + nv);
  const int64_t mult = dt == kF32 ? 16 : 32;
  const int64_t lanes = D / 2 / (dt == kF32 ? 4 : 8);  // threads per head row
  if (D < mult || D % mult || lanes > 32) return ROPE_ERR_PARAM_INVALID;
  if (q_gamma->ndim != 1 || q_gamma->shape[0] != D || k_gamma->ndim != 1 || k_gamma->shape[0] != D)
    return ROPE_ERR_PARAM_INVALID;
  if (cache->ndim != 2 || cache->shape[1] != D || cache->shape[0] < 1) return ROPE_ERR_PARAM_INVALID;
  const int64_t B = seq_lens->shape[0];
  if (B < 1 || B > (int64_t(1) << 30) || qsl->shape[0] != B + 1 || slot_mapping->shape[0] != T)
    return ROPE_ERR_PARAM_INVALID;
  if (q_out->ndim != 2 || q_out->shape[0] != T || q_out->shape[1] != nq * D) return ROPE_ERR_PARAM_INVALID;
  if (k_cache->ndim != 4 || v_cache->ndim != 4) return ROPE_ERR_PARAM_INVALID;
  const int64_t NB = k_cache->shape[0], BS = k_cache->shape[2];
  if (NB < 1 || BS < 1 || k_cache->shape[1] != nk || k_cache->shape[3] != D || v_cache->shape[0] != NB ||
      v_cache->shape[1] != nv || v_cache->shape[2] != BS || v_cache->shape[3] != D)
    return ROPE_ERR_PARAM_INVALID;
  int64_t slots = 0;  // NB * BS, also when a cache has no heads (and so no elements)
  if (__builtin_mul_overflow(NB, BS, &slots) || slots > kMaxElements) return ROPE_ERR_PARAM_INVALID;
  // head counts and the block size are kept in 32-bit fields by the kernel
  if (nq + nk + nv > (int64_t(1) << 30) || BS > (int64_t(1) << 30)) return ROPE_ERR_PARAM_INVALID;
  if (!(eps >= 0.0f) || !(eps < 1e30f)) return ROPE_ERR_PARAM_INVALID;
  for (const rope_tensor_t* t : all)
    if (!t->data && numel(t) > 0) return ROPE_ERR_PARAM_NULLPTR;
  // the outputs are written while every input is read: no output may share
  // memory with an input or with another output
  for (const rope_tensor_t* o : {q_out, k_cache, v_cache})
    for (const rope_tensor_t* t : all)
      if (t != o && tensors_overlap(o, t)) return ROPE_ERR_PARAM_INVALID;
  for (const rope_tensor_t* t : {qkv, q_gamma, k_gamma, cache, q_out, k_cache, v_cache})
    if (t->data && !aligned(t->data, 16)) return ROPE_ERR_PARAM_INVALID;
  for (const rope_tensor_t* t : {seq_lens, qsl, slot_mapping})
    if (!aligned(t->data, 8)) return ROPE_ERR_PARAM_INVALID;

  rope::QkvProblem p;
  p.qkv = qkv->data;
  p.q_gamma = q_gamma->data;
  p.k_gamma = k_gamma->data;
  p.cache = cache->data;
  p.seq_lens = static_cast<const int64_t*>(seq_lens->data);
  p.query_start_loc = static_cast<const int64_t*>(qsl->data);
  p.slot_mapping = static_cast<const int64_t*>(slot_mapping->data);
  p.q_out = q_out->data;
  p.k_cache = k_cache->data;
  p.v_cache = v_cache->data;
  p.dtype = dt;
  p.T = T;
  p.B = B;
  p.nq = nq;
  p.nk = nk;
  p.nv = nv;
  p.D = D;
  p.max_seq = cache->shape[0];
  p.num_blocks = NB;
  p.block_size = BS;
  p.eps = eps;
  return cuda_status(rope::launch_qkv(p, static_cast<cudaStream_t>(stream)));
}

// Frequencies scaled for long contexts; the formulas are in the header.
int frequencies(int64_t R, double base, const rope_scaling_t* s, double* inv_freq, double* scale) {
  if (!inv_freq || !scale) return ROPE_ERR_PARAM_NULLPTR;
  if (R < 2 || R > 2048 || R % 2 || !(base > 0) || !std::isfinite(base)) return ROPE_ERR_PARAM_INVALID;
  const int32_t kind = s ? s->kind : ROPE_SCALING_NONE;
  const int64_t F = R / 2;
  const double two_pi = 6.283185307179586476925;
  if (kind < ROPE_SCALING_NONE || kind > ROPE_SCALING_FACTORS) return ROPE_ERR_PARAM_INVALID;
  if (kind != ROPE_SCALING_NONE && kind != ROPE_SCALING_FACTORS && !(s->factor > 0 && std::isfinite(s->factor)))
    return ROPE_ERR_PARAM_INVALID;
  if ((kind == ROPE_SCALING_YARN || kind == ROPE_SCALING_WAVELENGTH) &&
      !(s->original_length > 0 && std::isfinite(s->original_length)))
    return ROPE_ERR_PARAM_INVALID;
  if (s && !(s->attention >= 0 && std::isfinite(s->attention))) return ROPE_ERR_PARAM_INVALID;
  double low = s ? s->low : 0, high = s ? s->high : 0;
  double ramp_from = 0, ramp_to = 0;
  if (kind == ROPE_SCALING_BASE) {
    if (R == 2) return ROPE_ERR_PARAM_INVALID;
    base *= std::pow(s->factor, (double)R / (double)(R - 2));
    if (!(base > 0) || !std::isfinite(base)) return ROPE_ERR_PARAM_INVALID;
  } else if (kind == ROPE_SCALING_YARN) {
    low = low == 0 ? 1 : low;
    high = high == 0 ? 32 : high;
    if (!(low > 0 && high > low && std::isfinite(high)) || base <= 1) return ROPE_ERR_PARAM_INVALID;
    auto index = [&](double turns) { return R * std::log(s->original_length / (two_pi * turns)) / (2 * std::log(base)); };
    ramp_from = std::fmax(std::floor(index(high)), 0);
    ramp_to = std::fmin(std::ceil(index(low)), (double)(R - 1));
  } else if (kind == ROPE_SCALING_WAVELENGTH) {
    if (!(low > 0 && high > low && std::isfinite(high))) return ROPE_ERR_PARAM_INVALID;
  } else if (kind == ROPE_SCALING_FACTORS) {
    if (!s->factors) return ROPE_ERR_PARAM_NULLPTR;
    for (int64_t i = 0; i < F; ++i)
      if (!(s->factors[i] > 0) || !std::isfinite(s->factors[i])) return ROPE_ERR_PARAM_INVALID;
  }
  for (int64_t i = 0; i < F; ++i) {
    double f = std::pow(base, -(double)(2 * i) / (double)R);
    if (kind == ROPE_SCALING_LINEAR) {
      f /= s->factor;
    } else if (kind == ROPE_SCALING_YARN) {
      const double r = std::fmin(std::fmax(((double)i - ramp_from) / std::fmax(ramp_to - ramp_from, 0.001), 0), 1);
      f = f / s->factor * r + f * (1 - r);
    } else if (kind == ROPE_SCALING_WAVELENGTH) {
      const double t = s->original_length * f / two_pi;
      const double keep = std::fmin(std::fmax((t - low) / (high - low), 0), 1);
      f = f * keep + f / s->factor * (1 - keep);
    } else if (kind == ROPE_SCALING_FACTORS) {
      f /= s->factors[i];
    }
    inv_freq[i] = f;
  }
  *scale = s && s->attention > 0                                ? s->attention
           : kind == ROPE_SCALING_YARN && s->factor > 1 ? 1 + 0.1 * std::log(s->factor)
                                                        : 1.0;
  return ROPE_OK;
}

// Checks of the cos/sin table calls (sin NULL: the cache layout), then the launch.
int table_call(const double* inv_freq, int64_t F, double scale, const rope_tensor_t* positions, int64_t first,
               bool interleave, const rope_tensor_t* cos, const rope_tensor_t* sin, void* stream) {
  if (!inv_freq) return ROPE_ERR_PARAM_NULLPTR;
  if (F < 1 || F > 1024 || !std::isfinite((float)scale)) return ROPE_ERR_PARAM_INVALID;
  for (int64_t i = 0; i < F; ++i)
    if (!(std::fabs(inv_freq[i]) <= 1e6)) return ROPE_ERR_PARAM_INVALID;
  if (!shape_ok(cos) || !is_float(cos->dtype) || cos->shape[cos->ndim - 1] != 2 * F) return ROPE_ERR_PARAM_INVALID;
  if (sin) {
    if (!shape_ok(sin) || sin->dtype != cos->dtype || sin->ndim != cos->ndim) return ROPE_ERR_PARAM_INVALID;
    for (int i = 0; i < cos->ndim; ++i)
      if (sin->shape[i] != cos->shape[i]) return ROPE_ERR_PARAM_INVALID;
  }
  const int64_t rows = numel(cos) / (2 * F);
  if (positions) {
    if (positions->dtype != kI64 || !shape_ok(positions) || numel(positions) != rows) return ROPE_ERR_PARAM_INVALID;
  }
  if (rows == 0) return ROPE_OK;
  if (!cos->data || (sin && !sin->data) || (positions && !positions->data)) return ROPE_ERR_PARAM_NULLPTR;
  const uintptr_t e = (uintptr_t)elem_size(cos->dtype);
  if (!aligned(cos->data, e) || (sin && !aligned(sin->data, e)) || (positions && !aligned(positions->data, 8)))
    return ROPE_ERR_PARAM_INVALID;
  if ((sin && tensors_overlap(cos, sin)) || (positions && tensors_overlap(positions, cos)) ||
      (positions && sin && tensors_overlap(positions, sin)))
    return ROPE_ERR_PARAM_INVALID;
  rope::TableProblem p;
  p.inv_freq = inv_freq;
  p.F = F;
  p.scale = scale;
  p.positions = positions ? static_cast<const int64_t*>(positions->data) : nullptr;
  p.first = first;
  p.rows = rows;
  p.cos = cos->data;
  p.sin = sin ? sin->data : nullptr;
  p.interleave = interleave;
  p.dtype = cos->dtype;
  return cuda_status(rope::launch_table(p, static_cast<cudaStream_t>(stream)));
}

// The mrope arguments of the cache-indexed calls: whether mrope is on, and the
// cumulative section ends.
int mrope_arguments(const int64_t* section, int64_t len, int64_t rotary_dim, int32_t cache_mode, bool* on,
                    int32_t (&end)[4]) {
  *on = section != nullptr && len > 0 && section[0] > 0;
  if (section != nullptr && len != 3 && len != 4) return ROPE_ERR_PARAM_INVALID;
  int64_t sum = 0;
  for (int64_t i = 0; section != nullptr && i < len; ++i) {
    if (section[i] < 0 || section[i] > rotary_dim) return ROPE_ERR_PARAM_INVALID;
    sum += section[i];
    end[i] = (int32_t)sum;
  }
  if (*on && 2 * sum != rotary_dim) return ROPE_ERR_PARAM_INVALID;
  if (cache_mode != 0 && cache_mode != 1) return ROPE_ERR_PARAM_INVALID;
  if (cache_mode == 1 && !(*on && len == 3)) return ROPE_ERR_PARAM_INVALID;
  return ROPE_OK;
}

// Byte range of `rows` rows of `width` elements, `stride` apart.
struct Range {
  uintptr_t at;
  int64_t bytes;
};

Range rows_range(const rope_tensor_t* t, int64_t stride) {
  const int64_t rows = t->shape[0], width = t->shape[1];
  if (rows < 1 || width < 1) return {reinterpret_cast<uintptr_t>(t->data), 0};
  return {reinterpret_cast<uintptr_t>(t->data), ((rows - 1) * stride + width) * elem_size(t->dtype)};
}

Range whole_range(const rope_tensor_t* t) {
  return {reinterpret_cast<uintptr_t>(t->data), numel(t) * elem_size(t->dtype)};
}

bool meet(const Range& x, const Range& y) { return ranges_overlap(x.at, x.bytes, y.at, y.bytes); }

// Checks of the append call, then the launch.
int append_call(const rope_tensor_t* positions, const rope_tensor_t* query, const rope_tensor_t* key,
                const rope_tensor_t* value, const rope_tensor_t* table, const rope_tensor_t* slots,
                const rope_tensor_t* query_out, const rope_tensor_t* k_cache, const rope_tensor_t* v_cache, int64_t D,
                int64_t R, int32_t is_neox, const int64_t* section, int64_t section_len, int32_t cache_mode,
                int64_t q_row_stride, int64_t k_row_stride, int64_t v_row_stride, void* stream) {
  for (const rope_tensor_t* t : {positions, key, value, table, slots, k_cache, v_cache})
    if (!t) return ROPE_ERR_PARAM_NULLPTR;
  if (query_out && !query) return ROPE_ERR_PARAM_NULLPTR;
  for (const rope_tensor_t* t : {positions, query, key, value, table, slots, query_out, k_cache, v_cache})
    if (t && !shape_ok(t)) return ROPE_ERR_PARAM_INVALID;
  const int32_t dt = key->dtype;
  if (!is_float(dt) || (table->dtype != dt && table->dtype != kF32)) return ROPE_ERR_PARAM_INVALID;
  for (const rope_tensor_t* t : {query, value, query_out, k_cache, v_cache})
    if (t && t->dtype != dt) return ROPE_ERR_PARAM_INVALID;
  if (positions->dtype != kI64 || slots->dtype != kI64 || slots->ndim != 1) return ROPE_ERR_PARAM_INVALID;
  // head size and rotary dim: 64-byte multiples; a head's row groups fit a block
  const int64_t mult = dt == kF32 ? 16 : 32;
  if (D <= 0 || D % mult || D > (dt == kF32 ? 1024 : 2048)) return ROPE_ERR_PARAM_INVALID;
  if (R <= 0 || R % mult || R > D) return ROPE_ERR_PARAM_INVALID;
  if (table->ndim != 2 || table->shape[0] < 1 || table->shape[1] != R) return ROPE_ERR_PARAM_INVALID;
  bool mrope = false;
  int32_t section_end[4] = {0, 0, 0, 0};
  const int st = mrope_arguments(section, section_len, R, cache_mode, &mrope, section_end);
  if (st != ROPE_OK) return st;
  // rows
  const int64_t T = key->shape[0];
  for (const rope_tensor_t* t : {query, key, value, query_out})
    if (t && (t->ndim != 2 || t->shape[0] != T || t->shape[1] < D || t->shape[1] % D)) return ROPE_ERR_PARAM_INVALID;
  if (slots->shape[0] != T) return ROPE_ERR_PARAM_INVALID;
  if (mrope ? positions->ndim != 2 || positions->shape[0] != section_len || positions->shape[1] != T
            : positions->ndim != 1 || positions->shape[0] != T)
    return ROPE_ERR_PARAM_INVALID;
  if (query_out && query_out->shape[1] != query->shape[1]) return ROPE_ERR_PARAM_INVALID;
  const int64_t per16 = 16 / elem_size(dt);
  int64_t strides[3] = {q_row_stride, k_row_stride, v_row_stride};
  const rope_tensor_t* rows[3] = {query, key, value};
  for (int i = 0; i < 3; ++i) {
    if (!rows[i]) continue;
    if (!strides[i]) strides[i] = rows[i]->shape[1];
    if (strides[i] < rows[i]->shape[1] || strides[i] % per16) return ROPE_ERR_PARAM_INVALID;
    if (strided_extent(T, strides[i], rows[i]->shape[1]) < 0) return ROPE_ERR_PARAM_INVALID;
  }
  const int64_t hq = query ? query->shape[1] / D : 0, hk = key->shape[1] / D, hv = value->shape[1] / D;
  // caches
  if (k_cache->ndim != 4 || v_cache->ndim != 4) return ROPE_ERR_PARAM_INVALID;
  const int64_t NB = k_cache->shape[0], BS = k_cache->shape[2];
  if (NB < 1 || BS < 1 || k_cache->shape[1] != hk || k_cache->shape[3] != D || v_cache->shape[0] != NB ||
      v_cache->shape[1] != hv || v_cache->shape[2] != BS || v_cache->shape[3] != D)
    return ROPE_ERR_PARAM_INVALID;
  if (hq + hk + hv > (int64_t(1) << 30) || BS > (int64_t(1) << 30)) return ROPE_ERR_PARAM_INVALID;
  if (T == 0) return ROPE_OK;
  for (const rope_tensor_t* t : {positions, query, key, value, table, slots, query_out, k_cache, v_cache})
    if (t && !t->data) return ROPE_ERR_PARAM_NULLPTR;
  for (const rope_tensor_t* t : {query, key, value, table, query_out, k_cache, v_cache})
    if (t && !aligned(t->data, 16)) return ROPE_ERR_PARAM_INVALID;
  if (!aligned(positions->data, 8) || !aligned(slots->data, 8)) return ROPE_ERR_PARAM_INVALID;
  // an output at its contiguous input is in place; a tensor that is written shares no memory with another
  const bool in_place = query && (!query_out || (query_out->data == query->data && strides[0] == query->shape[1]));
  const Range kr = rows_range(key, strides[1]), vr = rows_range(value, strides[2]);
  const Range read[] = {whole_range(positions), whole_range(table), whole_range(slots)};
  const Range caches[] = {whole_range(k_cache), whole_range(v_cache)};
  const Range qr = query ? rows_range(query, strides[0]) : Range{0, 0};
  const Range qo = !query ? Range{0, 0} : in_place ? qr : whole_range(query_out);
  for (const Range& r : read)
    if (meet(qo, r) || meet(caches[0], r) || meet(caches[1], r)) return ROPE_ERR_PARAM_INVALID;
  for (const Range& r : {kr, vr, qr, qo})
    if (meet(caches[0], r) || meet(caches[1], r)) return ROPE_ERR_PARAM_INVALID;
  if (meet(caches[0], caches[1])) return ROPE_ERR_PARAM_INVALID;
  if (query) {
    const int64_t e = elem_size(dt);
    if (in_place) {
      for (int i = 1; i < 3; ++i)
        if (rows_overlap(qr.at, strides[0] * e, query->shape[1] * e, i == 1 ? kr.at : vr.at, strides[i] * e,
                         rows[i]->shape[1] * e, T))
          return ROPE_ERR_PARAM_INVALID;
    } else if (meet(qo, qr) || meet(qo, kr) || meet(qo, vr)) {
      return ROPE_ERR_PARAM_INVALID;
    }
  }

  rope::AppendProblem p;
  p.positions = static_cast<const int64_t*>(positions->data);
  p.slot_mapping = static_cast<const int64_t*>(slots->data);
  p.query = query ? query->data : nullptr;
  p.key = key->data;
  p.value = value->data;
  p.table = table->data;
  p.query_out = !query ? nullptr : in_place ? query->data : query_out->data;
  p.k_cache = k_cache->data;
  p.v_cache = v_cache->data;
  p.dtype = dt;
  p.table_dtype = table->dtype;
  p.T = T;
  p.hq = hq;
  p.hk = hk;
  p.hv = hv;
  p.head_size = D;
  p.rotary_dim = R;
  p.max_seq = table->shape[0];
  p.num_blocks = NB;
  p.block_size = BS;
  p.is_neox = is_neox != 0;
  p.mrope_rows = mrope ? (int32_t)section_len : 0;
  for (int i = 0; i < 4; ++i) p.section_end[i] = section_end[i];
  p.cache_mode = cache_mode;
  p.q_stride = query ? strides[0] : 0;
  p.k_stride = strides[1];
  p.v_stride = strides[2];
  return cuda_status(rope::launch_append(p, static_cast<cudaStream_t>(stream)));
}

// Head counts, head size and row count that the attention takes (rows bounded so that the
// workspace's size stays in int64).
bool attend_sizes_ok(int64_t T, int64_t nq, int64_t nk, int64_t D, int32_t dt) {
  const int64_t mult = dt == kF32 ? 16 : 32;
  return is_float(dt) && nq >= 1 && nk >= 1 && nq <= (int64_t(1) << 16) && nq % nk == 0 && T >= 0 &&
         T <= (int64_t(1) << 31) && T * nq < (int64_t(1) << 31) - 512 && D >= mult && D % mult == 0 && D <= 512;
}

// Checks of the attention call, then the launch.
int attend_call(const rope_tensor_t* query, int64_t q_row_stride, const rope_tensor_t* k_cache,
                const rope_tensor_t* v_cache, const rope_tensor_t* block_table, const rope_tensor_t* seq_lens,
                const rope_tensor_t* qsl, const rope_tensor_t* prefix_blocks, int64_t P, float scale,
                const rope_tensor_t* out, const rope_tensor_t* lse, void* workspace, int64_t workspace_bytes,
                void* stream) {
  for (const rope_tensor_t* t : {query, k_cache, v_cache, block_table, seq_lens, qsl, out})
    if (!t) return ROPE_ERR_PARAM_NULLPTR;
  for (const rope_tensor_t* t : {query, k_cache, v_cache, block_table, seq_lens, qsl, prefix_blocks, out, lse})
    if (t && !shape_ok(t)) return ROPE_ERR_PARAM_INVALID;
  const int32_t dt = query->dtype;
  if (!is_float(dt)) return ROPE_ERR_PARAM_INVALID;
  for (const rope_tensor_t* t : {k_cache, v_cache, out})
    if (t->dtype != dt) return ROPE_ERR_PARAM_INVALID;
  for (const rope_tensor_t* t : {block_table, seq_lens, qsl, prefix_blocks})
    if (t && t->dtype != kI64) return ROPE_ERR_PARAM_INVALID;
  if (lse && lse->dtype != kF32) return ROPE_ERR_PARAM_INVALID;
  // caches and heads
  if (k_cache->ndim != 4 || v_cache->ndim != 4) return ROPE_ERR_PARAM_INVALID;
  for (int i = 0; i < 4; ++i)
    if (k_cache->shape[i] != v_cache->shape[i] || k_cache->shape[i] < 1) return ROPE_ERR_PARAM_INVALID;
  const int64_t NB = k_cache->shape[0], nk = k_cache->shape[1], BS = k_cache->shape[2], D = k_cache->shape[3];
  if (query->ndim != 2 || query->shape[1] < 1 || query->shape[1] % D) return ROPE_ERR_PARAM_INVALID;
  const int64_t T = query->shape[0], nq = query->shape[1] / D;
  if (!attend_sizes_ok(T, nq, nk, D, dt)) return ROPE_ERR_PARAM_INVALID;
  if (BS > (int64_t(1) << 30)) return ROPE_ERR_PARAM_INVALID;
  if (!q_row_stride) q_row_stride = query->shape[1];
  if (q_row_stride < query->shape[1] || q_row_stride % (16 / elem_size(dt))) return ROPE_ERR_PARAM_INVALID;
  if (strided_extent(T, q_row_stride, query->shape[1]) < 0) return ROPE_ERR_PARAM_INVALID;
  // batch
  if (seq_lens->ndim != 1 || qsl->ndim != 1 || block_table->ndim != 2) return ROPE_ERR_PARAM_INVALID;
  const int64_t B = seq_lens->shape[0], W = block_table->shape[1];
  const int64_t most = int64_t(1) << 30;
  if (B < 1 || B > most || qsl->shape[0] != B + 1 || block_table->shape[0] != B || W < 1)
    return ROPE_ERR_PARAM_INVALID;
  if (W > most / BS || P < 0 || P > most || P + W * BS >= 2 * most - 512) return ROPE_ERR_PARAM_INVALID;
  if (P > 0 && !prefix_blocks) return ROPE_ERR_PARAM_NULLPTR;
  if (P > 0 && numel(prefix_blocks) < (P + BS - 1) / BS) return ROPE_ERR_PARAM_INVALID;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return ROPE_ERR_PARAM_INVALID;
  // outputs
  if (out->ndim != 2 || out->shape[0] != T || out->shape[1] != nq * D) return ROPE_ERR_PARAM_INVALID;
  if (lse && (lse->ndim != 2 || lse->shape[0] != T || lse->shape[1] != nq)) return ROPE_ERR_PARAM_INVALID;
  if (T == 0) return ROPE_OK;
  if (!workspace) return ROPE_ERR_PARAM_NULLPTR;
  if (workspace_bytes < rope::attend_workspace(T, nq, nk, D, dt, P)) return ROPE_ERR_PARAM_INVALID;
  for (const rope_tensor_t* t : {query, k_cache, v_cache, block_table, seq_lens, qsl, out, lse})
    if (t && !t->data) return ROPE_ERR_PARAM_NULLPTR;
  if (P > 0 && !prefix_blocks->data) return ROPE_ERR_PARAM_NULLPTR;
  for (const rope_tensor_t* t : {query, k_cache, v_cache, out})
    if (!aligned(t->data, 16)) return ROPE_ERR_PARAM_INVALID;
  for (const rope_tensor_t* t : {block_table, seq_lens, qsl})
    if (!aligned(t->data, 8)) return ROPE_ERR_PARAM_INVALID;
  if ((P > 0 && !aligned(prefix_blocks->data, 8)) || (lse && !aligned(lse->data, 4)) || !aligned(workspace, 256))
    return ROPE_ERR_PARAM_INVALID;
  // what the call writes shares no memory with anything else of it
  const Range none = {0, 0};
  const Range written[] = {whole_range(out), lse ? whole_range(lse) : none,
                           {reinterpret_cast<uintptr_t>(workspace), workspace_bytes}};
  const Range read[] = {rows_range(query, q_row_stride), whole_range(k_cache), whole_range(v_cache),
                        whole_range(block_table), whole_range(seq_lens), whole_range(qsl),
                        P > 0 ? whole_range(prefix_blocks) : none};
  for (int i = 0; i < 3; ++i) {
    for (const Range& r : read)
      if (meet(written[i], r)) return ROPE_ERR_PARAM_INVALID;
    for (int j = 0; j < i; ++j)
      if (meet(written[i], written[j])) return ROPE_ERR_PARAM_INVALID;
  }

  rope::AttendProblem p;
  p.query = query->data;
  p.q_stride = q_row_stride;
  p.k_cache = k_cache->data;
  p.v_cache = v_cache->data;
  p.block_table = static_cast<const int64_t*>(block_table->data);
  p.seq_lens = static_cast<const int64_t*>(seq_lens->data);
  p.query_start_loc = static_cast<const int64_t*>(qsl->data);
  p.prefix_blocks = P > 0 ? static_cast<const int64_t*>(prefix_blocks->data) : nullptr;
  p.out = out->data;
  p.lse = lse ? static_cast<float*>(lse->data) : nullptr;
  p.workspace = workspace;
  p.dtype = dt;
  p.T = T;
  p.B = B;
  p.nq = nq;
  p.nk = nk;
  p.D = D;
  p.num_blocks = NB;
  p.block_size = BS;
  p.W = W;
  p.prefix_len = P;
  p.scale = scale;
  return cuda_status(rope::launch_attend(p, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int rope_inplace_partial(const rope_tensor_t* x, const rope_tensor_t* cos, const rope_tensor_t* sin,
                         int64_t rotary_mode, int64_t start, int64_t end, void* stream) {
  return inplace_call(x, cos, sin, rotary_mode, start, end, false, stream);
}

int rope_inplace_partial_backward(const rope_tensor_t* grad, const rope_tensor_t* cos, const rope_tensor_t* sin,
                                  int64_t rotary_mode, int64_t start, int64_t end, void* stream) {
  return inplace_call(grad, cos, sin, rotary_mode, start, end, true, stream);
}

int rope_with_sin_cos_cache(const rope_tensor_t* positions, const rope_tensor_t* query,
                            const rope_tensor_t* key, const rope_tensor_t* cos_sin_cache,
                            int64_t head_size, int64_t rotary_dim, int32_t is_neox,
                            const int64_t* mrope_section, int64_t mrope_section_len, void* stream) {
  return cache_call(positions, query, key, cos_sin_cache, head_size, rotary_dim, is_neox, mrope_section,
                    mrope_section_len, 0, 0, 0, nullptr, nullptr, stream);
}

int rope_with_sin_cos_cache_v2(const rope_tensor_t* positions, const rope_tensor_t* query,
                               const rope_tensor_t* key, const rope_tensor_t* cos_sin_cache,
                               int64_t head_size, int64_t rotary_dim, int32_t is_neox,
                               const int64_t* mrope_section, int64_t mrope_section_len, int32_t cache_mode,
                               int64_t query_row_stride, int64_t key_row_stride, const rope_tensor_t* query_out,
                               const rope_tensor_t* key_out, void* stream) {
  return cache_call(positions, query, key, cos_sin_cache, head_size, rotary_dim, is_neox, mrope_section,
                    mrope_section_len, cache_mode, query_row_stride, key_row_stride, query_out, key_out, stream);
}

int rope_qkv_rmsnorm_rope_cache(const rope_tensor_t* qkv, int64_t num_q_heads, int64_t num_k_heads,
                                int64_t num_v_heads, const rope_tensor_t* q_gamma, const rope_tensor_t* k_gamma,
                                float eps, const rope_tensor_t* cos_sin_cache, const rope_tensor_t* seq_lens,
                                const rope_tensor_t* query_start_loc, const rope_tensor_t* slot_mapping,
                                const rope_tensor_t* q_out, const rope_tensor_t* k_cache,
                                const rope_tensor_t* v_cache, void* stream) {
  return qkv_call(qkv, num_q_heads, num_k_heads, num_v_heads, q_gamma, k_gamma, eps, cos_sin_cache, seq_lens,
                  query_start_loc, slot_mapping, q_out, k_cache, v_cache, stream);
}

int rope_scaled_frequencies(int64_t rotary_dim, double base, const rope_scaling_t* scaling, double* inv_freq,
                            double* scale) {
  return frequencies(rotary_dim, base, scaling, inv_freq, scale);
}

int rope_scaled_cos_sin_cache(const double* inv_freq, int64_t num_freq, double scale, const rope_tensor_t* positions,
                              int64_t first_position, const rope_tensor_t* cache, void* stream) {
  if (!cache) return ROPE_ERR_PARAM_NULLPTR;
  return table_call(inv_freq, num_freq, scale, positions, first_position, false, cache, nullptr, stream);
}

int rope_scaled_cos_sin(const double* inv_freq, int64_t num_freq, double scale, const rope_tensor_t* positions,
                        int64_t first_position, int64_t rotary_mode, const rope_tensor_t* cos,
                        const rope_tensor_t* sin, void* stream) {
  if (!cos || !sin) return ROPE_ERR_PARAM_NULLPTR;
  if (rotary_mode != 0 && rotary_mode != 1) return ROPE_ERR_PARAM_INVALID;
  return table_call(inv_freq, num_freq, scale, positions, first_position, rotary_mode == 1, cos, sin, stream);
}

int rope_append_paged_kv(const rope_tensor_t* positions, const rope_tensor_t* query, const rope_tensor_t* key,
                         const rope_tensor_t* value, const rope_tensor_t* cos_sin_cache,
                         const rope_tensor_t* slot_mapping, const rope_tensor_t* query_out,
                         const rope_tensor_t* k_cache, const rope_tensor_t* v_cache, int64_t head_size,
                         int64_t rotary_dim, int32_t is_neox, const int64_t* mrope_section,
                         int64_t mrope_section_len, int32_t cache_mode, int64_t query_row_stride,
                         int64_t key_row_stride, int64_t value_row_stride, void* stream) {
  return append_call(positions, query, key, value, cos_sin_cache, slot_mapping, query_out, k_cache, v_cache, head_size,
                     rotary_dim, is_neox, mrope_section, mrope_section_len, cache_mode, query_row_stride,
                     key_row_stride, value_row_stride, stream);
}

int rope_paged_attention(const rope_tensor_t* query, int64_t query_row_stride, const rope_tensor_t* k_cache,
                         const rope_tensor_t* v_cache, const rope_tensor_t* block_table,
                         const rope_tensor_t* seq_lens, const rope_tensor_t* query_start_loc,
                         const rope_tensor_t* prefix_blocks, int64_t prefix_len, float scale,
                         const rope_tensor_t* out, const rope_tensor_t* lse, void* workspace,
                         int64_t workspace_bytes, void* stream) {
  return attend_call(query, query_row_stride, k_cache, v_cache, block_table, seq_lens, query_start_loc, prefix_blocks,
                     prefix_len, scale, out, lse, workspace, workspace_bytes, stream);
}

int rope_paged_attention_workspace(int64_t num_tokens, int64_t num_q_heads, int64_t num_k_heads, int64_t head_size,
                                   int32_t dtype, int64_t prefix_len, int64_t* bytes) {
  if (!bytes) return ROPE_ERR_PARAM_NULLPTR;
  if (prefix_len < 0 || !attend_sizes_ok(num_tokens, num_q_heads, num_k_heads, head_size, dtype))
    return ROPE_ERR_PARAM_INVALID;
  *bytes = rope::attend_workspace(num_tokens, num_q_heads, num_k_heads, head_size, dtype, prefix_len);
  return ROPE_OK;
}

int rope_get_device_error(void* stream, int32_t* code) {
  if (!code) return ROPE_ERR_PARAM_NULLPTR;
  uint32_t c = 0;
  const cudaError_t e = rope::read_and_clear_device_error(static_cast<cudaStream_t>(stream), &c);
  *code = (int32_t)c;
  return cuda_status(e);
}

const char* rope_status_string(int status) {
  switch (status) {
    case ROPE_OK:
      return "ROPE_OK";
    case ROPE_ERR_PARAM_NULLPTR:
      return "ROPE_ERR_PARAM_NULLPTR: a required tensor or its data pointer is NULL";
    case ROPE_ERR_PARAM_INVALID:
      return "ROPE_ERR_PARAM_INVALID: unsupported dtype, shape, slice, mode, section or alignment";
    case ROPE_ERR_CUDA:
      return "ROPE_ERR_CUDA: the CUDA runtime rejected a launch or query";
    default:
      return "unknown status";
  }
}

uint64_t rope_launch_count(void) { return rope::launch_count(); }

int rope_abi_version(void) { return ROPE_ABI_VERSION; }

}  // extern "C"
