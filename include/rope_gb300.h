/*
 * rope_gb300.h -- C ABI of the GB300 (sm_103a) rotary position embedding library.
 *
 * Operators, each an asynchronous call on a caller-given CUDA stream:
 *
 *   rope_inplace_partial          in-place partial-slice RoPE on a BSND tensor
 *                                 (interleave or half mode), and its backward
 *   rope_with_sin_cos_cache(_v2)  cos/sin-cache-indexed RoPE of query and key (rope /
 *                                 mrope, GPT-NeoX or GPT-J style; V2: interleaved mrope
 *                                 splice, strided inputs, separate outputs)
 *   rope_qkv_rmsnorm_rope_cache   fused QKV split + RMSNorm + RoPE + paged KV-cache write
 *   rope_scaled_cos_sin(_cache)   the cos/sin tables these operators read, from frequencies
 *                                 scaled for long contexts (rope_scaled_frequencies)
 *   rope_append_paged_kv          RoPE of query and key on the way to the output and to
 *                                 their slots of a paged KV cache (no norm)
 *   rope_paged_attention          attention over the paged KV cache, with a prefix shared by
 *                                 the whole batch read once for all
 *   rope_append_paged_kv_8bit     the append and the attention for a cache held in 8 bits, with a
 *   rope_paged_attention_8bit     scale for each block of tokens and head
 *   rope_rearrange_sequences      sequences of a paged cache forked, reordered, dropped and given room;
 *   rope_compact_pages            live pages moved to the front; pages copied in many tensors at once
 *   rope_copy_pages
 *
 * Sources (web pages, cited by title and section):
 *  [IPRM] "CANN ops-transformer 的 aclnnInplacePartialRotaryMul 算子：Inplace
 *         部分旋转位置编码接口详解与实现剖析"
 *  [RSCC] "CANN ops-transformer 旋转位置编码算子 RopeWithSinCosCache 深度解析：
 *         cache 化 RoPE 的计算原理与 aclnn 两段式调用实战"
 *  [QKV]  the "aclnnQkvRmsNormRopeCacheWithKScale" documentation page
 *
 * Memory and ownership.  Every tensor is described by a rope_tensor_t that the
 * caller owns; `data` is a DEVICE pointer to contiguous row-major storage,
 * borrowed for the duration of the call and of the work it enqueues.  All
 * tensors of a call live on the current device (cudaSetDevice), and `stream`
 * belongs to it: the launch goes to the current device.  The
 * library allocates nothing on the device, needs no workspace (except rope_paged_attention
 * and rope_paged_attention_8bit, whose caller gives them one), and never synchronises the
 * stream (except rope_get_device_error, which says so).  The two-phase
 * "GetWorkspaceSize, then execute" interface of the pages collapses to one call
 * because the workspace is always zero bytes.  (The fused op's kernel uses up to
 * 64 KB of on-chip shared memory per CTA; the first call that needs more than
 * 48 KB on a device raises the kernel's shared-memory limit there, once, with
 * cudaFuncSetAttribute.)
 *
 * Arithmetic.  Half-precision inputs are widened to binary32; each output is
 * a two-term dot product evaluated with Kahan's FMA-based difference of
 * products (relative error <= 2^-23, see Jeannerod, Louvet & Muller, Math. Comp.
 * 82 (2013)) and rounded once, to nearest even, to the output type.  Where
 * both products are exact in binary32 (query, key and the cache all binary16,
 * or all bfloat16, in the GPT-J and out-of-place cache kernels) it is one FMA
 * after an exact product: the correctly rounded binary32 value.  Results are
 * deterministic and do not depend on the launch shape.
 *
 * Errors.  Every argument check happens on the host before anything is
 * enqueued; a failed check returns a status and enqueues nothing.  A shape
 * whose element count (or a strided view's extent) overflows, or exceeds
 * INT64_MAX / 8, is ROPE_ERR_PARAM_INVALID.  So is a tensor the call rewrites
 * that shares memory with a tensor it reads or another one it writes (x with
 * cos or sin; in place, query with key, positions or the cache; an output of
 * the fused op with any other tensor of the call), whose result would depend
 * on the order in which threads run; query and key as disjoint column ranges
 * of one buffer, with one row stride, are accepted.  Status
 * values 161001 and 161002 are the ones [IPRM §返回值与错误码] lists
 * (ACLNN_ERR_PARAM_NULLPTR, ACLNN_ERR_PARAM_INVALID).  A CUDA launch error is
 * returned as ROPE_ERR_CUDA; errors that happen while the work runs surface at
 * the caller's next synchronisation, as with any CUDA launch.
 */
#ifndef ROPE_GB300_H_
#define ROPE_GB300_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ROPE_ABI_VERSION 4

typedef enum {
  ROPE_F32 = 0,  /* IEEE binary32 */
  ROPE_F16 = 1,  /* IEEE binary16 */
  ROPE_BF16 = 2, /* bfloat16 */
  ROPE_I64 = 3,  /* int64 (positions, slots, page numbers and the like) */
  ROPE_F8E4M3 = 4, /* 8-bit codes of a cache: sign, 4 exponent bits of bias 7, 3 of the fraction; 0x7f is NaN, no infinity */
  ROPE_E8M0 = 5,   /* scales of a cache of codes: byte b is 2^(b - 127), 255 is NaN; 0 here stands for 0 */
  ROPE_I32 = 6,    /* int32 (counts of holders of a page) */
  ROPE_U8 = 7      /* bytes of any meaning (rope_copy_pages) */
} rope_dtype_t;

/* A borrowed, contiguous, row-major device tensor of 1 to 4 dimensions. */
typedef struct {
  void* data;       /* device pointer; may be NULL only if the tensor is empty */
  int32_t dtype;    /* a rope_dtype_t value */
  int32_t ndim;     /* 1..4 */
  int64_t shape[4]; /* shape[i] for i < ndim; entries past ndim are ignored */
} rope_tensor_t;

enum {
  ROPE_OK = 0,
  ROPE_ERR_PARAM_NULLPTR = 161001, /* a required tensor (or its data) is NULL */
  ROPE_ERR_PARAM_INVALID = 161002, /* dtype, shape, slice, mode or alignment not supported */
  ROPE_ERR_CUDA = 561000           /* the CUDA runtime refused a call (launch or query) */
};

/* Codes reported by rope_get_device_error. */
enum {
  ROPE_DEVICE_OK = 0,
  ROPE_DEVICE_POSITION_OUT_OF_RANGE = 1, /* some position was < 0 or >= maxSeqLen */
  ROPE_DEVICE_SLOT_OUT_OF_RANGE = 2,     /* some KV-cache slot was >= blocks * block size, some page of a block
                                            table was outside the cache, or a sequence longer than its pages */
  ROPE_DEVICE_INDEX_OUT_OF_BOUNDS = 4,   /* bounds-checking builds only: a kernel formed an address
                                            outside the tensor it addresses (the access was skipped) */
  ROPE_DEVICE_PAGES_EXHAUSTED = 16,      /* rope_rearrange_sequences found fewer free pages than were asked for */
  ROPE_DEVICE_WAIT_EXPIRED = 8           /* a wait inside a kernel ran out (results are not valid); a defect of
                                            the library, never caused by the values of a tensor */
};

/*
 * In-place partial RoPE (interleave or half mode).
 * [IPRM §计算原理与公式, §partial_slice 局部旋转机制, §约束说明, §返回值与错误码]
 *
 * For every row r = (b, s, n) of x and every pair of the slice -- slot j and its
 * partner j', with j = start + 2p, j' = j + 1 in interleave mode (rotary_mode 1)
 * and j = start + i, j' = j + L/2 in half mode (rotary_mode 0) --
 *     x[r, j]  <- x[r, j]  * cos[r', j - start]  - x[r, j'] * sin[r', j - start]
 *     x[r, j'] <- x[r, j'] * cos[r', j' - start] + x[r, j]  * sin[r', j' - start]
 * (the page's  x = x*cos + x_rotate*sin  with x_rotate built from the negated
 * partners; interleave is the mode the page opens, half -- rotate_half over the
 * slice -- is the mode it declares), where r' is r broadcast into cos/sin's
 * [cB, cS, cN] dims.  Columns outside [start, end) are never read or written.
 *
 *   x            [B, S, N, D]; F32, F16 or BF16; D even, D <= 1024.  Rewritten in place.
 *   cos, sin     [cB, cS, cN, L] with L = end - start; each of cB, cS, cN is 1 or
 *                equal to x's B, S, N.  Same dtype as x, or F32 when x is F16/BF16
 *                (computed in binary32, the page's mixed-precision combination).
 *   rotary_mode  1 (interleave) or 0 (half); other values are rejected.
 *   start, end   the slice [start, end) of the D axis.  [0, 0] means the whole axis;
 *                any other start == end is a no-op that enqueues nothing.
 *                0 <= start <= end <= D, and end - start even.
 *   stream       a cudaStream_t (NULL: the legacy default stream).
 *
 * Returns ROPE_OK, ROPE_ERR_PARAM_NULLPTR, ROPE_ERR_PARAM_INVALID or ROPE_ERR_CUDA.
 * An empty x (some dim 0) is ROPE_OK and enqueues nothing.
 * Any element alignment is accepted.  Throughput: with 16-byte-aligned pointers
 * and a slice whose start and length are multiples of 16 bytes the kernel moves
 * 16-byte vectors; a slice that starts on a 128-byte boundary of the row touches
 * no more DRAM lines than it rotates, one that does not also fetches the line
 * holding its tail (about twice the DRAM reads for a 128-byte slice).
 */
int rope_inplace_partial(const rope_tensor_t* x, const rope_tensor_t* cos, const rope_tensor_t* sin,
                         int64_t rotary_mode, int64_t start, int64_t end, void* stream);

/*
 * Backward of rope_inplace_partial with respect to x, in place.
 * [IPRM §Python 接口与自动微分: the backward op computes the gradient of x only
 *  (cos/sin get none) and is a no-op for empty tensors and empty slices]
 *
 * `grad` holds dL/dy on entry and dL/dx on return.  Per pair (j, j') as above:
 *     grad[r, j]  <- grad[r, j]  * cos[r', j - start]  + grad[r, j'] * sin[r', j' - start]
 *     grad[r, j'] <- grad[r, j'] * cos[r', j' - start] - grad[r, j]  * sin[r', j - start]
 * i.e. the transpose of the forward map (for a true rotation, the inverse
 * rotation).  Arguments, checks and status values are those of
 * rope_inplace_partial, with `grad` in the place of x.
 */
int rope_inplace_partial_backward(const rope_tensor_t* grad, const rope_tensor_t* cos, const rope_tensor_t* sin,
                                  int64_t rotary_mode, int64_t start, int64_t end, void* stream);

/*
 * Cache-indexed RoPE of query and key, in place.
 * [RSCC §设计动机 (the three steps), §mrope 模式, §rope 模式, §rotate_half（GPT-NeoX style）,
 *  §rotate_interleaved（GPT-J style）, §约束说明, §入参校验逻辑]
 *
 * Per token t: gather cosSin = cache[positions[t]] (mrope: one row per positions
 * row), split it into cos = cosSin[:R/2] and sin = cosSin[R/2:] (mrope: index i
 * of cos and sin comes from the row of the section holding i), then rotate the
 * first R = rotary_dim columns of every head of query and key:
 *   NeoX (is_neox != 0), i < R/2:
 *     o[i] = x[i]*cos[i] - x[i+R/2]*sin[i];   o[i+R/2] = x[i+R/2]*cos[i] + x[i]*sin[i]
 *   GPT-J (is_neox == 0), i < R/2:
 *     o[2i] = x[2i]*cos[i] - x[2i+1]*sin[i];  o[2i+1] = x[2i+1]*cos[i] + x[2i]*sin[i]
 * Columns [R, head_size) of every head pass through: never read or written.
 *
 *   positions      I64; [numTokens] (rope) or [m, numTokens] (mrope, m = mrope_section_len).
 *                  8-byte aligned.
 *   query, key     2-D [numTokens, numQHeads*head_size] / [numTokens, numKHeads*head_size],
 *                  non-empty, same dtype (F32, F16 or BF16), 16-byte aligned.  Rewritten in
 *                  place (the page's queryOut/keyOut alias queryIn/keyIn).
 *   cos_sin_cache  2-D [maxSeqLen, R], same dtype as query, 16-byte aligned.
 *   head_size      a multiple of 32 (F16/BF16) or 16 (F32), dividing both row widths.
 *   rotary_dim     R; must equal cos_sin_cache.shape[1]; R <= head_size and a multiple of
 *                  32 (F16/BF16) or 16 (F32); at most 2048 (F16/BF16 NeoX), 1024 (F16/BF16
 *                  GPT-J, F32 NeoX) or 512 (F32 GPT-J).
 *   is_neox        nonzero: GPT-NeoX rotate_half; zero: GPT-J rotate_interleaved.
 *   mrope_section  HOST pointer to mrope_section_len int64 values, or NULL for rope mode.
 *                  mrope is on when the pointer is non-NULL and mrope_section[0] > 0;
 *                  then mrope_section_len is 3 or 4, every value >= 0, and
 *                  2 * sum == R.  A non-NULL section whose first value is 0 means rope.
 *   stream         a cudaStream_t (NULL: the legacy default stream).
 *
 * Positions outside [0, maxSeqLen) cannot be checked on the host: a token with such a
 * position is left untouched and ROPE_DEVICE_POSITION_OUT_OF_RANGE is recorded for
 * rope_get_device_error.
 *
 * Returns ROPE_OK, ROPE_ERR_PARAM_NULLPTR, ROPE_ERR_PARAM_INVALID or ROPE_ERR_CUDA.
 */
int rope_with_sin_cos_cache(const rope_tensor_t* positions, const rope_tensor_t* query,
                            const rope_tensor_t* key, const rope_tensor_t* cos_sin_cache,
                            int64_t head_size, int64_t rotary_dim, int32_t is_neox,
                            const int64_t* mrope_section, int64_t mrope_section_len, void* stream);

/*
 * Cache-indexed RoPE, V2 form: the V1 operation plus the interleaved mrope
 * splice, strided inputs and separate outputs.
 * [RSCC §V2 接口：cacheMode 扩展; §算子定义与属性 (qStride/kStride: row strides of
 *  query/key for non-contiguous inputs); §接口原型 (queryOut/keyOut)]
 *
 *   cache_mode        0: the sections are spliced in order, as in V1.
 *                     1: interleaved splice (three-section mrope only): cos and sin
 *                     start as the position row 0 values; indices i < 3*mrope_section[1]
 *                     with i % 3 == 1 take row 1, with i % 3 == 2 take row 2.
 *   query_row_stride  elements between the starts of consecutive query rows (0: the row
 *   key_row_stride    width, i.e. contiguous).  At least the row width, and a multiple of
 *                     16 bytes, so that query/key may be views into a fused QKV buffer.
 *   query_out,        NULL, NULL: rotate in place (only the first R columns of each head
 *   key_out           are written).  Otherwise contiguous [numTokens, ...] tensors of the
 *                     inputs' logical shape and dtype, 16-byte aligned, that receive the
 *                     whole rows: rotated columns and pass-through columns copied.  An
 *                     output equal to its input (same pointer, contiguous rows) means in
 *                     place; any other overlap of outputs with inputs is rejected.  Tokens
 *                     with an out-of-range position leave their output rows unwritten.
 *
 * Every other argument, check and status value is that of rope_with_sin_cos_cache.
 */
int rope_with_sin_cos_cache_v2(const rope_tensor_t* positions, const rope_tensor_t* query,
                               const rope_tensor_t* key, const rope_tensor_t* cos_sin_cache,
                               int64_t head_size, int64_t rotary_dim, int32_t is_neox,
                               const int64_t* mrope_section, int64_t mrope_section_len, int32_t cache_mode,
                               int64_t query_row_stride, int64_t key_row_stride, const rope_tensor_t* query_out,
                               const rope_tensor_t* key_out, void* stream);

/*
 * Fused QKV split + RMSNorm + RoPE + paged KV-cache write.
 * ["aclnnQkvRmsNormRopeCacheWithKScale" page, section 计算公式; its FP8
 *  quantisation and optional rotation matmul are not part of this call]
 *
 * Per token t of batch b (t in [query_start_loc[b], query_start_loc[b+1])):
 *   position = seq_lens[b] - (query_start_loc[b+1] - query_start_loc[b]) + (t - query_start_loc[b])
 *   cos, sin = the two halves of cos_sin_cache[position]
 *   for each of the Nq + Nk + Nv heads x of qkv[t] (D elements each):
 *     q and k heads:  y = x / sqrt(mean(x^2) + eps) * gamma   (q_gamma or k_gamma)
 *                     r = concat(y_lo*cos - y_hi*sin, y_hi*cos + y_lo*sin)
 *     q_out[t, h] = r;  k_cache[slot/BS, h, slot%BS, :] = r;  v_cache[slot/BS, h, slot%BS, :] = x (v heads)
 *   with slot = slot_mapping[t] and BS the cache block size.
 *
 *   qkv            [T, (Nq + Nk + Nv) * D]; F32, F16 or BF16; D a multiple of 32 (F16/BF16)
 *                  or 16 (F32), at most 512 (F16/BF16) or 256 (F32).
 *   q_gamma, k_gamma  [D], same dtype.      eps >= 0 (added to the mean of squares).
 *   cos_sin_cache  [maxSeq, D], same dtype: cos in the first half of a row, sin in the second.
 *   seq_lens       I64 [B]: tokens of each sequence including this call's; 1 <= B <= 2^30;
 *   query_start_loc I64 [B + 1]: first token of each batch in qkv, non-decreasing, from 0
 *                  to T (a batch may be empty).  Other values cannot make the kernel
 *                  access memory outside the tensors, but which batch a token is given
 *                  to is then unspecified;
 *   slot_mapping   I64 [T]: cache slot of each token; a negative slot writes no cache
 *                  (padding).
 *   q_out          [T, Nq * D] output; k_cache [NB, Nk, BS, D] and v_cache [NB, Nv, BS, D]
 *                  are updated in place at the tokens' slots only.  Nq + Nk + Nv and BS
 *                  are at most 2^30.
 * All float tensors 16-byte aligned, int64 tensors 8-byte aligned, all contiguous.
 * Computed in binary32 and rounded once per output element: the mean of squares, the
 * reciprocal square root, and the rotation with gamma folded into cos/sin,
 *   r_lo = (x_lo*(g_lo*cos) - x_hi*(g_hi*sin)) / rms,  r_hi = (x_hi*(g_hi*cos) + x_lo*(g_lo*sin)) / rms,
 * each a product, an FMA and the scaling (the terms already carry one rounding of
 * the normalisation, so the compensated difference of rope_with_sin_cos_cache would
 * not make the result more accurate).
 * A token whose position falls outside the table writes nothing and records
 * ROPE_DEVICE_POSITION_OUT_OF_RANGE; a slot at or past NB * BS writes no cache and
 * records ROPE_DEVICE_SLOT_OUT_OF_RANGE (q_out is still written).
 * Returns ROPE_OK, ROPE_ERR_PARAM_NULLPTR, ROPE_ERR_PARAM_INVALID or ROPE_ERR_CUDA.
 */
int rope_qkv_rmsnorm_rope_cache(const rope_tensor_t* qkv, int64_t num_q_heads, int64_t num_k_heads,
                                int64_t num_v_heads, const rope_tensor_t* q_gamma, const rope_tensor_t* k_gamma,
                                float eps, const rope_tensor_t* cos_sin_cache, const rope_tensor_t* seq_lens,
                                const rope_tensor_t* query_start_loc, const rope_tensor_t* slot_mapping,
                                const rope_tensor_t* q_out, const rope_tensor_t* k_cache,
                                const rope_tensor_t* v_cache, void* stream);

/*
 * Rotary frequencies scaled for long contexts (host arithmetic in binary64; no GPU).
 *
 * inv_freq[i] = base^(-2i/R) for i < F = R/2, changed by `scaling` (NULL: not at all):
 *   ROPE_SCALING_LINEAR      inv_freq[i] / factor
 *   ROPE_SCALING_BASE        base * factor^(R/(R-2)) in the place of base (R > 2; > 0, finite)
 *   ROPE_SCALING_YARN        mixed between inv_freq[i] and inv_freq[i] / factor along a ramp in i: with
 *                            i(n) = R/2 * ln(original_length / (2 pi n)) / ln(base), the index whose wave
 *                            makes n turns over the original length, the ramp goes from 0 (kept) at
 *                            max(0, floor(i(high))) to 1 (divided) at min(R - 1, ceil(i(low))); a ramp of no
 *                            width is 0.001 wide.  low and high are turns (0: 1 and 32).  base > 1.
 *   ROPE_SCALING_WAVELENGTH  with t = original_length * inv_freq[i] / (2 pi) turns over the original length:
 *                            kept where t >= high, divided by factor where t <= low, in between
 *                            inv_freq[i] * s + inv_freq[i] / factor * (1 - s), s = (t - low) / (high - low).
 *                            low < high.
 *   ROPE_SCALING_FACTORS     inv_freq[i] / factors[i]
 * *scale receives the factor of cos and sin: scaling->attention where that is > 0, else
 * 1 + 0.1 * ln(factor) for ROPE_SCALING_YARN with factor > 1, else 1.
 *
 *   rotary_dim  R: even, 2 to 2048.        base > 0, finite.
 *   factor > 0, original_length > 0 and factors (F values > 0) where the kind uses them.
 * Returns ROPE_OK, ROPE_ERR_PARAM_NULLPTR or ROPE_ERR_PARAM_INVALID.
 */
enum {
  ROPE_SCALING_NONE = 0,
  ROPE_SCALING_LINEAR = 1,
  ROPE_SCALING_BASE = 2,
  ROPE_SCALING_YARN = 3,
  ROPE_SCALING_WAVELENGTH = 4,
  ROPE_SCALING_FACTORS = 5
};

typedef struct {
  int32_t kind;           /* a ROPE_SCALING_* value */
  double factor;          /* how far the context is stretched */
  double original_length; /* positions the unscaled frequencies were made for */
  double low, high;       /* turns over the original length at the ends of the mixed range */
  double attention;       /* factor of cos and sin; 0: the kind's own */
  const double* factors;  /* ROPE_SCALING_FACTORS: R/2 HOST values */
} rope_scaling_t;

int rope_scaled_frequencies(int64_t rotary_dim, double base, const rope_scaling_t* scaling, double* inv_freq,
                            double* scale);

/*
 * cos/sin rows for given frequencies, in the layout of the cache-indexed operators
 * (rope_scaled_cos_sin_cache) or of the in-place one (rope_scaled_cos_sin).
 *
 * Row r stands for position p = first_position + (positions ? positions[r] : r), and
 * i < F = num_freq:
 *   cache:                     cache[r, i] = scale * cos(p * inv_freq[i]);  cache[r, F + i] = scale * sin(...)
 *   rotary_mode 0 (half):      cos[r, i] = cos[r, F + i] = scale * cos(p * inv_freq[i]);       sin likewise
 *   rotary_mode 1 (interleave) cos[r, 2i] = cos[r, 2i + 1] = scale * cos(p * inv_freq[i]);     sin likewise
 *
 *   inv_freq   HOST pointer to F binary64 frequencies (radians per position), |value| <= 1e6.  Read
 *              before the call returns.       1 <= F <= 1024.  scale: finite, rounded to binary32.
 *   positions  I64 device tensor of as many elements as there are rows, or NULL.
 *   cache      [rows, 2F] (or more leading dims); cos, sin: one shape, last dim 2F, e.g. [1, S, 1, 2F]
 *              for the in-place operator.  F32, F16 or BF16.  Element alignment; 16-byte-aligned
 *              tensors with F a multiple of 8 (F32: 4) are written in 16-byte pieces.
 *
 * The angle is kept as a 64-bit fraction of a turn: p * (inv_freq / 2 pi mod 1) mod 1 is exact in
 * integers for every int64 position but for the one rounding of inv_freq / 2 pi to 2^-64 turns (an
 * angle error of 2 pi p * 2^-65, 2e-13 at a million), so far positions are as exact as near ones.
 * sin and cos of the remainder are within 2 units in the last place in binary32, then scaled and rounded.
 * An empty output is ROPE_OK and enqueues nothing.  Outputs and positions must not share memory.
 * Returns ROPE_OK, ROPE_ERR_PARAM_NULLPTR, ROPE_ERR_PARAM_INVALID or ROPE_ERR_CUDA.
 */
int rope_scaled_cos_sin_cache(const double* inv_freq, int64_t num_freq, double scale, const rope_tensor_t* positions,
                              int64_t first_position, const rope_tensor_t* cache, void* stream);
int rope_scaled_cos_sin(const double* inv_freq, int64_t num_freq, double scale, const rope_tensor_t* positions,
                        int64_t first_position, int64_t rotary_mode, const rope_tensor_t* cos,
                        const rope_tensor_t* sin, void* stream);

/*
 * RoPE of query and key on the way to the query output and to a paged KV cache.
 *
 * The rotation of rope_with_sin_cos_cache_v2, and per token t with slot = slot_mapping[t] >= 0, BS the block size:
 *   query_out[t, h] = rotated query head
 *   k_cache[slot/BS, h, slot%BS, :] = rotated key head;  v_cache[slot/BS, h, slot%BS, :] = value head (copied)
 * The layout of the caches and the meaning of slots are those of rope_qkv_rmsnorm_rope_cache.
 *
 *   positions, cos_sin_cache, head_size, rotary_dim, is_neox, mrope_section, cache_mode: as in
 *                  rope_with_sin_cos_cache_v2, except that cos_sin_cache may also be F32 with F16/BF16
 *                  data (computed in binary32), and at most 1024 (F32) or 2048 for head_size.
 *   query          [T, numQHeads*head_size] or NULL (keys and values only).
 *   key, value     [T, numKHeads*head_size], [T, numVHeads*head_size]: same dtype as query.  Never written.
 *   *_row_stride   elements between the starts of consecutive rows (0: contiguous), at least the row
 *                  width, a multiple of 16 bytes: query, key and value may be column ranges of one buffer.
 *   slot_mapping   I64 [T]; a negative slot writes no cache (padding).  The slots of one call that are >= 0
 *                  are distinct: where two tokens name one slot, each 16-byte piece of it is one token's.
 *   query_out      contiguous [T, numQHeads*head_size]; NULL (or equal to a contiguous query): query is
 *                  rotated in place.  NULL without a query.
 *   k_cache, v_cache  [NB, numKHeads, BS, head_size], [NB, numVHeads, BS, head_size]: written at the slots
 *                  of this call only.
 * Float tensors 16-byte aligned, int64 tensors 8-byte aligned.  T == 0 is ROPE_OK and enqueues nothing.
 * A tensor the call writes shares no memory with any other of the call.
 * Each rotated element is rounded once: one FMA after an exact product where data and table are both
 * 16-bit, else the compensated difference of products.  A token with a position outside the table writes
 * nothing and records ROPE_DEVICE_POSITION_OUT_OF_RANGE; a slot at or past NB * BS writes no cache and
 * records ROPE_DEVICE_SLOT_OUT_OF_RANGE (query_out is still written).
 * Returns ROPE_OK, ROPE_ERR_PARAM_NULLPTR, ROPE_ERR_PARAM_INVALID or ROPE_ERR_CUDA.
 */
int rope_append_paged_kv(const rope_tensor_t* positions, const rope_tensor_t* query, const rope_tensor_t* key,
                         const rope_tensor_t* value, const rope_tensor_t* cos_sin_cache,
                         const rope_tensor_t* slot_mapping, const rope_tensor_t* query_out,
                         const rope_tensor_t* k_cache, const rope_tensor_t* v_cache, int64_t head_size,
                         int64_t rotary_dim, int32_t is_neox, const int64_t* mrope_section,
                         int64_t mrope_section_len, int32_t cache_mode, int64_t query_row_stride,
                         int64_t key_row_stride, int64_t value_row_stride, void* stream);

/*
 * Causal attention of a batch's new tokens over the paged KV cache, with an optional prefix that every
 * sequence shares.
 *
 * Token t of sequence b (query_start_loc[b] <= t < query_start_loc[b+1]) has position
 *   p = seq_lens[b] - (query_start_loc[b+1] - query_start_loc[b]) + (t - query_start_loc[b])
 * and sees the keys j <= p.  Key j sits in row j % BS of page prefix_blocks[j / BS] when j < prefix_len, else
 * in row (j - prefix_len) % BS of page block_table[b, (j - prefix_len) / BS].  Per query head h, with key head
 * g = h / (Nq / Nk):
 *   s_j = scale * <query[t, h], k_j[g]>;  out[t, h] = sum_j e^(s_j - lse) v_j[g];  lse[t, h] = ln(sum_j e^(s_j))
 * A row that sees no key gives out 0 and lse -infinity.  Keys and values that a row does not see have no
 * influence on it, NaN and infinities among them, nor have the rows of a page past a sequence's end.
 * Rows at or past query_start_loc[B] are left as they were.
 *
 * The keys and values of this call's own tokens are in the cache before the call
 * (rope_append_paged_kv, rope_qkv_rmsnorm_rope_cache).
 *
 *   query            [T, Nq*D], rows query_row_stride elements apart (0: contiguous; a multiple of 16 bytes);
 *                    F32, F16 or BF16; D a multiple of 32 (F16/BF16) or 16 (F32), at most 512;
 *                    Nq at most 65536, T * Nq below 2^31 - 512.
 *   k_cache, v_cache [NB, Nk, BS, D], same dtype; Nq a multiple of Nk.
 *   block_table      I64 [B, W]: pages of each sequence's own tokens; B >= 1, W >= 1, W * BS <= 2^30.
 *   seq_lens         I64 [B]: tokens of each sequence, prefix and this call's included.  Not negative.
 *   query_start_loc  I64 [B + 1], non-decreasing from 0 to at most T (a sequence may be empty).  Other values
 *                    cannot make the kernels access memory outside the tensors; which sequence a token
 *                    belongs to, and whether it is written, is then unspecified.
 *   prefix_blocks    I64, at least ceil(prefix_len / BS) pages, or NULL with prefix_len 0.
 *   prefix_len       0 to 2^30; prefix_len + W * BS below 2^31 - 512.
 *   scale            > 0 and finite.
 *   out              contiguous [T, Nq*D], query's dtype.      lse  F32 [T, Nq], or NULL.
 *   workspace        DEVICE pointer to workspace_bytes bytes, 256-byte aligned, at least what
 *                    rope_paged_attention_workspace says.  Used by this call only until its work is done;
 *                    its contents before and after mean nothing, and calls whose work may run at the same
 *                    time need workspaces of their own.
 *   stream           a cudaStream_t (NULL: the legacy default stream).
 * Float tensors 16-byte aligned (lse 4), int64 tensors 8-byte aligned.  T == 0 is ROPE_OK and enqueues nothing.
 * out, lse and the workspace share no memory with any other tensor of the call.
 *
 * Arithmetic: scores, softmax statistics and sums are binary32 (one running maximum and sum per row; partial
 * results over key ranges are joined in a fixed order, so results are deterministic).  With F16/BF16 data the
 * products run on the tensor cores, and the softmax weights e^(s_j - m) are rounded to the data's type before
 * the product with V: at most half a unit in the last place each, F16 weights below 2^-25 of the row's largest
 * by 2^-36 of it at most.  out is rounded once.
 * The products <query, k> are taken before scale and have to stay within binary32.  Where they do not (F32 and
 * BF16 reach that far): a row with a product of +infinity, or with none but of -infinity, is computed again with
 * the query scaled first; in other rows a key whose product is -infinity has weight 0.  A row of scores that are all
 * -infinity gives out 0 and lse -infinity.
 * Speed: W * BS stands for the number of keys a sequence can have where the kernels are chosen and where a launch
 * can be saved, so a block_table as narrow as the batch allows is the fastest (22 sequences of 1 or 2 tokens: 6.8 us,
 * with a table for long ones 8.2).  A row whose result is not finite, because a query, key or value that it sees is
 * not or a product leaves binary32, is computed again one key at a time, as all rows of heads over 256 are: about
 * 1 us a key for heads of 128, so that one such row of 8192 keys makes a call of 178 us one of 10 ms.
 * A page outside [0, NB), and tokens of a sequence past the W pages it has, are keys that no row sees; both
 * record ROPE_DEVICE_SLOT_OUT_OF_RANGE.
 * Returns ROPE_OK, ROPE_ERR_PARAM_NULLPTR, ROPE_ERR_PARAM_INVALID or ROPE_ERR_CUDA.
 */
int rope_paged_attention(const rope_tensor_t* query, int64_t query_row_stride, const rope_tensor_t* k_cache,
                         const rope_tensor_t* v_cache, const rope_tensor_t* block_table,
                         const rope_tensor_t* seq_lens, const rope_tensor_t* query_start_loc,
                         const rope_tensor_t* prefix_blocks, int64_t prefix_len, float scale,
                         const rope_tensor_t* out, const rope_tensor_t* lse, void* workspace,
                         int64_t workspace_bytes, void* stream);

/*
 * Bytes of workspace that rope_paged_attention needs on the current device for num_tokens query rows of
 * num_q_heads heads of head_size (a rope_dtype_t type), whatever the batch.  *bytes >= 256.  Without a prefix tens
 * of MB at most and 8 bytes a row; with one two binary32 results more (num_tokens * num_q_heads * (head_size + 2) *
 * 8 bytes: 2.2 GB for 65536 tokens of 32 heads of 128), which calls use where the prefix has a launch of its own.
 */
int rope_paged_attention_workspace(int64_t num_tokens, int64_t num_q_heads, int64_t num_k_heads, int64_t head_size,
                                   int32_t dtype, int64_t prefix_len, int64_t* bytes);

/*
 * RoPE of query and key on the way to the query output and to a paged KV cache of 8-bit codes.
 *
 * A cached value is code * 2^(b - 127), b being the scale byte of its block: the BS / S tokens of a page (S scale
 * blocks a page) of one head; b = 0 is a block of zeros, 255 is NaN.  The rotation is rope_append_paged_kv's; keys are
 * rotated with two roundings to binary32 an element (a code's step is 2^20 times as large), not to their type.  Then for
 * every scale block that the call writes, of the keys and of the values,
 *   most = max |x| over its values written that are finite;  e = the least integer with most <= 448 * 2^e
 *   byte = e + 127, from 1 to 254;  0 where most = 0
 * and where tokens stand in the block before the first one written: no less than the byte that was there, and where it
 * grew their codes become the nearest (ties to even) of code * 2^(old - new).  Written codes are the nearest of
 * x * 2^-e; a value that is not finite becomes NaN.  So a value is off by 2^-4 of itself at most, and by 2^(e - 10) where
 * that is more, once; the codes of tokens before are re-encoded exactly, but where 2^(old - new) makes them subnormal.
 *
 *   All arguments as in rope_append_paged_kv, and
 *   k_cache, v_cache  ROPE_F8E4M3 [NB, numKHeads, BS, head_size], [NB, numVHeads, BS, head_size].  head_size at most 512.
 *   k_scale, v_scale  ROPE_E8M0 [NB, numKHeads, S], [NB, numVHeads, S]; S divides BS.  Scales of blocks whose first
 *                     token the call writes need not be initialised.
 *   slot_mapping      The tokens of one scale block stand one after the other in the call, in the order of their slots
 *                     (tokens of a sequence in order do), and what a block holds before the first of them is kept.  Where
 *                     a call brings tokens to a block in more than one such run, the block's content is unspecified.
 *                     Rows of a block behind the last token written are not re-encoded.
 * Results, refusals and device errors otherwise as rope_append_paged_kv's.  Many tokens cost more than there (16384, 32 q,
 * 8 k and 8 v heads of 128: 84 us, 64.5): keys are rotated for the largest value and again for the codes.
 */
int rope_append_paged_kv_8bit(const rope_tensor_t* positions, const rope_tensor_t* query, const rope_tensor_t* key,
                              const rope_tensor_t* value, const rope_tensor_t* cos_sin_cache,
                              const rope_tensor_t* slot_mapping, const rope_tensor_t* query_out,
                              const rope_tensor_t* k_cache, const rope_tensor_t* v_cache,
                              const rope_tensor_t* k_scale, const rope_tensor_t* v_scale, int64_t head_size,
                              int64_t rotary_dim, int32_t is_neox, const int64_t* mrope_section,
                              int64_t mrope_section_len, int32_t cache_mode, int64_t query_row_stride,
                              int64_t key_row_stride, int64_t value_row_stride, void* stream);

/*
 * rope_paged_attention over a cache of codes (see rope_append_paged_kv_8bit): keys and values are code * 2^(b - 127).
 *
 *   All arguments as in rope_paged_attention (query and out F32, F16 or BF16), and
 *   k_cache, v_cache  ROPE_F8E4M3 [NB, Nk, BS, D].
 *   k_scale, v_scale  ROPE_E8M0 [NB, Nk, S]; S divides BS.
 *   workspace_bytes   at least what rope_paged_attention_8bit_workspace says.
 *
 * Arithmetic: as rope_paged_attention's, scores, statistics and sums in binary32.  The products run on the tensor cores
 * with binary16 operands, which hold codes exactly; scales come in as powers of two.  BF16 and F32 queries are taken
 * times a power of two that brings a row's largest element (where that is not below 2^-102) to about 2^8: BF16 exact
 * down to 2^-22 of it, off by 2^-33 of it below; F32 as a sum of two binary16 values, off by 2^-23 of an element or
 * 2^-33 of the largest.  Softmax weights are rounded to binary16, with F32 queries to the sum of two, together with V's
 * scale: with weights relative to the row's largest, and of a key whose V has 2^-n of the largest scale of V that the
 * row's part of the keys has had so far (a key that the row does not see among them), off by half a step, below
 * 2^(n - 29) by 2^(n - 40) at most, and never by more than the weight.  In calls with more than 16 rows a sequence and
 * key head the limits are 2^(n - 25) and 2^(n - 36), n being that of the largest of 32 keys that follow each other.
 * Scales that lie far apart leave binary16: rows that see such keys are computed again one key at a time, as rows are
 * whose result is not finite (about 1 us a key).  A row meets that where n is more than 15 for a key of more than 2^-30
 * of the largest weight (of less: weight 0); in calls with more than 16 rows a sequence and key head where it is more
 * than 10 for the largest scale of V of 32 keys that follow each other, and where among 32 such keys, some of which
 * the row sees, one's scale of K or V is below 2^-15 of the largest.  Blocks of zeros with the byte 0 count nowhere.
 * It meets it, too, where the scale of V grows beyond 2^90 of the first that the row's part of the keys had.
 * Speed: made for decoding, where the cache's bytes bound the call.  With more than 16 rows a sequence and key head the
 * codes are widened on the way, which costs more than their bytes save: 4 chunks of 1984 tokens behind 4096 take
 * 807 us, with rope_paged_attention over BF16 500.
 */
int rope_paged_attention_8bit(const rope_tensor_t* query, int64_t query_row_stride, const rope_tensor_t* k_cache,
                              const rope_tensor_t* v_cache, const rope_tensor_t* k_scale,
                              const rope_tensor_t* v_scale, const rope_tensor_t* block_table,
                              const rope_tensor_t* seq_lens, const rope_tensor_t* query_start_loc,
                              const rope_tensor_t* prefix_blocks, int64_t prefix_len, float scale,
                              const rope_tensor_t* out, const rope_tensor_t* lse, void* workspace,
                              int64_t workspace_bytes, void* stream);
int rope_paged_attention_8bit_workspace(int64_t num_tokens, int64_t num_q_heads, int64_t num_k_heads,
                                        int64_t head_size, int32_t dtype, int64_t prefix_len, int64_t* bytes);

/*
 * New sequences of old ones: forks (samples, beams), reordering, dropping, and room for what comes.
 *
 * Sequence b of the old batch has seq_lens[b] tokens, prefix_len of them in pages that all share and that stay out of
 * the tables, the others in the pages block_table[b, 0 ...], BS tokens a page.  ref_counts[page] says how many tables'
 * entries hold a page (and whoever else the program counts, a shared prefix say); 0 is a free page.
 * Row i of the new batch has the tokens of old row p = parents[i] (p < 0: only the prefix), and room for room[i] more:
 *   all old rows let go of their pages; a page that nobody then holds is free, with what follows taken into account;
 *   row i holds the whole pages of p;
 *   if p's last page is not full, the first row i that asks for it keeps it, provided nobody else holds it then; any other
 *   gets a fresh page, and (that page, the fresh one) is a pair of pages to be copied before the cache is written;
 *   fresh pages follow until the row has room: free pages are given out lowest first, rows in order.
 * copy_src and copy_dst receive the pairs in the order of rows, then -1.  counts[0] is their number, counts[1] how many
 * pages are free then.  new_seq_lens[i] = seq_lens[p] + room[i], also where sequence p ends within the prefix or is
 * empty (a row of a padded batch): room is first what is left of the prefix then.  Entries of the new table behind a
 * row's pages are left as they were.  With rope_copy_pages over every layer's caches the new batch is ready to be
 * written and read.
 * Where pages run out, the entries are -1 from there on, a pair's copy_dst too, and ROPE_DEVICE_PAGES_EXHAUSTED is
 * recorded.  A page number outside [0, NB), more tokens than a row's pages hold, and p >= B record
 * ROPE_DEVICE_SLOT_OUT_OF_RANGE; such pages are passed over, tokens past the table dropped, such a p is none.
 * A row's pages are those of its seq_lens.  A program that cuts a sequence short (drafted tokens that were refused) lets
 * go of pages that are then behind its end by itself, in ref_counts.
 *
 *   block_table I64 [B, W], new_block_table I64 [rows, new W]; seq_lens I64 [B]; parents, room (or NULL), new_seq_lens,
 *   copy_src, copy_dst I64 [rows], rows at most 8192; ref_counts, new_ref_counts I32 [NB], which may be one tensor;
 *   counts I64 [2].  W * BS, new W * BS, rows * new W, B and NB at most 2^30, W and new W below it.  B and rows may be 0.
 * What is written shares no memory with any other tensor of the call, new_ref_counts in the place of ref_counts apart.
 * Whole numbers: results are the same whatever the order in which threads run.
 */
int rope_rearrange_sequences(const rope_tensor_t* block_table, const rope_tensor_t* seq_lens,
                             const rope_tensor_t* ref_counts, const rope_tensor_t* parents, const rope_tensor_t* room,
                             const rope_tensor_t* new_block_table, const rope_tensor_t* new_seq_lens,
                             const rope_tensor_t* new_ref_counts, const rope_tensor_t* copy_src,
                             const rope_tensor_t* copy_dst, const rope_tensor_t* counts, int64_t block_size,
                             int64_t prefix_len, void* stream);

/*
 * Live pages to the front: with L pages held (ref_counts > 0), the k-th held page at or behind L goes to the k-th free
 * page before L, so that pages [L, NB) are free.  copy_src and copy_dst receive the moves, ascending, then -1;
 * counts[0] is their number, counts[1] is L.  Tables, prefix and counts follow; the pages themselves are moved by
 * rope_copy_pages.  Table entries behind a row's pages are left as they were.
 *
 *   block_table, new_block_table I64 [B, W]; seq_lens I64 [B]; ref_counts, new_ref_counts I32 [NB]; prefix_blocks,
 *   new_prefix_blocks I64, at least ceil(prefix_len / BS) pages (NULL with prefix_len 0); copy_src, copy_dst I64 [pairs],
 *   pairs at least NB / 2; counts I64 [2].  Each new tensor may be the old one.  Limits as rope_rearrange_sequences'.
 * An entry outside [0, NB), or of a page that ref_counts calls free, is copied as it is and records
 * ROPE_DEVICE_SLOT_OUT_OF_RANGE, as more tokens than a row's pages hold do.
 */
int rope_compact_pages(const rope_tensor_t* block_table, const rope_tensor_t* seq_lens,
                       const rope_tensor_t* ref_counts, const rope_tensor_t* prefix_blocks,
                       const rope_tensor_t* new_block_table, const rope_tensor_t* new_ref_counts,
                       const rope_tensor_t* new_prefix_blocks, const rope_tensor_t* copy_src,
                       const rope_tensor_t* copy_dst, const rope_tensor_t* counts, int64_t block_size,
                       int64_t prefix_len, void* stream);

/*
 * Page src[i] of every tensor to its page dst[i], i < count[0] (count NULL: all).  A pair with a negative number is passed
 * over; one outside [0, NB) too, and records ROPE_DEVICE_SLOT_OUT_OF_RANGE.
 *
 *   src, dst I64 [pairs]; count I64, at least one element.  A page that some pair writes is not of another pair of the
 *   call: where it is, each 16 bytes of it are of one of the states that it has on the way.
 *   tensors  HOST array of num_tensors descriptors (read before the call returns) of any type and shape whose first
 *            dimension is NB, the same for all: caches and scales of any number of layers.  No two share memory.
 */
int rope_copy_pages(const rope_tensor_t* src, const rope_tensor_t* dst, const rope_tensor_t* count,
                    const rope_tensor_t* tensors, int64_t num_tensors, void* stream);

/*
 * Takes the device-side error word of the current device (an atomic exchange
 * with zero, enqueued on `stream`), then synchronises `stream`.  *code receives
 * ROPE_DEVICE_OK or a bitwise OR of the ROPE_DEVICE_* codes recorded since the
 * previous read.  The word is shared by every stream and every caller of this
 * process on that device: a read returns (and clears) bits that kernels on other
 * streams recorded too, and no bit is lost between two reads.  Enqueues one
 * one-thread kernel (counted by rope_launch_count).  Returns ROPE_OK,
 * ROPE_ERR_PARAM_NULLPTR (code is NULL) or ROPE_ERR_CUDA.
 */
int rope_get_device_error(void* stream, int32_t* code);

/* A static, human-readable name for a status value (never NULL). */
const char* rope_status_string(int status);

/* Number of kernels this library has launched in this process (all devices). */
uint64_t rope_launch_count(void);

/* ROPE_ABI_VERSION of the built library. */
int rope_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ROPE_GB300_H_ */
