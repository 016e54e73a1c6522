// Shared by the attention kernels: the argument block, the sequence of a token, and where a
// key of a sequence sits in the paged cache.
#pragma once

#include <cfloat>
#include <cmath>

#include "rope_device.cuh"
#include "serving.h"

namespace rope {
namespace attend {

constexpr unsigned kSlotOutOfRange = 2u;

struct AttendArgs {
  int64_t T, B;
  int64_t q_stride;
  int64_t num_blocks;
  int64_t W;            // pages of a block table row
  int32_t nq, nk, G;    // G = nq / nk query heads share a key head
  int32_t D;
  int32_t block_size, bs_shift;  // bs_shift: log2(block_size), or -1
  int32_t P;            // keys of the shared prefix
  float scale_log2;     // scale * log2(e)
  Span q_span, k_span, v_span, bt_span, sl_span, qsl_span, pb_span, out_span, lse_span;
};

struct Pointers {
  const int64_t* block_table;
  const int64_t* seq_lens;
  const int64_t* qsl;
  const int64_t* prefix_blocks;
  unsigned int* err;
};

// Batch of token t: the largest b in [0, B) with query_start_loc[b] <= t.
__device__ __forceinline__ int64_t batch_of(int64_t t, const Pointers& g, const AttendArgs& a) {
  int64_t l = 0, h = a.B - 1;
  while (l < h) {
    const int64_t mid = (l + h + 1) >> 1;
    if (ldg(g.qsl + mid, a.qsl_span, g.err) <= t) l = mid; else h = mid - 1;
  }
  return l;
}

__device__ __forceinline__ int page_of(int j, const AttendArgs& a) {
  return a.bs_shift >= 0 ? j >> a.bs_shift : j / a.block_size;
}

// Cache row (page * Nk * BS + row of the page; the head's rows are head * BS further) of key
// j < P of the prefix, or of own key j - P of the sequence whose block table row is `table`.
// -1 when the page is outside the cache or the sequence has no such page.
__device__ __forceinline__ int64_t key_row(int j, const int64_t* table, const Pointers& g, const AttendArgs& a) {
  int64_t page;
  int i;
  if (j < a.P) {
    i = page_of(j, a);
    j -= i * a.block_size;
    page = ldg(g.prefix_blocks + i, a.pb_span, g.err);
  } else {
    j -= a.P;
    i = page_of(j, a);
    if (i >= a.W) return -1;
    j -= i * a.block_size;
    page = ldg(table + i, a.bt_span, g.err);
  }
  if (page < 0 || page >= a.num_blocks) return -1;
  return page * a.nk * a.block_size + j;
}

// The page that holds key j, or -1 (see key_row), and the key's row within it.
struct PageRow {
  int64_t page;
  int32_t row;
};

__device__ __forceinline__ PageRow page_row(int j, const int64_t* table, const Pointers& g, const AttendArgs& a) {
  if (j < a.P) {
    const int i = page_of(j, a);
    return {ldg(g.prefix_blocks + i, a.pb_span, g.err), j - i * a.block_size};
  }
  j -= a.P;
  const int i = page_of(j, a);
  if (i >= a.W) return {-1, 0};
  return {ldg(table + i, a.bt_span, g.err), j - i * a.block_size};
}

// ---------------------------------------------------------------------------
// How the work is cut.  A unit is a tile of M query rows of one sequence and key head (row r
// of a sequence is token r / G, head r % G of the key head's group) with the keys they see;
// or, in the launch over a shared prefix, a tile of M rows of the whole batch with the
// prefix's keys.  A unit's work is its number of key tiles and Cut::cost.  All units' work,
// one after the other, is cut into equal shares, one per CTA of the grid: a unit may be finished by
// several CTAs; each leaves its rows' partial (m, l, O) in one of its two slots (slot 1: the
// unit begins in this CTA, slot 0: it began in an earlier one), and the joining kernel adds
// them up in order.  Every CTA finds its share by itself from the lengths on the device:
// the cut needs no host copy of them and no extra launch.
//
// A unit of up to whole_tiles() tiles is not split: the CTA in which it begins finishes it.  A
// split costs writing and reading M rows of binary32 twice, about 3 tiles' time for 256 rows (68
// sequences of 45 tokens on 219, 8 rows a key head: 56 us with every unit split where the shares
// end, 43 with 4 tiles kept whole) and less than one for 16 or 64 (2 sequences of 14 tokens in
// binary32: 25 us split, 40 us whole).
// ---------------------------------------------------------------------------
struct Cut {
  int32_t lo;         // first key of the launch: P when the prefix has its own launch, else 0
  int32_t prefix;     // this launch is over the shared prefix: units of the whole batch, keys [0, P)
  int32_t shared;     // another launch covers the other keys: nothing is final here
  int32_t slot_rows;  // rows of a partial slot
  int32_t grid;       // CTAs of the launch
  int32_t whole;      // units of up to so many tiles are not split
  int32_t cost;       // what a unit costs beside its key tiles, in tiles (see unit_cost)
  int32_t solo;       // no unit is split and no joining kernel follows: no records
  int2* rec;          // [T * nq]: first and last CTA of the row's unit (16 bits each) and the row's
                      // place in the unit
  float* slots;       // [grid][2][slot_rows][D] O, then [grid][2][slot_rows][2] m, l
  float* dense;       // shared: [T * nq][D] O, then [T * nq][2] m, l, of units that one CTA finished
};

// Rows and keys of one sequence (or of the whole batch).  T * nq is below 2^31 - 512.
struct SeqWork {
  int32_t t0;       // first token
  int32_t rows;     // n * G
  int64_t pos0;     // position of token t0 (may be negative)
  int32_t hi;       // keys end here (clamped to the pages)
};

__device__ __forceinline__ SeqWork seq_work(int64_t b, const Pointers& g, const AttendArgs& a, const Cut& c) {
  SeqWork s;
  if (c.prefix) {
    const int64_t n = ldg(g.qsl + a.B, a.qsl_span, g.err);
    s.t0 = 0;
    s.rows = (int)(n < 0 ? 0 : n > a.T ? a.T : n) * a.G;
    s.pos0 = a.P;
    s.hi = a.P;
    return s;
  }
  int64_t t0 = ldg(g.qsl + b, a.qsl_span, g.err), t1 = ldg(g.qsl + b + 1, a.qsl_span, g.err);
  const int64_t len = ldg(g.seq_lens + b, a.sl_span, g.err);
  t0 = t0 < 0 ? 0 : t0 > a.T ? a.T : t0;
  t1 = t1 > a.T ? a.T : t1;
  const int n = t1 > t0 ? (int)(t1 - t0) : 0;
  const int64_t most = (int64_t)a.P + a.W * a.block_size;
  if (len > most && n > 0) atomicOr(g.err, kSlotOutOfRange);  // more tokens than pages
  s.t0 = (int)t0;
  s.rows = n * a.G;
  s.pos0 = len - n;
  s.hi = (int)(len < 0 ? 0 : len > most ? most : len);
  return s;
}

// Keys [lo, end) that the rows of tile i of a sequence see between them.
template <int M>
__device__ __forceinline__ int tile_end(const SeqWork& s, int i, const AttendArgs& a, const Cut& c) {
  if (c.prefix) return s.hi;
  const int last = (int)((unsigned)(min((i + 1) * M, s.rows) - 1) / (unsigned)a.G);  // last token of the tile
  const int64_t e = s.pos0 + last + 1;
  return (int)(e < c.lo ? c.lo : e > s.hi ? max(s.hi, c.lo) : e);
}

template <int M, int KT>
__device__ __forceinline__ int tile_work(const SeqWork& s, int i, const AttendArgs& a, const Cut& c) {
  const int keys = tile_end<M>(s, i, a, c) - c.lo;
  return keys <= KT ? 1 : (keys + KT - 1) / KT;  // a unit without keys is one (empty) tile
}

template <int M>
__device__ __forceinline__ int row_tiles(const SeqWork& s) {
  return (s.rows + M - 1) / M;
}

template <int M, int KT>
__device__ __forceinline__ int64_t seq_total(const SeqWork& s, const AttendArgs& a, const Cut& c) {
  const int tiles = row_tiles<M>(s);
  if (c.prefix) return (int64_t)tiles * (c.cost + tile_work<M, KT>(s, 0, a, c)) * a.nk;
  int64_t sum = (int64_t)tiles * c.cost;
  for (int i = 0; i < tiles; ++i) sum += tile_work<M, KT>(s, i, a, c);
  return sum * a.nk;
}

// Walk over the units of this CTA's share.
struct Walk {
  int32_t b;       // sequence
  SeqWork s;
  int32_t tiles;   // row tiles of the sequence
  int32_t i;       // row tile
  int32_t h;       // key head
  int32_t work;    // key tiles of the unit
  int32_t k0;      // first key tile of the unit in this CTA
  int64_t left;    // tiles of this CTA's share from (this unit, tile k0) on
  int64_t share;
  bool done;
};

// Units of at most so many tiles are not split.
inline int whole_tiles(int64_t M) { return M > 64 ? 4 : 1; }

// What a unit costs beside its key tiles (query rows in, results out), in tiles: it counts in the
// cut like key tiles that come before them, so that a CTA with many short units gets fewer tiles.
// (128 sequences of 31 to 1024 own keys: without it some CTAs took 67 us and most 45.  The call,
// which joins a prefix of 16384: 124.7 us with 0, 113.2 with 1, 110.4 with 2, 108.1 with 3.  32
// sequences of up to 5 tokens, heads of 256: 70.6, 68.1, 62.7, 62.2.  64 rows of binary32 have
// dearer tiles: 10 sequences of 8 tokens, heads of 160: 25.3 us with 1, 40.3 with 2.)
inline int unit_cost(int32_t dtype) { return dtype == kF32 ? 1 : 2; }

// Key tiles of the current unit in this CTA end here.
__device__ __forceinline__ int walk_k1(const Walk& w, const Cut& c) {
  return w.work <= c.whole ? w.work : (int)min((int64_t)w.work, w.k0 + w.left);
}

__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d) {
  return (n | d) >> 32 ? n / d : (int64_t)((uint32_t)n / (uint32_t)d);
}

// The next unit of the share; w.done at its end.
template <int M, int KT>
__device__ __forceinline__ void walk_next(Walk& w, const Pointers& g, const AttendArgs& a, const Cut& c) {
  w.left -= walk_k1(w, c) - w.k0 + c.cost;
  if (w.left <= 0) {
    w.done = true;
    return;
  }
  w.k0 = 0;
  if (++w.h < a.nk) return;
  w.h = 0;
  ++w.i;
  while (w.i >= w.tiles) {
    w.i = 0;
    if (++w.b >= (c.prefix ? 1 : (int)a.B)) {  // a share ends before the last sequence does: never, unless the lengths change under way
      w.done = true;
      return;
    }
    w.s = seq_work(w.b, g, a, c);
    w.tiles = row_tiles<M>(w.s);
  }
  w.work = tile_work<M, KT>(w.s, w.i, a, c);
}

// Sum over the CTA's NT threads and the exclusive prefix of each, through shared memory
// (`tmp`: NT / 32 + 1 values).  Ends with a barrier.
template <int NT>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* tmp, int64_t* before) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) tmp[w] = x;
  __syncthreads();
  int64_t off = 0, total = 0;
#pragma unroll
  for (int j = 0; j < NT / 32; ++j) {
    if (j < w) off += tmp[j];
    total += tmp[j];
  }
  __syncthreads();
  *before = off + x - v;
  return total;
}

// Finds this CTA's share.  All NT threads call it; `tmp` holds NT / 32 + 2 values.
template <int M, int KT, int NT>
__device__ __forceinline__ Walk find_share(const Pointers& g, const AttendArgs& a, const Cut& c, int64_t* tmp) {
  Walk w;
  const int nb = c.prefix ? 1 : (int)a.B;
  int64_t rest;
  if (nb <= 32) {  // every warp finds it by itself: no barrier, no second look at the lengths
    const int lane = threadIdx.x & 31;
    SeqWork s = {};
    int64_t mine = 0;
    if (lane < nb) {
      s = seq_work(lane, g, a, c);
      mine = seq_total<M, KT>(s, a, c);
    }
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int64_t y = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += y;
    }
    const int64_t total = __shfl_sync(0xffffffffu, upto, 31);
    // Few units, many CTAs: a unit of n tiles in shares of s takes s tiles' time and a join of n / s
    // parts, of which eight cost about 4/3 of a tile: s = sqrt(n / 6).  (Requests of 300 keys: 9 us in
    // single tiles, 11 in two; 2 heads of 4112 keys: 19 us in single tiles, 16 in two.)
    const int deep = lane < nb && s.rows > 0 ? tile_work<M, KT>(s, row_tiles<M>(s) - 1, a, c) : 1;
    const int least = (int)sqrtf((float)__reduce_max_sync(0xffffffffu, deep) * (1.0f / 6.0f));
    w.share = max(quotient(total + gridDim.x - 1, gridDim.x), (int64_t)max(least, 1));
    const int64_t at = w.share * blockIdx.x;
    w.left = min(w.share, total - at);
    w.done = at >= total;
    if (w.done) return w;
    w.b = __ffs(__ballot_sync(0xffffffffu, at < upto)) - 1;
    rest = at - __shfl_sync(0xffffffffu, upto - mine, w.b);
    w.s.t0 = __shfl_sync(0xffffffffu, s.t0, w.b);
    w.s.rows = __shfl_sync(0xffffffffu, s.rows, w.b);
    w.s.pos0 = __shfl_sync(0xffffffffu, s.pos0, w.b);
    w.s.hi = __shfl_sync(0xffffffffu, s.hi, w.b);
  } else {
    int64_t total = 0, before = 0, mine = 0;
    for (int base = 0; base < nb; base += NT) {
      const int b = base + threadIdx.x;
      mine = b < nb ? seq_total<M, KT>(seq_work(b, g, a, c), a, c) : 0;
      total += block_scan<NT>(mine, tmp, &before);
    }
    w.share = max(quotient(total + gridDim.x - 1, gridDim.x), (int64_t)1);
    const int64_t at = w.share * blockIdx.x;
    w.left = min(w.share, total - at);
    w.done = at >= total;
    if (w.done) return w;
    int64_t run = 0;
    for (int base = 0; base < nb; base += NT) {
      const int b = base + threadIdx.x;
      if (nb > NT) mine = b < nb ? seq_total<M, KT>(seq_work(b, g, a, c), a, c) : 0;
      const int64_t sum = nb > NT ? block_scan<NT>(mine, tmp, &before) : total;
      if (run + before <= at && at < run + before + mine) {
        tmp[0] = b;
        tmp[1] = at - run - before;
      }
      run += sum;
      if (run > at) break;
    }
    __syncthreads();
    w.b = (int)tmp[0];
    rest = tmp[1];
    __syncthreads();
    w.s = seq_work(w.b, g, a, c);
  }
  w.tiles = row_tiles<M>(w.s);
  if (c.prefix) {
    w.work = tile_work<M, KT>(w.s, 0, a, c);
    const int64_t row = (int64_t)(c.cost + w.work) * a.nk;
    w.i = (int)quotient(rest, row);
    rest -= w.i * row;
  } else {
    w.i = 0;
    for (;;) {
      w.work = tile_work<M, KT>(w.s, w.i, a, c);
      const int64_t row = (int64_t)(c.cost + w.work) * a.nk;
      if (rest < row) break;
      rest -= row;
      ++w.i;
    }
  }
  w.h = (int)quotient(rest, c.cost + w.work);
  w.k0 = (int)(rest - (int64_t)w.h * (c.cost + w.work)) - c.cost;
  if (w.k0 < 0) {  // the unit begins in this CTA, or (no more than a part of its cost is left) in the next
    w.left += w.k0;
    w.k0 = 0;
    w.done = w.left <= 0;
  }
  if (w.k0 > 0 && w.work <= c.whole) walk_next<M, KT>(w, g, a, c);  // the CTA before finishes it
  return w;
}


// The record of row r of a unit that begins in this CTA: its CTAs and the row's place.
__device__ __forceinline__ int2 unit_record(const Walk& w, int r, const Cut& c) {
  int last = blockIdx.x;
  if (w.work > c.whole && w.work > w.left) {  // the rest of the unit, in shares below its size
    const uint32_t rest = (uint32_t)(w.work - w.left);
    last += (int)((rest + (uint32_t)w.share - 1) / (uint32_t)w.share);
  }
  return make_int2(blockIdx.x | last << 16, r);
}

// Row r of a unit as (token, head of the group), by 32-bit arithmetic.
struct UnitRows {
  int32_t t0;   // token of the unit's first row
  int32_t rem;  // its head within the group
  int32_t rows;
};

template <int M>
__device__ __forceinline__ UnitRows unit_rows(const Walk& w, const AttendArgs& a) {
  const unsigned first = (unsigned)w.i * M;
  UnitRows u;
  const unsigned t = first / (unsigned)a.G;
  u.t0 = w.s.t0 + (int)t;
  u.rem = (int)(first - t * a.G);
  u.rows = min(M, w.s.rows - (int)first);
  return u;
}

struct RowAt {
  int64_t t;
  int32_t h;  // query head
};

__device__ __forceinline__ RowAt row_at(const UnitRows& u, int r, int key_head, const AttendArgs& a) {
  const unsigned x = (unsigned)(u.rem + r), tt = x / (unsigned)a.G;
  return {(int64_t)u.t0 + tt, key_head * a.G + (int)(x - tt * a.G)};
}

__device__ __forceinline__ float* slot_o(const Cut& c, const AttendArgs& a, int64_t cta, int slot) {
  return c.slots + (cta * 2 + slot) * c.slot_rows * a.D;
}

__device__ __forceinline__ float* slot_ml(const Cut& c, const AttendArgs& a, int64_t cta, int slot) {
  return c.slots + (int64_t)c.grid * 2 * c.slot_rows * a.D + (cta * 2 + slot) * c.slot_rows * 2;
}

// Keys j < limit are what the row of token t of the current unit's sequence sees.
__device__ __forceinline__ int row_limit(const Walk& w, int64_t t, const Pointers& g, const AttendArgs& a, const Cut& c) {
  int64_t p;
  if (c.prefix) {
    const int64_t b = batch_of(t, g, a);
    p = ldg(g.seq_lens + b, a.sl_span, g.err) - (ldg(g.qsl + b + 1, a.qsl_span, g.err) - t) + 1;
  } else {
    p = w.s.pos0 + (t - w.s.t0) + 1;
  }
  return (int)(p < 0 ? 0 : p > w.s.hi ? w.s.hi : p);
}

// 1 / l for the sum of weights of a row that this CTA finishes (in the launch over a prefix none does).
// A sum of 0 is 0 of a row without keys, but NaN, for mend_rows to find, of one with keys: the
// products of all of them may have left binary32 downwards where scaled they would not have.
__device__ __forceinline__ float inverse_sum(float l, const Walk& w, int64_t t) {
  if (l != 0.f) return 1.f / l;
  return w.s.hi > 0 && w.s.pos0 + (t - w.s.t0) >= 0 ? NAN : 0.f;
}

// One query row by one warp, a key at a time: keys the row does not see are not read at all.
template <typename T, int E>
__device__ __forceinline__ void attend_row(int64_t t, int h, const T* __restrict__ q, const T* __restrict__ kc,
                                           const T* __restrict__ vc, T* __restrict__ out, float* __restrict__ lse,
                                           const Pointers& g, const AttendArgs& a) {
  constexpr int KU = 4;
  const int lane = threadIdx.x & 31;
  const int64_t row = t * a.nq + h;
  const int kh = h / a.G;
  const int64_t b = batch_of(t, g, a);
  const int64_t end = ldg(g.qsl + b + 1, a.qsl_span, g.err);
  const int64_t len = ldg(g.seq_lens + b, a.sl_span, g.err);
  const int64_t most = (int64_t)a.P + a.W * a.block_size;
  if (len > most && lane == 0) atomicOr(g.err, kSlotOutOfRange);
  const int64_t seen64 = len - (end - t) + 1;  // keys the row sees
  const int seen = (int)(seen64 < 0 ? 0 : seen64 > most ? most : seen64);
  const int64_t* table = g.block_table + b * a.W;
  float qv[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int d = lane + 32 * e;
    o[e] = 0.f;
    qv[e] = d < a.D ? widen(ldg(q + t * a.q_stride + (int64_t)h * a.D + d, a.q_span, g.err)) * a.scale_log2 : 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j0 = 0; j0 < seen; j0 += KU) {
    int64_t at[KU];
    float s[KU];
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      const int64_t r = j0 + u < seen ? key_row(j0 + u, table, g, a) : -1;
      if (r < 0 && j0 + u < seen && lane == 0) atomicOr(g.err, kSlotOutOfRange);
      at[u] = r < 0 ? -1 : (r + (int64_t)kh * a.block_size) * a.D;
      s[u] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < KU; ++u)
      if (at[u] >= 0) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int d = lane + 32 * e;
          if (d < a.D) s[u] = fmaf(qv[e], widen(ldg(kc + at[u] + d, a.k_span, g.err)), s[u]);
        }
      }
#pragma unroll
    for (int sh = 16; sh > 0; sh /= 2)
#pragma unroll
      for (int u = 0; u < KU; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], sh);
    float top = m;
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      if (at[u] < 0) s[u] = -INFINITY;
      top = s[u] != s[u] ? s[u] : fmaxf(top, s[u]);
    }
    const float base = top == -INFINITY ? 0.f : top;  // no key seen yet: every weight is e^(-inf - 0) = 0
    const float keep = exp2f(m - base);
    l *= keep;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= keep;
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      if (at[u] < 0) continue;
      const float w = exp2f(s[u] - base);
      l += w;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int d = lane + 32 * e;
        if (d < a.D) o[e] = fmaf(w, widen(ldg(vc + at[u] + d, a.v_span, g.err)), o[e]);
      }
    }
    m = top;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int d = lane + 32 * e;
    T* p = out + row * a.D + d;
    if (d < a.D && access_ok(p, sizeof(T), a.out_span, g.err)) *p = narrow<T>(l == 0.f ? 0.f : o[e] * inv);
  }
  if (lse && lane == 0 && access_ok(lse + row, 4, a.lse_span, g.err))
    lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

// The rows that this CTA finished and whose result is not finite, once more key by key: a key that a
// row does not see has weight 0 in the unit kernels, and 0 * infinity or NaN of its value leaves NaN; and
// products of queries and keys beyond binary32 are infinite there, here queries are scaled before.
// All NT threads call it after a barrier; `tmp` as for find_share.
template <typename T, int DP, int M, int KT, int NT>
__device__ __forceinline__ void mend_rows(const T* __restrict__ q, const T* __restrict__ kc, const T* __restrict__ vc,
                                          T* __restrict__ out, float* __restrict__ lse, const Pointers& g,
                                          const AttendArgs& a, const Cut& c, int64_t* tmp) {
  const int lane = threadIdx.x & 31;
  Walk w = find_share<M, KT, NT>(g, a, c, tmp);
  while (!w.done) {
    const UnitRows u = unit_rows<M>(w, a);
    if (w.k0 == 0 && walk_k1(w, c) == w.work)
      for (int r = threadIdx.x >> 5; r < u.rows; r += NT / 32) {
        const RowAt at = row_at(u, r, w.h, a);
        const T* o = out + (at.t * a.nq + at.h) * a.D;
        bool fine = true;
        for (int d = lane; d < a.D; d += 32) fine = fine && fabsf(widen(o[d])) <= FLT_MAX;
        if (!__all_sync(0xffffffffu, fine)) attend_row<T, DP / 32>(at.t, at.h, q, kc, vc, out, lse, g, a);
      }
    walk_next<M, KT>(w, g, a, c);
  }
}

}  // namespace attend
}  // namespace rope
