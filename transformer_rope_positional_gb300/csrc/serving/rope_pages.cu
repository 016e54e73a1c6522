// Pages of a paged cache: sequences forked, reordered, dropped and given room; live pages moved to the front;
// pages copied in many tensors at once.
//
// The first two work on tables of page numbers and on how many times each page is held (ref_counts).  They are
// bound by latency: a handful of steps, each of which has to see all of the one before.  Each is one launch: of one CTA
// that keeps the counts in shared memory, so that a step is a few hundred nanoseconds, where they fit (kSmallPages) and
// there are few rows (kSmallRows, kSmallTable); else of one cluster of 8 CTAs with the counts in global memory.  Rows
// reordered, us, one CTA and cluster: 16 rows of 32 columns 7.1, 14.9; 64 of 256 13.7, 22.5; 256 of 64 16.7, 20.0; 256 of
// 256 19.4, 21.6; 384 of 64 21.4, 22.5; 512 of 64 26.7, 23.6; 1024 of 8 33.6, 23.5; 4096 of 4 145, 47.  Compacted: 16 of 32
// 4.8, 11.4; 64 of 256 17.5, 65; 256 of 256 23, 28; 1024 of 64 35, 43; 2048 of 8 55, 79; 4096 of 4 95, 101, of 1 92, 63;
// 8000 of 1 170, 105.  Caches that only the cluster takes: 256 rows of 512 in 200000 pages 35 and 158.  Free pages are
// given out lowest first, rows in order, so results do not depend on the order in which threads run.
//
// rearrange_sequences: every old row lets go of its pages; new row i takes the whole pages of its parent once
// more.  The page that is written on (the last, partly filled one) stays with the first of the new rows that
// claim it if nobody then holds it: rows claim it by atomicMin of row - kClaim in its count, which is then 0.
// The others get a copy.  Where fresh pages go is found the other way round: the r-th free page belongs to the
// row whose range of requests holds r.
//
// compact_pages: with L live pages, the k-th live page at or behind L goes to the k-th free page before L.
#include <algorithm>

#include "rope_device.cuh"
#include "serving.h"

namespace rope {
namespace {

constexpr unsigned kSlotOutOfRange = 2u;
constexpr unsigned kPagesExhausted = 16u;
constexpr int kCluster = 8;
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kClaim = 1 << 30;
constexpr int kKeeps = 1 << 30;  // a row keeps the page that it writes on (rows have fewer pages)
constexpr int64_t kSmallPages = 24576;  // 8 bytes each
constexpr int64_t kSmallRows = 384;     // reordered, old and new
constexpr int64_t kSmallTable = 2048;   // compacted

// The CTAs of a call: CL is 1 or kCluster.
template <int CL>
struct Team {
  static constexpr int kAll = CL * kThreads, kAllWarps = CL * kWarps;

  static __device__ __forceinline__ int rank() {
    if constexpr (CL == 1) return 0;
    uint32_t r;
    asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return (int)r;
  }

  // What any thread wrote before it, all see after it.
  static __device__ __forceinline__ void sync() {
    if constexpr (CL == 1)
      __syncthreads();
    else
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }

  // The word of CTA `rank` that is where `p` is in this one's shared memory.
  static __device__ __forceinline__ int peer(const int* p, int rank) {
    if constexpr (CL == 1) return *p;
    uint32_t at = (uint32_t)__cvta_generic_to_shared(p), far;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(at), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(far) : "memory");
    return v;
  }

  // Warps' ranges of pages: warp w of all has [w * per, min(NB, (w + 1) * per)), per a multiple of 32.
  static __device__ __forceinline__ int2 pages_of(int warp, int NB) {
    const int per = (NB + kAllWarps * 32 - 1) / (kAllWarps * 32) * 32;
    const int64_t from = (int64_t)warp * per;
    return make_int2((int)min(from, (int64_t)NB), (int)min(from + per, (int64_t)NB));
  }

  // Sum of `count` (a value a warp, in every CTA's shared memory) over all warps before `warp`, and over all.
  // Every warp calls it.
  static __device__ __forceinline__ int sum_before(const int* count, int warp, int* total) {
    const int lane = threadIdx.x & 31;
    int before = 0, all = 0;
#pragma unroll
    for (int r = 0; r < CL; ++r) {
      const int v = peer(count + lane, r);
      all += v;
      before += r * kWarps + lane < warp ? v : 0;
    }
    *total = __reduce_add_sync(0xffffffffu, all);
    return __reduce_add_sync(0xffffffffu, before);
  }
};

// For the first count(row).columns entries of every row of a table, a warp to a row, four rows at a time (their loads
// before the use of any): x = *(count(row).from + column), then use(row, column, x).
struct Entries {
  const int64_t* from;
  int columns;
};
template <int WARPS, typename N, typename F>
__device__ __forceinline__ void for_entries(int warp, int64_t rows, const Span& span, unsigned* err, N&& count, F&& use) {
  constexpr int U = 4;
  for (int64_t r0 = warp; r0 < rows; r0 += U * WARPS) {
    Entries n[U];
    int most = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      n[u] = {nullptr, 0};
      if (r0 + u * WARPS < rows) n[u] = count(r0 + u * WARPS);
      most = max(most, n[u].columns);
    }
    for (int c = threadIdx.x & 31; c < most; c += 32) {
      int64_t x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        x[u] = c < n[u].columns && access_ok(n[u].from + c, 8, span, err) ? *(const volatile int64_t*)(n[u].from + c) : 0;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c < n[u].columns) use(r0 + u * WARPS, c, x[u]);
    }
  }
}

// The pages of a sequence of this length: at most those of its row, whatever the length is.
template <typename P>
__device__ __forceinline__ int pages_of_length(int64_t len, const P& p, unsigned* err) {
  const int64_t own = max(len, p.prefix_len) - p.prefix_len, most = p.W * p.block_size;
  if (own > most) atomicOr(err, kSlotOutOfRange);
  return (int)((min(own, most) + p.block_size - 1) / p.block_size);
}

// Counts in shared memory (one CTA) or in global memory.
template <int CL>
__device__ __forceinline__ void add_to(int32_t* p, int32_t v) {
  if constexpr (CL == 1)
    asm volatile("red.shared.add.s32 [%0], %1;" ::"r"((unsigned)__cvta_generic_to_shared(p)), "r"(v) : "memory");
  else
    atomicAdd(p, v);
}
template <int CL>
__device__ __forceinline__ void min_to(int32_t* p, int32_t v) {
  if constexpr (CL == 1)
    asm volatile("red.shared.min.s32 [%0], %1;" ::"r"((unsigned)__cvta_generic_to_shared(p)), "r"(v) : "memory");
  else
    atomicMin(p, v);
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

// A word that others write meanwhile, in shared or global memory.
__device__ __forceinline__ int32_t now(const int32_t* p) { return *(const volatile int32_t*)p; }
__device__ __forceinline__ int64_t now(const int64_t* p) { return *(const volatile int64_t*)p; }

// ---------------------------------------------------------------------------
// New sequences of old ones
// ---------------------------------------------------------------------------
struct RearrangeArgs {
  RearrangeProblem p;
  Span table_span, lens_span, refs_span, parents_span, room_span, new_table_span, new_lens_span, new_refs_span, src_span,
      dst_span, counts_span;
};

struct RearrangeShared {
  int free_pages[kWarps];  // in the warp's range
  int2 sums[kWarps];
};

// What new row i takes of its parent.
struct Taken {
  int64_t parent;  // or -1
  int64_t len;     // of the parent
  int full, rest;  // whole pages, tokens on the page that is written on
  int64_t last;    // that page, or -1
};

__device__ __forceinline__ Taken taken_of(int i, const RearrangeArgs& a, unsigned* err) {
  const RearrangeProblem& p = a.p;
  Taken t = {ldg(p.parents + i, a.parents_span, err), p.prefix_len, 0, 0, -1};
  if (t.parent >= p.B) {
    atomicOr(err, kSlotOutOfRange);
    t.parent = -1;
  }
  if (t.parent < 0) {
    t.parent = -1;
    return t;
  }
  t.len = max(ldg(p.lens + t.parent, a.lens_span, err), (int64_t)0);
  int64_t own = max(t.len - p.prefix_len, (int64_t)0);
  const int64_t most = min(p.W, p.new_W) * p.block_size;
  if (own > most) {
    atomicOr(err, kSlotOutOfRange);
    own = most;
    t.len = p.prefix_len + own;
  }
  t.full = (int)(own / p.block_size);
  t.rest = (int)(own - (int64_t)t.full * p.block_size);
  if (t.rest) {
    const int64_t page = ldg(p.table + t.parent * p.W + t.full, a.table_span, err);
    if (page >= 0 && page < p.NB) t.last = page;
    else atomicOr(err, kSlotOutOfRange);
  }
  return t;
}

template <int CL>
__global__ void __launch_bounds__(kThreads) rearrange_kernel(RearrangeArgs a, unsigned int* err) {
  using All = Team<CL>;
  extern __shared__ __align__(16) unsigned char raw[];
  RearrangeShared& sm = *reinterpret_cast<RearrangeShared*>(raw);
  const RearrangeProblem& p = a.p;
  const int rank = All::rank(), me = rank * kThreads + threadIdx.x;
  const int lane = threadIdx.x & 31, cw = threadIdx.x >> 5, warp = rank * kWarps + cw;
  const int rows = (int)p.rows, NB = (int)p.NB;
  const int64_t bs = p.block_size;
  // the counts: one CTA's in shared memory, behind the rows' words
  int* const start = reinterpret_cast<int*>(raw + sizeof(RearrangeShared));  // first request of every row
  int* const have = start + rows + 1;                                        // pages that it has before, | kKeeps
  int* const pair = have + rows;                                             // its place among the copies, or -1
  int32_t* const refs = CL == 1 ? pair + rows : p.new_refs;
  auto ref_ok = [&](const int32_t* r) { return CL == 1 || access_ok(r, 4, a.new_refs_span, err); };
  wait_for_prior_grid();
  // (what a thread's row takes of its parent is three dependent loads: once, and on the way with the counts)
  const bool one_row = CL == 1 && rows <= kThreads;
  const Taken kept = one_row && me < rows ? taken_of(me, a, err) : Taken{-1, 0, 0, 0, -1};
  auto taken = [&](int i) { return one_row ? kept : taken_of(i, a, err); };
  for (int i = threadIdx.x; i < rows; i += kThreads) have[i] = taken(i).full;  // (of every CTA)
  // ---- counts as they were
  if (refs != p.refs) {
    for (int i = me; i < NB; i += All::kAll)
      if (ref_ok(refs + i)) *(volatile int32_t*)(refs + i) = access_ok(p.refs + i, 4, a.refs_span, err) ? p.refs[i] : 0;
    All::sync();
  }
  // ---- old rows let go
  auto pages_of_row = [&](int64_t b) -> Entries {
    return {p.table + b * p.W, pages_of_length(ldg(p.lens + b, a.lens_span, err), p, err)};
  };
  for_entries<All::kAllWarps>(warp, p.B, a.table_span, err, pages_of_row, [&](int64_t, int, int64_t page) {
    if (page < 0 || page >= p.NB) atomicOr(err, kSlotOutOfRange);
    else if (ref_ok(refs + page)) add_to<CL>(refs + page, -1);
  });
  All::sync();
  // ---- new rows take hold of whole pages
  auto whole_of_row = [&](int64_t i) -> Entries {
    const int n = have[i];
    return {n ? p.table + ldg(p.parents + i, a.parents_span, err) * p.W : nullptr, n};
  };
  for_entries<All::kAllWarps>(warp, rows, a.table_span, err, whole_of_row, [&](int64_t i, int c, int64_t page) {
    if (page < 0 || page >= p.NB) atomicOr(err, kSlotOutOfRange);
    else if (ref_ok(refs + page)) add_to<CL>(refs + page, 1);
    int64_t* const to = p.new_table + i * p.new_W + c;
    if (access_ok(to, 8, a.new_table_span, err)) *to = page;
  });
  All::sync();
  // ---- claims of pages that are written on
  for (int i = me; i < rows; i += All::kAll) {
    const Taken t = taken(i);
    if (t.last >= 0 && ref_ok(refs + t.last) && now(refs + t.last) <= 0) min_to<CL>(refs + t.last, i - kClaim);
  }
  All::sync();
  // ---- every CTA adds up what the rows keep, copy and ask for
  int2 run = make_int2(0, 0);  // requests, copies
  for (int base = 0; base < rows; base += kThreads) {
    const int i = base + threadIdx.x;
    int2 mine = make_int2(0, 0);
    int has = 0;
    bool copy = false, keeps_last = false;
    if (i < rows) {
      const Taken t = taken(i);
      const bool keeps = t.last >= 0 && ref_ok(refs + t.last) && now(refs + t.last) == i - kClaim;
      copy = t.rest > 0 && !keeps;
      has = t.full + keeps;
      keeps_last = keeps;
      const int64_t room = p.room ? max(ldg(p.room + i, a.room_span, err), (int64_t)0) : 0;
      // (a sequence that ends within the prefix has room there first)
      const int64_t most = p.prefix_len + p.new_W * bs, len = t.len + min(room, most - t.len);
      if (room > most - t.len && rank == 0) atomicOr(err, kSlotOutOfRange);
      const int64_t own = max(len - p.prefix_len, (int64_t)0);
      mine = make_int2((int)((own + bs - 1) / bs) - has, copy);
      if (rank == 0 && access_ok(p.new_lens + i, 8, a.new_lens_span, err)) p.new_lens[i] = len;
    }
    int2 upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, upto.x, d), y = __shfl_up_sync(0xffffffffu, upto.y, d);
      if (lane >= d) upto.x += x, upto.y += y;
    }
    __syncthreads();
    if (lane == 31) sm.sums[cw] = upto;
    __syncthreads();
    int2 sum = sm.sums[lane];
    const int2 own_sum = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, sum.x, d), y = __shfl_up_sync(0xffffffffu, sum.y, d);
      if (lane >= d) sum.x += x, sum.y += y;
    }
    const int before_x = __shfl_sync(0xffffffffu, sum.x - own_sum.x, cw);
    const int before_y = __shfl_sync(0xffffffffu, sum.y - own_sum.y, cw);
    if (i < rows) {
      start[i] = run.x + before_x + upto.x - mine.x;
      have[i] = has | (keeps_last ? kKeeps : 0);
      pair[i] = copy ? run.y + before_y + upto.y - 1 : -1;
    }
    run.x += __shfl_sync(0xffffffffu, sum.x, 31);
    run.y += __shfl_sync(0xffffffffu, sum.y, 31);
  }
  if (threadIdx.x == 0) start[rows] = run.x;
  All::sync();
  // ---- pages that are kept to be written on: off with the claims
  for (int i = me; i < rows; i += All::kAll) {
    if (!(have[i] & kKeeps)) continue;
    const int64_t page = taken(i).last;
    if (ref_ok(refs + page)) *(volatile int32_t*)(refs + page) = 1;
    int64_t* const to = p.new_table + i * p.new_W + (have[i] & ~kKeeps) - 1;
    if (access_ok(to, 8, a.new_table_span, err)) *to = page;
  }
  All::sync();
  // ---- free pages
  const int2 mine = All::pages_of(warp, NB);
  int free_pages = 0;
  for (int i = mine.x + lane; i < mine.y; i += 32) free_pages += ref_ok(refs + i) && now(refs + i) == 0;
  free_pages = warp_sum(free_pages);
  if (lane == 0) sm.free_pages[cw] = free_pages;
  All::sync();
  int all_free;
  int r0 = All::sum_before(sm.free_pages, warp, &all_free);
  const int asked = run.x;
  for (int base = mine.x; base < mine.y && r0 < asked; base += 32) {
    const int page = base + lane;
    const bool is_free = page < mine.y && ref_ok(refs + page) && now(refs + page) == 0;
    const uint32_t ones = __ballot_sync(0xffffffffu, is_free);
    const int r = r0 + __popc(ones & ((1u << lane) - 1u));
    r0 += __popc(ones);
    if (!is_free || r >= asked) continue;
    int lo = 0, hi = rows - 1;  // the last row that starts at or before r (rows without requests start with the next)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (start[mid] <= r) lo = mid;
      else hi = mid - 1;
    }
    const int j = r - start[lo];
    int64_t* const to = p.new_table + lo * p.new_W + (have[lo] & ~kKeeps) + j;
    if (access_ok(to, 8, a.new_table_span, err)) *to = page;
    refs[page] = 1;
    if (j == 0 && pair[lo] >= 0 && access_ok(p.dst + pair[lo], 8, a.dst_span, err)) p.dst[pair[lo]] = page;
  }
  // ---- pairs, requests that no page was left for, and the counts
  for (int i = me; i < rows; i += All::kAll) {
    const int at = pair[i], first = start[i], end = start[i + 1];
    if (at >= 0 && access_ok(p.src + at, 8, a.src_span, err)) {
      p.src[at] = taken(i).last;
      if (first >= all_free) p.dst[at] = -1;
    }
    if (i >= run.y && access_ok(p.src + i, 8, a.src_span, err)) p.src[i] = p.dst[i] = -1;
    for (int r = max(first, all_free); r < end; ++r) {
      int64_t* const to = p.new_table + i * p.new_W + (have[i] & ~kKeeps) + r - first;
      if (access_ok(to, 8, a.new_table_span, err)) *to = -1;
      atomicOr(err, kPagesExhausted);
    }
  }
  if (me == 0 && access_ok(p.counts, 16, a.counts_span, err)) {
    p.counts[0] = run.y;
    p.counts[1] = max(all_free - asked, 0);
  }
  All::sync();  // (nobody leaves while another reads its shared memory)
  if constexpr (CL == 1)
    for (int i = me; i < NB; i += All::kAll)
      if (access_ok(p.new_refs + i, 4, a.new_refs_span, err)) p.new_refs[i] = refs[i];
}

// ---------------------------------------------------------------------------
// Live pages to the front
// ---------------------------------------------------------------------------
struct CompactArgs {
  CompactProblem p;
  int64_t prefix_pages;
  Span table_span, lens_span, refs_span, new_table_span, new_refs_span, prefix_span, new_prefix_span, src_span, dst_span,
      counts_span;
};

template <int CL>
__global__ void __launch_bounds__(kThreads) compact_kernel(CompactArgs a, unsigned int* err) {
  using All = Team<CL>;
  __shared__ int live_of[kWarps], hole_of[kWarps], mover_of[kWarps];
  extern __shared__ __align__(16) unsigned char raw[];
  const CompactProblem& p = a.p;
  const int rank = All::rank(), me = rank * kThreads + threadIdx.x;
  const int lane = threadIdx.x & 31, cw = threadIdx.x >> 5, warp = rank * kWarps + cw;
  const int NB = (int)p.NB;
  // one CTA: the counts, where pages go, and the free pages in order, in shared memory
  int32_t* const held = reinterpret_cast<int32_t*>(raw);
  uint16_t* const moved_to = reinterpret_cast<uint16_t*>(held + (CL == 1 ? NB : 0));
  uint16_t* const hole_at = moved_to + (CL == 1 ? NB : 0);
  static_assert(kSmallPages < 65536, "page numbers in 16 bits");
  wait_for_prior_grid();
  auto ref_at = [&](int i) -> int32_t {
    if constexpr (CL == 1) return held[i];
    return access_ok(p.refs + i, 4, a.refs_span, err) ? now(p.refs + i) : 0;
  };
  if constexpr (CL == 1) {
    for (int i = me; i < NB; i += All::kAll) held[i] = access_ok(p.refs + i, 4, a.refs_span, err) ? p.refs[i] : 0;
    All::sync();
  }
  auto live_at = [&](int i) { return ref_at(i) > 0; };
  const int2 mine = All::pages_of(warp, NB);
  int n = 0;
  for (int i = mine.x + lane; i < mine.y; i += 32) n += live_at(i);
  n = warp_sum(n);
  if (lane == 0) live_of[cw] = n;
  All::sync();
  int L;
  All::sum_before(live_of, warp, &L);
  // ---- free pages before L, live ones at or behind it
  int holes = 0, movers = 0;
  for (int i = mine.x + lane; i < mine.y; i += 32) {
    const bool live = live_at(i);
    holes += !live && i < L;
    movers += live && i >= L;
  }
  holes = warp_sum(holes);
  movers = warp_sum(movers);
  if (lane == 0) {
    hole_of[cw] = holes;
    mover_of[cw] = movers;
  }
  All::sync();
  int all_holes, moved;
  int h0 = All::sum_before(hole_of, warp, &all_holes), m0 = All::sum_before(mover_of, warp, &moved);
  if (holes + movers > 0)
    for (int base = mine.x; base < mine.y; base += 32) {
      const int i = base + lane;
      const bool live = i < mine.y && live_at(i);
      const bool hole = i < mine.y && !live && i < L, mover = live && i >= L;
      const uint32_t hs = __ballot_sync(0xffffffffu, hole), ms = __ballot_sync(0xffffffffu, mover);
      const uint32_t before = (1u << lane) - 1u;
      if (hole) {
        const int k = h0 + __popc(hs & before);
        if (access_ok(p.dst + k, 8, a.dst_span, err)) *(volatile int64_t*)(p.dst + k) = i;
        if constexpr (CL == 1) hole_at[k] = (uint16_t)i;
      }
      if (mover) {
        const int k = m0 + __popc(ms & before);
        if (access_ok(p.src + k, 8, a.src_span, err)) *(volatile int64_t*)(p.src + k) = i;
        if constexpr (CL == 1) moved_to[i] = (uint16_t)k;  // (its rank: where that goes is known to all after the barrier)
      }
      h0 += __popc(hs);
      m0 += __popc(ms);
    }
  for (int64_t i = moved + me; i < p.pairs; i += All::kAll) {
    if (access_ok(p.src + i, 8, a.src_span, err)) p.src[i] = -1;
    if (access_ok(p.dst + i, 8, a.dst_span, err)) p.dst[i] = -1;
  }
  if (me == 0 && access_ok(p.counts, 16, a.counts_span, err)) {
    p.counts[0] = moved;
    p.counts[1] = L;
  }
  All::sync();
  // ---- tables
  auto to_of = [&](int64_t page) -> int64_t {  // where a page goes
    if (page < 0 || page >= p.NB || !live_at((int)page)) {
      atomicOr(err, kSlotOutOfRange);
      return page;
    }
    if (page < L) return page;
    if constexpr (CL == 1) return hole_at[moved_to[page]];
    int lo = 0, hi = moved - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (now(p.src + mid) < page) lo = mid + 1;
      else hi = mid;
    }
    return now(p.dst + lo);
  };
  auto pages_of_row = [&](int64_t b) -> Entries {
    return {p.table + b * p.W, pages_of_length(ldg(p.lens + b, a.lens_span, err), p, err)};
  };
  for_entries<All::kAllWarps>(warp, p.B, a.table_span, err, pages_of_row, [&](int64_t b, int c, int64_t page) {
    int64_t* const to = p.new_table + b * p.W + c;
    if (access_ok(to, 8, a.new_table_span, err)) *to = to_of(page);
  });
  for (int64_t i = me; i < a.prefix_pages; i += All::kAll) {
    const int64_t page = access_ok(p.prefix + i, 8, a.prefix_span, err) ? p.prefix[i] : 0;
    if (access_ok(p.new_prefix + i, 8, a.new_prefix_span, err)) p.new_prefix[i] = to_of(page);
  }
  // ---- counts (in place too: what is read of a page is read before it is written)
  if constexpr (CL > 1) All::sync();
  for (int i = me; i < L; i += All::kAll) {
    const int32_t v = ref_at(i);
    // (a free page gets the count of what moves there)
    if (v > 0 && access_ok(p.new_refs + i, 4, a.new_refs_span, err)) p.new_refs[i] = v;
  }
  for (int k = me; k < moved; k += All::kAll) {
    const int64_t from = now(p.src + k), to = now(p.dst + k);
    const int32_t v = ref_at((int)from);
    if (access_ok(p.new_refs + to, 4, a.new_refs_span, err)) p.new_refs[to] = v;
  }
  if constexpr (CL > 1) All::sync();
  for (int i = L + me; i < NB; i += All::kAll)
    if (access_ok(p.new_refs + i, 4, a.new_refs_span, err)) p.new_refs[i] = 0;
}

// One CTA, or one cluster of kCluster.
template <int CL, typename K, typename A>
cudaError_t launch_team(K kernel, size_t smem, const A& a, cudaStream_t stream) {
  unsigned int* err = nullptr;
  cudaError_t e = device_error_address(&err);
  if (e == cudaSuccess && smem > 48 * 1024) e = opt_in_shared(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CL);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CL;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL == 1 ? 1 : 2;
  e = cudaLaunchKernelEx(&cfg, kernel, a, err);
  count_launch();
  return e == cudaSuccess ? cudaGetLastError() : e;
}

// ---------------------------------------------------------------------------
// Pages copied
// ---------------------------------------------------------------------------
constexpr int kTensors = 64;   // of one launch
constexpr int kPiece = 4096;   // bytes that a warp copies at a time
constexpr int kCopyThreads = 256;

struct CopyArgs {
  const int64_t *src, *dst, *count;
  int64_t pairs, NB;
  int64_t pieces;  // of a pair, all tensors together
  int32_t tensors;
  CopyTensor t[kTensors];
  int32_t first[kTensors + 1];  // first piece of each tensor
  int32_t vec[kTensors];        // bytes of an access: 16, 8, 4, 2 or 1
  Span src_span, dst_span, count_span, span[kTensors];
};

template <typename V>
__device__ __forceinline__ void copy_piece(char* to, const char* from, int n, const Span& s, unsigned* err) {
  const int lane = threadIdx.x & 31;
  constexpr int U = 8;
  const V* x = reinterpret_cast<const V*>(from);
  V* y = reinterpret_cast<V*>(to);
  const int m = n / (int)sizeof(V);
  for (int i = lane; i < m; i += 32 * U) {
    V v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + 32 * u < m && access_ok(x + i + 32 * u, sizeof(V), s, err)) v[u] = __ldcs(x + i + 32 * u);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + 32 * u < m && access_ok(y + i + 32 * u, sizeof(V), s, err)) __stcs(y + i + 32 * u, v[u]);
  }
}

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyArgs a, unsigned int* err) {
  wait_for_prior_grid();
  const int lane = threadIdx.x & 31;
  int64_t pairs = a.pairs;
  if (a.count) pairs = max(min(ldg(a.count, a.count_span, err), pairs), (int64_t)0);
  const int64_t all = pairs * a.pieces, warps = (int64_t)gridDim.x * (kCopyThreads / 32);
  for (int64_t f = (int64_t)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); f < all; f += warps) {
    const int64_t pair = f / a.pieces;
    const int piece = (int)(f - pair * a.pieces);
    const int64_t from = ldg(a.src + pair, a.src_span, err), to = ldg(a.dst + pair, a.dst_span, err);
    if (from < 0 || to < 0 || from == to) continue;
    if (from >= a.NB || to >= a.NB) {
      if (lane == 0) atomicOr(err, kSlotOutOfRange);
      continue;
    }
    int lo = 0, hi = a.tensors - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.first[mid] <= piece) lo = mid;
      else hi = mid - 1;
    }
    const int64_t bytes = a.t[lo].bytes, off = (int64_t)(piece - a.first[lo]) * kPiece;
    const int n = (int)min((int64_t)kPiece, bytes - off);
    char* const y = a.t[lo].data + to * bytes + off;
    const char* const x = a.t[lo].data + from * bytes + off;
    switch (a.vec[lo]) {
      case 16:
        copy_piece<uint4>(y, x, n, a.span[lo], err);
        break;
      case 8:
        copy_piece<uint2>(y, x, n, a.span[lo], err);
        break;
      case 4:
        copy_piece<unsigned int>(y, x, n, a.span[lo], err);
        break;
      case 2:
        copy_piece<unsigned short>(y, x, n, a.span[lo], err);
        break;
      default:
        copy_piece<unsigned char>(y, x, n, a.span[lo], err);
    }
  }
}

}  // namespace

cudaError_t launch_rearrange(const RearrangeProblem& p, cudaStream_t stream) {
  RearrangeArgs a;
  a.p = p;
  a.table_span = make_span(p.table, p.B * p.W * 8);
  a.lens_span = make_span(p.lens, p.B * 8);
  a.refs_span = make_span(p.refs, p.NB * 4);
  a.parents_span = make_span(p.parents, p.rows * 8);
  a.room_span = make_span(p.room, p.rows * 8);
  a.new_table_span = make_span(p.new_table, p.rows * p.new_W * 8);
  a.new_lens_span = make_span(p.new_lens, p.rows * 8);
  a.new_refs_span = make_span(p.new_refs, p.NB * 4);
  a.src_span = make_span(p.src, p.rows * 8);
  a.dst_span = make_span(p.dst, p.rows * 8);
  a.counts_span = make_span(p.counts, 16);
  const size_t smem = sizeof(RearrangeShared) + (3 * p.rows + 1) * 4;
  if (p.NB <= kSmallPages && p.B <= kSmallRows && p.rows <= kSmallRows)
    return launch_team<1>(rearrange_kernel<1>, smem + p.NB * 4, a, stream);
  return launch_team<kCluster>(rearrange_kernel<kCluster>, smem, a, stream);
}

cudaError_t launch_compact(const CompactProblem& p, cudaStream_t stream) {
  CompactArgs a;
  a.p = p;
  a.prefix_pages = p.prefix ? (p.prefix_len + p.block_size - 1) / p.block_size : 0;
  a.table_span = make_span(p.table, p.B * p.W * 8);
  a.lens_span = make_span(p.lens, p.B * 8);
  a.refs_span = make_span(p.refs, p.NB * 4);
  a.new_table_span = make_span(p.new_table, p.B * p.W * 8);
  a.new_refs_span = make_span(p.new_refs, p.NB * 4);
  a.prefix_span = make_span(p.prefix, a.prefix_pages * 8);
  a.new_prefix_span = make_span(p.new_prefix, a.prefix_pages * 8);
  a.src_span = make_span(p.src, p.pairs * 8);
  a.dst_span = make_span(p.dst, p.pairs * 8);
  a.counts_span = make_span(p.counts, 16);
  if (p.NB <= kSmallPages && p.B <= kSmallTable)
    return launch_team<1>(compact_kernel<1>, p.NB * (4 + 2 + 2), a, stream);
  return launch_team<kCluster>(compact_kernel<kCluster>, 0, a, stream);
}

cudaError_t launch_copy_pages(const CopyProblem& p, cudaStream_t stream) {
  unsigned int* err = nullptr;
  const cudaError_t er = device_error_address(&err);
  if (er != cudaSuccess) return er;
  for (int64_t at = 0; at < p.num_tensors; at += kTensors) {
    CopyArgs a;
    a.src = p.src;
    a.dst = p.dst;
    a.count = p.count;
    a.pairs = p.pairs;
    a.NB = p.NB;
    a.tensors = (int32_t)std::min<int64_t>(kTensors, p.num_tensors - at);
    int64_t pieces = 0;
    for (int i = 0; i < a.tensors; ++i) {
      const CopyTensor& t = p.tensors[at + i];
      a.t[i] = t;
      a.first[i] = (int32_t)pieces;
      pieces += (t.bytes + kPiece - 1) / kPiece;
      const uintptr_t bits = reinterpret_cast<uintptr_t>(t.data) | (uintptr_t)t.bytes;
      a.vec[i] = bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : bits % 2 == 0 ? 2 : 1;
      a.span[i] = make_span(t.data, t.bytes * p.NB);
    }
    a.first[a.tensors] = (int32_t)pieces;
    a.pieces = pieces;
    a.src_span = make_span(p.src, p.pairs * 8);
    a.dst_span = make_span(p.dst, p.pairs * 8);
    a.count_span = make_span(p.count, 8);
    const int64_t warps = kCopyThreads / 32;
    const int64_t resident =
        (int64_t)sm_count() * resident_blocks(reinterpret_cast<const void*>(copy_pages_kernel), kCopyThreads);
    const int64_t grid = std::max<int64_t>(1, std::min((p.pairs * pieces + warps - 1) / warps, resident));
    const cudaError_t e = launch_overlapped(copy_pages_kernel, (unsigned)grid, kCopyThreads, stream, a, err);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace rope
