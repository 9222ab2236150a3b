// skv_pages.hip -- the paged KV cache: giving out, sharing, copying, compacting
// and freeing pages, writing tokens into them, and the way between pages and
// the coder's layout.  Contracts: skv.h.
//
// Page bookkeeping (extend, fork, truncate, compact) is integer work on short
// lists.  One workgroup plans a call: it checks the whole list first, so that
// a call that fails changes nothing, and works the order of a list out with
// prefix sums, so that the result does not depend on timing.  What has to be
// copied goes to a list that a second, wide launch works through.
//
// What bounds them.  The planning launches are chains of three or four dependent
// loads and as many barriers: fork 3 us (4 rows) to 5 (32 rows of 64 pages), extend
// 6.3 to 6.8, truncate 2.7 to 4.6, compaction's plan of 1000 pages 4.7.  What moves
// many symbols is bound by HBM: moving 250 of 1000 pages of 64 layers (2.07 GB read
// and written) 359 to 420 us from box to box, 5.8 to 4.9 TB/s; the coder's layout
// from 8192 tokens of 28 layers (0.94 GB) 150 us and back 163, 6.3 and 5.8 TB/s;
// 16376 tokens stored as e4m3 (101 MB) 21 us, 4.8 TB/s.  A copy of 4 GiB reaches 4.8
// to 4.9 TB/s here, a plain read 7.0.  The same tokens stored as bf16 (134 MB) take
// 43 us, 3.1 TB/s: that kernel's registers leave a SIMD two waves (the e4m3 one eight).
#include "skv_pages.hpp"

using namespace skv;

namespace {

constexpr int kPlan = 1024;  // threads of a planning workgroup
constexpr int kPlanWaves = kPlan / 64;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// symbols on their way through: past the caches
template <typename U>
__device__ __forceinline__ U take(const U *p) { return __builtin_nontemporal_load(p); }
template <typename U>
__device__ __forceinline__ void put(U *p, U v) { __builtin_nontemporal_store(v, p); }

// ---- workspace of the planning calls ----
enum { kHdrOk = 0, kHdrCopies = 1, kHdrLive = 2 };

struct PWork {
  int32_t *hdr;    // 16 words
  int32_t *mark;   // [max_seqs] long lists: last list place that names the row
  int32_t *cnt;    // [n_pages] extend, long lists: listed sharers of a page; compact: where a page went
  int32_t *owner;  // [n_pages] extend, long lists: the last of them
  int32_t *fl;     // [n_pages] extend: free pages in order
  int32_t *off;    // [max_seqs] extend, long lists: pages given out before a place's own
  int32_t *cow;    // [max_seqs] extend, long lists: 1 where the last page is copied
  int32_t *csrc;   // copies: source page, target page, tokens
  int32_t *cdst;
  int32_t *ctok;
  size_t total;
};

PWork carve_pages(const PGeo &g, void *base) {
  uint8_t *b = static_cast<uint8_t *>(base);
  size_t o = 0;
  auto take = [&](size_t words) {
    int32_t *p = reinterpret_cast<int32_t *>(b + o);
    o = (o + words * sizeof(int32_t) + 255) / 256 * 256;
    return p;
  };
  const size_t ns = (size_t)g.max_seqs, np = (size_t)g.n_pages;
  const size_t copies = ns > np ? ns : np;
  PWork w;
  w.hdr = take(16);
  w.mark = take(ns);
  w.cnt = take(np);
  w.owner = take(np);
  w.fl = take(np);
  w.off = take(ns);
  w.cow = take(ns);
  w.csrc = take(copies);
  w.cdst = take(copies);
  w.ctok = take(copies);
  w.total = o;
  return w;
}

// exclusive prefix sum over the workgroup's kPlan threads; total to all
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t &total, int64_t *lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  if (lane == 63) lds[wave] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) {
    const int64_t s = lds[w];
    before += w < wave ? s : 0;
    all += s;
  }
  __syncthreads();
  total = all;
  return before + x - v;
}

// errors seen by any thread of the workgroup, a bit per code, so that which one
// is reported does not depend on the threads' order
__device__ __forceinline__ void note(int *err, int code) { atomicOr(err, 1 << code); }

// after a barrier: true (for all threads alike) if the call ends here
__device__ __forceinline__ bool failed(const int *err, int32_t *hdr, int32_t *status) {
  __syncthreads();
  const int e = *err;
  __syncthreads();
  if (e == 0) return false;
  if (threadIdx.x == 0) {
    hdr[kHdrOk] = 0;
    hdr[kHdrCopies] = 0;
    set_status(status, __builtin_ctz((unsigned)e));
  }
  return true;
}

// holders of pages p .. p + 3 (p a multiple of 4); behind the last page 1, neither free nor counted on
__device__ __forceinline__ int4 refs_of(const PGeo &g, const skv_pages &a, int64_t p) {
  if (p + 4 <= g.n_pages) return *reinterpret_cast<const int4 *>(a.refs + p);
  int4 r = make_int4(1, 1, 1, 1);
  if (p < g.n_pages) r.x = a.refs[p];
  if (p + 1 < g.n_pages) r.y = a.refs[p + 1];
  if (p + 2 < g.n_pages) r.z = a.refs[p + 2];
  return r;
}

// ---- rows and pages named in a list of at most kPlan places: hash tables in LDS ----
constexpr int kSlots = 2 * kPlan;

__device__ __forceinline__ int slot_of(int32_t key) { return (int)(((uint32_t)key * 2654435761u) >> 21) & (kSlots - 1); }
// the slot of a key that is put in; `had`: it was there
__device__ __forceinline__ int put_key(int *keys, int32_t key, bool &had) {
  for (int i = slot_of(key);; i = (i + 1) & (kSlots - 1)) {  // at most half of the slots are ever taken
    const int old = atomicCAS(&keys[i], -1, key);
    had = old == key;
    if (old == -1 || had) return i;
  }
}
__device__ __forceinline__ bool has_key(const int *keys, int32_t key) {
  for (int i = slot_of(key);; i = (i + 1) & (kSlots - 1)) {
    const int k = keys[i];
    if (k == key || k == -1) return k == key;
  }
}
__device__ __forceinline__ void clear_keys(int *keys) {
  for (int i = threadIdx.x; i < kSlots; i += kPlan) keys[i] = -1;
}

// ---- extend ----
// Which listed sequences copy their last page: with c sharers in the list and r
// holders in all, every one of them where r > c, all but the last where r = c.
// That is what growing them one after another gives (each copy gives up one
// hold, and the last holder keeps the page), found without an order of events.
__global__ __launch_bounds__(kPlan) void k_plan_extend_long(PGeo g, skv_pages a, const int32_t *__restrict__ seqs,
                                                            const int32_t *__restrict__ n_new, int n, PWork w,
                                                            int32_t *status) {
  __shared__ int err;
  __shared__ int64_t lds[kPlanWaves];
  const int tid = threadIdx.x;
  if (tid == 0) err = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kPlan) {
    const int32_t s = seqs[i];
    if (s < 0) continue;
    if (s >= g.max_seqs) { note(&err, SKV_ERR_ARG); continue; }
    agent_store(&w.mark[s], i);
    const int32_t len = a.lens[s], add = n_new[i];
    if (len < 0 || len > g.max_tokens || add < 0) { note(&err, SKV_ERR_ARG); continue; }
    if ((int64_t)len + add > g.max_tokens) { note(&err, SKV_ERR_PAGES); continue; }
    if (add > 0 && (len & (g.P - 1))) {
      const int32_t pg = a.table[(int64_t)s * g.max_pages + (len >> g.log2P)];
      if (!good_page(pg, g) || a.refs[pg] < 1) { note(&err, SKV_ERR_ARG); continue; }
      agent_store(&w.cnt[pg], 0);
      agent_store(&w.owner[pg], -1);
    }
  }
  if (failed(&err, w.hdr, status)) return;
  for (int i = tid; i < n; i += kPlan) {
    const int32_t s = seqs[i];
    if (s < 0) continue;
    if (agent_load(&w.mark[s]) != i) { note(&err, SKV_ERR_ARG); continue; }
    const int32_t len = a.lens[s];
    if (n_new[i] > 0 && (len & (g.P - 1))) {
      const int32_t pg = a.table[(int64_t)s * g.max_pages + (len >> g.log2P)];
      atomicAdd(&w.cnt[pg], 1);
      atomicMax(&w.owner[pg], i);
    }
  }
  if (failed(&err, w.hdr, status)) return;
  // pages each place needs, and where its own begin in the order of the list
  int64_t need_all = 0, copies_all = 0;
  for (int base = 0; base < n; base += kPlan) {
    const int i = base + tid;
    const int32_t s = i < n ? seqs[i] : -1;
    int64_t need = 0, cow = 0;
    if (s >= 0) {
      const int32_t len = a.lens[s], add = n_new[i];
      need = pages_of(len + add, g) - pages_of(len, g);
      if (add > 0 && (len & (g.P - 1))) {
        const int32_t pg = a.table[(int64_t)s * g.max_pages + (len >> g.log2P)];
        const int32_t r = a.refs[pg], c = agent_load(&w.cnt[pg]);
        if (r < c) note(&err, SKV_ERR_ARG);  // fewer holds than holders
        cow = r > c || agent_load(&w.owner[pg]) != i;
      }
      need += cow;
    }
    int64_t t0, t1;
    const int64_t before = block_scan(need, t0, lds);
    const int64_t cbefore = block_scan(cow, t1, lds);
    if (i < n) {
      // an offset beyond the pool is not used: the call fails below
      agent_store(&w.off[i], (int32_t)min(need_all + before, (int64_t)INT32_MAX));
      agent_store(&w.cow[i], (int32_t)cow);
      if (cow) w.ctok[copies_all + cbefore] = i;  // the place, until the target is known
    }
    need_all += t0;
    copies_all += t1;
  }
  if (need_all > g.n_pages) note(&err, SKV_ERR_PAGES);
  if (failed(&err, w.hdr, status)) return;
  // the lowest free pages, in order
  int64_t found = 0;
  for (int64_t base = 0; base < g.n_pages && found < need_all; base += (int64_t)kPlan * 4) {
    const int64_t p = base + (int64_t)tid * 4;
    const int4 r = refs_of(g, a, p);
    const int f0 = r.x == 0, f1 = r.y == 0, f2 = r.z == 0, f3 = r.w == 0;
    int64_t t;
    int64_t at = found + block_scan(f0 + f1 + f2 + f3, t, lds);
    if (f0) { agent_store(&w.fl[at], (int32_t)p); ++at; }
    if (f1) { agent_store(&w.fl[at], (int32_t)p + 1); ++at; }
    if (f2) { agent_store(&w.fl[at], (int32_t)p + 2); ++at; }
    if (f3) { agent_store(&w.fl[at], (int32_t)p + 3); ++at; }
    found += t;
  }
  if (found < need_all) note(&err, SKV_ERR_PAGES);
  if (failed(&err, w.hdr, status)) return;
  // from here on the call succeeds: hand the pages out
  for (int64_t k = tid; k < need_all; k += kPlan) {
    int lo = 0, hi = n - 1;  // the last place whose pages begin at or before k
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (agent_load(&w.off[mid]) <= k) lo = mid;
      else hi = mid - 1;
    }
    const int i = lo;
    const int32_t s = seqs[i], len = a.lens[s], cow = agent_load(&w.cow[i]);
    const int64_t j = k - agent_load(&w.off[i]);
    const int32_t pg = agent_load(&w.fl[k]);
    a.refs[pg] = 1;
    if (!(cow && j == 0)) a.table[(int64_t)s * g.max_pages + pages_of(len, g) + (j - cow)] = pg;
  }
  for (int64_t c = tid; c < copies_all; c += kPlan) {
    const int i = agent_load(&w.ctok[c]);
    const int32_t s = seqs[i], len = a.lens[s];
    int32_t *entry = &a.table[(int64_t)s * g.max_pages + (len >> g.log2P)];
    const int32_t from = *entry, to = agent_load(&w.fl[agent_load(&w.off[i])]);
    *entry = to;
    atomicAdd(&a.refs[from], -1);
    w.csrc[c] = from;
    w.cdst[c] = to;
    w.ctok[c] = len & (g.P - 1);
  }
  __syncthreads();
  for (int i = tid; i < n; i += kPlan)
    if (seqs[i] >= 0) a.lens[seqs[i]] += n_new[i];
  if (tid == 0) {
    w.hdr[kHdrOk] = 1;
    w.hdr[kHdrCopies] = (int32_t)copies_all;
  }
}

// The same for lists of at most kPlan places, a thread to each: what the list
// says stays in registers, and rows and pages are found again in hash tables in
// LDS instead of through memory (2 to 32 rows: 6.0 to 6.7 us against 9 to 10.7).
constexpr int kFree = 2048;  // free pages that LDS holds; more go through the workspace

__global__ __launch_bounds__(kPlan) void k_plan_extend(PGeo g, skv_pages a, const int32_t *__restrict__ seqs,
                                                       const int32_t *__restrict__ n_new, int n, PWork w,
                                                       int32_t *status) {
  __shared__ int err;
  __shared__ int64_t lds[kPlanWaves];
  __shared__ int row_key[kSlots], page_key[kSlots], page_cnt[kSlots], page_last[kSlots];
  __shared__ int32_t off[kPlan], entry0[kPlan];  // by place: pages given out before its own; -1 - (last entry) or first new entry
  __shared__ int32_t place_row[kPlan];
  __shared__ int32_t fl[kFree];
  const int tid = threadIdx.x;
  const int32_t s = tid < n ? seqs[tid] : -1, add = tid < n ? n_new[tid] : 0;
  int4 held4 = refs_of(g, a, (int64_t)tid * 4);  // the first ones, long before they are looked at
  if (tid == 0) err = 0;
  clear_keys(row_key);
  clear_keys(page_key);
  clear_keys(page_last);
  for (int i = tid; i < kSlots; i += kPlan) page_cnt[i] = 0;
  __syncthreads();
  int32_t len = 0, page = -1, held = 0;
  if (s >= 0) {
    if (s >= g.max_seqs || add < 0) {
      note(&err, SKV_ERR_ARG);
    } else {
      len = a.lens[s];
      bool had;
      put_key(row_key, s, had);
      if (had || len < 0 || len > g.max_tokens) {
        note(&err, SKV_ERR_ARG);
      } else if ((int64_t)len + add > g.max_tokens) {
        note(&err, SKV_ERR_PAGES);
      } else if (add > 0 && (len & (g.P - 1))) {
        page = a.table[(int64_t)s * g.max_pages + (len >> g.log2P)];
        held = good_page(page, g) ? a.refs[page] : 0;
        if (held < 1) note(&err, SKV_ERR_ARG);
      }
    }
  }
  if (failed(&err, w.hdr, status)) return;
  int at = 0;
  if (page >= 0) {
    bool had;
    at = put_key(page_key, page, had);
    atomicAdd(&page_cnt[at], 1);
    atomicMax(&page_last[at], tid);
  }
  __syncthreads();
  int64_t need = s >= 0 ? pages_of(len + add, g) - pages_of(len, g) : 0;
  bool cow = false;
  if (page >= 0) {
    if (held < page_cnt[at]) note(&err, SKV_ERR_ARG);  // fewer holds than holders
    cow = held > page_cnt[at] || page_last[at] != tid;
    need += cow;
  }
  // pages in the upper part, copies in the lower: one sum for both
  int64_t all;
  const int64_t before = block_scan(need << 16 | (int64_t)cow, all, lds);
  const int64_t need_all = all >> 16;
  const int copies = (int)(all & 0xFFFF);
  if (need_all > g.n_pages) note(&err, SKV_ERR_PAGES);
  off[tid] = (int32_t)min(before >> 16, (int64_t)INT32_MAX);  // beyond the pool only where the call fails
  entry0[tid] = cow ? -1 - (len >> g.log2P) : pages_of(len, g);
  place_row[tid] = s;
  if (failed(&err, w.hdr, status)) return;
  // the lowest free pages, in order
  const bool in_lds = need_all <= kFree;
  int64_t found = 0;
  for (int64_t base = 0; base < g.n_pages && found < need_all; base += (int64_t)kPlan * 4) {
    const int64_t p = base + (int64_t)tid * 4;
    const int4 r = base == 0 ? held4 : refs_of(g, a, p);
    int64_t t;
    int64_t k = found + block_scan((r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0), t, lds);
    const int32_t rs[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (rs[c] == 0) {
        if (!in_lds) agent_store(&w.fl[k], (int32_t)p + c);
        else if (k < need_all) fl[k] = (int32_t)p + c;
        ++k;
      }
    }
    found += t;
  }
  if (found < need_all) note(&err, SKV_ERR_PAGES);
  if (failed(&err, w.hdr, status)) return;
  // from here on the call succeeds: hand the pages out
  auto freed = [&](int64_t k) { return in_lds ? fl[k] : agent_load(&w.fl[k]); };
  for (int64_t k = tid; k < need_all; k += kPlan) {
    int lo = 0, hi = n - 1;  // the last place whose pages begin at or before k
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (off[mid] <= k) lo = mid;
      else hi = mid - 1;
    }
    const int32_t pg = freed(k), e = entry0[lo];
    const int64_t j = k - off[lo];
    a.refs[pg] = 1;
    a.table[(int64_t)place_row[lo] * g.max_pages + (e < 0 ? -1 - e : e) + j] = pg;  // its copy takes the entry before its new ones
  }
  if (cow) {
    const int c = (int)(before & 0xFFFF);
    atomicAdd(&a.refs[page], -1);
    w.csrc[c] = page;
    w.cdst[c] = freed(off[tid]);
    w.ctok[c] = len & (g.P - 1);
  }
  if (s >= 0) a.lens[s] = len + add;
  if (tid == 0) {
    w.hdr[kHdrOk] = 1;
    w.hdr[kHdrCopies] = copies;
  }
}

// ---- the list of copies, all layers ----
// U: the unit of a copy, 16 bytes, or 8 where a token's row has no more.  A
// workgroup takes pieces of kCopyUnits units of one (copy, layer) at a time.
constexpr int kCopyUnits = 1024;

// STREAM: past the caches, for much data; a page copied for a sequence that grows is soon read again
template <typename U, int STREAM>
__device__ __forceinline__ void copy_pages(const PGeo &g, uint8_t *pool, const PWork &w, int64_t first, int64_t step) {
  const int64_t copies = w.hdr[kHdrCopies];
  const uint32_t ru = (uint32_t)g.row_bytes / sizeof(U);             // units of a row
  const uint32_t hu = (uint32_t)g.P * ru;                            // units of a (kv, head) of the page
  const int64_t lu = g.page_bytes / (int64_t)sizeof(U);              // units of a page of one layer
  const int64_t pieces = (lu + kCopyUnits - 1) / kCopyUnits;
  const int64_t items = copies * g.layers * pieces;
  for (int64_t it = first; it < items; it += step) {
    const int64_t piece = it % pieces, rest = it / pieces;
    const int64_t l = rest % g.layers, c = rest / g.layers;
    const uint32_t keep = (uint32_t)w.ctok[c] * ru;  // units of a (kv, head) that hold tokens
    const U *s = reinterpret_cast<const U *>(pool + (l * g.n_pages + w.csrc[c]) * g.page_bytes);
    U *d = reinterpret_cast<U *>(pool + (l * g.n_pages + w.cdst[c]) * g.page_bytes);
    const int64_t u0 = piece * kCopyUnits;
    for (int64_t u = u0 + threadIdx.x; u < min(u0 + kCopyUnits, lu); u += blockDim.x)
      if ((uint32_t)(u & (hu - 1)) < keep) {
        if (STREAM) put(d + u, take(s + u));
        else d[u] = s[u];
      }
  }
}

template <typename U>
__global__ __launch_bounds__(256) void k_copy_pages(PGeo g, uint8_t *pool, PWork w) {
  copy_pages<U, 0>(g, pool, w, blockIdx.x, gridDim.x);
}

// ---- fork, truncate ----
// One workgroup checks the list; where the rows are few it also changes them,
// a wave to each (32 rows of 64 pages: one launch of 4.7 us instead of 3.6 and 4.0),
// else a second launch does, a workgroup to each.
constexpr int kRowsAtOnce = 64;  // rows of 64 entries, four to a wave

__device__ __forceinline__ void fork_row(const PGeo &g, const skv_pages &a, int32_t s, int32_t d, int32_t len,
                                         int first, int step, int32_t *status) {
  const int32_t np = pages_of(len, g);
  for (int32_t k = first; k < np; k += step) {
    const int32_t pg = a.table[(int64_t)s * g.max_pages + k];
    a.table[(int64_t)d * g.max_pages + k] = pg;
    if (good_page(pg, g)) atomicAdd(&a.refs[pg], 1);
    else set_status(status, SKV_ERR_ARG);
  }
  if (first == 0) a.lens[d] = len;
}

// `len` was read by all of the row's threads before any writes the new one
__device__ __forceinline__ void truncate_row(const PGeo &g, const skv_pages &a, int32_t s, int32_t len, int32_t to,
                                             int first, int step, int32_t *status) {
  const int32_t np = pages_of(len, g);
  for (int32_t k = pages_of(to, g) + first; k < np; k += step) {
    int32_t *entry = &a.table[(int64_t)s * g.max_pages + k];
    const int32_t pg = *entry;
    *entry = -1;
    if (good_page(pg, g)) atomicSub(&a.refs[pg], 1);
    else set_status(status, SKV_ERR_ARG);
  }
  if (first == 0) a.lens[s] = to;
}

__global__ __launch_bounds__(kPlan) void k_check_fork(PGeo g, skv_pages a, const int32_t *__restrict__ src,
                                                      const int32_t *__restrict__ dst,
                                                      const int32_t *__restrict__ n_tokens, int n, int apply, PWork w,
                                                      int32_t *status) {
  __shared__ int err, keys[kSlots];
  if (threadIdx.x == 0) err = 0;
  clear_keys(keys);
  __syncthreads();
  const bool few = n <= kPlan;
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int32_t s = src[i], d = dst[i], to = n_tokens ? n_tokens[i] : 0;
    if (s < 0 || d < 0) continue;
    if (s >= g.max_seqs || d >= g.max_seqs) { note(&err, SKV_ERR_ARG); continue; }
    const int32_t len = a.lens[s];
    if (len < 0 || len > g.max_tokens || a.lens[d] != 0 || to < 0 || to > len) note(&err, SKV_ERR_ARG);
    if (few) {
      bool had;
      put_key(keys, d, had);
      if (had) note(&err, SKV_ERR_ARG);
    } else {
      agent_store(&w.mark[s], -1);
      agent_store(&w.mark[d], -1);
    }
  }
  __syncthreads();
  if (!few) {
    for (int i = threadIdx.x; i < n; i += kPlan)
      if (src[i] >= 0 && dst[i] >= 0 && src[i] < g.max_seqs && dst[i] < g.max_seqs) agent_store(&w.mark[dst[i]], i);
    __syncthreads();
  }
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int32_t s = src[i], d = dst[i];
    if (s < 0 || d < 0 || s >= g.max_seqs || d >= g.max_seqs) continue;
    if (few ? has_key(keys, s) : agent_load(&w.mark[d]) != i || agent_load(&w.mark[s]) != -1) note(&err, SKV_ERR_ARG);
  }
  if (failed(&err, w.hdr, status)) return;
  if (threadIdx.x == 0) w.hdr[kHdrOk] = 1;
  if (!apply) return;
  for (int i = threadIdx.x >> 6; i < n; i += kPlanWaves)
    if (src[i] >= 0 && dst[i] >= 0)
      fork_row(g, a, src[i], dst[i], n_tokens ? n_tokens[i] : a.lens[src[i]], threadIdx.x & 63, 64, status);
}

__global__ __launch_bounds__(256) void k_fork(PGeo g, skv_pages a, const int32_t *__restrict__ src,
                                              const int32_t *__restrict__ dst, const int32_t *__restrict__ n_tokens,
                                              PWork w, int32_t *status) {
  const int i = blockIdx.x;
  if (w.hdr[kHdrOk] == 0 || src[i] < 0 || dst[i] < 0) return;
  fork_row(g, a, src[i], dst[i], n_tokens ? n_tokens[i] : a.lens[src[i]], threadIdx.x, blockDim.x, status);
}

__global__ __launch_bounds__(kPlan) void k_check_truncate(PGeo g, skv_pages a, const int32_t *__restrict__ seqs,
                                                          const int32_t *__restrict__ keep, int n, int apply, PWork w,
                                                          int32_t *status) {
  __shared__ int err, keys[kSlots];
  if (threadIdx.x == 0) err = 0;
  clear_keys(keys);
  __syncthreads();
  const bool few = n <= kPlan;
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int32_t s = seqs[i], to = keep ? keep[i] : 0;
    if (s < 0) continue;
    if (s >= g.max_seqs) { note(&err, SKV_ERR_ARG); continue; }
    const int32_t len = a.lens[s];
    if (len < 0 || len > g.max_tokens || to < 0 || to > len) note(&err, SKV_ERR_ARG);
    if (few) {
      bool had;
      put_key(keys, s, had);
      if (had) note(&err, SKV_ERR_ARG);
    } else {
      agent_store(&w.mark[s], i);
    }
  }
  if (!few) {
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlan)
      if (seqs[i] >= 0 && seqs[i] < g.max_seqs && agent_load(&w.mark[seqs[i]]) != i) note(&err, SKV_ERR_ARG);
  }
  if (failed(&err, w.hdr, status)) return;
  if (threadIdx.x == 0) w.hdr[kHdrOk] = 1;
  if (!apply) return;
  for (int i = threadIdx.x >> 6; i < n; i += kPlanWaves)
    if (seqs[i] >= 0) truncate_row(g, a, seqs[i], a.lens[seqs[i]], keep ? keep[i] : 0, threadIdx.x & 63, 64, status);
}

__global__ __launch_bounds__(256) void k_truncate(PGeo g, skv_pages a, const int32_t *__restrict__ seqs,
                                                  const int32_t *__restrict__ keep, PWork w, int32_t *status) {
  const int i = blockIdx.x;
  if (w.hdr[kHdrOk] == 0 || seqs[i] < 0) return;
  const int32_t len = a.lens[seqs[i]];
  __syncthreads();
  truncate_row(g, a, seqs[i], len, keep ? keep[i] : 0, threadIdx.x, blockDim.x, status);
}

// ---- compact ----
// four pages to a thread; free and used pages are counted in the two halves of one sum
__global__ __launch_bounds__(kPlan) void k_plan_compact(PGeo g, skv_pages a, int32_t *n_live, PWork w) {
  __shared__ int64_t lds[kPlanWaves];
  const int tid = threadIdx.x;
  const int64_t step = (int64_t)kPlan * 4;
  const int4 first = refs_of(g, a, (int64_t)tid * 4);
  auto used_of = [&](int64_t p, const int4 &r) {  // a bit per page
    const int in = (int)max((int64_t)0, min((int64_t)4, g.n_pages - p));
    return ((r.x > 0) | (r.y > 0) << 1 | (r.z > 0) << 2 | (r.w > 0) << 3) & ((1 << in) - 1);
  };
  int64_t mine = 0, live;
  for (int64_t p = (int64_t)tid * 4; p < g.n_pages; p += step) mine += __builtin_popcount(used_of(p, p < step ? first : refs_of(g, a, p)));
  block_scan(mine, live, lds);
  int64_t holes = 0, movers = 0;
  for (int64_t base = 0; base < g.n_pages; base += step) {
    const int64_t p = base + (int64_t)tid * 4;
    const int used = used_of(p, base == 0 ? first : refs_of(g, a, p));
    const int in = (int)max((int64_t)0, min((int64_t)4, g.n_pages - p)), low = (int)max((int64_t)0, min((int64_t)4, live - p));
    const int hole = ~used & ((1 << low) - 1), mover = used & ~((1 << low) - 1);
    int64_t all;
    const int64_t before = block_scan((int64_t)__builtin_popcount(hole) << 32 | __builtin_popcount(mover), all, lds);
    int64_t h = holes + (before >> 32), m = movers + (int32_t)before;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (hole >> c & 1) agent_store(&w.cdst[h++], (int32_t)p + c);
      if (mover >> c & 1) agent_store(&w.csrc[m++], (int32_t)p + c);
      if (c >= low && c < in) w.cnt[p + c] = -1;  // its new place, once it has one
    }
    holes += all >> 32;
    movers += (int32_t)all;
  }
  __syncthreads();
  // as many free pages below n_live as used ones above it
  for (int64_t c = tid; c < movers; c += kPlan) {
    const int32_t from = agent_load(&w.csrc[c]), to = agent_load(&w.cdst[c]);
    a.refs[to] = a.refs[from];
    a.refs[from] = 0;
    w.cnt[from] = to;
    w.ctok[c] = g.P;
  }
  if (tid == 0) {
    *n_live = (int32_t)live;
    w.hdr[kHdrCopies] = (int32_t)movers;
    w.hdr[kHdrLive] = (int32_t)live;
  }
}

// pages that moved: their ids in the table; the other workgroups copy
template <typename U>
__global__ __launch_bounds__(256) void k_move_pages(PGeo g, skv_pages a, PWork w, int rename_blocks, int32_t *status) {
  if ((int)blockIdx.x >= rename_blocks) {
    copy_pages<U, 1>(g, static_cast<uint8_t *>(a.pool), w, blockIdx.x - rename_blocks, gridDim.x - rename_blocks);
    return;
  }
  const int32_t live = w.hdr[kHdrLive];
  for (int64_t s = blockIdx.x; s < g.max_seqs; s += rename_blocks) {
    const int32_t len = a.lens[s];
    if (len < 0 || len > g.max_tokens) {
      if (threadIdx.x == 0) set_status(status, SKV_ERR_ARG);
      continue;
    }
    const int32_t np = pages_of(len, g);
    for (int32_t k = threadIdx.x; k < np; k += blockDim.x) {
      int32_t *entry = &a.table[s * g.max_pages + k];
      const int32_t pg = *entry;
      if (!good_page(pg, g)) set_status(status, SKV_ERR_ARG);
      else if (pg >= live) {
        if (w.cnt[pg] >= 0) *entry = w.cnt[pg];
        else set_status(status, SKV_ERR_ARG);  // a page that refs calls free
      }
    }
  }
}

// ---- tokens in ----
// Bytes: two bf16 rows read and two rows written per token, once.  A thread
// takes 8 channels: 16 bytes in, 16 (bf16) or 8 (e4m3) out.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
  // the conversion instruction rounds to nearest even; a value past 448 is held
  // there before it, and a NaN, which min/max would replace, passes beside them
  const float x = a != a ? a : __builtin_fminf(__builtin_fmaxf(a, -448.0f), 448.0f);
  const float y = b != b ? b : __builtin_fminf(__builtin_fmaxf(b, -448.0f), 448.0f);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x, y, 0, false) & 0xFFFFu;
}

// Eight bf16 values over a scale, as e4m3.  The quotient is the correctly
// rounded one (the rounding to 4 bits would show a difference at ties), but a
// division costs a dozen instructions.  With y = 1 / s rounded, q = a y and the
// exact remainder r = q s - a (by fma), q - r y is that quotient for every bf16
// mantissa a over every fp32 mantissa s (all 2^30 pairs were tried), so long as
// nothing overflows, which the limits of 2^60 on s, 1 / s and |a| see to; a
// remainder that underflows belongs to a quotient far below e4m3's smallest value.
// With s > 0 zeros keep their signs.  Infinities, NaN and other scales take the
// division.  16376 tokens of 2048 values: 31 us with divisions, 21 without.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

struct Scale {
  float s, y;
  bool good;
  __device__ __forceinline__ explicit Scale(float scale) : s(scale), y(1.0f / scale), good(scale >= 0x1p-60f && scale <= 0x1p60f) {}
  __device__ __forceinline__ float over(float a) const {
    const float q = a * y;
    return __builtin_amdgcn_fmed3f(__builtin_fmaf(-__builtin_fmaf(q, s, -a), y, q), -448.0f, 448.0f);
  }
  __device__ __forceinline__ uint32_t four(uint32_t w0, uint32_t w1) const {
    const float a = __uint_as_float(w0 << 16), b = __uint_as_float(w0 & 0xFFFF0000u);
    const float c = __uint_as_float(w1 << 16), d = __uint_as_float(w1 & 0xFFFF0000u);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(over(c), over(d), __builtin_amdgcn_cvt_pk_fp8_f32(over(a), over(b), 0, false), true);
  }
  __device__ __forceinline__ uint32_t two(uint32_t w) const {
    return e4m3_pair(__uint_as_float(w << 16) / s, __uint_as_float(w & 0xFFFF0000u) / s);
  }
  __device__ __forceinline__ u32x2 eight(u32x4 x) const {
    u16x2 m = {0, 0};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t mag = x[c] & 0x7FFF7FFFu;
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, mag));
    }
    if (__builtin_amdgcn_ballot_w64(!good || max(m.x, m.y) > 0x5D80) == 0) return u32x2{four(x.x, x.y), four(x.z, x.w)};
    return u32x2{two(x.x) | two(x.y) << 16, two(x.z) | two(x.w) << 16};
  }
};

//
// A workgroup takes `tokens` tokens, 256 units of each at a time.  Where a token
// goes is a chain of four loads (row, length, table, holders), which one thread
// per token goes through while the symbols of all of them are on their way.
constexpr int kStoreTokens = 8;

template <int E4M3>
__global__ __launch_bounds__(256) void k_store(PGeo g, skv_pages a, int layer, const uint16_t *__restrict__ k,
                                               int64_t ks, const uint16_t *__restrict__ v, int64_t vs,
                                               const float *__restrict__ k_scale, const float *__restrict__ v_scale,
                                               const int32_t *__restrict__ seqs, const int32_t *__restrict__ pos,
                                               int64_t n, int tokens, int parts, int32_t *status) {
  __shared__ int64_t to[256];  // a token's place in the pool; -1: none
  const int half = g.heads * g.D / 8, units = 2 * half;  // units of a token
  const int at_once = parts > 1 ? 1 : 256 / units;       // tokens that the workgroup's threads cover
  const int64_t t0 = (int64_t)(blockIdx.x / (uint32_t)parts) * tokens;
  const int j = parts > 1 ? 0 : threadIdx.x / units;
  const int u = parts > 1 ? (int)(blockIdx.x % (uint32_t)parts) * 256 + threadIdx.x : threadIdx.x - j * units;
  const bool in = u < units && j < at_once;
  const int which = u >= half, hu = which ? u - half : u;
  u32x4 x[kStoreTokens];
#pragma unroll
  for (int r = 0; r < kStoreTokens; ++r) {
    const int64_t t = t0 + r * at_once + j;
    if (in && r * at_once + j < tokens && t < n) x[r] = take(reinterpret_cast<const u32x4 *>((which ? v + t * vs : k + t * ks) + hu * 8));
  }
  if (threadIdx.x < tokens) {
    const int64_t t = t0 + threadIdx.x;
    int64_t at = -1;
    const int32_t s = t < n ? seqs[t] : -1;
    if (s >= 0) {
      bool good = s < g.max_seqs;
      if (good) {
        const int32_t p = pos[t], len = a.lens[s];
        good = p >= 0 && p < len && len <= g.max_tokens;
        if (good) {
          const int32_t pg = a.table[(int64_t)s * g.max_pages + (p >> g.log2P)];
          good = good_page(pg, g) && a.refs[pg] == 1;
          if (good) at = ((int64_t)layer * g.n_pages + pg) * g.page_bytes + (int64_t)(p & (g.P - 1)) * g.row_bytes;
        }
      }
      if (!good) set_status(status, SKV_ERR_ARG);
    }
    to[threadIdx.x] = at;
  }
  __syncthreads();
  if (!in) return;
  const int h = hu * 8 >> g.log2D, c = hu * 8 & (g.D - 1);
  const float *sp = which ? v_scale : k_scale;
  const Scale sc(E4M3 && sp ? sp[h] : 1.0f);
  uint8_t *base = static_cast<uint8_t *>(a.pool) + (int64_t)(which * g.heads + h) * g.P * g.row_bytes + c * (E4M3 ? 1 : 2);
#pragma unroll
  for (int r = 0; r < kStoreTokens; ++r) {
    const int i = r * at_once + j;
    if (i >= tokens || to[i] < 0) continue;
    if (E4M3) {
      *reinterpret_cast<u32x2 *>(base + to[i]) = sc.eight(x[r]);
    } else {
      *reinterpret_cast<u32x4 *>(base + to[i]) = x[r];
    }
  }
}

// ---- pages <-> the coder's layout ----
// Bytes: each symbol read and written once.  A workgroup takes one (layer, kv,
// head) row's block of tokens; x and each page's part of the row are contiguous.
constexpr int kMoveTokens = 64;

template <typename U, int SCATTER>
__global__ __launch_bounds__(256) void k_reorder(PGeo g, skv_pages a, int seq, int32_t first, int64_t tokens,
                                                 int tiles, int64_t item0, uint8_t *x, int32_t *status) {
  const int32_t len = a.lens[seq];
  if (len < 0 || len > g.max_tokens || first + tokens > len) {
    if (threadIdx.x == 0) set_status(status, SKV_ERR_ARG);
    return;
  }
  const uint32_t ru = (uint32_t)g.row_bytes / sizeof(U);  // a power of two
  const int lr = __builtin_ctz(ru);
  const int rows = 2 * g.heads;
  const int64_t item = item0 + blockIdx.x, row = quotient(item, tiles), l = quotient(row, rows);
  const int kvh = (int)(row - l * rows);
  U *xr = reinterpret_cast<U *>(x) + (row * tokens << lr);
  const int64_t t0 = (item - row * tiles) * kMoveTokens;
  const uint32_t units = (uint32_t)min((int64_t)kMoveTokens, tokens - t0) << lr;
  for (uint32_t u = threadIdx.x; u < units; u += blockDim.x) {
    const int64_t t = t0 + (u >> lr);
    const uint32_t p = (uint32_t)(first + t);
    const int32_t pg = a.table[(int64_t)seq * g.max_pages + (p >> g.log2P)];
    if (!good_page(pg, g) || (SCATTER && a.refs[pg] != 1)) { set_status(status, SKV_ERR_ARG); continue; }
    U *c = reinterpret_cast<U *>(static_cast<uint8_t *>(a.pool) + (l * g.n_pages + pg) * g.page_bytes) +
           (((int64_t)kvh * g.P + (p & (g.P - 1))) << lr) + (u & (ru - 1));
    U *b = xr + (t0 << lr) + u;
    if (SCATTER) put(c, take(b));
    else put(b, take(c));
  }
}

__global__ void k_pages_reset(int32_t *table, int64_t entries, int32_t *lens, int64_t seqs, int32_t *refs, int64_t pages) {
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  for (int64_t i = at; i < entries; i += step) table[i] = -1;
  for (int64_t i = at; i < seqs; i += step) lens[i] = 0;
  for (int64_t i = at; i < pages; i += step) refs[i] = 0;
}

// ---- host side ----
int launched() { return hipGetLastError() == hipSuccess ? SKV_OK : SKV_ERR_HIP; }

// the checks that the planning calls share
int plan_args(const skv_pages_shape *shape, const skv_pages *pages, const void *list, int64_t n, void *workspace,
              size_t bytes, int32_t *status, PGeo &g, PWork &w) {
  int e = make_pgeo(shape, g);
  if (e != SKV_OK) return e;
  if ((e = check_pages(pages)) != SKV_OK) return e;
  if (!workspace || !aligned16(workspace) || !status || !aligned4(status)) return SKV_ERR_ARG;
  if (n < 0 || n > g.max_seqs || (n > 0 && (!list || !aligned4(list)))) return SKV_ERR_ARG;
  w = carve_pages(g, workspace);
  return bytes < w.total ? SKV_ERR_ARG : SKV_OK;
}

bool few_rows(const PGeo &g, int64_t n) { return n * ((g.max_pages + 63) / 64) <= kRowsAtOnce; }

// workgroups of a copy of `pages` pages at most, in all layers
int64_t copy_blocks(const PGeo &g, int64_t pages) {
  const int64_t unit = g.row_bytes >= 16 ? 16 : 8;
  const int64_t pieces = (g.page_bytes / unit + kCopyUnits - 1) / kCopyUnits;
  const int64_t most = (int64_t)device_cu_count() * 16;
  const __int128 items = (__int128)pages * g.layers * pieces;
  return items < most ? (int64_t)items : most;
}

}  // namespace

extern "C" int skv_pages_pool_size(const skv_pages_shape *shape, size_t *bytes) {
  PGeo g;
  int e = make_pgeo(shape, g);
  if (e != SKV_OK) return e;
  if (!bytes) return SKV_ERR_ARG;
  *bytes = (size_t)g.page_bytes * (size_t)g.n_pages * (size_t)g.layers;
  return SKV_OK;
}

extern "C" int skv_pages_workspace_size(const skv_pages_shape *shape, size_t *bytes) {
  PGeo g;
  int e = make_pgeo(shape, g);
  if (e != SKV_OK) return e;
  if (!bytes) return SKV_ERR_ARG;
  *bytes = carve_pages(g, nullptr).total;
  return SKV_OK;
}

extern "C" int skv_pages_reset(const skv_pages_shape *shape, const skv_pages *pages, void *stream) {
  PGeo g;
  int e = make_pgeo(shape, g);
  if (e != SKV_OK) return e;
  if ((e = check_pages(pages)) != SKV_OK) return e;
  const int64_t entries = g.max_seqs * g.max_pages;
  const int64_t blocks = (entries + g.n_pages + 255) / 256, most = (int64_t)device_cu_count() * 8;
  k_pages_reset<<<dim3((uint32_t)(blocks < most ? blocks : most)), 256, 0, static_cast<hipStream_t>(stream)>>>(
      pages->table, entries, pages->lens, g.max_seqs, pages->refs, g.n_pages);
  return launched();
}

extern "C" int skv_pages_extend(const skv_pages_shape *shape, const skv_pages *pages, const int32_t *seqs,
                                const int32_t *n_new, int64_t n, void *workspace, size_t workspace_bytes,
                                int32_t *status, void *stream) {
  PGeo g;
  PWork w;
  int e = plan_args(shape, pages, seqs, n, workspace, workspace_bytes, status, g, w);
  if (e != SKV_OK) return e;
  if (n == 0) return SKV_OK;
  if (!n_new || !aligned4(n_new)) return SKV_ERR_ARG;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (n <= kPlan) k_plan_extend<<<1, kPlan, 0, st>>>(g, *pages, seqs, n_new, (int)n, w, status);
  else k_plan_extend_long<<<1, kPlan, 0, st>>>(g, *pages, seqs, n_new, (int)n, w, status);
  if ((e = launched()) != SKV_OK) return e;
  const dim3 blocks((uint32_t)copy_blocks(g, n));
  uint8_t *pool = static_cast<uint8_t *>(pages->pool);
  if (g.row_bytes >= 16) k_copy_pages<u32x4><<<blocks, 256, 0, st>>>(g, pool, w);
  else k_copy_pages<u32x2><<<blocks, 256, 0, st>>>(g, pool, w);
  return launched();
}

extern "C" int skv_pages_fork(const skv_pages_shape *shape, const skv_pages *pages, const int32_t *src,
                              const int32_t *dst, const int32_t *n_tokens, int64_t n, void *workspace,
                              size_t workspace_bytes, int32_t *status, void *stream) {
  PGeo g;
  PWork w;
  int e = plan_args(shape, pages, src, n, workspace, workspace_bytes, status, g, w);
  if (e != SKV_OK) return e;
  if (n == 0) return SKV_OK;
  if (!dst || !aligned4(dst) || !aligned4(n_tokens)) return SKV_ERR_ARG;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool apply = few_rows(g, n);
  k_check_fork<<<1, kPlan, 0, st>>>(g, *pages, src, dst, n_tokens, (int)n, apply, w, status);
  if ((e = launched()) != SKV_OK || apply) return e;
  k_fork<<<dim3((uint32_t)n), 256, 0, st>>>(g, *pages, src, dst, n_tokens, w, status);
  return launched();
}

extern "C" int skv_pages_truncate(const skv_pages_shape *shape, const skv_pages *pages, const int32_t *seqs,
                                  const int32_t *keep, int64_t n, void *workspace, size_t workspace_bytes,
                                  int32_t *status, void *stream) {
  PGeo g;
  PWork w;
  int e = plan_args(shape, pages, seqs, n, workspace, workspace_bytes, status, g, w);
  if (e != SKV_OK) return e;
  if (n == 0) return SKV_OK;
  if (!aligned4(keep)) return SKV_ERR_ARG;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool apply = few_rows(g, n);
  k_check_truncate<<<1, kPlan, 0, st>>>(g, *pages, seqs, keep, (int)n, apply, w, status);
  if ((e = launched()) != SKV_OK || apply) return e;
  k_truncate<<<dim3((uint32_t)n), 256, 0, st>>>(g, *pages, seqs, keep, w, status);
  return launched();
}

extern "C" int skv_pages_compact(const skv_pages_shape *shape, const skv_pages *pages, int32_t *n_live,
                                 void *workspace, size_t workspace_bytes, int32_t *status, void *stream) {
  PGeo g;
  PWork w;
  int e = plan_args(shape, pages, nullptr, 0, workspace, workspace_bytes, status, g, w);
  if (e != SKV_OK) return e;
  if (!n_live || !aligned4(n_live)) return SKV_ERR_ARG;
  hipStream_t st = static_cast<hipStream_t>(stream);
  k_plan_compact<<<1, kPlan, 0, st>>>(g, *pages, n_live, w);
  if ((e = launched()) != SKV_OK) return e;
  const int64_t cus = device_cu_count();
  const int rename = (int)(g.max_seqs < cus ? g.max_seqs : cus);
  const dim3 blocks((uint32_t)(rename + copy_blocks(g, (g.n_pages + 1) / 2)));  // at most half the pages move
  if (g.row_bytes >= 16) k_move_pages<u32x4><<<blocks, 256, 0, st>>>(g, *pages, w, rename, status);
  else k_move_pages<u32x2><<<blocks, 256, 0, st>>>(g, *pages, w, rename, status);
  return launched();
}

extern "C" int skv_pages_store(const skv_pages_shape *shape, const skv_pages *pages, int64_t layer, const void *k,
                               int64_t k_stride, const void *v, int64_t v_stride, const float *k_scale,
                               const float *v_scale, const int32_t *seqs, const int32_t *pos, int64_t n,
                               int32_t *status, void *stream) {
  PGeo g;
  int e = make_pgeo(shape, g);
  if (e != SKV_OK) return e;
  if ((e = check_pages(pages)) != SKV_OK) return e;
  if (layer < 0 || layer >= g.layers || n < 0 || n > INT32_MAX || !status || !aligned4(status)) return SKV_ERR_ARG;
  if (n == 0) return SKV_OK;
  const int64_t row = (int64_t)g.heads * g.D;
  if (!k || !v || !seqs || !pos || !aligned16(k) || !aligned16(v) || !aligned4(seqs) || !aligned4(pos)) return SKV_ERR_ARG;
  if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8) return SKV_ERR_ARG;
  if (k_stride > INT64_MAX / 2 / n || v_stride > INT64_MAX / 2 / n) return SKV_ERR_ARG;
  if ((k_scale || v_scale) && g.fmt != SKV_SYM_E4M3) return SKV_ERR_ARG;
  if (!aligned4(k_scale) || !aligned4(v_scale)) return SKV_ERR_ARG;
  // as many tokens to a workgroup, up to eight rounds of its threads, as leave every CU four workgroups
  const int64_t units = 2 * row / 8, at_once = units <= 256 ? 256 / units : 1, parts = (units + 255) / 256;
  const int64_t want = n * parts / (device_cu_count() * 4);
  const int64_t rounds = want / at_once < 1 ? 1 : (want / at_once < kStoreTokens ? want / at_once : kStoreTokens);
  const int64_t tokens = rounds * at_once < 256 ? rounds * at_once : 256;
  const int64_t most = kMaxGrid / parts * tokens;  // of a launch
  hipStream_t st = static_cast<hipStream_t>(stream);
  for (int64_t t = 0; t < n; t += most) {
    const int64_t here = n - t < most ? n - t : most;
    const dim3 grid((uint32_t)((here + tokens - 1) / tokens * parts));
    const uint16_t *kp = static_cast<const uint16_t *>(k) + t * k_stride, *vp = static_cast<const uint16_t *>(v) + t * v_stride;
    if (g.fmt == SKV_SYM_E4M3)
      k_store<1><<<grid, 256, 0, st>>>(g, *pages, (int)layer, kp, k_stride, vp, v_stride, k_scale, v_scale, seqs + t, pos + t, here, (int)tokens, (int)parts, status);
    else
      k_store<0><<<grid, 256, 0, st>>>(g, *pages, (int)layer, kp, k_stride, vp, v_stride, nullptr, nullptr, seqs + t, pos + t, here, (int)tokens, (int)parts, status);
    if ((e = launched()) != SKV_OK) return e;
  }
  return SKV_OK;
}

namespace {
int reorder(const skv_pages_shape *shape, const skv_pages *pages, int64_t seq, int64_t first, int64_t tokens,
            void *x, int32_t *status, void *stream, bool scatter) {
  PGeo g;
  int e = make_pgeo(shape, g);
  if (e != SKV_OK) return e;
  if ((e = check_pages(pages)) != SKV_OK) return e;
  if (seq < 0 || seq >= g.max_seqs || first < 0 || tokens < 0 || !status || !aligned4(status)) return SKV_ERR_ARG;
  if (first > g.max_tokens || tokens > g.max_tokens - first) return SKV_ERR_ARG;
  if (tokens == 0) return SKV_OK;
  if (!x || !aligned16(x)) return SKV_ERR_ARG;
  const int tiles = (int)((tokens + kMoveTokens - 1) / kMoveTokens);
  const int64_t items = (int64_t)g.layers * 2 * g.heads * tiles;
  hipStream_t st = static_cast<hipStream_t>(stream);
  uint8_t *xb = static_cast<uint8_t *>(x);
  const int32_t f = (int32_t)first;
  const int sq = (int)seq;
  for (int64_t i = 0; i < items; i += kMaxGrid) {
    const dim3 grid((uint32_t)(items - i < kMaxGrid ? items - i : kMaxGrid));
    if (g.row_bytes >= 16) {
      if (scatter) k_reorder<u32x4, 1><<<grid, 256, 0, st>>>(g, *pages, sq, f, tokens, tiles, i, xb, status);
      else k_reorder<u32x4, 0><<<grid, 256, 0, st>>>(g, *pages, sq, f, tokens, tiles, i, xb, status);
    } else {
      if (scatter) k_reorder<u32x2, 1><<<grid, 256, 0, st>>>(g, *pages, sq, f, tokens, tiles, i, xb, status);
      else k_reorder<u32x2, 0><<<grid, 256, 0, st>>>(g, *pages, sq, f, tokens, tiles, i, xb, status);
    }
    if ((e = launched()) != SKV_OK) return e;
  }
  return SKV_OK;
}
}  // namespace

extern "C" int skv_pages_gather(const skv_pages_shape *shape, const skv_pages *pages, int64_t seq, int64_t first,
                                int64_t tokens, void *x, int32_t *status, void *stream) {
  return reorder(shape, pages, seq, first, tokens, x, status, stream, false);
}

extern "C" int skv_pages_scatter(const skv_pages_shape *shape, const skv_pages *pages, int64_t seq, int64_t first,
                                 int64_t tokens, const void *x, int32_t *status, void *stream) {
  return reorder(shape, pages, seq, first, tokens, const_cast<void *>(x), status, stream, true);
}
