// skv_pages.hpp -- geometry, argument checks and small device helpers shared by
// the paged cache's calls and the attention that reads it.
#pragma once

#include "skv_internal.hpp"

namespace skv {

// Everything a kernel needs to know about a paged cache.
struct PGeo {
  int64_t n_pages, max_seqs, max_pages;
  int64_t page_bytes;  // one page of one layer: 2 * heads * page_tokens * row_bytes, contiguous
  int layers, heads, D, P;
  int log2P, log2D;
  int fmt;
  int esz;             // bytes of a symbol
  int row_bytes;       // one token of one (kv, head): D * esz
  int32_t max_tokens;  // max_pages * P
};

// Workgroups of a launch at most, where the number follows the data: HIP launches
// fewer than 2^32 threads in all, which 2^24 workgroups of 256 would reach.  More
// are launched in turn.
constexpr int64_t kMaxGrid = 1 << 23;

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// shape checks and derived geometry; SKV_OK or an error
inline int make_pgeo(const skv_pages_shape *sh, PGeo &g) {
  if (!sh || sh->reserved != 0) return SKV_ERR_ARG;
  if (sh->layers < 1 || sh->layers > (1 << 20) || sh->kv_heads < 1 || sh->kv_heads > (1 << 16)) return SKV_ERR_ARG;
  if (sh->sym_fmt != SKV_SYM_BF16 && sh->sym_fmt != SKV_SYM_E4M3) return SKV_ERR_ARG;
  if (sh->head_dim < 1) return SKV_ERR_ARG;
  if (sh->head_dim % 8 != 0 || 512 % sh->head_dim != 0) return SKV_ERR_UNSUPPORTED;
  if (sh->page_tokens < 16 || sh->page_tokens > kChunkTokens || (sh->page_tokens & (sh->page_tokens - 1))) return SKV_ERR_ARG;
  if (sh->n_pages < 1 || sh->n_pages > (1 << 30) || sh->max_seqs < 1 || sh->max_seqs > (1 << 20)) return SKV_ERR_ARG;
  if (sh->max_pages < 1 || sh->max_pages > ((int64_t)1 << 30) / sh->page_tokens) return SKV_ERR_ARG;
  g.layers = (int)sh->layers;
  g.heads = (int)sh->kv_heads;
  g.D = (int)sh->head_dim;
  g.P = (int)sh->page_tokens;
  g.log2P = __builtin_ctz((unsigned)g.P);
  g.log2D = __builtin_ctz((unsigned)g.D);
  g.n_pages = sh->n_pages;
  g.max_seqs = sh->max_seqs;
  g.max_pages = sh->max_pages;
  g.fmt = sh->sym_fmt;
  g.esz = sh->sym_fmt == SKV_SYM_BF16 ? 2 : 1;
  g.row_bytes = g.D * g.esz;
  g.page_bytes = (int64_t)2 * g.heads * g.P * g.row_bytes;
  g.max_tokens = (int32_t)(g.max_pages * g.P);
  // the whole pool is addressed in 64 bits
  if ((__int128)g.page_bytes * g.n_pages * g.layers > ((__int128)1 << 62)) return SKV_ERR_ARG;
  return SKV_OK;
}

inline int check_pages(const skv_pages *p) {
  if (!p || !p->pool || !p->table || !p->lens || !p->refs) return SKV_ERR_ARG;
  if (!aligned16(p->pool) || !aligned4(p->table) || !aligned4(p->lens) || !aligned16(p->refs)) return SKV_ERR_ARG;
  return SKV_OK;
}

// ---- device helpers ----

__device__ __forceinline__ int32_t pages_of(int32_t tokens, const PGeo &g) {
  return (int32_t)(((uint32_t)tokens + (uint32_t)g.P - 1) >> g.log2P);
}

__device__ __forceinline__ bool good_page(int32_t pg, const PGeo &g) { return (uint32_t)pg < (uint64_t)g.n_pages; }

// a / b; of 32 bits where both are, as they are nearly always
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((uint64_t)a | (uint64_t)b) >> 32) return a / b;
  return (uint32_t)a / (uint32_t)b;
}

// agent-scope accesses: read and written in L2, past the CU's own cache
__device__ __forceinline__ int32_t agent_load(const int32_t *p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void agent_store(int32_t *p, int32_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace skv
