// skv_attend.hip -- attention of one new token per sequence over a paged cache.
// Contract: skv.h.
#include <math.h>

#include "skv_pages.hpp"

using namespace skv;

namespace {

struct AttendArgs {
  const uint16_t *q;
  int64_t q_stride;
  int q_heads;
  float scale;
  const float *k_scale, *v_scale;
  const int32_t *seqs;
  uint16_t *out;
  float *lse;
};

__device__ __forceinline__ float symbol_value(const uint8_t *row, int c, int fmt) {
  if (fmt == SKV_SYM_BF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(row)[c] << 16);
  return __builtin_amdgcn_cvt_f32_fp8((int)row[c], 0);
}

__device__ __forceinline__ uint16_t bf16_rne(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);
  return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

// One wave per (sequence, query head): a pass over the tokens, 64 at a time, a
// token per lane for the scores and a channel per lane for the sum, with the
// running maximum m and sum l of the softmax; the sum is scaled when m grows.
__global__ __launch_bounds__(64) void k_attend(PGeo g, skv_pages a, int layer, AttendArgs p, int32_t *status) {
  __shared__ float qs[512];
  __shared__ float ps[64];
  __shared__ int32_t pg_of[64];
  const int lane = threadIdx.x;
  const int64_t i = blockIdx.x / p.q_heads;
  const int j = blockIdx.x - (int)i * p.q_heads;
  const int32_t s = p.seqs[i];
  if (s < 0) return;
  if (s >= g.max_seqs) { set_status(status, SKV_ERR_ARG); return; }
  int32_t len = a.lens[s];
  if (len < 0 || len > g.max_tokens) {
    set_status(status, SKV_ERR_ARG);
    len = 0;
  }
  const int h = j / (p.q_heads / g.heads);
  for (int c = lane; c < g.D; c += 64) qs[c] = __uint_as_float((uint32_t)p.q[i * p.q_stride + (int64_t)j * g.D + c] << 16);
  __syncthreads();
  const float sc = p.scale * (p.k_scale ? p.k_scale[h] : 1.0f);
  const uint8_t *base = static_cast<const uint8_t *>(a.pool) + (int64_t)layer * g.n_pages * g.page_bytes;
  const int64_t koff = (int64_t)h * g.P * g.row_bytes, voff = koff + (int64_t)g.heads * g.P * g.row_bytes;
  float m = -INFINITY, l = 0.0f, o[8] = {};
  for (int32_t t0 = 0; t0 < len; t0 += 64) {
    const int32_t t = t0 + lane;
    const bool in = t < len;
    int32_t pg = in ? a.table[(int64_t)s * g.max_pages + (t >> g.log2P)] : 0;
    if (!good_page(pg, g)) {
      set_status(status, SKV_ERR_ARG);
      pg = 0;
    }
    float z = -INFINITY;
    if (in) {
      const uint8_t *kr = base + pg * g.page_bytes + koff + (int64_t)(t & (g.P - 1)) * g.row_bytes;
      float acc = 0.0f;
      for (int c = 0; c < g.D; ++c) acc = __builtin_fmaf(qs[c], symbol_value(kr, c, g.fmt), acc);
      z = acc * sc;
    }
    float mt = z;
    for (int d = 32; d; d >>= 1) mt = __builtin_fmaxf(mt, __shfl_xor(mt, d));
    const float mn = __builtin_fmaxf(m, mt), r = m == -INFINITY ? 0.0f : expf(m - mn);
    const float e = in && mn != -INFINITY ? expf(z - mn) : 0.0f;
    float et = e;
    for (int d = 32; d; d >>= 1) et += __shfl_xor(et, d);
    l = l * r + et;
    m = mn;
    ps[lane] = e;
    pg_of[lane] = pg;
    __syncthreads();
    for (int c = 0; c < 8; ++c) o[c] *= r;
    const int n = min(64, len - t0);
    for (int u = 0; u < n; ++u) {
      const uint8_t *vr = base + pg_of[u] * g.page_bytes + voff + (int64_t)((t0 + u) & (g.P - 1)) * g.row_bytes;
      for (int c = 0; c * 64 + lane < g.D; ++c) o[c] = __builtin_fmaf(ps[u], symbol_value(vr, c * 64 + lane, g.fmt), o[c]);
    }
    __syncthreads();
  }
  const float inv = l > 0.0f ? (p.v_scale ? p.v_scale[h] : 1.0f) / l : (l == 0.0f ? 0.0f : l);
  uint16_t *out = p.out + (i * p.q_heads + j) * g.D;
  for (int c = 0; c * 64 + lane < g.D; ++c) out[c * 64 + lane] = bf16_rne(o[c] * inv);
  if (p.lse && lane == 0) p.lse[i * p.q_heads + j] = m + logf(l);
}

}  // namespace

extern "C" int skv_attend_workspace_size(const skv_pages_shape *shape, int64_t q_heads, size_t *bytes) {
  PGeo g;
  int e = make_pgeo(shape, g);
  if (e != SKV_OK) return e;
  if (!bytes || q_heads < 1 || q_heads > (1 << 16) || q_heads % g.heads) return SKV_ERR_ARG;
  *bytes = 256;
  return SKV_OK;
}

extern "C" int skv_attend(const skv_pages_shape *shape, const skv_pages *pages, int64_t layer, const void *q,
                          int64_t q_stride, int64_t q_heads, float scale, const float *k_scale,
                          const float *v_scale, const int32_t *seqs, int64_t n, void *out, float *lse,
                          void *workspace, size_t workspace_bytes, int32_t *status, void *stream) {
  PGeo g;
  int e = make_pgeo(shape, g);
  if (e != SKV_OK) return e;
  if ((e = check_pages(pages)) != SKV_OK) return e;
  size_t need = 0;
  if ((e = skv_attend_workspace_size(shape, q_heads, &need)) != SKV_OK) return e;
  if (layer < 0 || layer >= g.layers || n < 0 || n > (1 << 20) || !status || !aligned4(status)) return SKV_ERR_ARG;
  if (!workspace || !aligned16(workspace) || workspace_bytes < need) return SKV_ERR_ARG;
  if (!isfinite(scale)) return SKV_ERR_ARG;
  if (n == 0) return SKV_OK;
  if (!q || !out || !seqs || !aligned16(q) || !aligned16(out) || !aligned4(seqs) || !aligned4(lse)) return SKV_ERR_ARG;
  if (q_stride < q_heads * g.D || q_stride % 8 || q_stride > INT64_MAX / 2 / n) return SKV_ERR_ARG;
  if ((k_scale || v_scale) && g.fmt != SKV_SYM_E4M3) return SKV_ERR_ARG;
  if (!aligned4(k_scale) || !aligned4(v_scale)) return SKV_ERR_ARG;
  if (n * q_heads > INT32_MAX) return SKV_ERR_ARG;
  AttendArgs p{static_cast<const uint16_t *>(q), q_stride, (int)q_heads, scale, k_scale, v_scale, seqs,
               static_cast<uint16_t *>(out), lse};
  k_attend<<<dim3((uint32_t)(n * q_heads)), 64, 0, static_cast<hipStream_t>(stream)>>>(g, *pages, (int)layer, p, status);
  return hipGetLastError() == hipSuccess ? SKV_OK : SKV_ERR_HIP;
}
