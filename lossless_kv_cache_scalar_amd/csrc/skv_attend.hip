// skv_attend.hip -- attention of one new token per sequence over a paged cache.
// Contract: skv.h.
//
// Work is cut into units: 32 tokens of one (sequence, KV head, tile of 16 query
// heads).  The units of a call, in that order, are dealt out evenly to the
// waves of the grid, a contiguous run to each, from the lengths on the device;
// so the split over a sequence's length follows the lengths of the moment, and
// one long sequence fills the chip as a batch of short ones does.  A row (sequence,
// KV head, tile) that lies in one wave's run is finished there; one that
// spans waves leaves partial sums, joined by a second launch.
//
// A wave keeps all of its state in registers: for each query head the running
// maximum m of the scores (times log2 e), the sum l of 2^(score - m), and the
// sum O of 2^(score - m) v.  Per unit: S^T = K Q^T by matrix instructions (rows:
// tokens, columns: heads), so that a lane holds eight tokens' scores of one
// head; the same lane's weights are then the operand of O^T += V^T P^T as they
// lie, and no value crosses lanes but the maximum.
#include <math.h>

#include "skv_pages.hpp"

using namespace skv;

namespace {

constexpr int kTile = 32;    // tokens of a unit
constexpr int kHeads = 16;   // query heads of a tile
constexpr int kMinUnits = 2; // units that a wave gets at least
constexpr int kWavesPerCu = 8;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct AttendArgs {
  const uint16_t *q;
  int64_t q_stride;
  float scale;
  const float *k_scale, *v_scale;
  const int32_t *seqs;
  int n;
  int q_heads, group, tiles_q;  // query heads, per KV head, tiles of 16 of them
  int kept;                     // heads of a partial sum: min(group, 16)
  int waves;                    // of the main launch
  uint16_t *out;
  float *lse;
  int slot;                     // floats of a partial sum: O [kept][D], m [kept], l [kept], rounded up to 4
  float *part;                  // [waves][2][slot]
  int4 *split;                  // [waves] the row that begins in a wave's run and ends in another's (Split)
};

// what a wave leaves about such a row: waves it spans (0: there is none) and
// where its first partial sum lies, its first query head's row in out, its
// heads, its KV head
__device__ __forceinline__ int4 split_of(int parts, int slot, int32_t qrow, int heads, int h) {
  return make_int4(parts << 1 | slot, qrow, heads, h);
}

// ---- the dealing out ----
// units of list place i; 0 for padding.  An empty sequence has one unit, whose
// only work is to write its zeros.
__device__ __forceinline__ int32_t place_len(const PGeo &g, const skv_pages &a, const AttendArgs &p, int i, bool &there,
                                             bool &bad) {
  there = false;
  bad = false;
  if (i >= p.n) return 0;
  const int32_t s = p.seqs[i];
  if (s < 0) return 0;
  if (s >= g.max_seqs) {
    bad = true;
    return 0;
  }
  there = true;
  const int32_t len = a.lens[s];
  if (len < 0 || len > g.max_tokens) {
    bad = true;
    return 0;
  }
  return len;
}

__device__ __forceinline__ int32_t tiles_of(int32_t len) { return len > 0 ? (int32_t)(((uint32_t)len + kTile - 1) / kTile) : 1; }

__device__ __forceinline__ int64_t wave_scan(int64_t v) {  // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up(v, d);
    if (lane >= d) v += y;
  }
  return v;
}

__device__ __forceinline__ int64_t lane_of(int64_t v, int l) {
  const int lo = __builtin_amdgcn_readlane((int)(uint32_t)v, l);
  const int hi = __builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), l);
  return (int64_t)((uint64_t)(uint32_t)hi << 32 | (uint32_t)lo);
}

// waves that take part: every one where there are units enough
__device__ __forceinline__ int64_t active_waves(int64_t units, int waves) {
  const int64_t n = units / kMinUnits;
  return n < 1 ? 1 : (n < waves ? n : waves);
}
__device__ __forceinline__ int64_t first_unit(int64_t w, int64_t units, int64_t active) { return w * units / active; }
// the wave whose run holds unit u
__device__ __forceinline__ int64_t wave_with(int64_t u, int64_t units, int64_t active) { return ((u + 1) * active - 1) / units; }

// ---- numbers ----
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));  // nearest even
}
// e4m3 bytes 2h, 2h + 1 of w as two bf16 (exact)
template <bool H>
__device__ __forceinline__ uint32_t bf16_of_e4m3(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, H));
}
// over the four lanes l, l ^ 16, l ^ 32, l ^ 48 that share a head
__device__ __forceinline__ float max_over_rows(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __builtin_fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __builtin_fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_over_rows(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
// m where it is a number to subtract: a row without any weight yet has m = -inf
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }

// ---- a unit's keys and values in registers ----
// K, operand A of a 16x16x32 product: lane l holds token l % 16, eight of 32
// channels by l / 16.  bf16: channels in order; e4m3: a 16-byte load holds the
// lane's channels of two products (which channels form a product does not
// matter as long as q takes the same ones).
template <int FMT, int D>
struct Keys {
  static constexpr int KB = D < 32 ? 1 : D / 32;                   // products
  static constexpr bool wide = FMT == 0 || D >= 64;                // 16-byte loads
  static constexpr int NL = FMT == 0 ? KB : (D >= 64 ? D / 64 : 1);  // loads per 16 tokens
  static constexpr int row = D * (FMT == 0 ? 2 : 1);
  u32x4 r[2][NL];

  __device__ __forceinline__ void load(const uint8_t *b0, const uint8_t *b1) {
    const int l = threadIdx.x & 63, t = l & 15, g = l >> 4;
    constexpr int bytes = wide ? 16 : 8;
    const bool in = (g + 1) * bytes <= row;  // a row shorter than a product's 32 channels
    const uint32_t off = (uint32_t)(t * row + g * bytes);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint8_t *b = s ? b1 : b0;
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        if (row >= 4 * bytes || in) {
          if (wide) {
            r[s][j] = *reinterpret_cast<const u32x4 *>(b + off + j * 64);
          } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(b + off);
            r[s][j] = u32x4{v.x, v.y, 0, 0};
          }
        } else {
          r[s][j] = u32x4{0, 0, 0, 0};
        }
      }
    }
  }
  __device__ __forceinline__ bf16x8 operand(int s, int j) const {
    if (FMT == 0) return __builtin_bit_cast(bf16x8, r[s][j]);
    const u32x4 v = r[s][wide ? j >> 1 : j];
    const uint32_t x = wide && (j & 1) ? v.z : v.x, y = wide && (j & 1) ? v.w : v.y;
    const u32x4 o = {bf16_of_e4m3<false>(x), bf16_of_e4m3<true>(x), bf16_of_e4m3<false>(y), bf16_of_e4m3<true>(y)};
    return __builtin_bit_cast(bf16x8, o);
  }
  // the first of the eight channels that product j takes in lane group g
  static __device__ __forceinline__ int channel(int j, int g) {
    if (FMT == 0 || D < 64) return j * 32 + g * 8;
    return (j >> 1) * 64 + g * 16 + (j & 1) * 8;
  }
};

// V^T, operand A of the second product: lane l holds channels CW (l % 16) .. of
// 128 (one per product), eight of the 32 tokens by l / 16: those whose weights
// the lane group holds, 4 g .. 4 g + 3 of either half.  Loaded along the channels,
// a whole row by 16 lanes; a byte permute turns two tokens' words into
// two channels' pairs.
template <int FMT, int D>
struct Values {
  static constexpr int CW = D < 16 ? 1 : (D < 128 ? D / 16 : 8);
  static constexpr int esz = FMT == 0 ? 2 : 1;
  static constexpr int bytes = CW * esz;
  static constexpr int W = bytes < 4 ? 1 : bytes / 4;
  static constexpr int row = D * esz;
  uint32_t w[8][W];

  __device__ __forceinline__ void load(const uint8_t *b0, const uint8_t *b1, int chunk) {
    const int l = threadIdx.x & 63, c = l & 15, g = l >> 4;
    const uint32_t off = (uint32_t)(4 * g * row + chunk * 128 * esz + c * bytes);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint8_t *b = (i < 4 ? b0 : b1) + off + (i & 3) * row;
      if (D >= 16 || c < D) {
        if (bytes == 16) {
          const u32x4 v = *reinterpret_cast<const u32x4 *>(b);
#pragma unroll
          for (int k = 0; k < W; ++k) w[i][k] = v[k];
        } else if (bytes == 8) {
          const uint2 v = *reinterpret_cast<const uint2 *>(b);
          w[i][0] = v.x;
          w[i][W - 1] = v.y;
        } else if (bytes == 4) {
          w[i][0] = *reinterpret_cast<const uint32_t *>(b);
        } else if (bytes == 2) {
          w[i][0] = *reinterpret_cast<const uint16_t *>(b);
        } else {
          w[i][0] = *b;
        }
      } else {
        w[i][0] = 0;
      }
    }
  }
  // tokens at and behind `left` of the unit's 32 count as zeros, whatever lies there
  __device__ __forceinline__ void cut(int left) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool in = (i >> 2) * 16 + 4 * g + (i & 3) < left;
#pragma unroll
      for (int k = 0; k < W; ++k) w[i][k] = in ? w[i][k] : 0;
    }
  }
  // operands of channels 2 q and 2 q + 1 of the lane's CW (CW = 1: the first alone)
  __device__ __forceinline__ void operands(int q, bf16x8 &even, bf16x8 &odd) const {
    u32x4 e, o;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if (FMT == 0) {
        e[d] = __builtin_amdgcn_perm(w[2 * d + 1][q], w[2 * d][q], 0x05040100u);
        o[d] = __builtin_amdgcn_perm(w[2 * d + 1][q], w[2 * d][q], 0x07060302u);
      } else {
        const uint32_t x = __builtin_amdgcn_perm(w[2 * d + 1][q >> 1], w[2 * d][q >> 1], q & 1 ? 0x07030602u : 0x05010400u);
        e[d] = bf16_of_e4m3<false>(x);
        o[d] = bf16_of_e4m3<true>(x);
      }
    }
    even = __builtin_bit_cast(bf16x8, e);
    odd = __builtin_bit_cast(bf16x8, o);
  }
};

// the page ids of a run of tokens, 64 in the lanes at a time
struct Ids {
  const int32_t *row;
  int32_t first, last;  // entry that lane 0 holds; the run's last
  int32_t v;
  int64_t n_pages;

  __device__ __forceinline__ void fetch(int32_t *status) {
    const int lane = threadIdx.x & 63;
    v = row[min(first + lane, last)];
    const bool good = (uint32_t)v < (uint64_t)n_pages;
    if (!good) {  // read page 0 in its place, and say so
      v = 0;
      set_status(status, SKV_ERR_ARG);
    }
  }
  // entries are asked for in order
  __device__ __forceinline__ int32_t at(int32_t entry, int32_t *status) {
    if (entry - first >= 64) {
      first = entry;
      fetch(status);
    }
    return __builtin_amdgcn_readlane(v, entry - first);
  }
};

template <int FMT, int D>
__global__ __launch_bounds__(64) void k_attend(PGeo g, skv_pages a, int layer, AttendArgs p, int32_t *status) {
  using K = Keys<FMT, D>;
  using V = Values<FMT, D>;
  constexpr int KB = K::KB, CW = V::CW;
  constexpr int NV = D < 128 ? 1 : D / 128;  // chunks of 128 channels
  constexpr int row = K::row;
  const int lane = threadIdx.x, hd = lane & 15, grp = lane >> 4;
  const int rows_of_place = g.heads * p.tiles_q;

  // units in all, and the place that this wave's run begins in
  int64_t before = 0;  // units of the places before the 64 at hand
  int chunk = 0;       // the first of them
  int32_t len_l = 0;
  int64_t upto = 0;    // units up to and with the lane's place
  bool there, bad;
  auto look = [&]() {
    len_l = place_len(g, a, p, chunk + lane, there, bad);
    upto = before + wave_scan(there ? (int64_t)tiles_of(len_l) * rows_of_place : 0);
  };
  for (;;) {
    look();
    if (bad && blockIdx.x == 0) set_status(status, SKV_ERR_ARG);
    if (chunk + 64 >= p.n) break;
    before = lane_of(upto, 63);
    chunk += 64;
  }
  const int64_t units = lane_of(upto, 63);
  const int64_t active = active_waves(units, p.waves);
  if (units == 0 || (int64_t)blockIdx.x >= active) {
    if (lane == 0) p.split[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }
  int64_t u = first_unit(blockIdx.x, units, active);
  const int64_t end = first_unit(blockIdx.x + 1, units, active);
  if (chunk > 0) {
    before = 0;
    chunk = 0;
    look();
  }
  const int64_t begun = u;
  int4 split = make_int4(0, 0, 0, 0);
  while (u < end) {
    // the place of unit u: the first whose units reach beyond it
    uint64_t beyond = __builtin_amdgcn_ballot_w64(upto > u);
    while (beyond == 0) {
      before = lane_of(upto, 63);
      chunk += 64;
      if (chunk >= p.n) {  // only where lengths change under the call
        if (lane == 0) p.split[blockIdx.x] = make_int4(0, 0, 0, 0);
        return;
      }
      look();
      beyond = __builtin_amdgcn_ballot_w64(upto > u);
    }
    const int at = __builtin_ctzll(beyond);
    const int i = chunk + at;
    const int32_t len = __builtin_amdgcn_readlane(len_l, at);
    const int32_t tiles = tiles_of(len);
    const int64_t in_place = u - (lane_of(upto, at) - (int64_t)tiles * rows_of_place);
    const int r = (int)(in_place / tiles);             // (KV head, tile of query heads)
    const int32_t ta = (int32_t)(in_place - (int64_t)r * tiles);
    const int32_t tb = (int32_t)min((int64_t)tiles, ta + (end - u));
    const int h = r / p.tiles_q, qt = r - h * p.tiles_q;
    const bool whole = ta == 0 && tb == tiles;
    const int slot = u == begun ? 0 : 1;
    const int heads = min(kHeads, p.group - qt * kHeads);  // of this tile
    if (ta == 0 && !whole)
      split = split_of((int)(wave_with(u + tiles - 1, units, active) - blockIdx.x + 1), slot,
                       (int32_t)((int64_t)i * p.q_heads + (int64_t)h * p.group + qt * kHeads), heads, h);
    u += tb - ta;

    const int64_t qrow = (int64_t)i * p.q_heads + (int64_t)h * p.group + qt * kHeads + hd;
    float m = -INFINITY, l = 0.0f;
    f32x4 o[NV * CW];
#pragma unroll
    for (int k = 0; k < NV * CW; ++k) o[k] = f32x4{0, 0, 0, 0};

    if (len > 0) {
      const int32_t s = p.seqs[i];
      bf16x8 qf[KB];
      const uint16_t *qp = p.q + (int64_t)i * p.q_stride + (int64_t)(h * p.group + qt * kHeads + hd) * D;
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        u32x4 v = {0, 0, 0, 0};
        const int c = K::channel(j, grp);
        if (hd < heads && c < D) v = *reinterpret_cast<const u32x4 *>(qp + c);
        qf[j] = __builtin_bit_cast(bf16x8, v);
      }
      const float sc = p.scale * (p.k_scale ? p.k_scale[h] : 1.0f) * 1.44269504088896340736f;

      Ids ids;
      ids.row = a.table + (int64_t)s * g.max_pages;
      ids.first = ta * kTile >> g.log2P;
      ids.last = (int32_t)((min((uint32_t)tb * kTile, (uint32_t)len) - 1) >> g.log2P);
      ids.n_pages = g.n_pages;
      ids.fetch(status);
      const uint8_t *kbase = static_cast<const uint8_t *>(a.pool) + (int64_t)layer * g.n_pages * g.page_bytes + (int64_t)h * g.P * row;
      const int64_t to_v = (int64_t)g.heads * g.P * row;
      // the two halves of a unit lie in one page each; a half without tokens reads the first one again
      auto half = [&](int32_t t, int b) {
        int32_t tok = t * kTile + 16 * b;
        tok = tok < len ? tok : t * kTile;
        return kbase + (int64_t)ids.at(tok >> g.log2P, status) * g.page_bytes + (tok & (g.P - 1)) * row;
      };

      K keys;
      const uint8_t *b0 = half(ta, 0), *b1 = half(ta, 1);
      keys.load(b0, b1);
      for (int32_t t = ta; t < tb; ++t) {
        const int left = len - t * kTile;  // tokens from here on
        V vals;
        vals.load(b0 + to_v, b1 + to_v, 0);
        const uint8_t *v0 = b0 + to_v, *v1 = b1 + to_v;
        f32x4 z[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
        for (int j = 0; j < KB; ++j)
#pragma unroll
          for (int b = 0; b < 2; ++b) z[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(keys.operand(b, j), qf[j], z[b], 0, 0, 0);
        if (t + 1 < tb) {
          b0 = half(t + 1, 0);
          b1 = half(t + 1, 1);
          keys.load(b0, b1);
        }
        float zs[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) zs[k] = z[k >> 2][k & 3] * sc;
        if (left < kTile) {
#pragma unroll
          for (int k = 0; k < 8; ++k) zs[k] = (k >> 2) * 16 + 4 * grp + (k & 3) < left ? zs[k] : -INFINITY;
          vals.cut(left);
        }
        float mt = zs[0];
#pragma unroll
        for (int k = 1; k < 8; ++k) mt = __builtin_fmaxf(mt, zs[k]);
        mt = __builtin_fmaxf(m, max_over_rows(mt));
        if (__builtin_amdgcn_ballot_w64(mt > m)) {
          const float f = __builtin_amdgcn_exp2f(m - base_of(mt));
          l *= f;
#pragma unroll
          for (int k = 0; k < NV * CW; ++k) o[k] *= f;
          m = mt;
        }
        const float mb = base_of(m);
        float e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = __builtin_amdgcn_exp2f(zs[k] - mb);
        l += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
        // weights as bf16: the matrix instruction's type; off by 2^-8 of themselves
        // at most, and their sum l is taken before
        const u32x4 pk = {pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]), pack_bf16(e[4], e[5]), pack_bf16(e[6], e[7])};
        const bf16x8 pf = __builtin_bit_cast(bf16x8, pk);
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          if (c > 0) {
            vals.load(v0, v1, c);
            if (left < kTile) vals.cut(left);
          }
#pragma unroll
          for (int k = 0; k < CW; k += 2) {
            bf16x8 even, odd;
            vals.operands(k >> 1, even, odd);
            o[c * CW + k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(even, pf, o[c * CW + k], 0, 0, 0);
            if (CW > 1) o[c * CW + (CW > 1 ? k + 1 : 0)] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(odd, pf, o[c * CW + (CW > 1 ? k + 1 : 0)], 0, 0, 0);
          }
        }
      }
      l = sum_over_rows(l);
    }

    // a lane has channels 128 c + CW (4 grp + x) + k of its head in o[c CW + k][x]
    if (hd < heads) {
      if (whole) {
        const float f = l == 0.0f ? 0.0f : (p.v_scale ? p.v_scale[h] : 1.0f) / l;
        uint16_t *op = p.out + qrow * D;
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int ch = 128 * c + CW * (4 * grp + x);
            if (CW == 1) {
              if (ch < D) op[ch] = (uint16_t)pack_bf16(o[0][x] * f, 0.0f);
            } else {
#pragma unroll
              for (int k = 0; k < CW; k += 2)
                *reinterpret_cast<uint32_t *>(op + ch + k) = pack_bf16(o[c * CW + k][x] * f, o[c * CW + (CW > 1 ? k + 1 : 0)][x] * f);
            }
          }
        if (p.lse && grp == 0) p.lse[qrow] = l == 0.0f ? -INFINITY : (m + __builtin_log2f(l)) * 0.693147180559945309417f;
      } else {
        float *pp = p.part + ((int64_t)blockIdx.x * 2 + slot) * p.slot;
        float *po = pp + hd * D;
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int k = 0; k < CW; ++k) {
              const int ch = 128 * c + CW * (4 * grp + x) + k;
              if (ch < D) po[ch] = o[c * CW + k][x];
            }
        if (grp == 0) {
          pp[p.kept * D + hd] = m;
          pp[p.kept * (D + 1) + hd] = l;
        }
      }
    }
  }
  if (lane == 0) p.split[blockIdx.x] = split;
}

// ---- the join ----
// out = sum_w 2^(m_w - M) O_w / sum_w 2^(m_w - M) l_w over the waves w that a row
// spans.  A workgroup takes 256 of the row's values, four to a lane; each of
// its waves runs through every fourth partial sum with a running maximum as the main
// kernel does, all loads of a round in flight at once, and the four are joined
// in LDS.  Workgroups of waves that leave no such row end after one load.
constexpr int kJoin = 256;

__global__ __launch_bounds__(kJoin) void k_attend_join(PGeo g, AttendArgs p) {
  const int64_t w0 = blockIdx.x;
  const int4 sp = p.split[w0];
  const int parts = sp.x >> 1;
  if (parts == 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int v = ((int)blockIdx.y * 64 + lane) * 4;  // the lane's first value of the row's heads * D
  if ((int)blockIdx.y * 256 >= sp.z * g.D) return;
  const bool in = v < sp.z * g.D;
  const int hd = in ? v / g.D : 0;
  // partial sum k: the first of wave w0 + k, but for the wave that the row begins inside of
  auto part = [&](int k) { return p.part + ((w0 + k) * 2 + (k == 0 ? sp.x & 1 : 0)) * p.slot; };
  float m = -INFINITY, l = 0.0f;
  f32x4 o = {0, 0, 0, 0};
  constexpr int R = 8;
  for (int k0 = wave; k0 < parts; k0 += 4 * R) {
    float ms[R], ls[R];
    f32x4 os[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int k = k0 + 4 * r;
      ms[r] = -INFINITY;
      ls[r] = 0.0f;
      os[r] = f32x4{0, 0, 0, 0};
      if (k < parts && in) {
        const float *pp = part(k);
        ms[r] = pp[p.kept * g.D + hd];
        ls[r] = pp[p.kept * (g.D + 1) + hd];
        os[r] = *reinterpret_cast<const f32x4 *>(pp + v);
      }
    }
    float mn = m;
#pragma unroll
    for (int r = 0; r < R; ++r) mn = __builtin_fmaxf(mn, ms[r]);
    const float mb = base_of(mn), f = __builtin_amdgcn_exp2f(m - mb);
    m = mn;
    l *= f;
    o *= f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float e = __builtin_amdgcn_exp2f(ms[r] - mb);
      l = __builtin_fmaf(e, ls[r], l);
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] = __builtin_fmaf(e, os[r][c], o[c]);
    }
  }
  __shared__ float sm[4][64], sl[4][64];
  __shared__ f32x4 so[4][64];
  sm[wave][lane] = m;
  sl[wave][lane] = l;
  so[wave][lane] = o;
  __syncthreads();
  if (wave > 0 || !in) return;
  const float mx = __builtin_fmaxf(__builtin_fmaxf(sm[0][lane], sm[1][lane]), __builtin_fmaxf(sm[2][lane], sm[3][lane]));
  const float mb = base_of(mx);
  l = 0.0f;
  o = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float e = __builtin_amdgcn_exp2f(sm[w][lane] - mb);
    l = __builtin_fmaf(e, sl[w][lane], l);
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = __builtin_fmaf(e, so[w][lane][c], o[c]);
  }
  const float f = l == 0.0f ? 0.0f : (p.v_scale ? p.v_scale[sp.w] : 1.0f) / l;
  const uint2 y = make_uint2(pack_bf16(o[0] * f, o[1] * f), pack_bf16(o[2] * f, o[3] * f));
  *reinterpret_cast<uint2 *>(p.out + (int64_t)sp.y * g.D + v) = y;
  if (p.lse && v - hd * g.D == 0) p.lse[sp.y + hd] = l == 0.0f ? -INFINITY : (mx + __builtin_log2f(l)) * 0.693147180559945309417f;
}

int attend_waves() { return device_cu_count() * kWavesPerCu; }
int slot_floats(const PGeo &g, int kept) { return kept * g.D + (2 * kept + 3) / 4 * 4; }

}  // namespace

extern "C" int skv_attend_workspace_size(const skv_pages_shape *shape, int64_t q_heads, size_t *bytes) {
  PGeo g;
  int e = make_pgeo(shape, g);
  if (e != SKV_OK) return e;
  if (!bytes || q_heads < 1 || q_heads > (1 << 16) || q_heads % g.heads) return SKV_ERR_ARG;
  const int64_t group = q_heads / g.heads;
  *bytes = (size_t)attend_waves() * (2 * sizeof(float) * (size_t)slot_floats(g, (int)(group < kHeads ? group : kHeads)) + sizeof(int4));
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
  AttendArgs p;
  p.q = static_cast<const uint16_t *>(q);
  p.q_stride = q_stride;
  p.scale = scale;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.seqs = seqs;
  p.n = (int)n;
  p.q_heads = (int)q_heads;
  p.group = (int)(q_heads / g.heads);
  p.tiles_q = (p.group + kHeads - 1) / kHeads;
  p.kept = p.group < kHeads ? p.group : kHeads;
  p.out = static_cast<uint16_t *>(out);
  p.lse = lse;
  p.slot = slot_floats(g, p.kept);
  // no more waves than the longest sequences the table holds could use
  const __int128 most = ((__int128)n * g.heads * p.tiles_q * ((g.max_tokens + (int64_t)kTile - 1) / kTile) + kMinUnits - 1) / kMinUnits;
  const int all = attend_waves();
  p.waves = most < all ? (int)most : all;
  p.split = static_cast<int4 *>(workspace);
  p.part = reinterpret_cast<float *>(p.split + all);
  const dim3 grid((uint32_t)p.waves);
  hipStream_t st = static_cast<hipStream_t>(stream);
#define SKV_ATTEND(F_, D_) case D_: k_attend<F_, D_><<<grid, 64, 0, st>>>(g, *pages, (int)layer, p, status); break
#define SKV_ATTEND_ALL(F_) \
  switch (g.D) { \
    SKV_ATTEND(F_, 8); SKV_ATTEND(F_, 16); SKV_ATTEND(F_, 32); SKV_ATTEND(F_, 64); \
    SKV_ATTEND(F_, 128); SKV_ATTEND(F_, 256); SKV_ATTEND(F_, 512); \
  }
  if (g.fmt == SKV_SYM_BF16) {
    SKV_ATTEND_ALL(0)
  } else {
    SKV_ATTEND_ALL(1)
  }
#undef SKV_ATTEND_ALL
#undef SKV_ATTEND
  if (hipGetLastError() != hipSuccess) return SKV_ERR_HIP;
  k_attend_join<<<dim3((uint32_t)p.waves, (uint32_t)((p.kept * g.D + 255) / 256)), kJoin, 0, st>>>(g, p);
  return hipGetLastError() == hipSuccess ? SKV_OK : SKV_ERR_HIP;
}
