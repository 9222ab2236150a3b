// skv_attend.hip -- attention of one new token per sequence over a paged cache.
// Contract: skv.h.
//
// Work is cut into units: 32 tokens of one row, a row being a sequence, a KV
// head and a tile of its query heads.  The units of a call, row by row, are
// dealt out evenly from the lengths on the device, a contiguous run to each
// workgroup; so the split over a sequence's length follows the lengths of the moment,
// and one long sequence fills the chip as a batch of short ones does.  Within a
// workgroup the run is dealt out to the waves in the same way: a wave works
// through its part alone, and a row that spans waves is joined in LDS at the end.
// A row that lies in one workgroup's run is finished there; one that spans
// workgroups leaves partial sums, joined by a second launch.
//
// A wave keeps all of its state in registers: for each query head the running
// maximum m of the scores (times log2 e), the sum l of 2^(score - m), and the
// sum O of 2^(score - m) v.  Per unit: S^T = K Q^T by matrix instructions (rows:
// tokens, columns: heads), so that a lane holds eight tokens' scores of one
// head; the same lane's weights are then the operand of O^T += V^T P^T as they
// lie, and no value crosses lanes but the maximum.
//
// What bounds it.  Up to 16 query heads to a KV head every cached symbol is read
// once and used for 1 to 32 operations a byte, far below what the matrix units need
// to be the limit: it is HBM.  64 sequences of up to 8192 tokens (64 query and 8 KV
// heads of 128, bf16, 1.08 GB): 168 us and 5 for the join, 6.2 TB/s, of the 7.0 that
// a plain read reaches here; inside the loop it is 6.85, the rest is the start (three
// dependent loads before the first key, 2.3 us), the last waves' tail (the older
// workgroup of a CU ends first) and the join.  16 sequences up to 32768 in e4m3
// (0.81 GB): 127 + 5 us.  One sequence of 2048 tokens (8.4 MB) takes 7.1 + 2.2 us,
// which is latency: a chain of six loads, two launches.  With more query heads each
// tile of 16 asks for the same keys and values, through the caches, and from 65 (33
// at 512 channels) on another row reads them from HBM again: 64 sequences of up to
// 8192 with 20 heads to each of 4 KV heads (0.54 GB) take 119 us, with 40 to each of
// 2 (0.27 GB) 86.  At 256 and 512 channels the values come 128 channels at a time,
// each asked for after the products of those before, and the loop waits for them:
// 64 sequences of up to 4096 over 8 KV heads of 256 in e4m3 (0.54 GB) take 112 us,
// of up to 2048 over 8 of 512 in bf16 (1.08 GB) 219.
#include <math.h>

#include "skv_pages.hpp"

using namespace skv;

namespace {

constexpr int kTile = 32;    // tokens of a unit
constexpr int kHeads = 16;   // query heads of a tile
// Units of a workgroup at least: one to a wave (captured in a graph, 8 KV heads of
// 128, one sequence of 2048 tokens in bf16: 8.9 us; with 2, 8 and 16 it is 9.4, 10.0
// and 12.0; 7 sequences of up to 301 over 2 KV heads of 64: 9.3, and 8.7, 11.1, 14.6).
constexpr int kMinUnits = 4;
// Workgroups are limited to kSplit sqrt(units * rows), see below.  At 1.5 the one
// sequence takes 11.3 us.  No limit at all is about as good: one sequence over one
// KV head takes 11.6 us instead of 12.6 at 8192 tokens, 17.2 instead of 16.2 at 32768,
// 27.6 instead of 28.0 at 131072.  Only the longest single rows want fewer: 2^20
// tokens of one KV head take 98 us at 1.5 and 108 at 3.
constexpr float kSplit = 3.0f;
constexpr int kLongRow = 32;  // units of a row, on average, that make it a long one
// waves of a workgroup (LDS holds two partial sums of each), and of a SIMD
// (registers: 256 or 512 to a wave)
__host__ __device__ constexpr int waves_of(int D) { return D <= 256 ? 4 : 2; }
__host__ __device__ constexpr int waves_per_simd(int fmt, int D) { return D <= 128 || (D == 256 && fmt == SKV_SYM_E4M3) ? 2 : 1; }
constexpr int kMaxRows = 1 << 16;  // list places of a call
constexpr int kLds = 160 * 1024;  // of a CU

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct AttendArgs {
  const uint16_t *q;
  int64_t q_stride;
  float scale;
  const float *k_scale, *v_scale;
  const int32_t *seqs;
  int n;
  int q_heads, group, tiles_q;  // query heads, per KV head, tiles of 16 of them
  int shared_q;                 // tiles of a row, a wave to each: 1, 2 or 4
  int kept;                     // heads of a row at most: min(group, 16 shared_q)
  int blocks, cus;              // of the main launch; compute units
  uint16_t *out;
  float *lse;
  int slot;                     // floats of a partial sum: O [kept][D], m [kept], l [kept], rounded up to 4
  float *part;                  // [block][2][slot]
  int4 *split;                  // [block] the row that begins in its run and ends in another's: workgroups that it
                                // spans (0: there is none) * 2 + place of the first partial sum, its first place in
                                // lse, its query heads, its KV head
};

// floats of a head's row in LDS: sixteen heads' rows then begin in different banks
__host__ __device__ constexpr int row_floats(int D) { return D + 4; }

// a row of which a wave has a part
struct Row {
  int64_t u0;      // its first unit
  int32_t tiles;   // its units; 0: no row
  int32_t at;      // its first place in lse
  int32_t heads, h;
};

// ---- the dealing out ----
// the sequence of a list place (-1: padding, or none that the cache has) and its length
struct Place {
  int32_t s, len;
};
__device__ __forceinline__ int32_t listed(const AttendArgs &p, int i) { return i < p.n ? p.seqs[i] : -1; }
__device__ __forceinline__ Place place_of(const PGeo &g, const skv_pages &a, int32_t s, bool &bad) {
  Place x = {-1, 0};
  bad = s >= g.max_seqs;
  if (s < 0 || bad) return x;
  x.s = s;
  x.len = a.lens[s];
  bad = x.len < 0 || x.len > g.max_tokens;
  if (bad) x.len = 0;
  return x;
}

// units of a row.  An empty sequence has one, whose only work is to write its zeros.
__device__ __forceinline__ int32_t tiles_of(int32_t len) { return len > 0 ? (int32_t)(((uint32_t)len + kTile - 1) / kTile) : 1; }

// inclusive prefix sum over the wave, by row shifts and row broadcasts in the vector unit
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false);  // row_shr:1
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false);  // row_bcast:15 into rows 1 and 3
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false);  // row_bcast:31 into rows 2 and 3
  return v;
}

__device__ __forceinline__ int64_t lane_of(int64_t v, int l) {
  const int lo = __builtin_amdgcn_readlane((int)(uint32_t)v, l);
  const int hi = __builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), l);
  return (int64_t)((uint64_t)(uint32_t)hi << 32 | (uint32_t)lo);
}

// Runs: of `units` units among `active` workgroups, the first `more` of which
// have each + 1 and the others `each`.
struct Runs {
  int64_t each, more;
  __device__ __forceinline__ Runs(int64_t units, int64_t active) : each(quotient(units, active)), more(units - each * active) {}
  __device__ __forceinline__ int64_t first(int64_t w) const { return w * each + min(w, more); }
  // the workgroup that has unit u
  __device__ __forceinline__ int64_t of(int64_t u) const {
    const int64_t big = more * (each + 1);
    return u < big ? quotient(u, each + 1) : more + quotient(u - big, each);
  }
};

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
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

// m where it is a number to subtract: a row without any weight yet has m = -inf
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }

// ---- a unit's keys and values in registers ----
// Where one tile of query heads reads each it goes past the caches: 7.0 TB/s against
// 6.1 for a plain read of 1 GiB, 169 us against 194 for the 64 sequences above.
// Several tiles read the same ones.  Sequences that share pages do too, but far
// apart in time; the memory-side cache serves them (32 forks of 8192 tokens, 8 KV
// heads of 128 in bf16: 122 us, 8.8 TB/s of what the rows read, 34 MB of it distinct).
template <int ONCE, typename T>
__device__ __forceinline__ T fetched(const uint8_t *p) {
  if (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const T *>(p));
  return *reinterpret_cast<const T *>(p);
}

// K, operand A of a 16x16x32 product: lane l holds token l % 16, eight of 32
// channels by l / 16.  bf16: channels in order; e4m3: a 16-byte load holds the
// lane's channels of two products (which channels form a product does not
// matter as long as q takes the same ones).
template <int FMT, int D, int ONCE>
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
            r[s][j] = fetched<ONCE, u32x4>(b + off + j * 64);
          } else {
            const u32x2 v = fetched<ONCE, u32x2>(b + off);
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
template <int FMT, int D, int ONCE>
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
          const u32x4 v = fetched<ONCE, u32x4>(b);
#pragma unroll
          for (int k = 0; k < W; ++k) w[i][k] = v[k];
        } else if (bytes == 8) {
          const u32x2 v = fetched<ONCE, u32x2>(b);
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

template <int FMT, int D, int ONCE>
__global__ __launch_bounds__(64 * waves_of(D), waves_per_simd(FMT, D)) void k_attend(PGeo g, skv_pages a, int layer, AttendArgs p,
                                                                                    int32_t *status) {
  using K = Keys<FMT, D, ONCE>;
  using V = Values<FMT, D, ONCE>;
  constexpr int KB = K::KB, CW = V::CW;
  constexpr int NV = D < 128 ? 1 : D / 128;  // chunks of 128 channels
  constexpr int row = K::row;
  constexpr int NW = waves_of(D);
  constexpr int LD = row_floats(D);
  constexpr bool ahead = D <= 256;           // the next unit's keys are asked for before this one's softmax
  // [NW][2][tile_heads][LD]: a wave's partial sums
  extern __shared__ float os[];
  const int tile_heads = min(p.group, kHeads);
  auto sum_at = [&](int w, int slot, int hd) { return os + ((w * 2 + slot) * tile_heads + hd) * LD; };
  __shared__ float sm[NW][2][kHeads], sl[NW][2][kHeads];
  __shared__ Row rows[NW][2];                // by part of the run
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, hd = lane & 15, grp = lane >> 4;

  // Units of 32 tokens in each 64 places of the list, by the waves in turn, four
  // times 64 places at once; and in all.
  const int rows_of_head = (p.tiles_q + p.shared_q - 1) / p.shared_q, rows_of_place = g.heads * rows_of_head;
  const int chunks = (p.n + 63) / 64;
  __shared__ uint32_t chunk_tiles[kMaxRows / 64];
  __shared__ int32_t chunk_places[kMaxRows / 64];
  bool bad;
  Place place;         // the lane's of the 64 places at hand
  uint32_t upto = 0;   // units of those, up to and with the lane's; 64 lengths of 2^30 at most: 2^31
  int64_t all = 0, places = 0;
  if (chunks == 1) {
    place = place_of(g, a, listed(p, lane), bad);
    upto = wave_scan(place.s >= 0 ? (uint32_t)tiles_of(place.len) : 0);
    all = (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
    places = __builtin_popcountll(__builtin_amdgcn_ballot_w64(place.s >= 0));
    if (bad && blockIdx.x == 0) set_status(status, SKV_ERR_ARG);
  } else {
    constexpr int R = 4;
    for (int c = wave; c < chunks; c += NW * R) {
      int32_t s[R];
      Place x[R];
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] = listed(p, (c + NW * r) * 64 + lane);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        x[r] = place_of(g, a, s[r], bad);
        if (bad && blockIdx.x == 0) set_status(status, SKV_ERR_ARG);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t t = wave_scan(x[r].s >= 0 ? (uint32_t)tiles_of(x[r].len) : 0);
        const int n = __builtin_popcountll(__builtin_amdgcn_ballot_w64(x[r].s >= 0));
        if (lane == 63 && c + NW * r < chunks) {
          chunk_tiles[c + NW * r] = t;
          chunk_places[c + NW * r] = n;
        }
      }
    }
    __syncthreads();
    for (int c = 0; c < chunks; c += 64) {
      // 64 sums of 2^31 at most: in two halves
      const uint32_t t = c + lane < chunks ? chunk_tiles[c + lane] : 0;
      all += (uint32_t)__builtin_amdgcn_readlane((int)wave_scan(t & 0xFFFF), 63);
      all += (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)wave_scan(t >> 16), 63) << 16;
      places += (uint32_t)__builtin_amdgcn_readlane((int)wave_scan(c + lane < chunks ? (uint32_t)chunk_places[c + lane] : 0), 63);
    }
  }
  const int64_t units = all * rows_of_place;
  // workgroups that take part: not so many that a row's join costs more than the
  // split saves.  With w of them a row is read in time ~ units / w and joined in
  // ~ w / rows; the sum is least where w^2 ~ units * rows.
  int64_t fit = min(units / kMinUnits, (int64_t)(kSplit * __builtin_amdgcn_sqrtf((float)units * (float)(places * rows_of_place))));
  // More than one for each CU pays where rows are short, so that workgroups wait
  // for first loads often (64 sequences up to 512 tokens: 23.1 us with two, 27.1
  // with one), or where there is much to read (up to 8192: 169 and 178); 8 sequences
  // of 2048 tokens take 20.5 with two and 18.9 with one, 4 of 8192 31.6 and 29.4.
  if (fit > p.cus && units >= kLongRow * places * rows_of_place) fit = max((int64_t)p.cus, min(fit, units / kLongRow));
  // and it is the same number for each: three for two CUs take as long as four
  if (fit > p.cus && fit < p.blocks) fit -= fit % p.cus;
  const int64_t active = fit < 1 ? 1 : (fit < p.blocks ? fit : p.blocks);
  if (units == 0 || (int64_t)blockIdx.x >= active) {
    if (threadIdx.x == 0) p.split[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }
  const Runs runs(units, active);
  const int64_t run = runs.first(blockIdx.x), run_end = runs.first(blockIdx.x + 1);
  // this wave's part of the run, and its tile of each row's query heads
  const int log2q = __builtin_ctz(p.shared_q), parts = NW >> log2q, log2p = __builtin_ctz(parts);
  const int my_part = __builtin_amdgcn_readfirstlane(wave >> log2q), my_tile = __builtin_amdgcn_readfirstlane(wave & (p.shared_q - 1));
  int64_t u = run + ((run_end - run) * my_part >> log2p);
  const int64_t begun = u, end = run + ((run_end - run) * (my_part + 1) >> log2p);
  if (my_tile == 0 && lane < 2) rows[my_part][lane].tiles = 0;
  int64_t before = 0;  // units of 32 tokens in the places before those at hand
  int chunk = 0;       // the 64 at hand
  bool looked = chunks == 1;
  while (u < end) {
    // the place of unit u: the first whose units reach beyond it
    while (chunks > 1 && chunk + 1 < chunks && (before + chunk_tiles[chunk]) * rows_of_place <= u) {
      before += chunk_tiles[chunk++];
      looked = false;
    }
    if (!looked) {
      place = place_of(g, a, listed(p, chunk * 64 + lane), bad);
      upto = wave_scan(place.s >= 0 ? (uint32_t)tiles_of(place.len) : 0);
      looked = true;
    }
    const uint64_t beyond = __builtin_amdgcn_ballot_w64((before + upto) * rows_of_place > u);
    if (beyond == 0) break;  // only where lengths change under the call
    const int at = __builtin_ctzll(beyond);
    const int i = chunk * 64 + at;
    const int32_t s = __builtin_amdgcn_readlane(place.s, at), len = __builtin_amdgcn_readlane(place.len, at);
    const int32_t tiles = tiles_of(len);
    const int64_t in_place = u - (before + (uint32_t)__builtin_amdgcn_readlane((int)upto, at) - tiles) * rows_of_place;
    const int r = (int)quotient(in_place, tiles);      // (KV head, its row)
    const int32_t ta = (int32_t)(in_place - (int64_t)r * tiles);
    const int32_t tb = (int32_t)min((int64_t)tiles, ta + (end - u));
    const int h = rows_of_head == 1 ? r : r / rows_of_head, q0 = (r - h * rows_of_head) * p.shared_q * kHeads;  // first query head of the row
    const int32_t row_at = (int32_t)((int64_t)i * p.q_heads + (int64_t)h * p.group + q0);
    const int row_heads = min(p.shared_q * kHeads, p.group - q0);
    const int heads = min(kHeads, row_heads - my_tile * kHeads);  // of the wave's tile; none where the row has no such
    const bool whole = ta == 0 && tb == tiles;
    const int slot = u == begun && !whole ? 0 : 1;
    if (!whole && my_tile == 0 && lane == 0) rows[my_part][slot] = Row{u - ta, tiles, row_at, row_heads, h};
    u += tb - ta;

    float m = -INFINITY, l = 0.0f;
    f32x4 o[NV * CW];
#pragma unroll
    for (int k = 0; k < NV * CW; ++k) o[k] = f32x4{0, 0, 0, 0};

    if (len > 0 && heads > 0) {
      bf16x8 qf[KB];
      const uint16_t *qp = p.q + (int64_t)i * p.q_stride + (int64_t)(h * p.group + q0 + my_tile * kHeads + hd) * D;
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        u32x4 v = {0, 0, 0, 0};
        const int c = K::channel(j, grp);
        if (hd < heads && c < D) v = *reinterpret_cast<const u32x4 *>(qp + c);
        qf[j] = __builtin_bit_cast(bf16x8, v);
      }
      const float sc = p.scale * (p.k_scale ? p.k_scale[h] : 1.0f) * kLog2e;

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
      if (ahead) keys.load(b0, b1);
      for (int32_t t = ta; t < tb; ++t) {
        const int left = len - t * kTile;  // tokens from here on
        if (!ahead) keys.load(b0, b1);
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
          if (ahead) keys.load(b0, b1);
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

    // To LDS: a lane has channels 128 c + CW (4 grp + x) + k of its head in o[c CW + k][x].
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (hd < heads) {
      float *const mine_at = sum_at(wave, slot, hd);
#pragma unroll
      for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int k = 0; k < CW; ++k) {
            const int ch = 128 * c + CW * (4 * grp + x) + k;
            if (D >= 16 || ch < D) mine_at[ch] = o[c * CW + k][x];
          }
      if (grp == 0) {
        sm[wave][slot][hd] = m;
        sl[wave][slot][hd] = l;
      }
    }
    if (whole) {  // written from there, in order
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      const float vs = p.v_scale ? p.v_scale[h] : 1.0f;
      for (int v = lane * 4; v < heads * D; v += 256) {
        const int hh = v / D, ch = v - hh * D;
        const int64_t q = row_at + my_tile * kHeads + hh;
        const float mx = sm[wave][1][hh], ls = sl[wave][1][hh], f = ls == 0.0f ? 0.0f : vs / ls;
        const f32x4 x = *reinterpret_cast<const f32x4 *>(sum_at(wave, 1, hh) + ch);
        *reinterpret_cast<uint2 *>(p.out + q * D + ch) = make_uint2(pack_bf16(x[0] * f, x[1] * f), pack_bf16(x[2] * f, x[3] * f));
        if (p.lse && ch == 0) p.lse[q] = ls == 0.0f ? -INFINITY : (mx + __builtin_log2f(ls)) * kLn2;
      }
    }
  }
  __syncthreads();

  // rows that span waves: parts of one row are neighbours among the parts' first and last rows
  int4 split = make_int4(0, 0, 0, 0);
  const Row mine = (&rows[0][0])[lane & (2 * NW - 1)];
  uint32_t todo = (uint32_t)__builtin_amdgcn_ballot_w64(lane < 2 * parts && mine.tiles > 0);
  while (todo) {
    const int k0 = __builtin_ctz(todo);
    const int64_t u0 = lane_of(mine.u0, k0);
    const int32_t tiles = __builtin_amdgcn_readlane(mine.tiles, k0), row_at = __builtin_amdgcn_readlane(mine.at, k0);
    const int row_heads = __builtin_amdgcn_readlane(mine.heads, k0), h = __builtin_amdgcn_readlane(mine.h, k0);
    const uint32_t of_row = todo & (uint32_t)__builtin_amdgcn_ballot_w64(mine.u0 == u0);
    todo &= ~of_row;
    const bool begins = u0 >= run, ends = u0 + tiles <= run_end;
    const int place = u0 <= run ? 0 : 1;
    if (begins && !ends) split = make_int4((int)(runs.of(u0 + tiles - 1) - blockIdx.x + 1) << 1 | place, row_at, row_heads, h);
    float *pp = p.part + ((int64_t)blockIdx.x * 2 + place) * p.slot;
    const float vs = p.v_scale ? p.v_scale[h] : 1.0f;
    for (int v = threadIdx.x * 4; v < row_heads * D; v += NW * 256) {
      const int hh = v / D, ch = v - hh * D, tile = hh / kHeads, hw = hh & (kHeads - 1);
      float ms[2 * NW], mx = -INFINITY, ls = 0.0f;
#pragma unroll
      for (int k = 0; k < 2 * NW; ++k) {
        ms[k] = of_row >> k & 1 ? sm[((k >> 1) << log2q) + tile][k & 1][hw] : -INFINITY;
        mx = __builtin_fmaxf(mx, ms[k]);
      }
      const float mb = base_of(mx);
      f32x4 ov = {0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < 2 * NW; ++k) {
        if (of_row >> k & 1) {
          const int w = ((k >> 1) << log2q) + tile;
          const float e = __builtin_amdgcn_exp2f(ms[k] - mb);
          ls = __builtin_fmaf(e, sl[w][k & 1][hw], ls);
          const f32x4 x = *reinterpret_cast<const f32x4 *>(sum_at(w, k & 1, hw) + ch);
#pragma unroll
          for (int c = 0; c < 4; ++c) ov[c] = __builtin_fmaf(e, x[c], ov[c]);
        }
      }
      if (begins && ends) {
        const float f = ls == 0.0f ? 0.0f : vs / ls;
        *reinterpret_cast<uint2 *>(p.out + (int64_t)(row_at + hh) * D + ch) = make_uint2(pack_bf16(ov[0] * f, ov[1] * f), pack_bf16(ov[2] * f, ov[3] * f));
        if (p.lse && ch == 0) p.lse[row_at + hh] = ls == 0.0f ? -INFINITY : (mx + __builtin_log2f(ls)) * kLn2;
      } else {
        *reinterpret_cast<f32x4 *>(pp + v) = ov;
        if (ch == 0) {
          pp[p.kept * D + hh] = mx;
          pp[p.kept * (D + 1) + hh] = ls;
        }
      }
    }
  }
  if (threadIdx.x == 0) p.split[blockIdx.x] = split;
}

// ---- the join ----
// out = sum_w 2^(m_w - M) O_w / sum_w 2^(m_w - M) l_w over the workgroups w that
// a row spans.  Up to eight are added up by a thread for each four values.  Of
// more, a workgroup takes 256 of the row's values, four to a lane; each of its
// waves runs through every fourth partial sum with a running maximum as the main
// kernel does, all loads of a round in flight at once, and the four are joined in
// LDS.  Where no such row begins it ends after one load.  Latency bounds it: 2.5 us
// for 16 partial sums of 8 rows, 3.5 for 1000 of 512 rows, 22 for 512 of one row.
constexpr int kJoinWaves = 4;

template <int R, int STEP, typename Part>
__device__ __forceinline__ void sum_parts(const Part &part, int first, int parts, bool in, int v, int at_m, int at_l, float &m,
                                          float &l, f32x4 &o) {
  for (int k0 = first; k0 < parts; k0 += STEP * R) {
    float ms[R], ls[R];
    f32x4 os[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int k = k0 + STEP * r;
      ms[r] = -INFINITY;
      ls[r] = 0.0f;
      os[r] = f32x4{0, 0, 0, 0};
      if (k < parts && in) {
        const float *pp = part(k);
        ms[r] = pp[at_m];
        ls[r] = pp[at_l];
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
}

__global__ __launch_bounds__(64 * kJoinWaves) void k_attend_join(PGeo g, AttendArgs p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int4 sp = p.split[blockIdx.x];
  const int parts = sp.x >> 1, values = sp.z * g.D;
  // partial sum k: the first of workgroup w + k, but for the one that the row begins inside of
  auto part = [&](int k) { return p.part + ((int64_t)(blockIdx.x + k) * 2 + (k == 0 ? sp.x & 1 : 0)) * p.slot; };
  auto write = [&](int v, float m, float l, f32x4 o) {
    const float f = l == 0.0f ? 0.0f : (p.v_scale ? p.v_scale[sp.w] : 1.0f) / l;
    *reinterpret_cast<u32x2 *>(p.out + (int64_t)sp.y * g.D + v) = u32x2{pack_bf16(o[0] * f, o[1] * f), pack_bf16(o[2] * f, o[3] * f)};
    if (p.lse && (v & (g.D - 1)) == 0) p.lse[sp.y + (v >> g.log2D)] = l == 0.0f ? -INFINITY : (m + __builtin_log2f(l)) * kLn2;
  };
  float m = -INFINITY, l = 0.0f;
  f32x4 o = {0, 0, 0, 0};
  if (parts <= 8) {  // a thread adds all of them up
    const int v = ((int)blockIdx.y * 64 * kJoinWaves + (int)threadIdx.x) * 4;
    if (parts == 0 || v >= values) return;
    const int at_m = p.kept * g.D + (v >> g.log2D);
    sum_parts<8, 1>(part, 0, parts, true, v, at_m, at_m + p.kept, m, l, o);
    write(v, m, l, o);
    return;
  }
  if ((int)blockIdx.y * 256 >= values) return;
  const int v = ((int)blockIdx.y * 64 + lane) * 4;  // the lane's first value of the row's heads * D
  const bool in = v < values;
  const int at_m = p.kept * g.D + (in ? v >> g.log2D : 0), at_l = at_m + p.kept;
  if (parts <= 8 * kJoinWaves) sum_parts<8, kJoinWaves>(part, wave, parts, in, v, at_m, at_l, m, l, o);
  else sum_parts<16, kJoinWaves>(part, wave, parts, in, v, at_m, at_l, m, l, o);
  __shared__ float sm[kJoinWaves][64], sl[kJoinWaves][64];
  __shared__ f32x4 so[kJoinWaves][64];
  sm[wave][lane] = m;
  sl[wave][lane] = l;
  so[wave][lane] = o;
  __syncthreads();
  if (wave > 0) return;
  m = -INFINITY;
#pragma unroll
  for (int w = 0; w < kJoinWaves; ++w) m = __builtin_fmaxf(m, sm[w][lane]);
  const float mb = base_of(m);
  l = 0.0f;
  o = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < kJoinWaves; ++w) {
    const float e = __builtin_amdgcn_exp2f(sm[w][lane] - mb);
    l = __builtin_fmaf(e, sl[w][lane], l);
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = __builtin_fmaf(e, so[w][lane][c], o[c]);
  }
  if (in) write(v, m, l, o);
}

struct Plan {
  int group, tiles_q, shared_q, kept, cus, blocks, slot, lds;
  int64_t bytes;
};

Plan attend_plan(const PGeo &g, int64_t q_heads) {
  Plan p;
  p.group = (int)(q_heads / g.heads);
  p.tiles_q = (p.group + kHeads - 1) / kHeads;
  p.shared_q = p.tiles_q == 1 ? 1 : (p.tiles_q == 2 ? 2 : waves_of(g.D));
  p.kept = p.group < kHeads * p.shared_q ? p.group : kHeads * p.shared_q;
  p.lds = waves_of(g.D) * 2 * (p.group < kHeads ? p.group : kHeads) * row_floats(g.D) * (int)sizeof(float);
  const int by_lds = kLds / (p.lds + 10 * 1024), by_regs = waves_per_simd(g.fmt, g.D) * 4 / waves_of(g.D);
  p.cus = device_cu_count();
  p.blocks = p.cus * (by_lds < by_regs ? by_lds : by_regs);
  p.slot = p.kept * g.D + (2 * p.kept + 3) / 4 * 4;
  p.bytes = p.blocks * ((int64_t)sizeof(int4) + 2 * (int64_t)sizeof(float) * p.slot);
  return p;
}

template <int FMT, int D>
void launch_attend(const PGeo &g, const skv_pages &pages, int layer, const AttendArgs &p, int lds, int32_t *status, hipStream_t st) {
  const dim3 grid((uint32_t)p.blocks), block(64 * waves_of(D));
  if (p.tiles_q == 1) k_attend<FMT, D, 1><<<grid, block, lds, st>>>(g, pages, layer, p, status);
  else k_attend<FMT, D, 0><<<grid, block, lds, st>>>(g, pages, layer, p, status);
}

}  // namespace

extern "C" int skv_attend_workspace_size(const skv_pages_shape *shape, int64_t q_heads, size_t *bytes) {
  PGeo g;
  int e = make_pgeo(shape, g);
  if (e != SKV_OK) return e;
  if (!bytes || q_heads < 1 || q_heads > (1 << 16) || q_heads % g.heads) return SKV_ERR_ARG;
  *bytes = (size_t)attend_plan(g, q_heads).bytes;
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
  if (layer < 0 || layer >= g.layers || n < 0 || n > kMaxRows || !status || !aligned4(status)) return SKV_ERR_ARG;
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
  const Plan plan = attend_plan(g, q_heads);
  p.group = plan.group;
  p.tiles_q = plan.tiles_q;
  p.shared_q = plan.shared_q;
  p.kept = plan.kept;
  p.slot = plan.slot;
  p.out = static_cast<uint16_t *>(out);
  p.lse = lse;
  // no more workgroups than the longest sequences that the table holds could use
  const __int128 units = (__int128)n * g.heads * plan.tiles_q * (((int64_t)g.max_tokens + kTile - 1) / kTile) / kMinUnits + 1;
  p.blocks = units < plan.blocks ? (int)units : plan.blocks;
  p.cus = plan.cus;
  p.split = static_cast<int4 *>(workspace);
  p.part = reinterpret_cast<float *>(p.split + p.blocks);
  hipStream_t st = static_cast<hipStream_t>(stream);
#define SKV_ATTEND(F_, D_) case D_: launch_attend<F_, D_>(g, *pages, (int)layer, p, plan.lds, status, st); break
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
  k_attend_join<<<dim3((uint32_t)p.blocks, (uint32_t)((p.kept * g.D + 255) / 256)), 64 * kJoinWaves, 0, st>>>(g, p);
  return hipGetLastError() == hipSuccess ? SKV_OK : SKV_ERR_HIP;
}
