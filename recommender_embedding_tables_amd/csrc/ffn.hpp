// Products of the experts' gated feed-forward: row groups, tiles, operands and
// epilogues that its kernels share.
#pragma once

#include "dense.hpp"

namespace embtab {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------- row groups
// Expert e's rows of the expert-ordered buffer.  Offsets that name no rows of
// the buffer give an empty or shortened group: no access leaves it.
struct Groups {
  const int32_t* offsets;  // [experts + 1], or null: one group of all rows
  int64_t rows, capacity;
  int32_t experts;
};
struct Group {
  int64_t first, count;
};

__device__ inline Group group_of(const Groups& g, int32_t e) {
  if (!g.offsets) return {0, g.rows};
  const int64_t from = g.offsets[e];
  int64_t n = (int64_t)g.offsets[e + 1] - from;
  const int64_t first = g.capacity ? g.capacity * e : from;
  if (g.capacity && n > g.capacity) n = g.capacity;
  if (first < 0 || first >= g.rows || n < 0) return {0, 0};
  return {first, n < g.rows - first ? n : g.rows - first};
}

// Most tiles of `tile` rows that the groups can need.
inline int64_t row_tiles_bound(const Groups& g, int64_t tile) {
  if (!g.offsets) return (g.rows + tile - 1) / tile;
  if (g.capacity) {
    const int64_t full = (g.rows + g.capacity - 1) / g.capacity;
    return (full < g.experts ? full : g.experts) * ((g.capacity + tile - 1) / tile);
  }
  // ceil(n / tile) <= (n + tile - 1) / tile over the groups that hold a row
  const int64_t used = g.rows < g.experts ? g.rows : g.experts;
  return (g.rows + used * (tile - 1)) / tile;
}

// ---------------------------------------------------------------- tile order
// Blocks go to the 8 XCDs in turn, each with an L2 of its own.  The order is cut
// into chunks which the XCDs take in turn: an XCD works on neighbouring tiles, and
// the tiles of a long group are spread over all of them.  Inside a group, panels
// of kPanel row tiles walk over the column tiles with the rows innermost.  Chunks
// of 32 tiles (8 row and 4 column tiles), one for each CU of an XCD, where every
// tile costs the same; weight gradients, whose tiles cost their expert's rows,
// take chunks of 8 and the longest expert first (32768 x 3328 x 1664 bf16, 16 experts
// with 0.3 to 3 times the mean's rows: 1156 us for both matrices, in chunks of 32 by
// expert 1463, with one run of tiles to each XCD 2125).
constexpr uint32_t kXcds = 8, kPanel = 8;
constexpr uint32_t kRowChunk = 32, kWeightChunk = 8;

__device__ inline bool place_of(uint32_t block, uint64_t all, uint32_t longest, uint64_t& place) {
  const uint64_t even = (all + kXcds - 1) / kXcds;
  const uint32_t chunk = even < longest ? (uint32_t)even : longest;
  if (chunk == 0) return false;
  const uint32_t i = block / kXcds;
  place = ((uint64_t)(i / chunk) * kXcds + block % kXcds) * chunk + i % chunk;
  return place < all;
}
// Blocks that hold the places of up to `most` tiles.
inline int64_t blocks_of(int64_t most, int64_t longest) {
  const int64_t whole = kXcds * (most > kXcds * longest ? longest : 1);
  return (most + whole - 1) / whole * whole;
}

__device__ inline void panel_tile(uint32_t local, uint32_t row_tiles, uint32_t col_tiles,
                                  uint32_t& rt, uint32_t& ct) {
  const uint32_t p = local / (kPanel * col_tiles), base = p * kPanel;
  const uint32_t high = row_tiles - base < kPanel ? row_tiles - base : kPanel;
  const uint32_t r = local - p * kPanel * col_tiles;
  rt = base + r % high;
  ct = r / high;
}

struct RowTile {
  int32_t expert;
  int64_t first, count;  // the group's rows
  uint32_t rt, ct;       // tile of the group's rows, tile of the columns
};

// The tile of a block; false where there is none.  Every wave finds it by
// itself from the groups' counts (64 experts a step).
__device__ inline bool find_row_tile(const Groups& g, uint32_t tile, uint32_t col_tiles,
                                     uint32_t block, RowTile& t) {
  if (!g.offsets) {
    const uint32_t n = (uint32_t)((g.rows + tile - 1) / tile);
    uint64_t place;
    if (!place_of(block, (uint64_t)n * col_tiles, kRowChunk, place)) return false;
    t.expert = 0;
    t.first = 0;
    t.count = g.rows;
    panel_tile((uint32_t)place, n, col_tiles, t.rt, t.ct);
    return true;
  }
  const int lane = threadIdx.x & 63;
  uint32_t total = 0;
  for (int32_t e0 = 0; e0 < g.experts; e0 += 64) {
    uint32_t n = 0;
    if (e0 + lane < g.experts)
      n = (uint32_t)((group_of(g, e0 + lane).count + tile - 1) / tile);
    total += (uint32_t)__builtin_amdgcn_readlane((int)wave_incl_scan(n), 63);
  }
  uint64_t place;
  if (!place_of(block, (uint64_t)total * col_tiles, kRowChunk, place)) return false;
  const uint32_t want = (uint32_t)(place / col_tiles);  // in row tiles of the groups in order
  uint32_t before = 0;
  for (int32_t e0 = 0; e0 < g.experts; e0 += 64) {
    uint32_t n = 0;
    if (e0 + lane < g.experts)
      n = (uint32_t)((group_of(g, e0 + lane).count + tile - 1) / tile);
    const uint32_t upto = before + wave_incl_scan(n);
    const uint64_t hit = __ballot(want < upto);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      t.expert = e0 + l;
      const uint32_t mine = (uint32_t)__builtin_amdgcn_readlane((int)n, l);
      const uint32_t start = (uint32_t)__builtin_amdgcn_readlane((int)upto, l) - mine;
      const Group gr = group_of(g, t.expert);
      t.first = gr.first;
      t.count = gr.count;
      panel_tile((uint32_t)(place - (uint64_t)start * col_tiles), mine, col_tiles, t.rt, t.ct);
      return true;
    }
    before = (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
  }
  return false;
}

// Two products of the experts' rows in one launch, C[p][m, n] = sum over one
// expert's rows of A[p][row, m] B[p][row, n], and the tile of them that a block
// computes.  Experts go in the order of their rows, the longest first (up to 64
// experts; more even out by themselves), so that no long one is left to the end.
template <class T>
struct WeightProducts {
  Groups groups;
  const T *A[2], *B[2];
  int64_t M[2], N[2];
  uint32_t row_tiles[2], col_tiles[2];
  uint32_t parts;  // that an expert's rows are cut into
};
struct WeightTile {
  int32_t expert, product;
  uint32_t part, rt, ct;
};

__device__ inline int32_t expert_by_rows(const Groups& g, int32_t place) {
  if (g.experts > 64) return place;
  const int lane = threadIdx.x & 63;
  const int32_t n = lane < g.experts ? (int32_t)group_of(g, lane).count : -1;
  int32_t before = 0;
  for (int32_t e = 0; e < g.experts; ++e) {
    const int32_t other = __builtin_amdgcn_readlane(n, e);
    before += other > n || (other == n && e < lane);
  }
  return (int32_t)__builtin_ctzll(__ballot(lane < g.experts && before == place));
}

template <class T>
__device__ inline bool find_weight_tile(const WeightProducts<T>& w, uint32_t block,
                                        WeightTile& t) {
  const uint32_t first = w.row_tiles[0] * w.col_tiles[0];
  const uint32_t tiles = first + w.row_tiles[1] * w.col_tiles[1];
  uint64_t place;
  if (!place_of(block, (uint64_t)tiles * w.parts * w.groups.experts, kWeightChunk, place))
    return false;
  const uint32_t matrix = (uint32_t)(place / tiles);
  uint32_t local = (uint32_t)(place - (uint64_t)matrix * tiles);
  t.expert = expert_by_rows(w.groups, (int32_t)(matrix / w.parts));
  t.part = matrix % w.parts;
  t.product = local >= first;
  if (t.product) local -= first;
  panel_tile(local, w.row_tiles[t.product], w.col_tiles[t.product], t.rt, t.ct);
  return true;
}

// Rows `from` .. `from + count` of expert e's group that part `part` adds up, in
// whole steps.
__device__ inline void part_rows(const Group& g, uint32_t parts, uint32_t part, int64_t step,
                                 int64_t& from, int64_t& count) {
  const int64_t per = ((g.count + parts - 1) / parts + step - 1) / step * step;
  from = per * part < g.count ? per * part : g.count;
  count = g.count - from < per ? g.count - from : per;
}

inline dim3 tile_grid(int64_t blocks, int threads) {
  const int64_t x = ((int64_t)1 << 31) / threads;  // fewer than 2^32 threads along x
  if (blocks <= x) return dim3((unsigned)blocks);
  return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}

// ---------------------------------------------------------------- activations
// act(v) and its slope for N values (one choice of the activation for all).
//
// e^-v as 2 to the power of -v log2(e) by the hardware.  The product's rounding
// would be |v| 2^-24 of the result: below 16-bit data's own rounding, while fp32
// takes it up again, e = the product's error with log2(e)'s second half, as
// 2^(p + e) = 2^p (1 + e ln 2) within 2^-37 (|e| < 2^-17).  1 / (1 + t) by the hardware's
// reciprocal (1 ulp), for fp32 with one Newton step below 2^126.  The hardware gives 0
// for results below 2^-126.
template <class T>
__device__ inline float exp_neg(float v) {
  constexpr float kLog = 1.44269504088896340736f, kLow = 1.92596299112661746887e-8f;
  const float p = v * -kLog;
  const float t = __builtin_amdgcn_exp2f(p);
  if constexpr (sizeof(T) == 2) return t;
  if (!(__builtin_fabsf(p) < 126.0f)) return t;  // 0 or infinite, nearly or in fact, or a NaN
  const float e = __builtin_fmaf(v, -kLow, __builtin_fmaf(v, -kLog, -p));
  return __builtin_fmaf(t, e * 0.69314718055994530942f, t);
}

template <class T>
__device__ inline void logistic(float v, float& s, float& rest) {  // s(v) and 1 - s(v)
  const float t = exp_neg<T>(v), x = 1.0f + t;
  s = __builtin_amdgcn_rcpf(x);
  if constexpr (sizeof(T) == 4)
    s = x < 0x1p126f ? __builtin_fmaf(__builtin_fmaf(-x, s, 1.0f), s, s) : s;
  rest = v > 0.0f ? t * s : 1.0f - s;  // 1 - s cancels where s is near 1
}

template <class T, int N>
__device__ inline void activate(int32_t act, const float (&v)[N], float (&a)[N],
                                float (&slope)[N]) {
  if (act == EMB_ACT_SILU || act == EMB_ACT_SIGMOID) {
    const bool silu = act == EMB_ACT_SILU;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s, rest;
      logistic<T>(v[i], s, rest);
      a[i] = silu ? v[i] * s : s;
      slope[i] = silu ? s + v[i] * (s * rest) : s * rest;
    }
  } else if (act == EMB_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float cdf = 0.5f * erfcf(v[i] * -0.70710678118654752440f);
      a[i] = v[i] * cdf;
      slope[i] = cdf + v[i] * (0.39894228040143267794f * expf(-0.5f * v[i] * v[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      a[i] = v[i] <= 0.0f ? 0.0f : v[i];
      slope[i] = v[i] <= 0.0f ? 0.0f : 1.0f;
    }
  }
}

// ---------------------------------------------------------------- values
// W neighbouring values in memory, 8 or 16 bytes (or twice 16), and the first n of
// them.
template <class T, int W>
struct Span {
  static constexpr int kPer = W < kVec<T> ? W : kVec<T>;
  Raw<T, kPer> r[W / kPer];
  __device__ inline float get(int i) const { return r[i / kPer].get(i % kPer); }
};

template <int W, class T>
__device__ inline void store_span(T* p, const float (&v)[W], int64_t n) {
  typedef Span<T, W> S;
  if (n >= W) {
#pragma unroll
    for (int k = 0; k < W / S::kPer; ++k) {
      Raw<T, S::kPer> r;
      r.set_all(v + k * S::kPer);
      store_raw<T, S::kPer>(p + k * S::kPer, r);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < W; ++i)
    if (i < n) p[i] = from_f32<T>(v[i]);
}

// zeros behind the first n
template <int W, class T>
__device__ inline Span<T, W> load_span(const T* p, int64_t n) {
  typedef Span<T, W> S;
  S s;
  if (n >= W) {
#pragma unroll
    for (int k = 0; k < W / S::kPer; ++k) s.r[k] = load_raw<T, S::kPer>(p + k * S::kPer);
    return s;
  }
  float f[W];
#pragma unroll
  for (int i = 0; i < W; ++i) f[i] = i < n ? to_f32(p[i]) : 0.0f;
#pragma unroll
  for (int k = 0; k < W / S::kPer; ++k) s.r[k].set_all(f + k * S::kPer);
  return s;
}

// ---------------------------------------------------------------- epilogues
// Of W neighbouring columns from n on, in a row of the buffer.  row(): its places;
// held(): what is read there, for callers that have these loads on their way before
// they are needed.
struct NothingHeld {};

template <class T>
struct StoreEpilogue {
  static constexpr bool kDual = false;
  T* out;
  int64_t width;
  struct Row {
    T* out;
  };
  template <int W>
  using Held = NothingHeld;
  __device__ inline Row row(int64_t r) const { return {out + r * width}; }
  template <int W>
  __device__ inline Held<W> held(const Row&, int64_t) const {
    return {};
  }
  template <int W>
  __device__ inline void store(const Row& r, int64_t n, const float (&v)[W],
                               const Held<W>&) const {
    store_span(r.out + n, v, width - n);
  }
};

// The activated product from both projections.
template <class T>
struct ActEpilogue {
  static constexpr bool kDual = true;
  T *gu, *a;  // gu: null where it is not kept
  int64_t width;
  int32_t act;
  struct Row {
    T *gu, *a;
  };
  template <int W>
  using Held = NothingHeld;
  __device__ inline Row row(int64_t r) const {
    return {gu ? gu + r * 2 * width : nullptr, a + r * width};
  }
  template <int W>
  __device__ inline Held<W> held(const Row&, int64_t) const {
    return {};
  }
  template <int W>
  __device__ inline void product(const Row& r, int64_t n, const float (&g)[W],
                                 const float (&u)[W], float (&p)[W]) const {
    if (r.gu) {
      store_span(r.gu + n, g, width - n);
      store_span(r.gu + width + n, u, width - n);
    }
    float slope[W];
    activate<T>(act, g, p, slope);
#pragma unroll
    for (int i = 0; i < W; ++i) p[i] *= u[i];
    store_span(r.a + n, p, width - n);
  }
  template <int W>
  __device__ inline void store(const Row& r, int64_t n, const float (&g)[W], const float (&u)[W],
                               const Held<W>&) const {
    float p[W];
    product(r, n, g, u, p);
  }
};

// The pre-activations' gradients from the product's.
template <class T>
struct ActGradEpilogue {
  static constexpr bool kDual = false;
  const T* gu;
  T* dgu;
  int64_t width;
  int32_t act;
  struct Row {
    const T* gu;
    T* dgu;
  };
  template <int W>
  struct Held {
    Span<T, W> g, u;
  };
  __device__ inline Row row(int64_t r) const {
    return {gu + r * 2 * width, dgu + r * 2 * width};
  }
  template <int W>
  __device__ inline Held<W> held(const Row& r, int64_t n) const {
    return {load_span<W>(r.gu + n, width - n), load_span<W>(r.gu + width + n, width - n)};
  }
  template <int W>
  __device__ inline void gradients(const float (&da)[W], const Held<W>& h, float (&dg)[W],
                                   float (&du)[W]) const {
    float g[W], f[W], slope[W];
#pragma unroll
    for (int i = 0; i < W; ++i) g[i] = h.g.get(i);
    activate<T>(act, g, f, slope);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      dg[i] = da[i] * h.u.get(i) * slope[i];
      du[i] = da[i] * f[i];
    }
  }
  template <int W>
  __device__ inline void store(const Row& r, int64_t n, const float (&da)[W],
                               const Held<W>& h) const {
    float dg[W], du[W];
    gradients(da, h, dg, du);
    store_span(r.dgu + n, dg, width - n);
    store_span(r.dgu + width + n, du, width - n);
  }
};

// Weight gradients: the expert's matrices, or the parts' sums, [expert][part].
template <class Out>
struct WeightEpilogue {
  Out* out[2];
};

// Four results of a matrix instruction, or of two whose columns follow each other.
__device__ inline void put4(float* v, f32x4 x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = x[i];
}

// ---------------------------------------------------------------- matrix steps
template <class T>
__device__ inline f32x4 mfma_16x16x32(i16x8 a, i16x8 b, f32x4 c) {
  if constexpr (__is_same(T, f16_t))
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Of 16 lanes, each naming four neighbouring values of one of four rows (lane i:
// row i / 4, values 4 (i % 4) on), lane i gets the four rows' values of column i.
__device__ inline i16x4 lds_read_columns(const uint16_t* p) {
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (lds_i16x4*)(__attribute__((address_space(3))) void*)p);
}

}  // namespace embtab
