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
// take chunks of 8.
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
// act(v) and its slope.  16-bit data takes the hardware's exponential and
// reciprocal (within a few 2^-23, far below its own rounding).
struct ActValue {
  float a, slope;
};

template <class T>
__device__ inline void logistic(float v, float& s, float& rest) {  // s(v) and 1 - s(v)
  float t;
  if constexpr (sizeof(T) == 4) {
    t = expf(-v);
    s = 1.0f / (1.0f + t);
  } else {
    t = __builtin_amdgcn_exp2f(v * -1.44269504088896340736f);
    s = __builtin_amdgcn_rcpf(1.0f + t);
  }
  rest = v > 0.0f ? t * s : 1.0f - s;  // 1 - s cancels where s is near 1
}

template <class T>
__device__ inline ActValue act_value(int32_t act, float v) {
  if (act == EMB_ACT_SILU) {
    float s, rest;
    logistic<T>(v, s, rest);
    return {v * s, s + v * (s * rest)};
  }
  if (act == EMB_ACT_GELU) {
    const float cdf = 0.5f * erfcf(v * -0.70710678118654752440f);
    return {v * cdf, cdf + v * (0.39894228040143267794f * expf(-0.5f * v * v))};
  }
  if (act == EMB_ACT_RELU) return {v <= 0.0f ? 0.0f : v, v <= 0.0f ? 0.0f : 1.0f};
  float s, rest;
  logistic<T>(v, s, rest);
  return {s, s * rest};
}

// ---------------------------------------------------------------- stores
// The first n of four neighbouring values, each rounded once.
template <class T>
__device__ inline void store4(T* p, f32x4 v, int64_t n) {
  if (n >= 4) {
    if constexpr (sizeof(T) == 4) {
      Raw<float> r;
#pragma unroll
      for (int i = 0; i < 4; ++i) r.w[i] = __float_as_uint(v[i]);
      store_raw(p, r);
    } else {
      Raw<T, 4> r;
      const float f[4] = {v[0], v[1], v[2], v[3]};
      r.set_all(f);
      store_raw<T, 4>(p, r);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) p[i] = from_f32<T>(v[i]);
}

// The first n of four neighbouring values, then zeros.
template <class T>
__device__ inline Raw<T, 4> load_part4(const T* p, int64_t n) {
  if (n >= 4) return load_raw<T, 4>(p);
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = i < n ? to_f32(p[i]) : 0.0f;
  Raw<T, 4> r;
  r.set_all(f);
  return r;
}

// ---------------------------------------------------------------- epilogues
// Of four neighbouring columns from n on, of `width`, in row `row` of the buffer.  held(): what it reads of
// them, for callers that have these loads on their way before they are needed.
struct NothingHeld {};

template <class T>
struct StoreEpilogue {
  static constexpr bool kDual = false;
  T* out;
  int64_t width;
  typedef NothingHeld Held;
  __device__ inline Held held(int64_t, int64_t) const { return {}; }
  __device__ inline void operator()(int64_t row, int64_t n, f32x4 v, Held) const {
    store4(out + row * width + n, v, width - n);
  }
};

// Weight gradients: the expert's matrices, or the parts' sums, [expert][part].
template <class Out>
struct WeightEpilogue {
  Out* out[2];
  __device__ inline void operator()(int32_t product, int64_t matrix, int64_t M, int64_t N,
                                    int64_t m, int64_t n, f32x4 v) const {
    store4(out[product] + (matrix * M + m) * N + n, v, N - n);
  }
};

// The activated product from both projections.
template <class T>
struct ActEpilogue {
  static constexpr bool kDual = true;
  T *gu, *a;  // gu: null where it is not kept
  int64_t width;
  int32_t act;
  typedef NothingHeld Held;
  __device__ inline Held held(int64_t, int64_t) const { return {}; }
  __device__ inline f32x4 product(int64_t row, int64_t n, f32x4 g, f32x4 u) const {
    const int64_t have = width - n;
    if (gu) {
      store4(gu + row * 2 * width + n, g, have);
      store4(gu + (row * 2 + 1) * width + n, u, have);
    }
    f32x4 p;
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = act_value<T>(act, g[i]).a * u[i];
    store4(a + row * width + n, p, have);
    return p;
  }
  __device__ inline void operator()(int64_t row, int64_t n, f32x4 g, f32x4 u, Held) const {
    product(row, n, g, u);
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
  struct Held {
    Raw<T, 4> g, u;
  };
  __device__ inline Held held(int64_t row, int64_t n) const {
    return {load_part4(gu + row * 2 * width + n, width - n),
            load_part4(gu + (row * 2 + 1) * width + n, width - n)};
  }
  __device__ inline void gradients(f32x4 da, const Held& h, f32x4& dg, f32x4& du) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const ActValue f = act_value<T>(act, h.g.get(i));
      dg[i] = da[i] * h.u.get(i) * f.slope;
      du[i] = da[i] * f.a;
    }
  }
  __device__ inline void operator()(int64_t row, int64_t n, f32x4 da, const Held& h) const {
    const int64_t have = width - n;
    f32x4 dg, du;
    gradients(da, h, dg, du);
    store4(dgu + row * 2 * width + n, dg, have);
    store4(dgu + (row * 2 + 1) * width + n, du, have);
  }
};

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
