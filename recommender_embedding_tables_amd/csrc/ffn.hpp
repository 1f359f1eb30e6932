// Products of the experts' gated feed-forward: row groups, tiles, operands and
// epilogues that its kernels share.
#pragma once

#include "dense.hpp"

namespace embtab {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
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
// Blocks go to the 8 XCDs in turn, each with an L2 of its own: block b takes
// place (b mod 8) * per + b / 8 of the order, so that an XCD works on
// neighbouring tiles.  Inside a group, panels of kPanel row tiles walk over the
// column tiles with the rows innermost: 32 blocks of an XCD share 8 row and 4
// column tiles.
constexpr uint32_t kXcds = 8, kPanel = 8;

__device__ inline bool place_of(uint32_t block, uint64_t all, uint64_t& place) {
  const uint64_t per = (all + kXcds - 1) / kXcds;
  const uint64_t i = block / kXcds;
  place = (block % kXcds) * per + i;
  return i < per && place < all;
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
    if (!place_of(block, (uint64_t)n * col_tiles, place)) return false;
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
  if (!place_of(block, (uint64_t)total * col_tiles, place)) return false;
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

template <class T>
__device__ inline f32x4 load4(const T* p, int64_t n) {
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (n >= 4) {
    if constexpr (sizeof(T) == 4) {
      const Raw<float> r = load_raw(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = r.get(i);
    } else {
      const Raw<T, 4> r = load_raw<T, 4>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = r.get(i);
    }
    return v;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) v[i] = to_f32(p[i]);
  return v;
}

// ---------------------------------------------------------------- epilogues
// Of four neighbouring columns from n on, of `width`, in row `row` (of the
// buffer; of the expert's matrix for weight gradients).
template <class T>
struct StoreEpilogue {
  static constexpr bool kDual = false;
  T* out;
  int64_t width, expert_stride;
  __device__ inline void operator()(int32_t e, int64_t row, int64_t n, f32x4 v) const {
    store4(out + e * expert_stride + row * width + n, v, width - n);
  }
};

// Partial sums of weight gradients, one matrix per part.
struct PartEpilogue {
  static constexpr bool kDual = false;
  float* out;
  int64_t width, expert_stride;
  __device__ inline void operator()(int32_t e, int64_t row, int64_t n, f32x4 v) const {
    store4(out + e * expert_stride + row * width + n, v, width - n);
  }
};

// The activated product from both projections.
template <class T>
struct ActEpilogue {
  static constexpr bool kDual = true;
  T *gu, *a;  // gu: null where it is not kept
  int64_t width;
  int32_t act;
  __device__ inline void operator()(int32_t, int64_t row, int64_t n, f32x4 g, f32x4 u) const {
    const int64_t have = width - n;
    if (gu) {
      store4(gu + row * 2 * width + n, g, have);
      store4(gu + (row * 2 + 1) * width + n, u, have);
    }
    f32x4 p;
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = act_value<T>(act, g[i]).a * u[i];
    store4(a + row * width + n, p, have);
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
  __device__ inline void operator()(int32_t, int64_t row, int64_t n, f32x4 da) const {
    const int64_t have = width - n;
    const f32x4 g = load4(gu + row * 2 * width + n, have);
    const f32x4 u = load4(gu + (row * 2 + 1) * width + n, have);
    f32x4 dg, du;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const ActValue f = act_value<T>(act, g[i]);
      dg[i] = da[i] * u[i] * f.slope;
      du[i] = da[i] * f.a;
    }
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
