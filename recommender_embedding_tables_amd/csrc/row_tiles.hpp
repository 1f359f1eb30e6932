// Rows of up to 8192 values on the threads of a block: which threads share a
// row, their columns, and sums over them.  Of the kernels that normalise rows
// (gated_norm.hip, rows_int8.hip).
#pragma once

#include "dense.hpp"

namespace embtab {

constexpr int kMaxWaves = 16;
constexpr int kCus = 256;

// 1 / sqrt(x) by the hardware instruction (1 ulp), which takes no denormals:
// those are scaled up by 2^64 first.
__device__ inline float inv_sqrt(float x) {
  const bool tiny = x < 0x1p-100f;
  return __builtin_amdgcn_rsqf(tiny ? x * 0x1p64f : x) * (tiny ? 0x1p32f : 1.0f);
}

// How the rows lie on the threads: tpr threads share a row (8 .. 64 lanes of
// a wave, or, MULTI, the whole block), each holding V vectors of it, at most 8
// values: the backward pass holds about 15 registers for each.
struct Shape {
  int32_t tpr, threads, vecs, multi;
  int32_t rows_per_block() const { return multi ? 1 : threads / tpr; }
  int32_t waves() const { return threads / 64; }
};

template <class T>
Shape shape_of(int32_t dim) {
  const int nvec = (dim + kVec<T> - 1) / kVec<T>;
  Shape s{8, 256, 1, 0};
  while (s.tpr < 64 && s.tpr < nvec) s.tpr *= 2;
  if (nvec <= 64) return s;
  s.vecs = sizeof(T) == 4 ? 2 : 1;
  if (nvec <= 64 * s.vecs) return s;
  s.multi = 1;
  s.tpr = s.threads = ((nvec + s.vecs - 1) / s.vecs + 63) / 64 * 64;
  return s;
}

template <int CTRL>
__device__ inline float dpp(float v) {
  return __uint_as_float(
      (uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}

// Sum over groups of tpr (8, 16, 32 or 64) neighbouring lanes, in every lane:
// quads, half rows and rows by lane permutations, then pairs of rows and the
// halves of the wave by row swaps; no LDS.  Both lanes of a pair add the same
// two values, so the lanes' results have the same bits.
__device__ inline float lanes_sum(float v, int tpr) {
  v += dpp<0xB1>(v);   // quad_perm 1,0,3,2
  v += dpp<0x4E>(v);   // quad_perm 2,3,0,1
  v += dpp<0x141>(v);  // the other quad of 8
  if (tpr >= 16) v += dpp<0x140>(v);  // the other half of 16
  if (tpr >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if (tpr >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// Sums of N values over the threads of a row.  MULTI rows pass through LDS,
// with one barrier: the calls of a kernel alternate between two buffers, so a
// wave that writes for the next sum never meets one that still reads this
// one.  Lane l then takes wave l % 16's part (zero for a wave the block does
// not have) and the 16 are added as above.
struct SumBuffers {
  float part[2][3][kMaxWaves];
};

template <bool MULTI, int N>
__device__ inline void row_sum(float (&v)[N], int tpr, SumBuffers& lds, uint32_t& turn) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = lanes_sum(v[k], MULTI ? 64 : tpr);
  if (!MULTI) return;
  float(*part)[kMaxWaves] = lds.part[turn];
  turn ^= 1u;
  if ((threadIdx.x & 63u) == 0u)
#pragma unroll
    for (int k = 0; k < N; ++k) part[k][threadIdx.x >> 6] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = lanes_sum(part[k][threadIdx.x % kMaxWaves], kMaxWaves);
}

template <bool MULTI>
__device__ inline void clear_sums(SumBuffers& lds) {
  if (!MULTI) return;
  for (uint32_t i = threadIdx.x; i < 2u * 3u * kMaxWaves; i += blockDim.x)
    (&lds.part[0][0][0])[i] = 0.0f;
  __syncthreads();
}

// The columns of one thread: vector v starts at col[v].  A vector that would
// pass the row's end is moved back to end with it (TAIL: the width is not a
// multiple of the vector); its elements before skip[v] belong to the vector
// before and are left out of sums, and stored twice with the same value.  A
// vector past the row (skip = its width) repeats the last one and stores
// nothing.
template <class T, int V, bool TAIL>
struct Columns {
  uint32_t col[V], skip[V];
  __device__ Columns(uint32_t lane, uint32_t tpr, uint32_t dim) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t c = (lane + v * tpr) * (uint32_t)kVec<T>;
      col[v] = c + kVec<T> <= dim ? c : dim - kVec<T>;
      skip[v] = c >= dim ? kVec<T> : c - col[v];
    }
  }
  __device__ bool any(int v) const { return skip[v] < kVec<T>; }
  // of a vector with any(v)
  __device__ bool owns(int v, int e) const { return !TAIL || (uint32_t)e >= skip[v]; }
};

// Blocks for rows, so that a CU holds waves_per_cu waves, in whole blocks and at
// least one: the blocks walk over the rows.
inline unsigned grid_of(int64_t rows, const Shape& s, int waves_per_cu) {
  const int64_t g = (rows + s.rows_per_block() - 1) / s.rows_per_block();
  const int per_cu = waves_per_cu / s.waves() > 1 ? waves_per_cu / s.waves() : 1;
  const int64_t most = (int64_t)kCus * per_cu;
  return (unsigned)(g < most ? g : most);
}

}  // namespace embtab
