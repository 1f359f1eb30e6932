// The residual's addition, the norm of the sum and its row-wise 8-bit codes in
// one pass, for gfx950.
//
// Per row of D values, every step in fp32:
//   y = x + block                              (stored rounded once)
//   r = rsqrt(mean(y^2) + eps),  h = (y * r) * w
//   amax = max |h|;  code = round-to-nearest-even(h * (127 / amax)),
//   scale = amax / 127;  codes and scale 0 where amax is 0
// h is formed from the unrounded y and never stored.  127 / amax passes fp32's
// range below 2^-121: such a row is scaled up by 2^64 first, exactly.  A row
// with a value that is not finite, or whose squares pass fp32's range, has no
// codes: all 0, with a NaN for its scale, so that it cannot pass unseen.
//
// Bound by memory: two streams read, one written, and a byte per value.  A
// row's vectors stay in the registers of the threads that share it, so the sum,
// the maximum and the codes come from one read (row_tiles.hpp), and a thread's
// next row is loaded with the stores of this one.  65536 x 3328 bf16: 291 us, 5.2 TB/s
// (1529 MB by the counters, none twice).
#include "row_tiles.hpp"

namespace embtab {

namespace {

// Waves on each CU (in whole blocks, at least one block).
constexpr int kNormWaves = 14;

typedef u2 u2_at1 __attribute__((aligned(1)));
typedef uint32_t u1_at1 __attribute__((aligned(1)));

template <int CTRL>
__device__ inline uint32_t dpp_max(uint32_t v) {
  const uint32_t o =
      (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
  return v > o ? v : o;
}

// Largest over groups of tpr neighbouring lanes, in every lane (as lanes_sum).
__device__ inline uint32_t lanes_max(uint32_t v, int tpr) {
  v = dpp_max<0xB1>(v);
  v = dpp_max<0x4E>(v);
  v = dpp_max<0x141>(v);
  if (tpr >= 16) v = dpp_max<0x140>(v);
  if (tpr >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = r[0] > r[1] ? r[0] : r[1];
  }
  if (tpr >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = r[0] > r[1] ? r[0] : r[1];
  }
  return v;
}

// Largest over the threads of a row; for rows of a block (MULTI) through the
// buffers of row_sum, in turn with it.
template <bool MULTI>
__device__ inline uint32_t row_max(uint32_t v, int tpr, SumBuffers& lds, uint32_t& turn) {
  v = lanes_max(v, MULTI ? 64 : tpr);
  if (!MULTI) return v;
  float* part = lds.part[turn][0];
  turn ^= 1u;
  if ((threadIdx.x & 63u) == 0u) part[threadIdx.x >> 6] = __uint_as_float(v);
  __syncthreads();
  return lanes_max(__float_as_uint(part[threadIdx.x % kMaxWaves]), kMaxWaves);
}

template <class T, int V, bool MULTI, bool TAIL>
__global__ __launch_bounds__(MULTI ? 1024 : 256) void k_add_norm_int8(
    const T* x, const T* block, const float* __restrict__ w, int64_t rows, uint32_t dim,
    int32_t tpr, float eps, T* y, int8_t* __restrict__ codes, float* __restrict__ scales) {
  constexpr int N = kVec<T>;
  __shared__ SumBuffers lds;
  uint32_t turn = 0;
  const uint32_t lane = MULTI ? threadIdx.x : threadIdx.x % (uint32_t)tpr;
  const uint32_t rpb = MULTI ? 1u : blockDim.x / (uint32_t)tpr;
  const uint32_t mine = MULTI ? 0u : threadIdx.x / (uint32_t)tpr;
  const Columns<T, V, TAIL> c(lane, (uint32_t)tpr, dim);
  const float inv = 1.0f / (float)dim;
  const int64_t step = (int64_t)gridDim.x * rpb, last = rows - 1;
  int64_t r = (int64_t)blockIdx.x * rpb + mine;
  Raw<T> in[2][V];
  const auto load = [&](int64_t row) {
    const size_t at = (size_t)row * dim;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      in[0][v] = load_raw<T, N, true>(x + at + c.col[v]);
      in[1][v] = load_raw<T, N, true>(block + at + c.col[v]);
    }
  };
  load(r < last ? r : last);
  float weight[V][N];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < N; e += 4) {
      const Raw<float> q = load_raw(w + c.col[v] + e);
#pragma unroll
      for (int i = 0; i < 4; ++i) weight[v][e + i] = q.get(i);
    }
  clear_sums<MULTI>(lds);
  // every thread of a block takes the same number of rounds (barriers)
  for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < rows; r0 += step, r += step) {
    float h[V][N];
    float s[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        h[v][e] = in[0][v].get(e) + in[1][v].get(e);
        const float t = c.any(v) && c.owns(v, e) ? h[v][e] : 0.0f;
        s[0] = __builtin_fmaf(t, t, s[0]);
      }
    if (r0 + step < rows) load(r + step < last ? r + step : last);
    row_sum<MULTI, 1>(s, tpr, lds, turn);
    // y may be x or block: by now every thread of the row has its values
    const size_t at = (size_t)r * dim;
    if (r < rows)
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (c.any(v)) {
          Raw<T> o;
          o.set_all(h[v]);
          store_raw<T, N, true>(y + at + c.col[v], o);
        }
    const float ry = inv_sqrt(s[0] * inv + eps);
    // The bits of non-negative floats are ordered as they are, infinity and NaN
    // above the finite ones.
    uint32_t top = (__float_as_uint(s[0]) & 0x7FFFFFFFu) >= 0x7F800000u ? 0x7FC00000u : 0u;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        h[v][e] = (h[v][e] * ry) * weight[v][e];
        const uint32_t b = __float_as_uint(h[v][e]) & 0x7FFFFFFFu;
        top = b > top ? b : top;  // a vector past the row repeats one inside it
      }
    top = row_max<MULTI>(top, tpr, lds, turn);
    if (r >= rows) continue;
    const float amax = __uint_as_float(top);
    const bool none = top == 0u || top >= 0x7F800000u;
    const float up = amax < 0x1p-100f ? 0x1p64f : 1.0f;
    const float to_code = none ? 0.0f : 127.0f / (amax * up);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!c.any(v)) continue;
      uint32_t words[N / 4];
#pragma unroll
      for (int k = 0; k < N / 4; ++k) {
        words[k] = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float q = none ? 0.0f : __builtin_rintf((h[v][4 * k + i] * up) * to_code);
          words[k] |= ((uint32_t)(int32_t)q & 0xFFu) << (8 * i);
        }
      }
      int8_t* p = codes + at + c.col[v];
      if constexpr (N == 8)
        __builtin_nontemporal_store(u2{words[0], words[1]}, reinterpret_cast<u2_at1*>(p));
      else
        __builtin_nontemporal_store(words[0], reinterpret_cast<u1_at1*>(p));
    }
    if (lane == 0)
      scales[r] = top >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : amax / 127.0f;
  }
}

template <class T, int V, bool MULTI, bool TAIL>
hipError_t add_norm_shape(const AddNorm& a, const Shape& sh, void* y, int8_t* codes,
                          float* scales, hipStream_t s) {
  const unsigned blocks = grid_of(a.rows, sh, kNormWaves);
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL((k_add_norm_int8<T, V, MULTI, TAIL>), dim3(blocks),
                     dim3((unsigned)sh.threads), 0, s, static_cast<const T*>(a.x),
                     static_cast<const T*>(a.block), a.w, a.rows, (uint32_t)a.dim, sh.tpr, a.eps,
                     static_cast<T*>(y), codes, scales);
  return hipGetLastError();
}

template <class T>
hipError_t add_norm_t(const AddNorm& a, void* y, int8_t* codes, float* scales, hipStream_t s) {
  constexpr int V = sizeof(T) == 4 ? 2 : 1;
  const Shape sh = shape_of<T>(a.dim);
  const bool tail = a.dim % kVec<T> != 0;
  if (sh.multi)
    return tail ? add_norm_shape<T, V, true, true>(a, sh, y, codes, scales, s)
                : add_norm_shape<T, V, true, false>(a, sh, y, codes, scales, s);
  if (sh.vecs == V)
    return tail ? add_norm_shape<T, V, false, true>(a, sh, y, codes, scales, s)
                : add_norm_shape<T, V, false, false>(a, sh, y, codes, scales, s);
  return tail ? add_norm_shape<T, 1, false, true>(a, sh, y, codes, scales, s)
              : add_norm_shape<T, 1, false, false>(a, sh, y, codes, scales, s);
}

}  // namespace

hipError_t launch_add_norm_int8(const AddNorm& a, int32_t dtype, void* y, int8_t* codes,
                                float* scales, hipStream_t s) {
  switch (dtype) {
    case EMB_F32: return add_norm_t<float>(a, y, codes, scales, s);
    case EMB_BF16: return add_norm_t<bf16_t>(a, y, codes, scales, s);
    default: return add_norm_t<f16_t>(a, y, codes, scales, s);
  }
}

}  // namespace embtab
