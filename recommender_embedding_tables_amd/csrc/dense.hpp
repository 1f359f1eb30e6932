// Element types of the dense operators (gradient clip, expert routing, gated
// norm), 16-byte accesses at element alignment, and their launchers.
#pragma once

#include "embtab_internal.hpp"
#include "grid.hpp"

namespace embtab {

// bf16 and fp16 values in memory; arithmetic is always in fp32 or wider.
struct bf16_t {
  uint16_t bits;
};
struct f16_t {
  _Float16 value;
};

typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
// Rows of odd width start at any element: a 16-byte global access needs no
// more than element alignment on gfx950, so no row takes a narrower path for
// its address.
typedef u4 u4_at2 __attribute__((aligned(2)));
typedef u2 u2_at2 __attribute__((aligned(2)));

__device__ inline float to_f32(float x) { return x; }
__device__ inline float to_f32(bf16_t x) { return __uint_as_float((uint32_t)x.bits << 16); }
__device__ inline float to_f32(f16_t x) { return (float)x.value; }

// One rounding to nearest even (NaN stays NaN).
template <class T>
__device__ inline T from_f32(float x);
template <>
__device__ inline float from_f32<float>(float x) {
  return x;
}
template <>
__device__ inline bf16_t from_f32<bf16_t>(float x) {
  return bf16_t{__builtin_bit_cast(uint16_t, (__bf16)x)};
}
template <>
__device__ inline f16_t from_f32<f16_t>(float x) {
  return f16_t{(_Float16)x};
}

// Elements of one 16-byte vector.
template <class T>
constexpr int kVec = 16 / (int)sizeof(T);

// N consecutive elements held as 32-bit words (N * sizeof(T) = 8 or 16 bytes).
template <class T, int N = kVec<T>>
struct Raw {
  static constexpr int kWords = N * (int)sizeof(T) / 4;
  static_assert(kWords == 2 || kWords == 4, "8 or 16 bytes");
  uint32_t w[kWords];

  __device__ inline float get(int i) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[i]);
    } else {
      const uint32_t h = w[i >> 1];
      if constexpr (__is_same(T, bf16_t)) {
        return __uint_as_float((i & 1) ? (h & 0xFFFF0000u) : (h << 16));
      } else {
        return (float)__builtin_bit_cast(_Float16, (uint16_t)((i & 1) ? (h >> 16) : h));
      }
    }
  }
  __device__ inline void set_all(const float* v) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      if constexpr (sizeof(T) == 4) {
        w[k] = __float_as_uint(v[k]);
      } else {
        const uint32_t lo = __builtin_bit_cast(uint16_t, from_f32<T>(v[2 * k]));
        const uint32_t hi = __builtin_bit_cast(uint16_t, from_f32<T>(v[2 * k + 1]));
        w[k] = lo | (hi << 16);
      }
    }
  }
};

template <class T, int N = kVec<T>, bool NT = false>
__device__ inline Raw<T, N> load_raw(const T* p) {
  Raw<T, N> r;
  if constexpr (Raw<T, N>::kWords == 4) {
    const u4_at2* q = reinterpret_cast<const u4_at2*>(p);
    const u4 x = NT ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = x[i];
  } else {
    const u2_at2* q = reinterpret_cast<const u2_at2*>(p);
    const u2 x = NT ? __builtin_nontemporal_load(q) : *q;
    r.w[0] = x[0];
    r.w[1] = x[1];
  }
  return r;
}

template <class T, int N = kVec<T>, bool NT = false>
__device__ inline void store_raw(T* p, const Raw<T, N>& r) {
  if constexpr (Raw<T, N>::kWords == 4) {
    u4_at2* q = reinterpret_cast<u4_at2*>(p);
    const u4 x = {r.w[0], r.w[1], r.w[2], r.w[3]};
    if (NT) __builtin_nontemporal_store(x, q);
    else *q = x;
  } else {
    u2_at2* q = reinterpret_cast<u2_at2*>(p);
    const u2 x = {r.w[0], r.w[1]};
    if (NT) __builtin_nontemporal_store(x, q);
    else *q = x;
  }
}

// Blocks of a kernel of 256 threads a block, which finds its index with
// block_index().
inline dim3 row_grid(int64_t blocks) {
  const Grid g = fold_grid(blocks);
  return dim3(g.x, g.y);
}
__device__ inline uint32_t block_index() { return blockIdx.y * gridDim.x + blockIdx.x; }

inline bool dtype_ok(int32_t t) { return t == EMB_F32 || t == EMB_BF16 || t == EMB_F16; }
inline size_t dtype_size(int32_t t) { return t == EMB_F32 ? 4 : 2; }

// ---------------------------------------------------------------- launchers
// grad_norm.hip
size_t grad_workspace_bytes(const emb_tensor_t* grads, int32_t n);
hipError_t launch_clip_grad_norm(const emb_tensor_t* grads, const emb_tensor_t* out, int32_t n,
                                 const double* extra, int32_t num_extra, float max_norm,
                                 float* norm_out, char* ws, hipStream_t s);

// segment_reduce.hip, on a prepared workspace
hipError_t launch_grad_reduce(const Handle& h, const Plan& p, const uint32_t* keys,
                              const uint32_t* perm, bool mean, const float* grad_out,
                              float* sums, double* sqnorm, char* ws, hipStream_t s);
hipError_t launch_adagrad_rows(const Handle& h, const Plan& p, const uint32_t* keys,
                               const float* sums, const float* scale, float lr, float eps,
                               char* ws, hipStream_t s);

// expert.hip
size_t expert_workspace_bytes(int64_t tokens, int32_t topk, int32_t experts);
hipError_t launch_expert_sort(const int64_t* ids, int64_t tokens, int32_t topk, int32_t experts,
                              int64_t capacity, int32_t* offsets, int32_t* src, int32_t* pos,
                              char* ws, hipStream_t s);
hipError_t launch_expert_dispatch(const void* x, const int32_t* pos, const int32_t* src,
                                  int64_t tokens, int32_t topk, int64_t rows, int32_t dim,
                                  int32_t dtype, void* xs, hipStream_t s);
hipError_t launch_expert_combine(const void* ys, const int32_t* pos, const float* weights,
                                 int64_t tokens, int32_t topk, int64_t rows, int32_t dim,
                                 int32_t dtype, void* y, hipStream_t s);
hipError_t launch_expert_combine_backward(const void* dy, const void* ys, const int32_t* pos,
                                          const int32_t* src, const float* weights,
                                          int64_t tokens, int32_t topk, int64_t rows, int32_t dim,
                                          int32_t dtype, void* dys, float* dweights,
                                          hipStream_t s);

// gated_norm.hip
struct GatedNorm {
  const void *x, *block, *gate;           // gate: null, [rows] or [rows, dim]
  const float *w_post, *scale, *w_pre;    // w_post null: no norm before the gate
  int64_t rows;
  int32_t dim, gate_kind;                 // EMB_GATE_* without the sigmoid bit
  bool sigmoid;
  float eps;
};
size_t gated_norm_workspace_bytes(int64_t rows, int32_t dim);
hipError_t launch_gated_norm_forward(const GatedNorm& a, int32_t dtype, void* y, void* h,
                                     hipStream_t s);
hipError_t launch_gated_norm_backward(const GatedNorm& a, int32_t dtype, const void* dy,
                                      const void* dh, void* dx, void* dblock, void* dgate,
                                      float* dw_post, float* dscale, float* dw_pre, char* ws,
                                      hipStream_t s);

}  // namespace embtab
