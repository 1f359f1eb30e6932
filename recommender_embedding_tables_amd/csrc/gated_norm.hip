// A block's output normalised, gated, scaled and added to the residual, with
// the norm of the sum for the next block, and the gradients, for gfx950.
//
// Per row of D values, every step in fp32:
//   r_o = rsqrt(mean(o^2) + eps),  u = o * r_o * w_post    (u = o without w_post)
//   a = gate or sigmoid(gate), per row or per element       (1 without a gate)
//   y = x + scale * a * u
//   r_y = rsqrt(mean(y^2) + eps),  h = y * r_y * w_pre
// y is rounded once, when it is stored; h is formed from the unrounded y.
//
// Backward, from the stored y and the upstream dy and dh (nothing else is kept
// by the forward), with yhat = y * r_y and ohat = o * r_o:
//   q = dh * w_pre;   t = dy + r_y * (q - yhat * mean(q * yhat))     (= dx)
//   du = scale * a * t
//   dblock = r_o * (p - ohat * mean(p * ohat)),  p = du * w_post     (du without w_post)
//   da = t * scale * u, summed over the row for a row gate;  times a * (1 - a)
//        for a sigmoid gate
//   dw_post = sum_rows du * ohat;  dscale = sum_rows t * a * u;
//   dw_pre = sum_rows dh * yhat
//
// Bound by memory: each stream is read or written once.  A row's vectors live
// in the registers of the threads that share it (lanes of one wave for short
// rows, the whole block for long ones), so the statistics and the results come
// from one read.  The blocks walk over rows and keep the weights of their
// columns, and in the backward pass the columns' sums, in registers.  The sums
// of a block go to the workspace and a second kernel adds them in block order:
// no atomics, the result does not depend on timing.
#include "dense.hpp"

namespace embtab {

namespace {

constexpr int kMaxBlocksForward = 2048;
constexpr int kMaxBlocksBackward = 512;
constexpr int kMaxWaves = 16;

__device__ inline float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// How the rows lie on the threads: tpr threads share a row (8 .. 64 lanes of
// a wave, or, MULTI, the whole block), each holding V vectors of it.
struct Shape {
  int32_t tpr, threads, vecs, multi;
  int32_t rows_per_block() const { return multi ? 1 : threads / tpr; }
};

template <class T>
Shape shape_of(int32_t dim) {
  const int nvec = (dim + kVec<T> - 1) / kVec<T>;
  Shape s{8, 256, 1, 0};
  while (s.tpr < 64 && s.tpr < nvec) s.tpr *= 2;
  if (nvec <= 64) return s;
  if (nvec <= 128) {
    s.vecs = 2;
    return s;
  }
  s.multi = 1;
  s.vecs = nvec <= 1024 ? 1 : 2;
  s.tpr = s.threads = ((nvec + s.vecs - 1) / s.vecs + 63) / 64 * 64;
  return s;
}

// Sums of N values over the threads of a row.  MULTI rows pass through LDS;
// the caller alternates between two buffers, so one barrier per sum suffices.
template <bool MULTI, int N>
__device__ inline void row_sum(float (&v)[N], int tpr, float (*lds)[kMaxWaves]) {
  if (MULTI) {
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) v[k] += __shfl_xor(v[k], o, 64);
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63u) == 0u)
#pragma unroll
      for (int k = 0; k < N; ++k) lds[k][threadIdx.x >> 6] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float t = 0.0f;
      for (int w = 0; w < waves; ++w) t += lds[k][w];
      v[k] = t;
    }
  } else {
    for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor(v[k], o, 64);
  }
}

// The columns of one thread: vector v starts at col[v]; elements before
// skip[v] belong to the vector before it (the last vector of a row is moved
// back to end with the row) or to none (skip = the vector's width).
template <class T, int V>
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
  __device__ bool owns(int v, int e) const { return (uint32_t)e >= skip[v]; }
};

template <class T, int V>
__device__ inline void load_weights(const float* w, const Columns<T, V>& c,
                                    float (&out)[V][kVec<T>]) {
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e) out[v][e] = w ? w[c.col[v] + e] : 1.0f;
}

template <class T, int V, bool MULTI>
__global__ __launch_bounds__(MULTI ? 1024 : 256) void k_gated_norm_forward(
    const T* x, const T* block, const T* gate, const float* __restrict__ w_post,
    const float* __restrict__ scale, const float* __restrict__ w_pre, int64_t rows, uint32_t dim,
    int32_t tpr, int32_t gate_kind, bool sig, float eps, T* y, T* h) {
  constexpr int N = kVec<T>;
  __shared__ float lds[2][1][kMaxWaves];
  const uint32_t lane = MULTI ? threadIdx.x : threadIdx.x % (uint32_t)tpr;
  const uint32_t rpb = MULTI ? 1u : blockDim.x / (uint32_t)tpr;
  const Columns<T, V> c(lane, (uint32_t)tpr, dim);
  const float inv = 1.0f / (float)dim;
  float wpost[V][N], sc[V][N], wpre[V][N];
  load_weights<T, V>(w_post, c, wpost);
  load_weights<T, V>(scale, c, sc);
  load_weights<T, V>(w_pre, c, wpre);
  const int64_t step = (int64_t)gridDim.x * rpb;
  // every thread of a block takes the same number of rounds (barriers)
  for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < rows; r0 += step) {
    const int64_t r = MULTI ? r0 : r0 + threadIdx.x / (uint32_t)tpr;
    const bool live = r < rows;
    const size_t at = (size_t)(live ? r : rows - 1) * dim;
    Raw<T> rx[V], ro[V], rg[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      ro[v] = load_raw<T, N, true>(block + at + c.col[v]);
      rx[v] = load_raw<T, N, true>(x + at + c.col[v]);
      if (gate_kind == EMB_GATE_ELEMENT) rg[v] = load_raw<T, N, true>(gate + at + c.col[v]);
    }
    float a_row = 1.0f;
    if (gate_kind == EMB_GATE_ROW) {
      a_row = to_f32(gate[live ? r : rows - 1]);
      if (sig) a_row = sigmoid(a_row);
    }
    float ro_s = 1.0f;
    if (w_post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float o = c.owns(v, e) ? ro[v].get(e) : 0.0f;
          s[0] = __builtin_fmaf(o, o, s[0]);
        }
      row_sum<MULTI, 1>(s, tpr, lds[0]);
      ro_s = 1.0f / sqrtf(s[0] * inv + eps);
    }
    float yv[V][N];
    float s[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        float a = a_row;
        if (gate_kind == EMB_GATE_ELEMENT) a = sig ? sigmoid(rg[v].get(e)) : rg[v].get(e);
        const float u = (ro[v].get(e) * ro_s) * wpost[v][e];
        yv[v][e] = __builtin_fmaf(sc[v][e] * a, u, rx[v].get(e));
        const float t = c.owns(v, e) ? yv[v][e] : 0.0f;
        s[0] = __builtin_fmaf(t, t, s[0]);
      }
    row_sum<MULTI, 1>(s, tpr, lds[1]);
    const float ry = 1.0f / sqrtf(s[0] * inv + eps);
    // Without w_post a MULTI round has one barrier: the next round must not
    // write lds[1] while a slower wave still reads it.
    if (MULTI && !w_post) __syncthreads();
    if (!live) continue;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!c.any(v)) continue;
      Raw<T> o;
      o.set_all(yv[v]);
      store_raw<T, N, true>(y + at + c.col[v], o);
      float hv[N];
#pragma unroll
      for (int e = 0; e < N; ++e) hv[e] = (yv[v][e] * ry) * wpre[v][e];
      o.set_all(hv);
      store_raw<T, N, true>(h + at + c.col[v], o);
    }
  }
}

template <class T, int V, bool MULTI>
__global__ __launch_bounds__(MULTI ? 1024 : 256) void k_gated_norm_backward(
    const T* y, const T* block, const T* gate, const float* __restrict__ w_post,
    const float* __restrict__ scale, const float* __restrict__ w_pre, const T* dy, const T* dh,
    int64_t rows, uint32_t dim, int32_t tpr, int32_t gate_kind, bool sig, float eps, T* dx,
    T* dblock, T* dgate, float* __restrict__ parts) {
  constexpr int N = kVec<T>;
  __shared__ float lds[2][3][kMaxWaves];
  const uint32_t lane = MULTI ? threadIdx.x : threadIdx.x % (uint32_t)tpr;
  const uint32_t rpb = MULTI ? 1u : blockDim.x / (uint32_t)tpr;
  const Columns<T, V> c(lane, (uint32_t)tpr, dim);
  const float inv = 1.0f / (float)dim;
  float wpost[V][N], sc[V][N], wpre[V][N];
  load_weights<T, V>(w_post, c, wpost);
  load_weights<T, V>(scale, c, sc);
  load_weights<T, V>(w_pre, c, wpre);
  float s_post[V][N], s_scale[V][N], s_pre[V][N];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < N; ++e) s_post[v][e] = s_scale[v][e] = s_pre[v][e] = 0.0f;
  const int64_t step = (int64_t)gridDim.x * rpb;
  for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < rows; r0 += step) {
    const int64_t r = MULTI ? r0 : r0 + threadIdx.x / (uint32_t)tpr;
    const bool live = r < rows;
    const size_t at = (size_t)(live ? r : rows - 1) * dim;
    Raw<T> ry_[V], ro[V], rg[V], rdy[V], rdh[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      ry_[v] = load_raw<T, N, true>(y + at + c.col[v]);
      ro[v] = load_raw<T, N, true>(block + at + c.col[v]);
      rdh[v] = load_raw<T, N, true>(dh + at + c.col[v]);
      rdy[v] = load_raw<T, N, true>(dy + at + c.col[v]);
      if (gate_kind == EMB_GATE_ELEMENT) rg[v] = load_raw<T, N, true>(gate + at + c.col[v]);
    }
    float a_row = 1.0f;
    if (gate_kind == EMB_GATE_ROW) {
      a_row = to_f32(gate[live ? r : rows - 1]);
      if (sig) a_row = sigmoid(a_row);
    }
    // sums of y^2, q * y and o^2
    float s1[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const bool own = c.owns(v, e);
        const float yy = own ? ry_[v].get(e) : 0.0f, o = own ? ro[v].get(e) : 0.0f;
        s1[0] = __builtin_fmaf(yy, yy, s1[0]);
        s1[1] = __builtin_fmaf(rdh[v].get(e) * wpre[v][e], yy, s1[1]);
        s1[2] = __builtin_fmaf(o, o, s1[2]);
      }
    row_sum<MULTI, 3>(s1, tpr, lds[0]);
    const float ry = 1.0f / sqrtf(s1[0] * inv + eps);
    const float mq = (s1[1] * ry) * inv;  // mean(q * yhat)
    const float ro_s = w_post ? 1.0f / sqrtf(s1[2] * inv + eps) : 1.0f;
    // t, and the sums of p * ohat and t * scale * u over the row
    float s2[2] = {0.0f, 0.0f};
    float tv[V][N];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const bool own = live && c.owns(v, e);
        const float yhat = ry_[v].get(e) * ry, dhv = rdh[v].get(e);
        const float t = __builtin_fmaf(ry, dhv * wpre[v][e] - yhat * mq, rdy[v].get(e));
        float a = a_row;
        if (gate_kind == EMB_GATE_ELEMENT) a = sig ? sigmoid(rg[v].get(e)) : rg[v].get(e);
        const float ohat = ro[v].get(e) * ro_s, u = ohat * wpost[v][e];
        const float ts = t * sc[v][e];
        tv[v][e] = t;
        if (own) {
          s2[0] = __builtin_fmaf(ts * a, u, s2[0]);
          s2[1] = __builtin_fmaf(ts, u, s2[1]);
          s_post[v][e] = __builtin_fmaf(ts * a, ohat, s_post[v][e]);
          s_scale[v][e] = __builtin_fmaf(t * a, u, s_scale[v][e]);
          s_pre[v][e] = __builtin_fmaf(dhv, yhat, s_pre[v][e]);
        }
      }
    row_sum<MULTI, 2>(s2, tpr, lds[1]);
    const float mp = s2[0] * inv;  // mean(p * ohat)
    if (!live) continue;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!c.any(v)) continue;
      float o1[N], o2[N], o3[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float t = tv[v][e];
        float a = a_row;
        if (gate_kind == EMB_GATE_ELEMENT) a = sig ? sigmoid(rg[v].get(e)) : rg[v].get(e);
        const float ohat = ro[v].get(e) * ro_s, u = ohat * wpost[v][e];
        const float ts = t * sc[v][e];
        const float p = (ts * a) * wpost[v][e];
        o1[e] = t;
        o2[e] = w_post ? ro_s * (p - ohat * mp) : p;
        o3[e] = sig ? (ts * u) * (a * (1.0f - a)) : ts * u;
      }
      Raw<T> o;
      o.set_all(o1);
      store_raw<T, N, true>(dx + at + c.col[v], o);
      o.set_all(o2);
      store_raw<T, N, true>(dblock + at + c.col[v], o);
      if (gate_kind == EMB_GATE_ELEMENT) {
        o.set_all(o3);
        store_raw<T, N, true>(dgate + at + c.col[v], o);
      }
    }
    if (gate_kind == EMB_GATE_ROW && lane == 0)
      dgate[r] = from_f32<T>(sig ? s2[1] * (a_row * (1.0f - a_row)) : s2[1]);
  }
  // the block's column sums: [3][dim] of this block
  float* out = parts + (size_t)blockIdx.x * 3u * dim;
  if (MULTI) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (c.owns(v, e)) {
          out[c.col[v] + e] = s_post[v][e];
          out[dim + c.col[v] + e] = s_scale[v][e];
          out[2u * dim + c.col[v] + e] = s_pre[v][e];
        }
  } else {
    // the block's row groups hold sums of the same columns: added through LDS
    __shared__ float acc[256 * V * N];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      float(&s)[V][N] = k == 0 ? s_post : k == 1 ? s_scale : s_pre;
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < N; ++e)  // [group][v][e][lane]
          acc[(((threadIdx.x / (uint32_t)tpr) * V + v) * N + e) * (uint32_t)tpr + lane] = s[v][e];
      __syncthreads();
      if (threadIdx.x < (uint32_t)tpr) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (c.owns(v, e)) {
              float t = 0.0f;
              for (uint32_t g = 0; g < rpb; ++g)
                t += acc[((g * V + v) * N + e) * (uint32_t)tpr + lane];
              out[(uint32_t)k * dim + c.col[v] + e] = t;
            }
      }
    }
  }
}

// dst[c] = sum over the blocks of parts[block][c], in block order per group of
// blocks and then over the groups; 64 columns per block, 16 groups.
constexpr int kSumGroups = 16;
__global__ __launch_bounds__(64 * kSumGroups) void k_gated_norm_column_sums(
    const float* __restrict__ parts, uint32_t blocks, uint32_t dim, float* __restrict__ dw_post,
    float* __restrict__ dscale, float* __restrict__ dw_pre) {
  __shared__ float lds[kSumGroups][64];
  const uint32_t col = blockIdx.x * 64u + (threadIdx.x & 63u), g = threadIdx.x >> 6;
  const uint32_t width = 3u * dim;
  float s = 0.0f;
  if (col < width)
    for (uint32_t b = g; b < blocks; b += kSumGroups) s += parts[(size_t)b * width + col];
  lds[g][threadIdx.x & 63u] = s;
  __syncthreads();
  if (g != 0 || col >= width) return;
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < kSumGroups; ++i) t += lds[i][threadIdx.x];
  const uint32_t k = col / dim, j = col - k * dim;
  float* dst = k == 0 ? dw_post : k == 1 ? dscale : dw_pre;
  if (dst) dst[j] = t;
}

unsigned grid_of(int64_t rows, int32_t rpb, int most) {
  const int64_t g = (rows + rpb - 1) / rpb;
  return (unsigned)(g < most ? g : most);
}

template <class T>
hipError_t forward_t(const GatedNorm& a, void* y, void* h, hipStream_t s) {
  const Shape sh = shape_of<T>(a.dim);
  const dim3 grid(grid_of(a.rows, sh.rows_per_block(), kMaxBlocksForward)),
      threads((unsigned)sh.threads);
#define EMBTAB_GN(V_, M_)                                                                       \
  hipLaunchKernelGGL((k_gated_norm_forward<T, V_, M_>), grid, threads, 0, s,                    \
                     static_cast<const T*>(a.x), static_cast<const T*>(a.block),                \
                     static_cast<const T*>(a.gate), a.w_post, a.scale, a.w_pre, a.rows,         \
                     (uint32_t)a.dim, sh.tpr, a.gate_kind, a.sigmoid, a.eps, static_cast<T*>(y), \
                     static_cast<T*>(h))
  if (sh.multi) {
    if (sh.vecs == 1) EMBTAB_GN(1, true);
    else EMBTAB_GN(2, true);
  } else {
    if (sh.vecs == 1) EMBTAB_GN(1, false);
    else EMBTAB_GN(2, false);
  }
#undef EMBTAB_GN
  return hipGetLastError();
}

template <class T>
hipError_t backward_t(const GatedNorm& a, const void* dy, const void* dh, void* dx, void* dblock,
                      void* dgate, float* dw_post, float* dscale, float* dw_pre, float* parts,
                      hipStream_t s) {
  const Shape sh = shape_of<T>(a.dim);
  const unsigned blocks = grid_of(a.rows, sh.rows_per_block(), kMaxBlocksBackward);
  const dim3 grid(blocks), threads((unsigned)sh.threads);
#define EMBTAB_GN(V_, M_)                                                                        \
  hipLaunchKernelGGL((k_gated_norm_backward<T, V_, M_>), grid, threads, 0, s,                    \
                     static_cast<const T*>(a.x), static_cast<const T*>(a.block),                 \
                     static_cast<const T*>(a.gate), a.w_post, a.scale, a.w_pre,                  \
                     static_cast<const T*>(dy), static_cast<const T*>(dh), a.rows,               \
                     (uint32_t)a.dim, sh.tpr, a.gate_kind, a.sigmoid, a.eps,                     \
                     static_cast<T*>(dx), static_cast<T*>(dblock), static_cast<T*>(dgate), parts)
  if (blocks) {
    if (sh.multi) {
      if (sh.vecs == 1) EMBTAB_GN(1, true);
      else EMBTAB_GN(2, true);
    } else {
      if (sh.vecs == 1) EMBTAB_GN(1, false);
      else EMBTAB_GN(2, false);
    }
  }
#undef EMBTAB_GN
  const uint32_t width = 3u * (uint32_t)a.dim;
  hipLaunchKernelGGL(k_gated_norm_column_sums, dim3((width + 63u) / 64u), dim3(64 * kSumGroups),
                     0, s, parts, blocks, (uint32_t)a.dim, dw_post, dscale, dw_pre);
  return hipGetLastError();
}

}  // namespace

// One [3][dim] fp32 part per block of the backward kernel.
size_t gated_norm_workspace_bytes(int64_t rows, int32_t dim) {
  const int64_t blocks = rows < kMaxBlocksBackward ? rows : kMaxBlocksBackward;
  return (sizeof(float) * 3u * (size_t)dim * (size_t)blocks + 256) & ~(size_t)255;
}

hipError_t launch_gated_norm_forward(const GatedNorm& a, int32_t dtype, void* y, void* h,
                                     hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  switch (dtype) {
    case EMB_F32: return forward_t<float>(a, y, h, s);
    case EMB_BF16: return forward_t<bf16_t>(a, y, h, s);
    default: return forward_t<f16_t>(a, y, h, s);
  }
}

hipError_t launch_gated_norm_backward(const GatedNorm& a, int32_t dtype, const void* dy,
                                      const void* dh, void* dx, void* dblock, void* dgate,
                                      float* dw_post, float* dscale, float* dw_pre, char* ws,
                                      hipStream_t s) {
  float* parts = reinterpret_cast<float*>(ws);
#define EMBTAB_GB(T_) \
  backward_t<T_>(a, dy, dh, dx, dblock, dgate, dw_post, dscale, dw_pre, parts, s)
  switch (dtype) {
    case EMB_F32: return EMBTAB_GB(float);
    case EMB_BF16: return EMBTAB_GB(bf16_t);
    default: return EMBTAB_GB(f16_t);
  }
#undef EMBTAB_GB
}

}  // namespace embtab
