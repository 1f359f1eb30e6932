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
// Bound by memory: each stream is read or written once (by the counters too; a
// one-shot device copy reaches 6.5 TB/s here).  A row's vectors live in the registers of the threads
// that share it (lanes of one wave for short rows, the whole block for long
// ones), so the statistics and the results come from one read, and the loads
// of a thread's next row are issued with the stores of this one.  Issuing them
// a row ahead, into a second set of registers, left fewer waves and gained
// nothing (same rows: 214 us against 210 on the same buffers).  The blocks walk over rows
// and keep the weights of their columns, and in the backward pass the columns'
// sums.  The sums of a block go to the workspace and a second kernel adds them
// in block order: no atomics, the result does not depend on timing.
//
// Element-wise sigmoid gate, norm before the gate:
//   forward   32768 x 3328 bf16   182 us, 6.0 TB/s (210 us where all five
//             streams begin at the same offset of a large power of two)
//   backward  16384 x 3328 bf16   167 to 178 us, 4.9 to 5.2 TB/s by the streams'
//             places, 6 us of it the column sums
// What moved them there: sums by lane permutations in place of LDS shuffles,
// the hardware's exponential and reciprocal for 16-bit gates, weights in LDS.
#include "row_tiles.hpp"

namespace embtab {

namespace {

typedef float fv4 __attribute__((ext_vector_type(4)));

// Waves a launch puts on each of the 256 CUs, in whole blocks and at least one:
// few blocks that walk over many rows each, so that the weights and column sums
// are set up once.  Measured on 65536 x 512 bf16 rows (blocks of 4 waves):
// forward 61 us with 3 blocks, 68 with 7; backward, whose blocks leave 12 * dim
// bytes of sums each, 112 us with 2, 122 with 4.  A row that takes a whole block
// wants two blocks to hide its barriers, and has them up to 7 waves in the
// forward, 8 in the backward; with one, 109 million bf16 values take 240 us
// forward in rows of 4096 and 217 in rows of 6656, 183 with two in rows of 3584
// (fp32: 202, 200 and 202).
constexpr int kForwardWaves = 14, kBackwardWaves = 8, kBackwardBlockRowWaves = 16;

// e^-v.  For 16-bit data one product and the hardware exponential, within
// (1.5 |v| + 2) * 2^-24 and so far below the data's own rounding up to |v| = 87,
// where it is 0 or infinite; fp32 takes the library's exponential.
template <class T>
__device__ inline float exp_neg(float v) {
  if constexpr (sizeof(T) == 4) return expf(-v);
  return __builtin_amdgcn_exp2f(v * -1.44269504088896340736f);
}

// a (1 - a) for a = 1 / (1 + t), t = e^-v.  1 - a cancels where a is near 1 (in
// fp32 one percent is lost at v = 12, all of it at 17), so an open gate takes it
// as t a.
__device__ inline float sigmoid_slope(float v, float t, float a) {
  return a * (v > 0.0f ? t * a : 1.0f - a);
}

// A gate's factor: a = v, or 1 / (1 + e^-v) (for 16-bit data with the hardware
// reciprocal; infinite gates give 0 and 1, a NaN stays one), and da/dv.
struct Factor {
  float a, slope;
};
template <class T>
__device__ inline Factor gate_factor(float v, bool sig) {
  if (!sig) return {v, 1.0f};
  const float t = exp_neg<T>(v);
  float a;
  if constexpr (sizeof(T) == 4) a = 1.0f / (1.0f + t);
  else a = __builtin_amdgcn_rcpf(1.0f + t);
  return {a, sigmoid_slope(v, t, a)};
}

// A thread's share of the fp32 weight vectors, 1 where the vector is null.  A
// wave's rows keep it in registers; a block's rows (MULTI) in LDS, [value / 4]
// [thread] in 16-byte steps without bank conflicts, each thread its own and so
// without barriers: 24 registers less, without which the backward pass spills.
template <class T, int V, bool MULTI>
struct Weights {
  float w[V][kVec<T>];
  template <bool TAIL>
  __device__ inline void load(const float* p, const Columns<T, V, TAIL>& c) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < kVec<T>; e += 4) {
        const Raw<float> r = p ? load_raw(p + c.col[v] + e) : Raw<float>{};
#pragma unroll
        for (int i = 0; i < 4; ++i) w[v][e + i] = p ? r.get(i) : 1.0f;
      }
  }
  __device__ inline fv4 get(int v, int e) const {  // values e .. e + 3 of vector v
    return fv4{w[v][e], w[v][e + 1], w[v][e + 2], w[v][e + 3]};
  }
};

template <class T, int V>
struct Weights<T, V, true> {
  fv4* mine;
  template <bool TAIL>
  __device__ inline void load(const float* p, const Columns<T, V, TAIL>& c) {
    Weights<T, V, false> r;
    r.load(p, c);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < kVec<T>; e += 4)
        mine[(v * kVec<T> + e) / 4 * blockDim.x] =
            fv4{r.w[v][e], r.w[v][e + 1], r.w[v][e + 2], r.w[v][e + 3]};
  }
  __device__ inline fv4 get(int v, int e) const {
    return mine[(v * kVec<T> + e) / 4 * blockDim.x];
  }
};

template <class T, int V, bool MULTI>
__device__ inline void place_weights(Weights<T, V, MULTI> (&w)[3]) {
  if constexpr (MULTI) {
    extern __shared__ fv4 weights_lds[];
#pragma unroll
    for (int k = 0; k < 3; ++k)
      w[k].mine = weights_lds + k * (V * kVec<T> / 4) * blockDim.x + threadIdx.x;
  }
}

// One row's vectors of S streams, and its gate value for a row gate.
template <class T, int V, int S>
struct RowData {
  Raw<T> in[S][V], gate[V];
  float row_gate;

  template <bool TAIL>
  __device__ inline void load(const T* const (&p)[S], const T* g, int32_t gate_kind, int64_t r,
                              uint32_t dim, const Columns<T, V, TAIL>& c) {
    const size_t at = (size_t)r * dim;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int s = 0; s < S; ++s) in[s][v] = load_raw<T, kVec<T>, true>(p[s] + at + c.col[v]);
      if (gate_kind == EMB_GATE_ELEMENT)
        gate[v] = load_raw<T, kVec<T>, true>(g + at + c.col[v]);
    }
    row_gate = gate_kind == EMB_GATE_ROW ? to_f32(g[r]) : 1.0f;
  }

  // The gate's factors and slopes (those of a row gate in every place).
  __device__ inline void factors(int32_t gate_kind, bool sig, float (&a)[V][kVec<T>],
                                 float (&slope)[V][kVec<T>]) const {
    const Factor row = gate_factor<T>(row_gate, sig && gate_kind == EMB_GATE_ROW);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < kVec<T>; ++e) {
        const Factor f =
            gate_kind == EMB_GATE_ELEMENT ? gate_factor<T>(gate[v].get(e), sig) : row;
        a[v][e] = f.a;
        slope[v][e] = f.slope;
      }
  }
};

enum { kPost = 0, kScale = 1, kPre = 2 };  // the weight vectors

template <class T, int V, bool MULTI, bool TAIL>
__global__ __launch_bounds__(MULTI ? 1024 : 256) void k_gated_norm_forward(
    const T* x, const T* block, const T* gate, const float* __restrict__ w_post,
    const float* __restrict__ scale, const float* __restrict__ w_pre, int64_t rows, uint32_t dim,
    int32_t tpr, int32_t gate_kind, bool sig, float eps, T* y, T* h) {
  constexpr int N = kVec<T>;
  __shared__ SumBuffers lds;
  uint32_t turn = 0;
  const uint32_t lane = MULTI ? threadIdx.x : threadIdx.x % (uint32_t)tpr;
  const uint32_t rpb = MULTI ? 1u : blockDim.x / (uint32_t)tpr;
  const uint32_t mine = MULTI ? 0u : threadIdx.x / (uint32_t)tpr;
  const Columns<T, V, TAIL> c(lane, (uint32_t)tpr, dim);
  const float inv = 1.0f / (float)dim;
  const T* const in[2] = {x, block};
  const int64_t step = (int64_t)gridDim.x * rpb, last = rows - 1;
  RowData<T, V, 2> cur;
  int64_t r = (int64_t)blockIdx.x * rpb + mine;
  cur.load(in, gate, gate_kind, r < last ? r : last, dim, c);
  Weights<T, V, MULTI> w[3];
  place_weights<T, V, MULTI>(w);
  w[kPost].load(w_post, c);
  w[kScale].load(scale, c);
  w[kPre].load(w_pre, c);
  clear_sums<MULTI>(lds);
  // every thread of a block takes the same number of rounds (barriers)
  for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < rows; r0 += step, r += step) {
    float a[V][N], slope[V][N];
    cur.factors(gate_kind, sig, a, slope);
    float ro_s = 1.0f;
    if (w_post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (c.any(v))
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const float o = c.owns(v, e) ? cur.in[1][v].get(e) : 0.0f;
            s[0] = __builtin_fmaf(o, o, s[0]);
          }
      row_sum<MULTI, 1>(s, tpr, lds, turn);
      ro_s = inv_sqrt(s[0] * inv + eps);
    }
    float yv[V][N];
    float s[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (c.any(v))
#pragma unroll
        for (int e0 = 0; e0 < N; e0 += 4) {
          const fv4 wpost = w[kPost].get(v, e0), sc = w[kScale].get(v, e0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = e0 + i;
            const float u = (cur.in[1][v].get(e) * ro_s) * wpost[i];
            yv[v][e] = __builtin_fmaf(sc[i] * a[v][e], u, cur.in[0][v].get(e));
            const float t = c.owns(v, e) ? yv[v][e] : 0.0f;
            s[0] = __builtin_fmaf(t, t, s[0]);
          }
        }
    row_sum<MULTI, 1>(s, tpr, lds, turn);
    const float ry = inv_sqrt(s[0] * inv + eps);
    if (r < rows) {
      const size_t at = (size_t)r * dim;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!c.any(v)) continue;
        Raw<T> o;
        o.set_all(yv[v]);
        store_raw<T, N, true>(y + at + c.col[v], o);
        float hv[N];
#pragma unroll
        for (int e0 = 0; e0 < N; e0 += 4) {
          const fv4 wpre = w[kPre].get(v, e0);
#pragma unroll
          for (int i = 0; i < 4; ++i) hv[e0 + i] = (yv[v][e0 + i] * ry) * wpre[i];
        }
        o.set_all(hv);
        store_raw<T, N, true>(h + at + c.col[v], o);
      }
    }
    if (r0 + step < rows)
      cur.load(in, gate, gate_kind, r + step < last ? r + step : last, dim, c);
  }
}

template <class T, int V, bool MULTI, bool TAIL>
__global__ __launch_bounds__(MULTI ? 1024 : 256) void k_gated_norm_backward(
    const T* y, const T* block, const T* gate, const float* __restrict__ w_post,
    const float* __restrict__ scale, const float* __restrict__ w_pre, const T* dy, const T* dh,
    int64_t rows, uint32_t dim, int32_t tpr, int32_t gate_kind, bool sig, float eps, T* dx,
    T* dblock, T* dgate, float* __restrict__ parts) {
  constexpr int N = kVec<T>;
  enum { Y = 0, O = 1, DH = 2, DY = 3 };
  // The slopes of an element gate stay in registers from the factors on; the
  // fp32 blocks of up to 1024 threads have none left (41 spilled, 8000 columns
  // 235 us against 220) and form them again where they are used.
  constexpr bool kHeld = !(MULTI && sizeof(T) == 4);
  __shared__ SumBuffers lds;
  uint32_t turn = 0;
  const uint32_t lane = MULTI ? threadIdx.x : threadIdx.x % (uint32_t)tpr;
  const uint32_t rpb = MULTI ? 1u : blockDim.x / (uint32_t)tpr;
  const uint32_t mine = MULTI ? 0u : threadIdx.x / (uint32_t)tpr;
  const Columns<T, V, TAIL> c(lane, (uint32_t)tpr, dim);
  const float inv = 1.0f / (float)dim;
  const T* const in[4] = {y, block, dh, dy};
  const int64_t step = (int64_t)gridDim.x * rpb, last = rows - 1;
  RowData<T, V, 4> cur;
  int64_t r = (int64_t)blockIdx.x * rpb + mine;
  cur.load(in, gate, gate_kind, r < last ? r : last, dim, c);
  Weights<T, V, MULTI> w[3];
  place_weights<T, V, MULTI>(w);
  w[kPost].load(w_post, c);
  w[kScale].load(scale, c);
  w[kPre].load(w_pre, c);
  float s_post[V][N], s_scale[V][N], s_pre[V][N];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < N; ++e) s_post[v][e] = s_scale[v][e] = s_pre[v][e] = 0.0f;
  clear_sums<MULTI>(lds);
  for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < rows; r0 += step, r += step) {
    const bool live = r < rows;
    float a[V][N], slope[V][N];
    cur.factors(gate_kind, sig, a, slope);
    // sums of y^2, q * y and o^2
    float s1[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (c.any(v))
#pragma unroll
        for (int e0 = 0; e0 < N; e0 += 4) {
          const fv4 wpre = w[kPre].get(v, e0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = e0 + i;
            const bool own = c.owns(v, e);
            const float yy = cur.in[Y][v].get(e), o = cur.in[O][v].get(e);
            const float q = cur.in[DH][v].get(e) * wpre[i];
            s1[0] = own ? __builtin_fmaf(yy, yy, s1[0]) : s1[0];
            s1[1] = own ? __builtin_fmaf(q, yy, s1[1]) : s1[1];
            s1[2] = own ? __builtin_fmaf(o, o, s1[2]) : s1[2];
          }
        }
    row_sum<MULTI, 3>(s1, tpr, lds, turn);
    const float ry = inv_sqrt(s1[0] * inv + eps);
    const float mq = (s1[1] * ry) * inv;  // mean(q * yhat)
    const float ro_s = w_post ? inv_sqrt(s1[2] * inv + eps) : 1.0f;
    // t, and the sums of p * ohat and t * scale * u over the row
    float s2[2] = {0.0f, 0.0f};
    float tv[V][N];
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (c.any(v) && live)
#pragma unroll
        for (int e0 = 0; e0 < N; e0 += 4) {
          const fv4 wpost = w[kPost].get(v, e0), sc = w[kScale].get(v, e0),
                    wpre = w[kPre].get(v, e0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = e0 + i;
            const float yhat = cur.in[Y][v].get(e) * ry, dhv = cur.in[DH][v].get(e);
            const float t =
                __builtin_fmaf(ry, dhv * wpre[i] - yhat * mq, cur.in[DY][v].get(e));
            const float ohat = cur.in[O][v].get(e) * ro_s, u = ohat * wpost[i];
            const float ts = t * sc[i];
            tv[v][e] = t;
            if (c.owns(v, e)) {
              s2[0] = __builtin_fmaf(ts * a[v][e], u, s2[0]);
              s2[1] = __builtin_fmaf(ts, u, s2[1]);
              s_post[v][e] = __builtin_fmaf(ts * a[v][e], ohat, s_post[v][e]);
              s_scale[v][e] = __builtin_fmaf(t * a[v][e], u, s_scale[v][e]);
              s_pre[v][e] = __builtin_fmaf(dhv, yhat, s_pre[v][e]);
            }
          }
        }
    row_sum<MULTI, 2>(s2, tpr, lds, turn);
    const float mp = s2[0] * inv;  // mean(p * ohat)
    if (live) {
      const size_t at = (size_t)r * dim;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!c.any(v)) continue;
        Raw<T> o;
        o.set_all(tv[v]);
        store_raw<T, N, true>(dx + at + c.col[v], o);
        float ov[N], gv[N];
#pragma unroll
        for (int e0 = 0; e0 < N; e0 += 4) {
          const fv4 wpost = w[kPost].get(v, e0), sc = w[kScale].get(v, e0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = e0 + i;
            const float ohat = cur.in[O][v].get(e) * ro_s, ts = tv[v][e] * sc[i];
            const float p = (ts * a[v][e]) * wpost[i], da = ts * (ohat * wpost[i]);
            ov[e] = w_post ? ro_s * (p - ohat * mp) : p;
            gv[e] = kHeld ? da * slope[v][e] : da;
          }
        }
        o.set_all(ov);
        store_raw<T, N, true>(dblock + at + c.col[v], o);
        if (gate_kind == EMB_GATE_ELEMENT) {
          if (!kHeld && sig)
#pragma unroll
            for (int e = 0; e < N; ++e) {
              const float g = cur.gate[v].get(e);
              gv[e] *= sigmoid_slope(g, exp_neg<T>(g), a[v][e]);
            }
          o.set_all(gv);
          store_raw<T, N, true>(dgate + at + c.col[v], o);
        }
      }
      if (gate_kind == EMB_GATE_ROW && lane == 0)
        dgate[r] = from_f32<T>(s2[1] * gate_factor<T>(cur.row_gate, sig).slope);
    }
    if (r0 + step < rows)
      cur.load(in, gate, gate_kind, r + step < last ? r + step : last, dim, c);
  }
  // the block's column sums: [3][dim] of this block
  float* out = parts + (size_t)blockIdx.x * 3u * dim;
  if (MULTI) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (c.any(v))
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (c.owns(v, e)) {
            out[c.col[v] + e] = s_post[v][e];
            out[dim + c.col[v] + e] = s_scale[v][e];
            out[2u * dim + c.col[v] + e] = s_pre[v][e];
          }
  } else {
    // the block's row groups hold sums of the same columns: added through LDS,
    // in the order of the groups
    __shared__ float acc[3][V * N][256];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        acc[0][v * N + e][threadIdx.x] = s_post[v][e];
        acc[1][v * N + e][threadIdx.x] = s_scale[v][e];
        acc[2][v * N + e][threadIdx.x] = s_pre[v][e];
      }
    __syncthreads();
    // one group of threads per sum: 256 / tpr groups take the 3 * V * N in turn
    for (uint32_t k = mine; k < 3u * V * N; k += rpb) {
      const uint32_t which = k / (V * N), ve = k % (V * N), v = ve / N, e = ve % N;
      const uint32_t at = (lane + v * (uint32_t)tpr) * N;
      if (at >= dim) continue;
      const uint32_t col = at + N <= dim ? at : dim - N;
      if (col + e < at) continue;
      float t = 0.0f;
      for (uint32_t g = 0; g < rpb; ++g) t += acc[which][ve][g * (uint32_t)tpr + lane];
      out[which * dim + col + e] = t;
    }
  }
}

// dst[c] = sum over the blocks of parts[block][c]: 32 columns per block, 32
// groups of threads that take every 32nd part, eight loads in flight each, and
// the groups in order.
constexpr int kSumCols = 32, kSumGroups = 32, kSumAhead = 8;
__global__ __launch_bounds__(kSumCols* kSumGroups) void k_gated_norm_column_sums(
    const float* __restrict__ parts, uint32_t blocks, uint32_t dim, float* __restrict__ dw_post,
    float* __restrict__ dscale, float* __restrict__ dw_pre) {
  __shared__ float lds[kSumGroups][kSumCols];
  const uint32_t lane = threadIdx.x % kSumCols, g = threadIdx.x / kSumCols;
  const uint32_t col = blockIdx.x * kSumCols + lane, width = 3u * dim;
  float s = 0.0f;
  if (col < width)
    for (uint32_t b = g; b < blocks; b += kSumGroups * kSumAhead) {
      float v[kSumAhead];
#pragma unroll
      for (int i = 0; i < kSumAhead; ++i) {
        const uint32_t at = b + i * kSumGroups;
        v[i] = at < blocks ? parts[(size_t)at * width + col] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kSumAhead; ++i) s += v[i];
    }
  lds[g][lane] = s;
  __syncthreads();
  if (g != 0 || col >= width) return;
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < kSumGroups; ++i) t += lds[i][lane];
  const uint32_t k = col / dim, j = col - k * dim;
  float* dst = k == 0 ? dw_post : k == 1 ? dscale : dw_pre;
  if (dst) dst[j] = t;
}

int backward_waves(const Shape& s) {
  return s.multi ? kBackwardBlockRowWaves : kBackwardWaves;
}

// Launch of KERNEL on a shape; a block's rows keep their weights in dynamic
// LDS, which passes the default limit of 64 KB beyond 682 threads.
template <class T, class Kernel, class... Args>
hipError_t launch_rows(Kernel kernel, const Shape& sh, unsigned blocks, hipStream_t s,
                       Args... args) {
  const size_t lds = sh.multi ? (size_t)sh.vecs * kVec<T> * 12u * sh.threads : 0u;
  if (lds > 64u * 1024u) {
    const hipError_t e =
        hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3(blocks), dim3((unsigned)sh.threads), lds, s, args...);
  return hipGetLastError();
}

// CALL(V, MULTI, TAIL) of a shape.
#define EMBTAB_GN_TAIL(V_, M_, CALL)             \
  do {                                           \
    if (a.dim % kVec<T>) return CALL(V_, M_, true); \
    return CALL(V_, M_, false);                  \
  } while (0)
#define EMBTAB_GN_SHAPE(CALL)                              \
  do {                                                     \
    constexpr int kV = sizeof(T) == 4 ? 2 : 1;             \
    if (sh.multi) EMBTAB_GN_TAIL(kV, true, CALL);          \
    if (sh.vecs == kV) EMBTAB_GN_TAIL(kV, false, CALL);    \
    EMBTAB_GN_TAIL(1, false, CALL);                        \
  } while (0)

template <class T>
hipError_t forward_t(const GatedNorm& a, void* y, void* h, hipStream_t s) {
  const Shape sh = shape_of<T>(a.dim);
  const unsigned blocks = grid_of(a.rows, sh, kForwardWaves);
#define EMBTAB_GN(V_, M_, TAIL_)                                                                 \
  launch_rows<T>(k_gated_norm_forward<T, V_, M_, TAIL_>, sh, blocks, s,                          \
                 static_cast<const T*>(a.x), static_cast<const T*>(a.block),                     \
                 static_cast<const T*>(a.gate), a.w_post, a.scale, a.w_pre, a.rows,              \
                 (uint32_t)a.dim, sh.tpr, a.gate_kind, a.sigmoid, a.eps, static_cast<T*>(y),     \
                 static_cast<T*>(h))
  EMBTAB_GN_SHAPE(EMBTAB_GN);
#undef EMBTAB_GN
}

template <class T>
hipError_t backward_rows(const GatedNorm& a, const Shape& sh, unsigned blocks, const void* dy,
                         const void* dh, void* dx, void* dblock, void* dgate, float* parts,
                         hipStream_t s) {
#define EMBTAB_GN(V_, M_, TAIL_)                                                                 \
  launch_rows<T>(k_gated_norm_backward<T, V_, M_, TAIL_>, sh, blocks, s,                         \
                 static_cast<const T*>(a.x), static_cast<const T*>(a.block),                     \
                 static_cast<const T*>(a.gate), a.w_post, a.scale, a.w_pre,                      \
                 static_cast<const T*>(dy), static_cast<const T*>(dh), a.rows, (uint32_t)a.dim,  \
                 sh.tpr, a.gate_kind, a.sigmoid, a.eps, static_cast<T*>(dx),                     \
                 static_cast<T*>(dblock), static_cast<T*>(dgate), parts)
  EMBTAB_GN_SHAPE(EMBTAB_GN);
#undef EMBTAB_GN
}
#undef EMBTAB_GN_SHAPE
#undef EMBTAB_GN_TAIL

template <class T>
hipError_t backward_t(const GatedNorm& a, const void* dy, const void* dh, void* dx, void* dblock,
                      void* dgate, float* dw_post, float* dscale, float* dw_pre, float* parts,
                      hipStream_t s) {
  const Shape sh = shape_of<T>(a.dim);
  const unsigned blocks = grid_of(a.rows, sh, backward_waves(sh));
  if (blocks) {
    const hipError_t e =
        backward_rows<T>(a, sh, blocks, dy, dh, dx, dblock, dgate, parts, s);
    if (e != hipSuccess) return e;
  }
  const uint32_t width = 3u * (uint32_t)a.dim;
  hipLaunchKernelGGL(k_gated_norm_column_sums, dim3((width + kSumCols - 1) / kSumCols),
                     dim3(kSumCols * kSumGroups), 0, s, parts, blocks, (uint32_t)a.dim, dw_post,
                     dscale, dw_pre);
  return hipGetLastError();
}

}  // namespace

// One [3][dim] fp32 part per block of the backward kernel, of whichever type
// takes more blocks.
size_t gated_norm_workspace_bytes(int64_t rows, int32_t dim) {
  const Shape wide = shape_of<float>(dim), narrow = shape_of<bf16_t>(dim);
  const size_t a = grid_of(rows, wide, backward_waves(wide));
  const size_t b = grid_of(rows, narrow, backward_waves(narrow));
  return (sizeof(float) * 3u * (size_t)dim * (a > b ? a : b) + 256) & ~(size_t)255;
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
