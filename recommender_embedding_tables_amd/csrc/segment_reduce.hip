// Deduplicated gradients of a prepared batch, and the Adagrad step of its
// rows from them, for gfx950: the fused reduction and step in two parts, so
// that a clip by the global norm (which needs every row's gradient first) can
// stand between them.
//
//   sums[u] = sum over the occurrences of distinct row u of c_b * grad_out[b]
//   sqnorm  = sum over u and columns of sums[u]^2, in 64 bits
//   step:   g = scale * sums[u];  G += g^2;  W -= lr * g / (sqrt(G) + eps)
//
// Bound by memory: one gradient row per occurrence read, one row per distinct
// row written; the step then reads and writes rows of the distinct rows only,
// where a second pass over the occurrences would gather every gradient row
// again.  26 tables, D = 128, 1.7 million occurrences of 342 thousand rows: the
// reduction 194 us (5.5 TB/s over its 1.08 GB), the step 158 us (5.9 TB/s over
// its 0.94 GB).  The sums are stored through the caches, where the step finds
// part of them again: past them the step takes 174 us.  Eight gradient rows in
// flight per sub-group instead of four change neither time.
//
// The sorted positions are cut into chunks, one sub-group of lanes each, and
// blocks of chunks, as for the fused step.  A run inside a chunk is summed in
// registers and stored.  A run over several chunks of a block leaves its parts
// in LDS, and the sub-group of the chunk where it ends adds them in chunk
// order.  A run over several blocks leaves one part per block in the
// workspace (part_tail of the block where it starts, part_head of the later
// ones), and a second launch adds those, one block per run: a row with tens of
// thousands of occurrences is split over the whole chip.  Every sum has a
// fixed order.
#include "dense.hpp"

namespace embtab {

namespace {

__device__ inline double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

__device__ inline void add_squares(double& acc, const f4 x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) acc = __builtin_fma((double)x[i], (double)x[i], acc);
}

// Sum over the block's 256 threads; valid in thread 0.
__device__ inline double block_sum_256(double v, double* lds4) {
  v = wave_sum(v);
  if ((threadIdx.x & 63u) == 0u) lds4[threadIdx.x >> 6] = v;
  __syncthreads();
  return (lds4[0] + lds4[1]) + (lds4[2] + lds4[3]);
}

struct ReduceIn {
  const uint32_t *keys, *perm, *sgr, *misc, *chunk_base, *head_base;
  const float *sscale, *grad;
  uint32_t n, sentinel, nbags, B, T;
  int32_t D;
};

template <int SG, int VEC, bool MEAN, bool REUSE>
__global__ __launch_bounds__(256) void k_grad_reduce(const ReduceIn in,
                                                     float* __restrict__ sums,
                                                     float* __restrict__ part_head,
                                                     float* __restrict__ part_tail,
                                                     double* __restrict__ sq_block) {
  constexpr int MPL = chunk_rounds<SG>();
  constexpr int UF = VEC > 1 ? 2 : (SG < 4 ? SG : 4);  // positions in flight
  constexpr uint32_t CH = SG * MPL;
  constexpr int SGPB = 256 / SG;
  __shared__ f4 s_in[SGPB][SG * VEC];   // part of the run that entered the chunk
  __shared__ f4 s_out[SGPB][SG * VEC];  // part of the run that starts in it and leaves it
  __shared__ uint32_t s_in_u[SGPB], s_out_u[SGPB];
  __shared__ uint32_t s_in_ends[SGPB];
  __shared__ double lds4[4];
  const int lane = threadIdx.x % SG, sg = threadIdx.x / SG;
  const uint32_t D4 = (uint32_t)in.D >> 2;
  const uint32_t c = blockIdx.x * SGPB + sg, k0 = c * CH;
  const uint32_t k1 = k0 + CH < in.n ? k0 + CH : in.n;
  const bool one_hot = !batch_not_one_hot(in.misc);
  uint32_t in_u = kNoRow, out_u = kNoRow, in_ends = 0u;
  double sq = 0.0;
  if (k0 < in.n) {
    const uint32_t key_prev = k0 > 0 ? in.keys[k0 - 1] : kNoRow;
    const uint32_t key_next = k1 < in.n ? in.keys[k1] : kNoRow;
    uint32_t u = in.head_base[k0 >> 8] + in.chunk_base[c];
    uint32_t mkey[MPL], mgr[MPL];
    float msc[MPL];
#pragma unroll
    for (int i = 0; i < MPL; ++i) {
      const uint32_t k = k0 + i * SG + lane;
      mkey[i] = kNoRow;
      mgr[i] = kNoRow;
      msc[i] = 1.0f;
      if (k < k1) {
        mkey[i] = in.keys[k];
        if (one_hot) {
          const uint32_t v = in.perm[k];
          if (v < in.n) mgr[i] = one_hot_grad_row(v, in.B, in.T);
        } else {
          mgr[i] = in.sgr[k];
          if (MEAN) msc[i] = in.sscale[k];
        }
      }
    }
    f4 acc[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) acc[v] = f4{0.f, 0.f, 0.f, 0.f};
    // whether the run being summed entered the chunk from the one before
    bool entered = (uint32_t)__shfl((int)mkey[0], 0, SG) == key_prev;
    if (entered) u -= 1u;  // that run's head was counted before the chunk
#pragma unroll
    for (int i = 0; i < MPL; ++i) {
      for (int l0 = 0; l0 < SG; l0 += UF) {
        uint32_t kk[UF + 1], gr[UF];
        float cc[UF];
#pragma unroll
        for (int q = 0; q < UF; ++q) {
          kk[q] = (uint32_t)__shfl((int)mkey[i], l0 + q, SG);
          gr[q] = (uint32_t)__shfl((int)mgr[i], l0 + q, SG);
          cc[q] = MEAN ? __shfl(msc[i], l0 + q, SG) : 1.0f;
        }
        if (kk[0] >= in.sentinel) break;  // the rest of the chunk holds no valid key
        uint32_t nx = key_next;
        if (l0 + UF < SG) nx = (uint32_t)__shfl((int)mkey[i], l0 + UF, SG);
        else if (i + 1 < MPL) nx = (uint32_t)__shfl((int)mkey[(i + 1) < MPL ? i + 1 : i], 0, SG);
        kk[UF] = nx;
        f4 g[UF][VEC];
#pragma unroll
        for (int q = 0; q < UF; ++q)
#pragma unroll
          for (int v = 0; v < VEC; ++v) {
            const uint32_t d4 = (uint32_t)(lane + v * SG);
            // a position no bag wrote (bad offsets) may name any row: it adds 0
            const bool ok = kk[q] < in.sentinel && gr[q] < in.nbags && d4 < D4;
            g[q][v] = REUSE ? load4_or_zero(in.grad, gr[q], (uint32_t)in.D, d4, ok)
                            : load4_nt_or_zero(in.grad, gr[q], (uint32_t)in.D, d4, ok);
          }
#pragma unroll
        for (int q = 0; q < UF; ++q) {
          if (kk[q] >= in.sentinel) continue;
          const uint32_t p = k0 + (uint32_t)(i * SG + l0 + q);
#pragma unroll
          for (int v = 0; v < VEC; ++v) acc[v] += MEAN ? g[q][v] * cc[q] : g[q][v];
          const uint32_t nxt = p + 1 == k1 ? key_next : kk[q + 1];
          const bool ends = nxt != kk[q];
          if (!ends && p + 1 != k1) continue;
          if (ends && !entered) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
              const uint32_t d4 = (uint32_t)(lane + v * SG);
              if (d4 < D4) {
                *reinterpret_cast<f4*>(sums + (size_t)u * in.D + 4 * d4) = acc[v];
                add_squares(sq, acc[v]);
              }
            }
          } else if (entered) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) s_in[sg][lane + v * SG] = acc[v];
            in_u = u;
            in_ends = ends ? 1u : 0u;
          } else {
#pragma unroll
            for (int v = 0; v < VEC; ++v) s_out[sg][lane + v * SG] = acc[v];
            out_u = u;
          }
          if (ends) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) acc[v] = f4{0.f, 0.f, 0.f, 0.f};
            entered = false;
            ++u;
          }
        }
      }
    }
  }
  if (lane == 0) {
    s_in_u[sg] = in_u;
    s_out_u[sg] = out_u;
    s_in_ends[sg] = in_ends;
  }
  __syncthreads();
  // The sub-group of the last chunk that a run reaches inside the block adds
  // its parts: the chunk where it ends, or the block's last.
  const bool closes_in = in_u != kNoRow && (in_ends || sg == SGPB - 1);
  const bool closes_out = out_u != kNoRow && sg == SGPB - 1;
  if (closes_in) {
    int j = sg;  // first chunk of the block that the run enters
    while (j > 0 && s_in_u[j - 1] == in_u) --j;
    const bool starts = j > 0 && s_out_u[j - 1] == in_u;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const uint32_t d4 = (uint32_t)(lane + v * SG);
      if (d4 >= D4) continue;
      f4 t = starts ? s_out[j - 1][d4] : f4{0.f, 0.f, 0.f, 0.f};
      for (int i = j; i <= sg; ++i) t += s_in[i][d4];
      if (starts && in_ends) {
        *reinterpret_cast<f4*>(sums + (size_t)in_u * in.D + 4 * d4) = t;
        add_squares(sq, t);
      } else {
        float* dst = starts ? part_tail : part_head;
        *reinterpret_cast<f4*>(dst + (size_t)blockIdx.x * in.D + 4 * d4) = t;
      }
    }
  }
  if (closes_out) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const uint32_t d4 = (uint32_t)(lane + v * SG);
      if (d4 < D4)
        *reinterpret_cast<f4*>(part_tail + (size_t)blockIdx.x * in.D + 4 * d4) = s_out[sg][d4];
    }
  }
  sq = block_sum_256(sq, lds4);
  if (threadIdx.x == 0) sq_block[blockIdx.x] = sq;
}

// Block b finishes the run that starts in reduction block b and leaves it.
template <int SG, int VEC>
__global__ __launch_bounds__(256) void k_grad_spans(const uint32_t* __restrict__ span_u,
                                                    const uint32_t* __restrict__ seg_off,
                                                    const float* __restrict__ part_head,
                                                    const float* __restrict__ part_tail,
                                                    uint32_t n, uint32_t bp, int32_t D,
                                                    float* __restrict__ sums,
                                                    double* __restrict__ sq_span) {
  constexpr int SGPB = 256 / SG;
  __shared__ f4 s_part[SGPB][SG * VEC];
  __shared__ double lds4[4];
  const uint32_t b = blockIdx.x;
  const uint32_t u = (uint64_t)(b + 1) * bp < n ? span_u[b + 1] : kNoRow;
  const bool mine = u != kNoRow && seg_off[u] / bp == b;
  if (!mine) {
    if (threadIdx.x == 0) sq_span[b] = 0.0;
    return;
  }
  const uint32_t last = (seg_off[u + 1] - 1u) / bp;
  const int lane = threadIdx.x % SG, sg = threadIdx.x / SG;
  const uint32_t D4 = (uint32_t)D >> 2;
  f4 t[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v)
    t[v] = sg == 0 ? load4_or_zero(part_tail, b, (uint32_t)D, lane + v * SG,
                                   (uint32_t)(lane + v * SG) < D4)
                   : f4{0.f, 0.f, 0.f, 0.f};
  for (uint32_t i = b + 1 + sg; i <= last; i += 4 * SGPB) {
    f4 x[4][VEC];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        x[q][v] = load4_or_zero(part_head, i + q * SGPB, (uint32_t)D, lane + v * SG,
                                i + q * SGPB <= last && (uint32_t)(lane + v * SG) < D4);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int v = 0; v < VEC; ++v) t[v] += x[q][v];
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v) s_part[sg][lane + v * SG] = t[v];
  __syncthreads();
  double sq = 0.0;
  if (sg == 0) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const uint32_t d4 = (uint32_t)(lane + v * SG);
      if (d4 >= D4) continue;
      f4 r = t[v];
      for (int i = 1; i < SGPB; ++i) r += s_part[i][d4];
      *reinterpret_cast<f4*>(sums + (size_t)u * D + 4 * d4) = r;
      add_squares(sq, r);
    }
  }
  sq = block_sum_256(sq, lds4);
  if (threadIdx.x == 0) sq_span[b] = sq;
}

__global__ __launch_bounds__(1024) void k_sum_doubles(const double* __restrict__ v, uint32_t n,
                                                      double* __restrict__ out) {
  __shared__ double lds[16];
  double s = 0.0;
  for (uint32_t i = threadIdx.x; i < n; i += 1024) s += v[i];
  s = wave_sum(s);
  if ((threadIdx.x & 63u) == 0u) lds[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  double t = 0.0;
  for (int i = 0; i < 16; ++i) t += lds[i];
  out[0] = t;
}

// One sub-group per distinct row; up to 2^32 - 1 rows, so the blocks past kGridX
// go along y (a block index times the rows of a block stays below 2^32 there:
// 2^32 / rows is a multiple of kGridX).  The square root and the reciprocal are the
// hardware instructions (each within 1 ulp), as in the fused step.
template <int SG, int VEC>
__global__ __launch_bounds__(256) void k_adagrad_rows(
    const uint32_t* __restrict__ keys, const uint32_t* __restrict__ seg_off,
    const uint32_t* __restrict__ misc, const float* __restrict__ sums,
    const float* __restrict__ scale, float* __restrict__ W, float* __restrict__ G,
    uint32_t most, uint32_t sentinel, int32_t D, float lr, float eps) {
  const uint32_t u = block_index() * (256 / SG) + threadIdx.x / SG;
  const float s = scale ? scale[0] : 1.0f;
  if (s == 0.0f || u >= most || u >= misc[kMiscNumUnique]) return;
  const uint32_t lane = threadIdx.x % SG, D4 = (uint32_t)D >> 2;
  f4 g[VEC], w[VEC], a[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) {  // under way while the row is looked up
    const uint32_t d4 = lane + v * SG;
    g[v] = load4_nt_or_zero(sums, u, (uint32_t)D, d4, d4 < D4);
  }
  const uint32_t row = keys[seg_off[u]];
  if (row >= sentinel) return;
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    const uint32_t d4 = lane + v * SG;
    w[v] = load4_or_zero(W, row, (uint32_t)D, d4, d4 < D4);
    a[v] = load4_nt_or_zero(G, row, (uint32_t)D, d4, d4 < D4);
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    const uint32_t d4 = lane + v * SG;
    if (d4 >= D4) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float gi = s * g[v][i];
      const float A = __builtin_fmaf(gi, gi, a[v][i]);
      w[v][i] = w[v][i] - (lr * gi) * __builtin_amdgcn_rcpf(__builtin_amdgcn_sqrtf(A) + eps);
      a[v][i] = A;
    }
    *reinterpret_cast<f4*>(W + (size_t)row * D + 4 * d4) = w[v];
    __builtin_nontemporal_store(a[v], reinterpret_cast<f4*>(G + (size_t)row * D + 4 * d4));
  }
}

template <int SG, int VEC>
hipError_t reduce_t(const Handle& h, const Plan& p, const ReduceIn& in, bool mean, float* sums,
                    double* sqnorm, char* ws, hipStream_t s) {
  const unsigned blocks = (unsigned)((p.nnz + p.bp - 1) / p.bp);
  float* ph = reinterpret_cast<float*>(ws + p.part_head);
  float* pt = reinterpret_cast<float*>(ws + p.part_tail);
  // the sums of squares, two per block: the counts' space (4 bytes per
  // occurrence and at least 256 bytes, a block covers 256 occurrences or more)
  double* sq = reinterpret_cast<double*>(ws + p.counts);
  const bool reuse = mean || p.nnz != p.B * (int64_t)h.T;  // a cache policy only
  if (mean)
    hipLaunchKernelGGL((k_grad_reduce<SG, VEC, true, true>), dim3(blocks), dim3(256), 0, s, in,
                       sums, ph, pt, sq);
  else if (reuse)
    hipLaunchKernelGGL((k_grad_reduce<SG, VEC, false, true>), dim3(blocks), dim3(256), 0, s, in,
                       sums, ph, pt, sq);
  else
    hipLaunchKernelGGL((k_grad_reduce<SG, VEC, false, false>), dim3(blocks), dim3(256), 0, s, in,
                       sums, ph, pt, sq);
  hipLaunchKernelGGL((k_grad_spans<SG, VEC>), dim3(blocks), dim3(256), 0, s,
                     reinterpret_cast<const uint32_t*>(ws + p.span_u),
                     reinterpret_cast<const uint32_t*>(ws + p.seg_off), ph, pt, (uint32_t)p.nnz,
                     p.bp, h.D, sums, sq + blocks);
  hipLaunchKernelGGL(k_sum_doubles, dim3(1), dim3(1024), 0, s, sq, 2u * blocks, sqnorm);
  return hipGetLastError();
}

template <int SG, int VEC>
hipError_t step_t(const Handle& h, const Plan& p, const uint32_t* keys, const float* sums,
                  const float* scale, float lr, float eps, char* ws, hipStream_t s) {
  const int64_t most = p.nnz < h.total_rows ? p.nnz : h.total_rows;
  constexpr int kRows = 256 / SG;
  hipLaunchKernelGGL((k_adagrad_rows<SG, VEC>), row_grid((most + kRows - 1) / kRows), dim3(256),
                     0, s, keys, reinterpret_cast<const uint32_t*>(ws + p.seg_off),
                     reinterpret_cast<const uint32_t*>(ws + p.misc), sums, scale, h.W, h.G,
                     (uint32_t)most, (uint32_t)h.total_rows, h.D, lr, eps);
  return hipGetLastError();
}

}  // namespace

// CALL(SG, VEC) for the sub-group shape of rows of D values.
#define EMBTAB_BY_SHAPE(D_, CALL)              \
  switch (subgroup_lanes(D_)) {                \
    case 1: return CALL(1, 1);                 \
    case 2: return CALL(2, 1);                 \
    case 4: return CALL(4, 1);                 \
    case 8: return CALL(8, 1);                 \
    case 16: return CALL(16, 1);               \
    case 32: return CALL(32, 1);               \
    default:                                   \
      switch (vec_per_lane(D_)) {              \
        case 1: return CALL(64, 1);            \
        case 2: return CALL(64, 2);            \
        case 3: return CALL(64, 3);            \
        default: return CALL(64, 4);           \
      }                                        \
  }

hipError_t launch_grad_reduce(const Handle& h, const Plan& p, const uint32_t* keys,
                              const uint32_t* perm, bool mean, const float* grad_out,
                              float* sums, double* sqnorm, char* ws, hipStream_t s) {
  if (p.nnz == 0 || p.B == 0) {
    hipLaunchKernelGGL(k_sum_doubles, dim3(1), dim3(1024), 0, s,
                       static_cast<const double*>(nullptr), 0u, sqnorm);
    return hipGetLastError();
  }
  ReduceIn in;
  in.keys = keys;
  in.perm = perm;
  in.sgr = reinterpret_cast<const uint32_t*>(ws + p.sgr);
  in.misc = reinterpret_cast<const uint32_t*>(ws + p.misc);
  in.chunk_base = reinterpret_cast<const uint32_t*>(ws + p.chunk_base);
  in.head_base = reinterpret_cast<const uint32_t*>(ws + p.head_base);
  in.sscale = reinterpret_cast<const float*>(ws + p.sscale);
  in.grad = grad_out;
  in.n = (uint32_t)p.nnz;
  in.sentinel = (uint32_t)h.total_rows;
  in.nbags = (uint32_t)(p.B * h.T);
  in.B = (uint32_t)p.B;
  in.T = (uint32_t)h.T;
  in.D = h.D;
#define EMBTAB_REDUCE(SG_, VEC_) reduce_t<SG_, VEC_>(h, p, in, mean, sums, sqnorm, ws, s)
  EMBTAB_BY_SHAPE(h.D, EMBTAB_REDUCE)
#undef EMBTAB_REDUCE
}

hipError_t launch_adagrad_rows(const Handle& h, const Plan& p, const uint32_t* keys,
                               const float* sums, const float* scale, float lr, float eps,
                               char* ws, hipStream_t s) {
  if (p.nnz == 0 || p.B == 0) return hipSuccess;
#define EMBTAB_STEP(SG_, VEC_) step_t<SG_, VEC_>(h, p, keys, sums, scale, lr, eps, ws, s)
  EMBTAB_BY_SHAPE(h.D, EMBTAB_STEP)
#undef EMBTAB_STEP
}

}  // namespace embtab
