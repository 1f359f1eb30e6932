// Choices sorted by expert, rows copied into expert order and back with their
// weights, and the gradients of both, for gfx950.
//
// A token i has k choices of an expert each; choice i*k + j goes to a row of
// the expert-ordered buffer.  Rows of one expert are contiguous and keep the
// order of their choices (a stable counting sort), so every output is
// determined by the input alone:
//   row(choice) = start[e] + rank            without a capacity
//               = e * capacity + rank        with one; rank >= capacity: dropped
// with rank the number of earlier choices of the same expert and start the
// exclusive sum of the experts' counts.
//
//   dispatch           xs[r] = x[src[r] / k], 0 where src[r] < 0
//   combine            y[i] = sum_j w[i,j] * ys[pos[i,j]]
//   combine backward   dys[r] = w[src[r]] * dy[src[r] / k], 0 where src[r] < 0
//                      dw[i,j] = sum_c dy[i,c] * ys[pos[i,j],c]
//   dispatch backward  dx[i] = sum_j dxs[pos[i,j]]     (combine with weights 1)
// A dropped choice (pos < 0) contributes nothing and has a zero dw; a pos that
// names no row is taken as dropped, so no access leaves the buffers.
//
// The row kernels are bound by memory (a one-shot device copy reaches 6.5 TB/s
// here, rows written in scattered order 5.1 to 5.3).  They walk tokens, not
// rows: a token's row is read once and serves its k choices from registers,
// where a walk over the rows would read it k times.  Outputs are stored past the
// caches, which they would only sweep: the forward of 65536 tokens with two of
// 64 experts, 3328 x bf16, takes 490 us (5.3 TB/s) against 520, the gradients of
// 16384 tokens with four 274 us of kernels (5.5 TB/s; 276 to 292 a pass) against
// 313.
#include "dense.hpp"

namespace embtab {

namespace {

// ---------------------------------------------------------------- sort
// Tiles of 1024 choices, one block each; wave w owns the contiguous quarter w
// of its tile.
constexpr int kTileThreads = 256;
constexpr int kTileRounds = 4;
constexpr int kTile = kTileThreads * kTileRounds;
constexpr int kMaxExperts = 1024;
// Up to this many tiles every block of the scatter adds the tiles' counts
// itself (counts [tile][expert], one row per tile) and the scan's launch is
// saved: sort, dispatch and combine of 4096 tokens with two choices take 19 us
// against 21.5, of 16384 tokens 22.5 against 23.8; with more tiles the adding
// takes as long as the scan (counts [expert][tile]).
constexpr uint32_t kDirectTiles = 32;

__device__ inline uint32_t expert_block_scan(uint32_t v, uint32_t* total, uint32_t* lds4) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const uint32_t x = wave_incl_scan(v);
  if (lane == 63) lds4[w] = x;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    before += i < w ? lds4[i] : 0u;
    all += lds4[i];
  }
  __syncthreads();
  *total = all;
  return x - v + before;
}

__global__ __launch_bounds__(kTileThreads) void k_expert_hist(const int64_t* __restrict__ ids,
                                                              uint32_t n, uint32_t experts,
                                                              uint32_t ntiles,
                                                              uint32_t* __restrict__ tile_hist) {
  __shared__ uint32_t cnt[kMaxExperts];
  for (uint32_t e = threadIdx.x; e < experts; e += kTileThreads) cnt[e] = 0u;
  __syncthreads();
  const uint32_t base = blockIdx.x * kTile + threadIdx.x;
#pragma unroll
  for (int r = 0; r < kTileRounds; ++r) {
    const uint32_t c = base + r * kTileThreads;
    const int64_t id = c < n ? ids[c] : -1;
    if (id >= 0 && id < (int64_t)experts) atomicAdd(&cnt[id], 1u);
  }
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < experts; e += kTileThreads)
    tile_hist[ntiles <= kDirectTiles ? (size_t)blockIdx.x * experts + e
                                     : (size_t)e * ntiles + blockIdx.x] = cnt[e];
}

// One block per expert: exclusive scan of its counts over the tiles.
__global__ __launch_bounds__(kTileThreads) void k_expert_scan(uint32_t* __restrict__ tile_hist,
                                                              uint32_t ntiles,
                                                              uint32_t* __restrict__ totals) {
  __shared__ uint32_t lds4[4];
  uint32_t* row = tile_hist + (size_t)blockIdx.x * ntiles;
  uint32_t carry = 0;
  for (uint32_t base = 0; base < ntiles; base += kTileThreads) {
    const uint32_t i = base + threadIdx.x;
    const uint32_t v = i < ntiles ? row[i] : 0u;
    uint32_t total;
    const uint32_t ex = expert_block_scan(v, &total, lds4);
    if (i < ntiles) row[i] = carry + ex;
    carry += total;
  }
  if (threadIdx.x == 0) totals[blockIdx.x] = carry;
}

__global__ __launch_bounds__(kTileThreads) void k_expert_scatter(
    const int64_t* __restrict__ ids, uint32_t n, uint32_t experts, int nbits, int64_t capacity,
    int64_t rows, uint32_t ntiles, const uint32_t* __restrict__ tile_off,
    const uint32_t* __restrict__ totals, int32_t* __restrict__ offsets,
    int32_t* __restrict__ src, int32_t* __restrict__ pos) {
  __shared__ uint32_t wcnt[4][kMaxExperts];
  __shared__ uint32_t kept[kMaxExperts];       // choices kept per expert
  __shared__ uint32_t first[kMaxExperts + 1];  // exclusive sums of the kept counts
  __shared__ uint32_t lds4[4];
  const uint32_t w = threadIdx.x >> 6, lane = threadIdx.x & 63u;
  for (uint32_t i = threadIdx.x; i < experts; i += kTileThreads)
    wcnt[0][i] = wcnt[1][i] = wcnt[2][i] = wcnt[3][i] = 0u;
  __syncthreads();
  const uint32_t base = blockIdx.x * kTile + w * (kTileRounds * 64) + lane;
  uint32_t key[kTileRounds], rank[kTileRounds];
#pragma unroll
  for (int r = 0; r < kTileRounds; ++r) {
    const uint32_t c = base + r * 64;
    const int64_t id = c < n ? ids[c] : -1;
    key[r] = id >= 0 && id < (int64_t)experts ? (uint32_t)id : kNoRow;
  }
  // rank inside the wave's quarter: its rounds go in choice order
#pragma unroll
  for (int r = 0; r < kTileRounds; ++r) {
    const bool valid = key[r] != kNoRow;
    uint64_t m = __ballot(valid);
    for (int b = 0; b < nbits; ++b) {
      const bool bit = (key[r] >> b) & 1u;
      const uint64_t bb = __ballot(bit);
      m &= bit ? bb : ~bb;
    }
    const uint32_t below = lanes_below(m);
    uint32_t old = 0u;
    if (valid) old = wcnt[w][key[r]];
    // the group's lanes have read before its first lane writes, and the next
    // round reads what this one wrote
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (valid && below == 0u) wcnt[w][key[r]] = old + (uint32_t)__popcll(m);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    rank[r] = old + below;
  }
  __syncthreads();
  // per expert: offset of each wave's quarter, and the kept totals
  const bool solo = ntiles == 1u;  // a single tile's counts are the totals
  uint32_t carry = 0;
  for (uint32_t e0 = 0; e0 < experts; e0 += kTileThreads) {
    const uint32_t e = e0 + threadIdx.x;
    uint32_t keep = 0u;
    if (e < experts) {
      const uint32_t c0 = wcnt[0][e], c1 = wcnt[1][e], c2 = wcnt[2][e], c3 = wcnt[3][e];
      uint32_t t0 = 0u, all = 0u;  // choices of the earlier tiles and of all
      if (solo) {
        all = c0 + c1 + c2 + c3;
      } else if (ntiles <= kDirectTiles) {
#pragma unroll 8
        for (uint32_t t = 0; t < ntiles; ++t) {
          const uint32_t v = tile_off[(size_t)t * experts + e];
          t0 += t < blockIdx.x ? v : 0u;
          all += v;
        }
      } else {
        t0 = tile_off[(size_t)e * ntiles + blockIdx.x];
        all = totals[e];
      }
      wcnt[0][e] = t0;
      wcnt[1][e] = t0 + c0;
      wcnt[2][e] = t0 + c0 + c1;
      wcnt[3][e] = t0 + c0 + c1 + c2;
      keep = all;
      if (capacity && (int64_t)keep > capacity) keep = (uint32_t)capacity;
      kept[e] = keep;
    }
    uint32_t total;
    const uint32_t ex = expert_block_scan(keep, &total, lds4);
    if (e < experts) first[e] = carry + ex;
    carry += total;
  }
  if (threadIdx.x == 0) first[experts] = carry;
  __syncthreads();
  if (blockIdx.x == 0)
    for (uint32_t e = threadIdx.x; e <= experts; e += kTileThreads) offsets[e] = (int32_t)first[e];
#pragma unroll
  for (int r = 0; r < kTileRounds; ++r) {
    const uint32_t c = base + r * 64;
    if (c >= n) continue;
    int32_t p = -1;
    if (key[r] != kNoRow) {
      const uint32_t k = wcnt[w][key[r]] + rank[r];
      if (!capacity) p = (int32_t)(first[key[r]] + k);
      else if ((int64_t)k < capacity) p = (int32_t)((int64_t)key[r] * capacity + k);
      if (p >= 0) src[p] = (int32_t)c;
    }
    pos[c] = p;
  }
  // rows without a choice, spread over the blocks
  for (int64_t row = (int64_t)blockIdx.x * kTileThreads + threadIdx.x; row < rows;
       row += (int64_t)gridDim.x * kTileThreads) {
    const bool empty = capacity ? (uint64_t)(row % capacity) >= kept[row / capacity]
                                : (uint64_t)row >= carry;
    if (empty) src[row] = -1;
  }
}

// ---------------------------------------------------------------- rows
// The vector that starts at column c of a row of `dim` elements (c a multiple
// of the vector width, below dim).  A last vector that would pass the row's
// end is moved back to end there: it then repeats elements of the one before,
// which copies write twice with the same value and sums mask out.
template <class T>
__device__ inline uint32_t vec_column(uint32_t v, uint32_t dim) {
  const uint32_t c = v * (uint32_t)kVec<T>;
  return c + kVec<T> <= dim ? c : dim - kVec<T>;
}

constexpr int kRowThreads = 256;

constexpr int kRowVecs = 4;          // vectors in flight per thread
constexpr uint32_t kWideVecs = 64;   // vectors of a row that takes a wave of its own
constexpr uint32_t kZeroRows = 64;   // rows checked by one zero-fill block

// Fills the rows of [first, first + kZeroRows) that hold no choice with zeros.
template <class T>
__device__ inline void zero_empty_rows(const int32_t* __restrict__ src, int64_t first,
                                       int64_t rows, uint32_t dim, T* __restrict__ out) {
  const uint32_t lane = threadIdx.x & 63u;
  Raw<T> z;
#pragma unroll
  for (int i = 0; i < 4; ++i) z.w[i] = 0u;
  const uint32_t nvec = (dim + kVec<T> - 1) / kVec<T>;
  for (uint32_t i = threadIdx.x >> 6; i < kZeroRows; i += kRowThreads / 64) {
    const int64_t r = first + i;
    if (r >= rows) return;
    if (src[r] >= 0) continue;
    T* p = out + (size_t)r * dim;
    for (uint32_t v = lane; v < nvec; v += 64) store_raw(p + vec_column<T>(v, dim), z);
  }
}

// Block b < token_blocks copies tpb tokens; the later blocks zero the empty
// rows.
template <class T>
__global__ __launch_bounds__(kRowThreads) void k_expert_dispatch(
    const T* __restrict__ x, const int32_t* __restrict__ pos, const int32_t* __restrict__ src,
    int64_t tokens, uint32_t topk, int64_t rows, uint32_t dim, uint32_t nvec, uint32_t tpb,
    uint32_t token_blocks, T* __restrict__ xs) {
  const uint32_t block = block_index();
  if (block >= token_blocks) {
    zero_empty_rows(src, (int64_t)(block - token_blocks) * kZeroRows, rows, dim, xs);
    return;
  }
  const int64_t t0 = (int64_t)block_index() * tpb;
  const uint32_t nt = tokens - t0 < (int64_t)tpb ? (uint32_t)(tokens - t0) : tpb;
  const uint32_t all = nt * nvec;
  for (uint32_t i0 = threadIdx.x; i0 < all; i0 += kRowThreads * kRowVecs) {
    Raw<T> r[kRowVecs];
    uint32_t tok[kRowVecs], col[kRowVecs];
#pragma unroll
    for (int u = 0; u < kRowVecs; ++u) {
      const uint32_t i = i0 + u * kRowThreads < all ? i0 + u * kRowThreads : all - 1;
      tok[u] = i / nvec;
      col[u] = vec_column<T>(i - tok[u] * nvec, dim);
      r[u] = load_raw<T, kVec<T>, true>(x + (size_t)(t0 + tok[u]) * dim + col[u]);
    }
#pragma unroll
    for (int u = 0; u < kRowVecs; ++u) {
      if (i0 + u * kRowThreads >= all) break;
      const int32_t* p = pos + (size_t)(t0 + tok[u]) * topk;
      for (uint32_t j = 0; j < topk; ++j)
        if ((uint32_t)p[j] < (uint32_t)rows)
          store_raw<T, kVec<T>, true>(xs + (size_t)p[j] * dim + col[u], r[u]);
    }
  }
}

// The same with one wave per token for rows that fill its lanes (kWideVecs):
// its choices are scalars.
template <class T>
__global__ __launch_bounds__(kRowThreads) void k_expert_dispatch_wide(
    const T* __restrict__ x, const int32_t* __restrict__ pos, const int32_t* __restrict__ src,
    int64_t tokens, uint32_t topk, int64_t rows, uint32_t dim, uint32_t nvec,
    uint32_t token_blocks, T* __restrict__ xs) {
  const uint32_t block = block_index();
  if (block >= token_blocks) {
    zero_empty_rows(src, (int64_t)(block - token_blocks) * kZeroRows, rows, dim, xs);
    return;
  }
  const uint32_t lane = threadIdx.x & 63u;
  const int64_t tok = (int64_t)block_index() * (kRowThreads / 64) +
                      __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (tok >= tokens) return;
  const int32_t* p = pos + (size_t)tok * topk;
  for (uint32_t v0 = 0; v0 < nvec; v0 += 64u * kRowVecs) {
    Raw<T> r[kRowVecs];
    uint32_t col[kRowVecs];
#pragma unroll
    for (int u = 0; u < kRowVecs; ++u) {
      const uint32_t v = v0 + u * 64u + lane;
      col[u] = vec_column<T>(v < nvec ? v : nvec - 1u, dim);
      r[u] = load_raw<T, kVec<T>, true>(x + (size_t)tok * dim + col[u]);
    }
    for (uint32_t j = 0; j < topk; ++j) {
      if ((uint32_t)p[j] >= (uint32_t)rows) continue;
      T* row = xs + (size_t)p[j] * dim;
#pragma unroll
      for (int u = 0; u < kRowVecs; ++u)
        if (v0 + u * 64u + lane < nvec) store_raw<T, kVec<T>, true>(row + col[u], r[u]);
    }
  }
}

// K choices summed in the order of j, each product and sum in fp32, one
// rounding at the end.
template <class T, int K, bool WEIGHTED>
__global__ __launch_bounds__(kRowThreads) void k_expert_combine(
    const T* __restrict__ ys, const int32_t* __restrict__ pos, const float* __restrict__ weights,
    int64_t tokens, uint32_t topk, uint32_t rows, uint32_t dim, uint32_t nvec, uint32_t tpb,
    T* __restrict__ y) {
  const int64_t t0 = (int64_t)block_index() * tpb;
  if (t0 >= tokens) return;
  const uint32_t nt = tokens - t0 < (int64_t)tpb ? (uint32_t)(tokens - t0) : tpb;
  const uint32_t all = nt * nvec;
  for (uint32_t i = threadIdx.x; i < all; i += kRowThreads) {
    const uint32_t tok = i / nvec, col = vec_column<T>(i - tok * nvec, dim);
    float acc[kVec<T>];
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e) acc[e] = 0.0f;
    for (uint32_t j0 = 0; j0 < topk; j0 += K) {
      Raw<T> r[K];
      float wt[K];
      bool on[K];
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const size_t c = (size_t)(t0 + tok) * topk + j0 + j;
        const int32_t p = j0 + j < topk ? pos[c] : -1;
        on[j] = (uint32_t)p < rows;
        wt[j] = WEIGHTED && on[j] ? weights[c] : 1.0f;
        if (on[j]) r[j] = load_raw<T, kVec<T>, true>(ys + (size_t)p * dim + col);
      }
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (on[j]) {
#pragma unroll
          for (int e = 0; e < kVec<T>; ++e)
            acc[e] = WEIGHTED ? __builtin_fmaf(wt[j], r[j].get(e), acc[e]) : acc[e] + r[j].get(e);
        }
    }
    Raw<T> o;
    o.set_all(acc);
    store_raw<T, kVec<T>, true>(y + (size_t)(t0 + tok) * dim + col, o);
  }
}

// The same with one wave per token, for rows that fill its lanes (kWideVecs):
// the choices are then scalars, their loads and branches cost the wave once, and
// U vectors of every choice are in flight.  65536 tokens of two 3328 x bf16
// rows: 227 us, against 248 with the vectors of a few tokens spread over the
// block, which short rows keep (their lanes would idle here).
template <class T, int K, bool WEIGHTED>
__global__ __launch_bounds__(kRowThreads) void k_expert_combine_wide(
    const T* __restrict__ ys, const int32_t* __restrict__ pos, const float* __restrict__ weights,
    int64_t tokens, uint32_t topk, uint32_t rows, uint32_t dim, uint32_t nvec,
    T* __restrict__ y) {
  constexpr int U = K <= 4 ? 4 : 2;
  const uint32_t lane = threadIdx.x & 63u;
  const int64_t tok = (int64_t)block_index() * (kRowThreads / 64) +
                      __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (tok >= tokens) return;
  T* row = y + (size_t)tok * dim;
  for (uint32_t v0 = 0; v0 < nvec; v0 += 64u * U) {
    float acc[U][kVec<T>];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < kVec<T>; ++e) acc[u][e] = 0.0f;
    uint32_t col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t v = v0 + u * 64u + lane;
      col[u] = vec_column<T>(v < nvec ? v : nvec - 1u, dim);
    }
    for (uint32_t j0 = 0; j0 < topk; j0 += K) {
      Raw<T> r[K][U];
      float wt[K];
      bool on[K];
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const size_t c = (size_t)tok * topk + j0 + j;
        const int32_t p = j0 + j < topk ? pos[c] : -1;
        on[j] = (uint32_t)p < rows;
        wt[j] = WEIGHTED && on[j] ? weights[c] : 1.0f;
        if (on[j])
#pragma unroll
          for (int u = 0; u < U; ++u)
            r[j][u] = load_raw<T, kVec<T>, true>(ys + (size_t)p * dim + col[u]);
      }
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (on[j])
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < kVec<T>; ++e)
              acc[u][e] = WEIGHTED ? __builtin_fmaf(wt[j], r[j][u].get(e), acc[u][e])
                                   : acc[u][e] + r[j][u].get(e);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (v0 + u * 64u + lane < nvec) {
        Raw<T> o;
        o.set_all(acc[u]);
        store_raw<T, kVec<T>, true>(row + col[u], o);
      }
  }
}

// `lanes` lanes per token, the whole wave (WIDE: the choices are scalars) or, for
// rows of fewer vectors, the power of two that holds them (65536 tokens of four
// 128 x bf16 rows, both gradients: 59 us, and 75 with a wave each).  Its
// row of dy is read once per K choices; the products with the choices' rows are
// summed per lane and then over the token's lanes, and the weighted rows are
// written on the way.
template <class T, int K, bool WIDE>
__global__ __launch_bounds__(kRowThreads) void k_expert_combine_backward(
    const T* __restrict__ dy, const T* __restrict__ ys, const int32_t* __restrict__ pos,
    const int32_t* __restrict__ src, const float* __restrict__ weights, int64_t tokens,
    uint32_t topk, int64_t rows, uint32_t dim, uint32_t nvec, uint32_t lanes,
    uint32_t token_blocks, T* __restrict__ dys, float* __restrict__ dweights) {
  const uint32_t block = block_index();
  if (block >= token_blocks) {
    zero_empty_rows(src, (int64_t)(block - token_blocks) * kZeroRows, rows, dim, dys);
    return;
  }
  if (WIDE) lanes = 64u;
  const uint32_t lane = threadIdx.x & (lanes - 1u);
  uint32_t mine = threadIdx.x / lanes;
  if (WIDE) mine = __builtin_amdgcn_readfirstlane(mine);
  const int64_t tok = (int64_t)block_index() * (kRowThreads / lanes) + mine;
  if (tok >= tokens) return;
  const T* row = dy + (size_t)tok * dim;
  for (uint32_t j0 = 0; j0 < topk; j0 += K) {
    float dot[K], wt[K];
    int32_t p[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const size_t c = (size_t)tok * topk + j0 + j;
      p[j] = j0 + j < topk ? pos[c] : -1;
      if ((uint32_t)p[j] >= (uint32_t)rows) p[j] = -1;
      wt[j] = p[j] >= 0 ? weights[c] : 0.0f;
      dot[j] = 0.0f;
    }
    for (uint32_t v = lane; v < nvec; v += lanes) {
      const uint32_t col = vec_column<T>(v, dim);
      const uint32_t skip = v * kVec<T> - col;  // elements the vector before has counted
      const Raw<T> g = load_raw<T>(row + col);
      Raw<T> r[K];
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (p[j] >= 0) r[j] = load_raw<T, kVec<T>, true>(ys + (size_t)p[j] * dim + col);
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (p[j] >= 0) {
          float out[kVec<T>];
#pragma unroll
          for (int e = 0; e < kVec<T>; ++e) {
            const float a = g.get(e);
            out[e] = wt[j] * a;
            dot[j] = (uint32_t)e >= skip ? __builtin_fmaf(a, r[j].get(e), dot[j]) : dot[j];
          }
          Raw<T> o;
          o.set_all(out);
          store_raw<T, kVec<T>, true>(dys + (size_t)p[j] * dim + col, o);
        }
    }
#pragma unroll
    for (int j = 0; j < K; ++j) {
      float d = dot[j];
      for (uint32_t o = lanes >> 1; o > 0; o >>= 1) d += __shfl_xor(d, (int)o, 64);
      if (lane == 0 && j0 + j < topk) dweights[(size_t)tok * topk + j0 + j] = d;
    }
  }
}

uint32_t vectors(uint32_t dim, int per) { return (dim + per - 1) / per; }

// Tokens of one block: about kRowVecs vectors per thread.
uint32_t tokens_per_block(uint32_t nvec) {
  const uint32_t t = (kRowThreads * kRowVecs) / nvec;
  return t < 1u ? 1u : t;
}

template <class T>
hipError_t dispatch_t(const void* x, const int32_t* pos, const int32_t* src, int64_t tokens,
                      int32_t topk, int64_t rows, int32_t dim, void* xs, hipStream_t s) {
  const uint32_t nvec = vectors((uint32_t)dim, kVec<T>), tpb = tokens_per_block(nvec);
  const bool wide = nvec >= kWideVecs;
  const uint32_t per = wide ? kRowThreads / 64 : tpb;
  const int64_t tb = (tokens + per - 1) / per, zb = (rows + kZeroRows - 1) / kZeroRows;
  if (tb + zb == 0) return hipSuccess;
  if (wide)
    hipLaunchKernelGGL((k_expert_dispatch_wide<T>), row_grid(tb + zb), dim3(kRowThreads),
                       0, s, static_cast<const T*>(x), pos, src, tokens, (uint32_t)topk, rows,
                       (uint32_t)dim, nvec, (uint32_t)tb, static_cast<T*>(xs));
  else
    hipLaunchKernelGGL((k_expert_dispatch<T>), row_grid(tb + zb), dim3(kRowThreads), 0, s,
                       static_cast<const T*>(x), pos, src, tokens, (uint32_t)topk, rows,
                       (uint32_t)dim, nvec, tpb, (uint32_t)tb, static_cast<T*>(xs));
  return hipGetLastError();
}

template <class T, int K>
hipError_t combine_k(const void* ys, const int32_t* pos, const float* weights, int64_t tokens,
                     int32_t topk, int64_t rows, int32_t dim, void* y, hipStream_t s) {
  const uint32_t nvec = vectors((uint32_t)dim, kVec<T>);
  const uint32_t tpb = tokens_per_block(nvec);
  const dim3 grid = row_grid((tokens + tpb - 1) / tpb);
  if (nvec >= kWideVecs) {
    const dim3 wgrid = row_grid((tokens + kRowThreads / 64 - 1) / (kRowThreads / 64));
    if (weights)
      hipLaunchKernelGGL((k_expert_combine_wide<T, K, true>), wgrid, dim3(kRowThreads), 0,
                         s, static_cast<const T*>(ys), pos, weights, tokens, (uint32_t)topk,
                         (uint32_t)rows, (uint32_t)dim, nvec, static_cast<T*>(y));
    else
      hipLaunchKernelGGL((k_expert_combine_wide<T, K, false>), wgrid, dim3(kRowThreads),
                         0, s, static_cast<const T*>(ys), pos, weights, tokens, (uint32_t)topk,
                         (uint32_t)rows, (uint32_t)dim, nvec, static_cast<T*>(y));
    return hipGetLastError();
  }
  if (weights)
    hipLaunchKernelGGL((k_expert_combine<T, K, true>), grid, dim3(kRowThreads), 0, s,
                       static_cast<const T*>(ys), pos, weights, tokens, (uint32_t)topk,
                       (uint32_t)rows, (uint32_t)dim, nvec, tpb, static_cast<T*>(y));
  else
    hipLaunchKernelGGL((k_expert_combine<T, K, false>), grid, dim3(kRowThreads), 0, s,
                       static_cast<const T*>(ys), pos, weights, tokens, (uint32_t)topk,
                       (uint32_t)rows, (uint32_t)dim, nvec, tpb, static_cast<T*>(y));
  return hipGetLastError();
}

template <class T>
hipError_t combine_t(const void* ys, const int32_t* pos, const float* weights, int64_t tokens,
                     int32_t topk, int64_t rows, int32_t dim, void* y, hipStream_t s) {
  if (topk == 1) return combine_k<T, 1>(ys, pos, weights, tokens, topk, rows, dim, y, s);
  if (topk == 2) return combine_k<T, 2>(ys, pos, weights, tokens, topk, rows, dim, y, s);
  if (topk <= 4) return combine_k<T, 4>(ys, pos, weights, tokens, topk, rows, dim, y, s);
  return combine_k<T, 8>(ys, pos, weights, tokens, topk, rows, dim, y, s);
}

template <class T, int K>
hipError_t combine_backward_k(const void* dy, const void* ys, const int32_t* pos,
                              const int32_t* src, const float* weights, int64_t tokens,
                              int32_t topk, int64_t rows, int32_t dim, void* dys,
                              float* dweights, hipStream_t s) {
  const uint32_t nvec = vectors((uint32_t)dim, kVec<T>);
  uint32_t lanes = 1;
  while (lanes < 64u && lanes < nvec) lanes *= 2;
  const int64_t per = kRowThreads / lanes;
  const int64_t tb = (tokens + per - 1) / per, zb = (rows + kZeroRows - 1) / kZeroRows;
  if (tb + zb == 0) return hipSuccess;
#define EMBTAB_CB(WIDE_)                                                                       \
  hipLaunchKernelGGL((k_expert_combine_backward<T, K, WIDE_>), row_grid(tb + zb),              \
                     dim3(kRowThreads), 0, s, static_cast<const T*>(dy),                       \
                     static_cast<const T*>(ys), pos, src, weights, tokens, (uint32_t)topk,     \
                     rows, (uint32_t)dim, nvec, lanes, (uint32_t)tb, static_cast<T*>(dys),     \
                     dweights)
  if (lanes == 64u) EMBTAB_CB(true);
  else EMBTAB_CB(false);
#undef EMBTAB_CB
  return hipGetLastError();
}

template <class T>
hipError_t combine_backward_t(const void* dy, const void* ys, const int32_t* pos,
                              const int32_t* src, const float* weights, int64_t tokens,
                              int32_t topk, int64_t rows, int32_t dim, void* dys,
                              float* dweights, hipStream_t s) {
#define EMBTAB_CB(K_) \
  combine_backward_k<T, K_>(dy, ys, pos, src, weights, tokens, topk, rows, dim, dys, dweights, s)
  if (topk == 1) return EMBTAB_CB(1);
  if (topk == 2) return EMBTAB_CB(2);
  if (topk <= 4) return EMBTAB_CB(4);
  return EMBTAB_CB(8);
#undef EMBTAB_CB
}

size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }

}  // namespace

// tile_hist [experts][tiles], then totals [experts]; at most 2^31 choices.
size_t expert_workspace_bytes(int64_t tokens, int32_t topk, int32_t experts) {
  const size_t tiles = (size_t)((tokens * topk + kTile - 1) / kTile);
  return align256(sizeof(uint32_t) * (size_t)experts * tiles) +
         align256(sizeof(uint32_t) * (size_t)experts);
}

hipError_t launch_expert_sort(const int64_t* ids, int64_t tokens, int32_t topk, int32_t experts,
                              int64_t capacity, int32_t* offsets, int32_t* src, int32_t* pos,
                              char* ws, hipStream_t s) {
  const uint32_t n = (uint32_t)(tokens * topk);
  const int64_t rows = capacity ? capacity * experts : (int64_t)n;
  // an empty batch still writes the offsets and the empty rows
  const uint32_t tiles = n ? (n + kTile - 1) / kTile : 1u;
  uint32_t* hist = reinterpret_cast<uint32_t*>(ws);
  uint32_t* totals = reinterpret_cast<uint32_t*>(
      ws + align256(sizeof(uint32_t) * (size_t)experts * (n ? tiles : 0u)));
  int nbits = 0;
  while ((1 << nbits) < experts) ++nbits;
  if (tiles > 1u) {
    hipLaunchKernelGGL(k_expert_hist, dim3(tiles), dim3(kTileThreads), 0, s, ids, n,
                       (uint32_t)experts, tiles, hist);
    if (tiles > kDirectTiles)
      hipLaunchKernelGGL(k_expert_scan, dim3((unsigned)experts), dim3(kTileThreads), 0, s, hist,
                         tiles, totals);
  }
  hipLaunchKernelGGL(k_expert_scatter, dim3(tiles), dim3(kTileThreads), 0, s, ids, n,
                     (uint32_t)experts, nbits, capacity, rows, tiles, hist, totals, offsets, src,
                     pos);
  return hipGetLastError();
}

hipError_t launch_expert_dispatch(const void* x, const int32_t* pos, const int32_t* src,
                                  int64_t tokens, int32_t topk, int64_t rows, int32_t dim,
                                  int32_t dtype, void* xs, hipStream_t s) {
  switch (dtype) {
    case EMB_F32: return dispatch_t<float>(x, pos, src, tokens, topk, rows, dim, xs, s);
    case EMB_BF16: return dispatch_t<bf16_t>(x, pos, src, tokens, topk, rows, dim, xs, s);
    default: return dispatch_t<f16_t>(x, pos, src, tokens, topk, rows, dim, xs, s);
  }
}

hipError_t launch_expert_combine(const void* ys, const int32_t* pos, const float* weights,
                                 int64_t tokens, int32_t topk, int64_t rows, int32_t dim,
                                 int32_t dtype, void* y, hipStream_t s) {
  if (tokens == 0) return hipSuccess;
  switch (dtype) {
    case EMB_F32: return combine_t<float>(ys, pos, weights, tokens, topk, rows, dim, y, s);
    case EMB_BF16: return combine_t<bf16_t>(ys, pos, weights, tokens, topk, rows, dim, y, s);
    default: return combine_t<f16_t>(ys, pos, weights, tokens, topk, rows, dim, y, s);
  }
}

hipError_t launch_expert_combine_backward(const void* dy, const void* ys, const int32_t* pos,
                                          const int32_t* src, const float* weights,
                                          int64_t tokens, int32_t topk, int64_t rows, int32_t dim,
                                          int32_t dtype, void* dys, float* dweights,
                                          hipStream_t s) {
  switch (dtype) {
    case EMB_F32:
      return combine_backward_t<float>(dy, ys, pos, src, weights, tokens, topk, rows, dim, dys,
                                       dweights, s);
    case EMB_BF16:
      return combine_backward_t<bf16_t>(dy, ys, pos, src, weights, tokens, topk, rows, dim, dys,
                                        dweights, s);
    default:
      return combine_backward_t<f16_t>(dy, ys, pos, src, weights, tokens, topk, rows, dim, dys,
                                       dweights, s);
  }
}

}  // namespace embtab
