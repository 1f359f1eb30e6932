// Grouped matrix products of few rows (serving): the weights' bytes bound them,
// for gfx950.
//
// C[m, n] = sum_k A(m, k) B(n, k), both with k innermost.  A block takes 16
// columns (of both projections for a dual epilogue) of up to 64 rows of one
// expert, so that a weight is read once for all of them, and its four waves take
// turns in k; their sums are added in order through LDS.  Nothing else passes
// through LDS: a fragment of a matrix instruction is 16 or 32 neighbouring bytes
// of a row, in any order of k as long as both operands share it, so a lane loads
// its own, and the four lanes of a row read a line together.  fp32 takes the fp32
// matrix instructions, which keep up with the memory at these rows.
//
// 64 rows that use 15 of 32 experts, 3328 x 1664 bf16: 336 and 168 MB of weights in 71
// and 39 us (4.7 and 4.3 TB/s); 18 experts 72 and 41 us (the blocks' last round is
// fuller); 16 rows of 8 experts, 512 x 1024: 6.3 and 5.2 us, which are a few dependent
// waits.
#pragma once

#include "ffn.hpp"

namespace embtab {

constexpr int kFewRows = 64, kFewCols = 16, kFewWaves = 4;

template <class T>
struct FewStep {
  // k values of a step, and 16-byte vectors of a lane's part of it
  static constexpr int kVecs = sizeof(T) == 2 ? 2 : 1;
  static constexpr int kLane = kVec<T> * kVecs, kK = 4 * kLane;
  Raw<T> r[kVecs];

  __device__ inline void load(const T* p) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) r[v] = load_raw(p + v * kVec<T>);
  }
  // A row's values from k on, of K: a vector that ends past the row is the row's last
  // one, with zeros for what comes before its own first value (k counts once, in any
  // order).  No branch, at whose end the compiler would wait for the load (64 experts
  // of 479 x 1000 with 2 rows each, bf16: 67 us against 78).
  __device__ inline void load_end(const T* row, uint32_t k, int32_t K) {
    constexpr int kPerWord = 4 / (int)sizeof(T);
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int32_t at = (int32_t)k + v * kVec<T>, end = K - kVec<T>;
      const int32_t drop = at - end;  // values, none or less where the vector is inside
      r[v] = load_raw(row + (drop > 0 ? end : at));
#pragma unroll
      for (int w = 0; w < Raw<T>::kWords; ++w) {
        if (w * kPerWord < drop) r[v].w[w] &= (w + 1) * kPerWord > drop ? 0xFFFF0000u : 0u;
      }
    }
  }
  static __device__ inline f32x4 product(const FewStep& b, const FewStep& a, f32x4 c) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
        c = mfma_16x16x32<T>(__builtin_bit_cast(i16x8, b.r[v]), __builtin_bit_cast(i16x8, a.r[v]),
                             c);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(b.r[0].get(e), a.r[0].get(e), c, 0, 0, 0);
    }
    return c;
  }
};

// The wave's sums of MT x 16 rows and COLS sets of 16 columns.
template <class T, int MT, int COLS>
__device__ inline void few_sums(const T* const (&a)[MT], const T* const (&b)[COLS], int32_t K,
                                uint32_t wave, uint32_t q, f32x4 (&acc)[MT][COLS]) {
  typedef FewStep<T> Step;
  // Steps whose loads are under way together: two, in 16 waves a CU (32 rows of 18
  // experts, 3328 x 1664 bf16: 72 + 41 us against 78 + 41 with four in 12 waves, the
  // weights' loads past the caches)
  constexpr int kAhead = 2;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int c = 0; c < COLS; ++c) acc[i][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const uint32_t lane_k = q * Step::kLane;
  int32_t k0 = wave * Step::kK;
  constexpr int32_t kTurn = kFewWaves * Step::kK;
  for (; k0 + (kAhead - 1) * kTurn + Step::kK <= K; k0 += kAhead * kTurn) {
    Step sa[kAhead][MT], sb[kAhead][COLS];
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
#pragma unroll
      for (int c = 0; c < COLS; ++c) sb[s][c].load(b[c] + k0 + s * kTurn + lane_k);
#pragma unroll
      for (int i = 0; i < MT; ++i) sa[s][i].load(a[i] + k0 + s * kTurn + lane_k);
    }
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int c = 0; c < COLS; ++c) acc[i][c] = Step::product(sb[s][c], sa[s][i], acc[i][c]);
  }
  const auto products = [&](const Step (&sa)[MT], const Step (&sb)[COLS]) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int c = 0; c < COLS; ++c) acc[i][c] = Step::product(sb[c], sa[i], acc[i][c]);
  };
  for (; k0 + Step::kK <= K; k0 += kTurn) {
    Step sa[MT], sb[COLS];
#pragma unroll
    for (int c = 0; c < COLS; ++c) sb[c].load(b[c] + (k0 + lane_k));
#pragma unroll
    for (int i = 0; i < MT; ++i) sa[i].load(a[i] + (k0 + lane_k));
    products(sa, sb);
  }
  if (k0 < K) {  // the last turn's, of one wave
    Step sa[MT], sb[COLS];
#pragma unroll
    for (int c = 0; c < COLS; ++c) sb[c].load_end(b[c], k0 + lane_k, K);
#pragma unroll
    for (int i = 0; i < MT; ++i) sa[i].load_end(a[i], k0 + lane_k, K);
    products(sa, sb);
  }
}

template <class T, int MT, class Epilogue>
__device__ inline void few_rows(const RowTile& t, const T* __restrict__ A,
                                const T* __restrict__ B, int32_t K, int64_t N, int64_t b_stride,
                                const Epilogue& epilogue, f32x4* lds) {
  constexpr int COLS = Epilogue::kDual ? 2 : 1;
  const uint32_t lane = threadIdx.x & 63u, q = lane >> 4, i16 = lane & 15u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)t.rt * kFewRows, n0 = (int64_t)t.ct * kFewCols;
  const int64_t last = t.count - 1 - m0, last_n = N - 1 - n0;
  const T *a[MT], *b[COLS];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t m = i * 16 + i16;
    a[i] = A + (t.first + m0 + (m < last ? m : last)) * K;
  }
#pragma unroll
  for (int c = 0; c < COLS; ++c)
    b[c] = B + t.expert * b_stride + (n0 + ((int64_t)i16 < last_n ? i16 : last_n) + c * N) * K;
  f32x4 acc[MT][COLS];
  few_sums<T, MT, COLS>(a, b, K, wave, q, acc);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int c = 0; c < COLS; ++c) lds[((wave * MT + i) * COLS + c) * 64 + lane] = acc[i][c];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    if (i % kFewWaves != (int)wave) continue;
    f32x4 sum[COLS];
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
      sum[c] = lds[(i * COLS + c) * 64 + lane];
#pragma unroll
      for (int w = 1; w < kFewWaves; ++w) sum[c] += lds[((w * MT + i) * COLS + c) * 64 + lane];
    }
    const int64_t m = m0 + i * 16 + i16, n = n0 + q * 4;
    if (m >= t.count || n >= N) continue;
    const typename Epilogue::Row row = epilogue.row(t.first + m);
    const auto held = epilogue.template held<4>(row, n);
    float v[4], u[4];
    put4(v, sum[0]);
    if constexpr (Epilogue::kDual) {
      put4(u, sum[1]);
      epilogue.store(row, n, v, u, held);
    } else {
      epilogue.store(row, n, v, held);
    }
  }
}

template <class T, class Epilogue>
__global__ __launch_bounds__(64 * kFewWaves, 4) void k_ffn_few_rows(
    const Groups groups, const T* __restrict__ A, const T* __restrict__ B, int32_t K, int64_t N,
    int64_t b_stride, uint32_t col_tiles, const Epilogue epilogue) {
  __shared__ f32x4 lds[kFewWaves * 4 * (Epilogue::kDual ? 2 : 1) * 64];
  RowTile t;
  if (!find_row_tile(groups, kFewRows, col_tiles, block_index(), t)) return;
  const int64_t rows = t.count - (int64_t)t.rt * kFewRows;
  if (rows <= 16) few_rows<T, 1>(t, A, B, K, N, b_stride, epilogue, lds);
  else if (rows <= 32) few_rows<T, 2>(t, A, B, K, N, b_stride, epilogue, lds);
  else few_rows<T, 4>(t, A, B, K, N, b_stride, epilogue, lds);
}

}  // namespace embtab
