// Grouped matrix products for any width and alignment: tiles of 128 x 128 that
// pass through registers into LDS, for gfx950.
//
// C[m, n] = sum_k A(m, k) B(n, k) over one expert's rows.  An operand lies in
// memory with k innermost (KC) or with its own index innermost (OC):
//   forward        A = x, a (KC)      B = the weights [n, k] (KC)
//   to the input   A = dy, dgu (KC)   B = the weights [k, n] (OC)
//   weights        A = dgu, dy (OC)   B = x, a (OC), k over the expert's rows
// 16-bit values go to the matrix instructions as they are.  An fp32 value is the
// exact sum of three bf16 (8 bits each, rounded to nearest, so that the second is
// up to 2^-8 of the value and the third up to 2^-17), and of the nine products the
// six that can reach 2^-17 are taken, the smaller ones first: what is left out is
// below 2^-24 of a product, and the sums are in fp32.  That runs at a
// sixth of the bf16 rate, 2.6 times that of the fp32 matrix instructions.  (An
// infinite fp32 value leaves NaN in its sums.)
//
// A thread's vectors of the next step are on their way while the matrix
// instructions of this one run.  Rows and columns past the end are read inside
// the matrix and not stored; k past the end is zero on both sides.
//
// Several blocks on a CU hide each other's waits: 32 experts of 1664 x 1024 with 1024
// rows each take 1.68 ms forward in fp32 (200 TFLOP/s; the fp32 matrix instructions
// end at 157), and one block on a CU waits for most of its time (ffn_planes.hpp).
#pragma once

#include "ffn.hpp"

namespace embtab {

constexpr int kTileO = 128, kTileK = 32, kTileThreads = 256;

template <class T>
constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1;

// A KC plane has rows of 32 values, an OC plane rows of 128.  The four 16-byte
// pieces of a KC row are turned so that the 16 lanes that a 16-byte read serves at
// once (rows 0 to 3 and 12 to 15 of one piece with 4 to 11 of the next) meet no
// bank twice, the 32-byte pieces of an OC row so that eight rows of 32 bytes do not.
constexpr int kPlaneValues = kTileO * kTileK;

__device__ inline uint32_t kc_turn(uint32_t row) { return (row & 8u) ? 3u : 0u; }
__device__ inline uint32_t oc_turn(uint32_t k) { return ((k & 3u) | ((k >> 1) & 4u)) << 1; }

// One operand's share of a thread: its vectors of a tile, loaded and written.
template <class T, bool KC>
struct Staged {
  static constexpr int V = kVec<T>;
  static constexpr int kVecs = kTileO * kTileK / V / kTileThreads;
  static constexpr int kPer = (KC ? kTileK : kTileO) / V;  // vectors of a tile's row
  const T* p[kVecs];
  int32_t have[kVecs];  // OC: values of the vector inside the matrix
  bool whole;           // OC: the tile lies inside it
  Raw<T> r[kVecs];

  // row(i): memory offset of the operand's index i of the tile (KC)
  template <class Row>
  __device__ inline void init_kc(const T* base, Row row) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t v = threadIdx.x + i * kTileThreads;
      p[i] = base + row(v / kPer) + (v % kPer) * V;
    }
  }
  // index o0 .. of `limit`, rows of ld values (OC)
  __device__ inline void init_oc(const T* base, int64_t ld, int64_t o0, int64_t limit) {
    whole = o0 + kTileO <= limit;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t v = threadIdx.x + i * kTileThreads;
      const int64_t o = o0 + (v % kPer) * V;
      const int64_t n = limit - o;
      have[i] = n >= V ? V : n > 0 ? (int32_t)n : 0;
      p[i] = base + (int64_t)(v / kPer) * ld + (n > 0 ? o : 0);
    }
  }

  __device__ inline Raw<T> part(const T* q, int32_t n) const {  // n < V values, then zeros
    float f[V];
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = e < n ? to_f32(q[e]) : 0.0f;
    Raw<T> x;
    x.set_all(f);
    return x;
  }

  // k0 .. of K; ld as in init_oc.  A step inside the matrix takes no branch for
  // each vector, at whose end the compiler would wait for the load.
  __device__ inline void load(int64_t k0, int64_t K, int64_t ld) {
    if (k0 + kTileK <= K && (KC || whole)) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) r[i] = load_raw(p[i] + (KC ? k0 : k0 * ld));
      return;
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t v = threadIdx.x + i * kTileThreads;
      if (KC) {
        const int64_t n = K - k0 - (int64_t)(v % kPer) * V;
        if (n >= V) r[i] = load_raw(p[i] + k0);
        else r[i] = part(p[i] + k0, n > 0 ? (int32_t)n : 0);
      } else {
        const int32_t n = k0 + (v / kPer) < K ? have[i] : 0;
        if (n == V) r[i] = load_raw(p[i] + k0 * ld);
        else r[i] = part(p[i] + k0 * ld, n);
      }
    }
  }

  __device__ inline void write(uint16_t* lds) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t v = threadIdx.x + i * kTileThreads;
      const uint32_t row = v / kPer, c = (v % kPer) * V;
      const uint32_t at = KC ? row * kTileK + (((c >> 3) ^ kc_turn(row)) << 3) + (c & 7u)
                             : row * kTileO + (((c >> 3) ^ oc_turn(row)) << 3) + (c & 7u);
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<u4*>(lds + at) = u4{r[i].w[0], r[i].w[1], r[i].w[2], r[i].w[3]};
      } else {
        uint32_t words[3][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f32x2 v = {r[i].get(2 * h), r[i].get(2 * h + 1)};
#pragma unroll
          for (int q = 0; q < 3; ++q) {
            const uint32_t w =
                __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
            words[q][h] = w;
            v[0] -= __uint_as_float(w << 16);
            v[1] -= __uint_as_float(w & 0xFFFF0000u);
          }
        }
#pragma unroll
        for (int q = 0; q < 3; ++q)
          *reinterpret_cast<u2*>(lds + q * kPlaneValues + at) = u2{words[q][0], words[q][1]};
      }
    }
  }
};

// Lane's eight k values of one index: 16 indexes from o0 on, k = 8 (lane / 16) on.
template <bool KC>
__device__ inline i16x8 tile_fragment(const uint16_t* lds, uint32_t o0, uint32_t lane) {
  const uint32_t i = lane & 15u, q = lane >> 4;
  if (KC)
    return *reinterpret_cast<const i16x8*>(lds + (o0 + i) * kTileK + ((q ^ kc_turn(i)) << 3));
  i16x4 h[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t k = q * 8 + j * 4 + (i >> 2), c = o0 + (i & 3u) * 4;
    h[j] = lds_read_columns(lds + k * kTileO + (((c >> 3) ^ oc_turn(k)) << 3) + (c & 4u));
  }
  return __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
}

// The columns' operand is the first of the matrix instruction: a lane's four
// results are neighbouring columns of one row.
template <class T, bool A_KC, bool B_KC>
struct TileProduct {
  static constexpr int P = kPlanes<T>;
  static constexpr int kBuffers = P == 1 ? 2 : 1;
  static constexpr int kLds = kBuffers * 2 * P * kPlaneValues;  // 16-bit values

  // acc[fm][fn]; col(fn): the first index in the B tile of the wave's fragment fn
  template <class Col>
  __device__ static inline void run(Staged<T, A_KC>& a, Staged<T, B_KC>& b, int64_t K,
                                    int64_t lda, int64_t ldb, uint32_t wave_m, Col col,
                                    uint16_t* lds, f32x4 (&acc)[4][4]) {
    const uint32_t lane = threadIdx.x & 63u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (K <= 0) return;
    constexpr int kOne = P * kPlaneValues;
    a.load(0, K, lda);
    b.load(0, K, ldb);
    a.write(lds);
    b.write(lds + kOne);
    __syncthreads();
    uint32_t buffer = 0;
    for (int64_t k0 = 0; k0 < K; k0 += kTileK) {
      const bool more = k0 + kTileK < K;
      if (more) {
        a.load(k0 + kTileK, K, lda);
        b.load(k0 + kTileK, K, ldb);
      }
      const uint16_t* la = lds + buffer * 2 * kOne;
      const uint16_t* lb = la + kOne;
      i16x8 fb[P][4];
#pragma unroll
      for (int q = 0; q < P; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          fb[q][j] = tile_fragment<B_KC>(lb + q * kPlaneValues, col(j), lane);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        i16x8 fa[P];
#pragma unroll
        for (int q = 0; q < P; ++q)
          fa[q] = tile_fragment<A_KC>(la + q * kPlaneValues, wave_m + i * 16, lane);
        if constexpr (P == 1) {
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = mfma_16x16x32<T>(fb[0][j], fa[0], acc[i][j]);
        } else {
          constexpr int kSix[6][2] = {{2, 0}, {0, 2}, {1, 1}, {1, 0}, {0, 1}, {0, 0}};
#pragma unroll
          for (int s = 0; s < 6; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[i][j] = mfma_16x16x32<T>(fb[kSix[s][0]][j], fa[kSix[s][1]], acc[i][j]);
        }
      }
      if (!more) break;
      if (kBuffers == 1) __syncthreads();
      else buffer ^= 1u;
      a.write(lds + buffer * 2 * kOne);
      b.write(lds + buffer * 2 * kOne + kOne);
      __syncthreads();
    }
  }
};

// Row operands: C[row, n] over one expert's rows.  A: [rows, K]; B: the expert's
// weights, [n, K] (B_KC; both projections' rows for a dual epilogue) or [K, n].
template <class T, bool B_KC, class Epilogue>
__global__ __launch_bounds__(kTileThreads, 2) void k_ffn_rows(
    const Groups groups, const T* __restrict__ A, const T* __restrict__ B, int64_t K, int64_t N,
    int64_t b_stride, uint32_t col_tiles, const Epilogue epilogue) {
  typedef TileProduct<T, true, B_KC> Product;
  __shared__ __attribute__((aligned(16))) uint16_t lds[Product::kLds];
  constexpr int kCols = Epilogue::kDual ? kTileO / 2 : kTileO;
  RowTile t;
  if (!find_row_tile(groups, kTileO, col_tiles, block_index(), t)) return;
  const int64_t m0 = (int64_t)t.rt * kTileO, n0 = (int64_t)t.ct * kCols;
  const int64_t first = t.first, last = t.count - 1 - m0, last_n = N - 1 - n0;
  Staged<T, true> a;
  a.init_kc(A + (first + m0) * K,
            [&](uint32_t i) { return (int64_t)(i < last ? i : last) * K; });
  const T* be = B + t.expert * b_stride;
  Staged<T, B_KC> b;
  if constexpr (B_KC)
    b.init_kc(be + n0 * K, [&](uint32_t i) {
      const uint32_t j = i % kCols;
      return ((int64_t)(j < last_n ? j : last_n) + (i / kCols) * N) * K;
    });
  else
    b.init_oc(be, N, n0, N);
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const uint32_t wm = (wave & 1u) * 64u, wn = (wave >> 1) * (kCols / 2);
  f32x4 acc[4][4];
  Product::run(a, b, K, K, N, wm,
               [&](int j) {
                 return Epilogue::kDual ? wn + (j & 1) * 16u + (j >> 1) * (uint32_t)kCols
                                        : wn + j * 16u;
               },
               lds, acc);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + wm + i * 16 + (lane & 15u);
    if (m >= t.count) continue;
    const typename Epilogue::Row row = epilogue.row(first + m);
#pragma unroll
    for (int j = 0; j < (Epilogue::kDual ? 2 : 4); ++j) {
      const int64_t n = n0 + wn + j * 16 + (lane >> 4) * 4;
      if (n >= N) continue;
      const auto held = epilogue.template held<4>(row, n);
      float v[4], u[4];
      put4(v, acc[i][j]);
      if constexpr (Epilogue::kDual) {
        put4(u, acc[i][j + 2]);
        epilogue.store(row, n, v, u, held);
      } else {
        epilogue.store(row, n, v, held);
      }
    }
  }
}

// Weight gradients.
template <class T, class Out>
__global__ __launch_bounds__(kTileThreads, 2) void k_ffn_weights(const WeightProducts<T> w,
                                                                 const WeightEpilogue<Out> out) {
  typedef TileProduct<T, false, false> Product;
  __shared__ __attribute__((aligned(16))) uint16_t lds[Product::kLds];
  WeightTile t;
  if (!find_weight_tile(w, block_index(), t)) return;
  const Group g = group_of(w.groups, t.expert);
  int64_t from, K;
  part_rows(g, w.parts, t.part, kTileK, from, K);
  const int64_t M = w.M[t.product], N = w.N[t.product];
  const int64_t m0 = (int64_t)t.rt * kTileO, n0 = (int64_t)t.ct * kTileO;
  Staged<T, false> a, b;
  a.init_oc(w.A[t.product] + (g.first + from) * M, M, m0, M);
  b.init_oc(w.B[t.product] + (g.first + from) * N, N, n0, N);
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const uint32_t wm = (wave & 1u) * 64u, wn = (wave >> 1) * 64u;
  f32x4 acc[4][4];
  Product::run(a, b, K, M, N, wm, [&](int j) { return wn + j * 16u; }, lds, acc);
  Out* to = out.out[t.product] + ((int64_t)t.expert * w.parts + t.part) * M * N;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + wm + i * 16 + (lane & 15u);
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + wn + j * 16 + (lane >> 4) * 4;
      float v[4];
      put4(v, acc[i][j]);
      if (n < N) store_span(to + m * N + n, v, N - n);
    }
  }
}

}  // namespace embtab
