// Grouped matrix products of fp32 values that are cut into three bf16 planes
// before, for gfx950.
//
// The tiles of ffn_tiles.hpp cut an fp32 value into bf16 each time it enters a
// tile, which costs a vector instruction for every matrix instruction's cycle.
// Where a value enters several tiles its planes are made once instead (6 bytes a
// value, rows padded with zeros to a multiple of 8, so that any width and
// alignment will do), the products' results leave theirs as they are stored, and
// the tiles load planes straight into LDS, three or four stages ahead, which a block
// alone on its CU needs, or two where two blocks share one.  The six products and their order are those of ffn_tiles.hpp.
//
// 4096 x 479 from 1000: 36 us (the tiles above 50), forward of that size 99 us, of
// which the outputs' and planes' 92 MB are 15; a stage takes 1.0 to 1.2 us where its
// matrix instructions take 0.4 (64 rows) and 0.7 (128 rows): planes move 6 bytes a
// value, 10 TB/s over the card.
#pragma once

#include "ffn_wide.hpp"

namespace embtab {

__host__ __device__ inline int64_t padded(int64_t n) { return (n + 7) & ~(int64_t)7; }

// An fp32 matrix's planes: [3][rows][ld] bf16.
struct Planes {
  bf16_t* p;
  int64_t ld, size;  // values of a row, of a plane
};

__device__ inline void cut_planes(float a, float b, uint32_t (&w)[3]) {
  f32x2 v = {a, b};
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    w[q] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    v[0] -= __uint_as_float(w[q] << 16);
    v[1] -= __uint_as_float(w[q] & 0xFFFF0000u);
  }
}

// The planes of the first `have` of four values, then zeros up to `to` of them.
__device__ inline void store_planes4(const Planes& o, int64_t at, float (&v)[4], int64_t have,
                                     int64_t to) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = i < have ? v[i] : 0.0f;
  uint32_t lo[3], hi[3];
  cut_planes(v[0], v[1], lo);
  cut_planes(v[2], v[3], hi);
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    uint16_t* p = reinterpret_cast<uint16_t*>(o.p) + q * o.size + at;
    if (to >= 4) {
      *reinterpret_cast<u2_at2*>(p) = u2{lo[q], hi[q]};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < to) p[i] = (uint16_t)((i < 2 ? lo[q] : hi[q]) >> (16 * (i & 1)));
    }
  }
}

// Matrices cut in one launch.
constexpr int kMaxCuts = 5;
struct Cuts {
  const float* src[kMaxCuts];
  Planes dst[kMaxCuts];
  int64_t width[kMaxCuts];
  int64_t first[kMaxCuts + 1];  // vectors of 8 values before each matrix
  int32_t count;
};

// (a template, so that of the sources that include this only the fp32 one holds it)
template <class T>
__global__ __launch_bounds__(256) void k_ffn_cut(const Cuts c) {
  const int64_t v = (int64_t)block_index() * 256 + threadIdx.x;
  if (v >= c.first[c.count]) return;
  int m = 0;
#pragma unroll
  for (int i = 1; i < kMaxCuts; ++i) m += i < c.count && v >= c.first[i];
  const float* src = c.src[0];
  Planes dst = c.dst[0];
  int64_t width = c.width[0], first = 0;
#pragma unroll
  for (int i = 1; i < kMaxCuts; ++i)
    if (i == m) {
      src = c.src[i];
      dst = c.dst[i];
      width = c.width[i];
      first = c.first[i];
    }
  const int64_t per = dst.ld / 8, row = (v - first) / per, col = (v - first - row * per) * 8;
  const float* p = src + row * width + col;
  float f[8];
  if (col + 8 <= width) {
    const Raw<float> a = load_raw(p), b = load_raw(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = a.get(i);
      f[4 + i] = b.get(i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = col + i < width ? p[i] : 0.0f;
  }
  uint32_t w[4][3];
#pragma unroll
  for (int i = 0; i < 4; ++i) cut_planes(f[2 * i], f[2 * i + 1], w[i]);
#pragma unroll
  for (int q = 0; q < 3; ++q)
    *reinterpret_cast<u4*>(dst.p + q * dst.size + row * dst.ld + col) =
        u4{w[0][q], w[1][q], w[2][q], w[3][q]};
}

// ---------------------------------------------------------------- epilogues
// All also cover the columns that pad a row of planes, which can begin a tile of their
// own.  kReads: whether it reads as much as it stores.
struct ActPlanesEpilogue : ActEpilogue<float> {
  static constexpr bool kReads = false;
  Planes planes;  // of a
  struct Row {
    ActEpilogue<float>::Row values;
    int64_t at;
  };
  __host__ __device__ inline int64_t columns() const { return planes.ld; }
  __device__ inline Row row(int64_t r) const {
    return {ActEpilogue<float>::row(r), r * planes.ld};
  }
  __device__ inline NothingHeld held4(const Row&, int64_t) const { return {}; }
  __device__ inline void store4(const Row& r, int64_t n, const float (&g)[4], const float (&u)[4],
                                const NothingHeld&) const {
    float p[4];
    product(r.values, n, g, u, p);
    store_planes4(planes, r.at + n, p, width - n, planes.ld - n);
  }
};

struct ActGradPlanesEpilogue : ActGradEpilogue<float> {
  static constexpr bool kReads = true;
  Planes planes;  // of dgu, which is not stored itself
  struct Row {
    ActGradEpilogue<float>::Row values;
    int64_t at;
  };
  __host__ __device__ inline int64_t columns() const { return planes.ld - width; }
  __device__ inline Row row(int64_t r) const {
    return {ActGradEpilogue<float>::row(r), r * planes.ld};
  }
  __device__ inline Held<4> held4(const Row& r, int64_t n) const { return held<4>(r.values, n); }
  __device__ inline void store4(const Row& r, int64_t n, const float (&da)[4],
                                const Held<4>& h) const {
    float dg[4], du[4];
    gradients(da, h, dg, du);
    store_planes4(planes, r.at + n, dg, width - n, width - n);
    store_planes4(planes, r.at + width + n, du, width - n, planes.ld - width - n);
  }
};

struct StorePlanesEpilogue : StoreEpilogue<float> {
  static constexpr bool kReads = false;
  __host__ __device__ inline int64_t columns() const { return width; }
  __device__ inline NothingHeld held4(const Row&, int64_t) const { return {}; }
  __device__ inline void store4(const Row& r, int64_t n, const float (&v)[4],
                                const NothingHeld& h) const {
    store(r, n, v, h);
  }
};

// ---------------------------------------------------------------- product
template <bool KC, int O, int THREADS>
struct StageLoads {
  static constexpr int kVecs = O * kHalfK / 8 / THREADS;
  const char* p[kVecs];
  int32_t left[kVecs];  // k values (KC) or rows (OC) from the vector's first on

  // row(i): offset in values of the operand's index i (KC)
  template <class T, class Row>
  __device__ inline void init_kc(const T* base, int64_t K, Row row) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t v = threadIdx.x + i * THREADS, r = v >> 2;
      const uint32_t c = (v & 3u) ^ kc_turn(r);
      p[i] = reinterpret_cast<const char*>(base + row(r) + c * 8);
      left[i] = (int32_t)K - (int32_t)(c * 8);
    }
  }
  template <class T>
  __device__ inline void init_oc(const T* base, int64_t ld, int64_t o0, int64_t limit,
                                 int64_t K) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t v = threadIdx.x + i * THREADS, k = v / (O / 8);
      const uint32_t c = v % (O / 8) ^ oc_turn(k);
      const int64_t o = o0 + c * 8;
      p[i] = reinterpret_cast<const char*>(base + (int64_t)k * ld + (o < limit ? o : 0));
      left[i] = o < limit ? (int32_t)K - (int32_t)k : 0;
    }
  }
  // Vector i of the next stage, `offset` bytes on, to the wave's place `lds` (a byte
  // address).  In assembly, which the compiler does not wait for: it would have
  // every load land before each read of LDS.  No register is written.
  __device__ inline void issue(int i, uint32_t lds, int64_t offset = 0) const {
    const char* q = left[i] > 0 ? p[i] + offset : reinterpret_cast<const char*>(kZeroVector);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(
                     lds + i * THREADS * 16),
                 "v"(q)
                 : "m0");
  }
  // step: bytes from one stage to the next
  __device__ inline void advance(int i, int64_t step) {
    p[i] += step;
    left[i] -= kHalfK;
  }
};

template <bool KC, int O>
struct Fragments {
  uint32_t base, turn;
  __device__ inline Fragments(uint32_t o0, uint32_t lane) {
    const uint32_t i = lane & 15u, q = lane >> 4;
    if (KC) {
      base = ((o0 + i) * kHalfK + ((q ^ kc_turn(i)) << 3)) * 2;
      turn = 0;
    } else {
      const uint32_t k = q * 8 + (i >> 2);
      base = k * O * 2 + (i & 3u) * 8;
      turn = (o0 * 2) ^ (oc_turn(k) << 4);
    }
  }
  __device__ inline i16x8 read(uint32_t stage, uint32_t delta) const {
    typedef __attribute__((address_space(3))) i16x8 lds_i16x8;
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
    if (KC) return *(const lds_i16x8*)(uintptr_t)(base + stage + delta * (kHalfK * 2));
    const uint32_t at = (turn ^ (delta * 2)) + (base + stage);
    const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(uintptr_t)at);
    const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_i16x4*)(uintptr_t)(at + 4 * O * 2));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

// Tiles of OM x 128 by waves of 64 x 32: 128 rows by eight waves and a ring of
// three stages, 64 rows by four and a ring of four (144 KB of LDS either way) or, two
// blocks a CU, of two.  A stage holds 32 k of both operands' planes.
template <bool A_KC, bool B_KC, int OM, int RING>
struct PlaneProduct {
  static constexpr int WM = OM / 64, WN = 4, kThreads = 64 * WM * WN, kRing = RING;
  static constexpr int FM = 4, FN = 2;
  typedef StageLoads<A_KC, OM, kThreads> LoadsA;
  typedef StageLoads<B_KC, kTileO, kThreads> LoadsB;
  static constexpr int kLoads = 3 * (LoadsA::kVecs + LoadsB::kVecs);
  static constexpr uint32_t kPlaneA = OM * kHalfK * 2, kPlaneB = kTileO * kHalfK * 2;
  static constexpr uint32_t kStage = 3 * (kPlaneA + kPlaneB);

  // size_a, size_b: bytes of a plane
  template <class Delta>
  __device__ static inline void run(LoadsA& a, LoadsB& b, int64_t step_a, int64_t step_b,
                                    int64_t size_a, int64_t size_b, int32_t stages,
                                    const Fragments<A_KC, OM>& at_a,
                                    const Fragments<B_KC, kTileO>& at_b, Delta delta_b,
                                    uint16_t* lds, f32x4 (&acc)[FM][FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (stages <= 0) return;
    const uint32_t ring = lds_address(lds);
    const uint32_t mine = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
    const auto issue = [&](int load, uint32_t stage) {  // of kLoads: a's vectors, then b's
      if (load < 3 * LoadsA::kVecs) {
        const int q = load % 3, l = load / 3;
        a.issue(l, stage + mine + q * kPlaneA, q * size_a);
        if (q == 2) a.advance(l, step_a);
      } else {
        const int q = load % 3, l = load / 3 - LoadsA::kVecs;
        b.issue(l, stage + mine + 3 * kPlaneA + q * kPlaneB, q * size_b);
        if (q == 2) b.advance(l, step_b);
      }
    };
    const auto after = [&](uint32_t stage) {
      return stage == ring + (kRing - 1) * kStage ? ring : stage + kStage;
    };
    i16x8 fa[2][FM][3], fb[2][FN][3];
    const auto read = [&](int set, int r, uint32_t stage) {  // fragment r: b's, then a's
      const int q = r % 3, f = r / 3;
      if (f < FN) fb[set][f][q] = at_b.read(stage + 3 * kPlaneA + q * kPlaneB, delta_b(f));
      else fa[set][f - FN][q] = at_a.read(stage + q * kPlaneA, (f - FN) * 16);
    };
    constexpr int kReads = 3 * (FM + FN);
#pragma unroll
    for (int s = 0; s < kRing; ++s)
#pragma unroll
      for (int l = 0; l < kLoads; ++l) issue(l, ring + s * kStage);
    stage_landed<(kRing - 1) * kLoads>();
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(0, r, ring);
    constexpr int kSix[6][2] = {{2, 0}, {0, 2}, {1, 1}, {1, 0}, {0, 1}, {0, 0}};
    // At a step, its fragments are read by every wave, the next stage has landed, and
    // its own place takes the stage after the ring's last.  Loads and the next
    // fragments' reads go between the matrix instructions.
    const auto step = [&](auto set, uint32_t now) {
      constexpr int cur = decltype(set)::value;
      stage_landed<(kRing - 2) * kLoads>();
      const uint32_t next = after(now);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int h = 0; h < 3; ++h) {
          const int g = i * 3 + h;  // of 12 groups of four matrix instructions
#pragma unroll
          for (int r = 2 * g; r < 2 * g + 2; ++r)
            if (r < kReads) read(cur ^ 1, r, next);
          if (g < kLoads) issue(g, now);
#pragma unroll
          for (int s = 2 * h; s < 2 * h + 2; ++s)
#pragma unroll
            for (int j = 0; j < FN; ++j)
              acc[i][j] = mfma_16x16x32<bf16_t>(fb[cur][j][kSix[s][0]], fa[cur][i][kSix[s][1]],
                                                acc[i][j]);
          __builtin_amdgcn_sched_barrier(0);
        }
      return next;
    };
    static_assert(kReads <= 24 && kLoads <= 12, "all of them inside a step");
    uint32_t now = ring;
    for (int32_t t = 0; t < stages; t += 2) {
      now = step(std::integral_constant<int, 0>{}, now);
      if (t + 1 == stages) break;
      now = step(std::integral_constant<int, 1>{}, now);
    }
    // no load into LDS may outlive the block
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
};

// As k_ffn_rows, from planes: A [rows, K], B the expert's weights.
template <bool B_KC, class Epilogue, int OM, int RING>
__global__ __launch_bounds__(OM * 4) void k_ffn_rows_planes(
    const Groups groups, const Planes A, const Planes B, int64_t N, int64_t b_rows,
    uint32_t col_tiles, const Epilogue epilogue) {
  typedef PlaneProduct<true, B_KC, OM, RING> Product;
  constexpr int FM = Product::FM, FN = Product::FN;
  __shared__ __attribute__((aligned(16))) uint16_t lds[Product::kRing * Product::kStage / 2];
  constexpr int kCols = Epilogue::kDual ? kTileO / 2 : kTileO;
  RowTile t;
  if (!find_row_tile(groups, OM, col_tiles, block_index(), t)) return;
  const int64_t m0 = (int64_t)t.rt * OM, n0 = (int64_t)t.ct * kCols, K = A.ld;
  const int64_t first = t.first, last = t.count - 1 - m0, last_n = N - 1 - n0;
  typename Product::LoadsA a;
  a.init_kc(A.p + (first + m0) * A.ld, K,
            [&](uint32_t i) { return (int64_t)(i < last ? i : last) * A.ld; });
  const bf16_t* be = B.p + t.expert * b_rows * B.ld;
  typename Product::LoadsB b;
  if constexpr (B_KC)
    b.init_kc(be + n0 * B.ld, K, [&](uint32_t i) {
      const uint32_t j = i % kCols;
      return ((int64_t)(j < last_n ? j : last_n) + (i / kCols) * N) * B.ld;
    });
  else
    b.init_oc(be, B.ld, n0, B.ld, b_rows);
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const uint32_t wm = wave % Product::WM * 64;
  const uint32_t wn = wave / Product::WM * (kCols / Product::WN);
  f32x4 acc[FM][FN];
  Product::run(a, b, kHalfK * 2, B_KC ? kHalfK * 2 : kHalfK * 2 * B.ld, A.size * 2, B.size * 2,
               (int32_t)((K + kHalfK - 1) / kHalfK), Fragments<true, OM>(wm, lane),
               Fragments<B_KC, kTileO>(wn, lane),
               [](int j) {
                 return Epilogue::kDual
                            ? (uint32_t)(j % (FN / 2) * 16 + j / (FN / 2) * kCols)
                            : (uint32_t)(j * 16);
               },
               lds, acc);
  // What the epilogue reads is on its way before the first row is stored; rows and
  // columns past the end read inside the matrix.
  constexpr int kOut = Epilogue::kDual ? FN / 2 : FN;
  const auto row_of = [&](int i) { return m0 + wm + i * 16 + (lane & 15u); };
  const auto col_of = [&](int j) { return n0 + wn + j * 16 + (lane >> 4) * 4; };
  decltype(epilogue.held4(epilogue.row(0), 0)) held[FM][kOut];
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const auto row = epilogue.row(first + (row_of(i) < t.count ? row_of(i) : t.count - 1));
#pragma unroll
    for (int j = 0; j < kOut; ++j)
      held[i][j] = epilogue.held4(row, col_of(j) < N ? col_of(j) : N - 1);
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    if (row_of(i) >= t.count) continue;
    const typename Epilogue::Row row = epilogue.row(first + row_of(i));
#pragma unroll
    for (int j = 0; j < kOut; ++j) {
      if (col_of(j) >= epilogue.columns()) continue;
      float v[4], u[4];
      put4(v, acc[i][j]);
      if constexpr (Epilogue::kDual) {
        put4(u, acc[i][j + FN / 2]);
        epilogue.store4(row, col_of(j), v, u, held[i][j]);
      } else {
        epilogue.store4(row, col_of(j), v, held[i][j]);
      }
    }
  }
}

// As k_ffn_weights, from planes.
struct WeightPlanes {
  Planes A[2], B[2];
};
template <class Out, int OM>
__global__ __launch_bounds__(OM * 4) void k_ffn_weights_planes(
    const WeightProducts<float> w, const WeightPlanes planes, const WeightEpilogue<Out> out) {
  typedef PlaneProduct<false, false, OM, 3> Product;
  constexpr int FM = Product::FM, FN = Product::FN;
  __shared__ __attribute__((aligned(16))) uint16_t lds[Product::kRing * Product::kStage / 2];
  WeightTile t;
  if (!find_weight_tile(w, block_index(), t)) return;
  const Group g = group_of(w.groups, t.expert);
  int64_t from, K;
  part_rows(g, w.parts, t.part, kHalfK, from, K);
  const int64_t M = w.M[t.product], N = w.N[t.product];
  const int64_t m0 = (int64_t)t.rt * OM, n0 = (int64_t)t.ct * kTileO;
  const Planes A = t.product ? planes.A[1] : planes.A[0];
  const Planes B = t.product ? planes.B[1] : planes.B[0];
  typename Product::LoadsA a;
  typename Product::LoadsB b;
  a.init_oc(A.p + (g.first + from) * A.ld, A.ld, m0, A.ld, K);
  b.init_oc(B.p + (g.first + from) * B.ld, B.ld, n0, B.ld, K);
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const uint32_t wm = wave % Product::WM * 64;
  const uint32_t wn = wave / Product::WM * (kTileO / Product::WN);
  f32x4 acc[FM][FN];
  Product::run(a, b, kHalfK * 2 * A.ld, kHalfK * 2 * B.ld, A.size * 2, B.size * 2,
               (int32_t)((K + kHalfK - 1) / kHalfK), Fragments<false, OM>(wm, lane),
               Fragments<false, kTileO>(wn, lane), [](int j) { return (uint32_t)(j * 16); }, lds,
               acc);
  Out* to = out.out[t.product] + ((int64_t)t.expert * w.parts + t.part) * M * N;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m = m0 + wm + i * 16 + (lane & 15u);
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int64_t n = n0 + wn + j * 16 + (lane >> 4) * 4;
      float v[4];
      put4(v, acc[i][j]);
      if (n < N) store_span(to + m * N + n, v, N - n);
    }
  }
}

}  // namespace embtab
