// Grouped matrix products of 16-bit values in tiles of 256 x 256, for gfx950.
#pragma once

#include <utility>

#include "ffn_tiles.hpp"

namespace embtab {

constexpr int kWideO = 256, kWideK = 32;
constexpr int kRing = 5;                              // stages of LDS
constexpr int kWideValues = kWideO * kWideK;          // of one operand's stage
constexpr int kStageValues = 2 * kWideValues;

// Sixteen bytes of zeros that vectors past the end are taken from.
__device__ const uint32_t kZeroVector[4] = {0u, 0u, 0u, 0u};

// Loads of one operand straight into LDS: THREADS threads, kVecs vectors each a
// stage.  The place of a vector in LDS is the thread's own (the hardware puts a
// wave's 64 vectors one after another), so the turning that keeps the reads free
// of bank conflicts is in the address read from.
template <bool KC, int O, int THREADS>
struct StageLoads {
  static constexpr int kVecs = O * kWideK / 8 / THREADS;
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
    left[i] -= kWideK;
  }
};

// All but the last LEFT loads of every wave have landed, and every wave has its
// fragments: what they were read from may be written.
template <int LEFT>
__device__ inline void stage_landed() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(LEFT) : "memory");
}

__device__ inline uint32_t lds_address(const void* p) {
  typedef __attribute__((address_space(3))) const void lds_void;
  return (uint32_t)(uintptr_t)(lds_void*)p;
}

// A lane's fragments: 16 indexes from o0 + delta on, with delta a multiple of 16
// in the bits below o0's.  Bytes from the operand's stage on.
template <bool KC, int O>
struct Fragments {
  uint32_t base, turn;
  __device__ inline Fragments(uint32_t o0, uint32_t lane) {
    const uint32_t i = lane & 15u, q = lane >> 4;
    if (KC) {
      base = ((o0 + i) * kWideK + ((q ^ kc_turn(i)) << 3)) * 2;
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
    if (KC) return *(const lds_i16x8*)(uintptr_t)(base + stage + delta * (kWideK * 2));
    const uint32_t at = (turn ^ (delta * 2)) + (base + stage);
    const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(uintptr_t)at);
    const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_i16x4*)(uintptr_t)(at + 4 * O * 2));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

template <class T, bool A_KC, bool B_KC, int WM, int WN>
struct WideProduct {
  static constexpr int kThreads = 64 * WM * WN;
  static constexpr int FM = kWideO / WM / 16, FN = kWideO / WN / 16;
  typedef StageLoads<A_KC, kWideO, kThreads> LoadsA;
  typedef StageLoads<B_KC, kWideO, kThreads> LoadsB;
  static constexpr int kLoads = LoadsA::kVecs + LoadsB::kVecs;

  // acc[fm][fn]; delta_b(fn): of the wave's fragment fn
  template <class Delta>
  __device__ static inline void run(LoadsA& a, LoadsB& b, int64_t step_a, int64_t step_b,
                                    int32_t stages, const Fragments<A_KC, kWideO>& at_a,
                                    const Fragments<B_KC, kWideO>& at_b, Delta delta_b, uint16_t* lds,
                                    f32x4 (&acc)[FM][FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (stages <= 0) return;
    constexpr uint32_t kStage = kStageValues * 2, kOperand = kWideValues * 2;
    const uint32_t ring = lds_address(lds);
    const uint32_t mine = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
    const auto issue = [&](int load, uint32_t stage) {
      if (load < LoadsA::kVecs) {
        a.issue(load, stage + mine);
        a.advance(load, step_a);
      } else {
        b.issue(load - LoadsA::kVecs, stage + mine + kOperand);
        b.advance(load - LoadsA::kVecs, step_b);
      }
    };
    const auto after = [&](uint32_t stage) {
      return stage == ring + (kRing - 1) * kStage ? ring : stage + kStage;
    };
    i16x8 fa[2][FM], fb[2][FN];
#pragma unroll
    for (int s = 0; s < kRing - 1; ++s)
#pragma unroll
      for (int l = 0; l < kLoads; ++l) issue(l, ring + s * kStage);
    stage_landed<(kRing - 2) * kLoads>();
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[0][j] = at_b.read(ring + kOperand, delta_b(j));
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[0][i] = at_a.read(ring, i * 16);
    // A stage's matrix instructions, with the reads of the next stage's fragments
    // and the loads of a later one between them.
    constexpr int kReads = (FM + FN + FM - 3) / (FM - 2);  // a row, none in the last two
    const auto step = [&](auto set, uint32_t next, uint32_t in) {
      constexpr int now = decltype(set)::value;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int r = i * kReads; r < (i + 1) * kReads; ++r) {
          if (r < FN) fb[now ^ 1][r] = at_b.read(next + kOperand, delta_b(r));
          else if (r < FN + FM) fa[now ^ 1][r - FN] = at_a.read(next, (r - FN) * 16);
        }
        if ((i + 1) * kLoads / FM > i * kLoads / FM) issue(i * kLoads / FM, in);
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = mfma_16x16x32<T>(fb[now][j], fa[now][i], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // Two stages to a barrier.  At stage t's, the fragments of t are read, t + 1
    // and t + 2 have landed, t + 3 is on its way, and t + 4 and t + 5 are sent to
    // the places of t - 1 and t.
    uint32_t now = ring;
    for (int32_t t = 0; t < stages; t += 2) {
      stage_landed<kLoads>();
      const uint32_t next = after(now), second = after(next);
      const uint32_t before = now == ring ? ring + (kRing - 1) * kStage : now - kStage;
      step(std::integral_constant<int, 0>{}, next, before);
      if (t + 1 == stages) break;
      step(std::integral_constant<int, 1>{}, second, now);
      now = second;
    }
    // no load into LDS may outlive the block
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
};

template <class T, bool B_KC, class Epilogue, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void k_ffn_rows_wide(
    const Groups groups, const T* __restrict__ A, const T* __restrict__ B, int64_t K, int64_t N,
    int64_t b_stride, uint32_t col_tiles, const Epilogue epilogue) {
  typedef WideProduct<T, true, B_KC, WM, WN> Product;
  constexpr int FM = Product::FM, FN = Product::FN;
  __shared__ __attribute__((aligned(16))) uint16_t lds[kRing * kStageValues];
  constexpr int kCols = Epilogue::kDual ? kWideO / 2 : kWideO;
  RowTile t;
  if (!find_row_tile(groups, kWideO, col_tiles, block_index(), t)) return;
  const int64_t m0 = (int64_t)t.rt * kWideO, n0 = (int64_t)t.ct * kCols;
  const int64_t first = t.first, last = t.count - 1 - m0, last_n = N - 1 - n0;
  typename Product::LoadsA a;
  a.init_kc(A + (first + m0) * K, K,
            [&](uint32_t i) { return (int64_t)(i < last ? i : last) * K; });
  const T* be = B + t.expert * b_stride;
  typename Product::LoadsB b;
  if constexpr (B_KC)
    b.init_kc(be + n0 * K, K, [&](uint32_t i) {
      const uint32_t j = i % kCols;
      return ((int64_t)(j < last_n ? j : last_n) + (i / kCols) * N) * K;
    });
  else
    b.init_oc(be, N, n0, N, K);
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const uint32_t wm = wave % WM * (kWideO / WM), wn = wave / WM * (kCols / WN);
  const Fragments<true, kWideO> at_a(wm, lane);
  const Fragments<B_KC, kWideO> at_b(wn, lane);
  f32x4 acc[FM][FN];
  Product::run(a, b, kWideK * 2, B_KC ? kWideK * 2 : (int64_t)kWideK * 2 * N,
               (int32_t)((K + kWideK - 1) / kWideK), at_a, at_b,
               [](int j) {
                 return Epilogue::kDual
                            ? (uint32_t)(j % (FN / 2) * 16 + j / (FN / 2) * kCols)
                            : (uint32_t)(j * 16);
               },
               lds, acc);
  // What the epilogue reads for a row is on its way while the row before is
  // stored; rows and columns past the end read inside the matrix.
  constexpr int kOut = Epilogue::kDual ? FN / 2 : FN;
  typename Epilogue::Held held[2][kOut];
  const auto row_of = [&](int i) { return m0 + wm + i * 16 + (lane & 15u); };
  const auto col_of = [&](int j) { return n0 + wn + j * 16 + (lane >> 4) * 4; };
  const auto hold = [&](int i) {
    const int64_t m = row_of(i) < t.count ? row_of(i) : t.count - 1;
#pragma unroll
    for (int j = 0; j < kOut; ++j)
      held[i & 1][j] = epilogue.held(first + m, col_of(j) < N ? col_of(j) : N - 1);
  };
  hold(0);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    if (i + 1 < FM) hold(i + 1);
    const int64_t m = row_of(i);
    if (m >= t.count) continue;
#pragma unroll
    for (int j = 0; j < kOut; ++j) {
      const int64_t n = col_of(j);
      if (n >= N) continue;
      if constexpr (Epilogue::kDual)
        epilogue(first + m, n, acc[i][j], acc[i][j + FN / 2], held[i & 1][j]);
      else
        epilogue(first + m, n, acc[i][j], held[i & 1][j]);
    }
  }
}

template <class T, class Out, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void k_ffn_weights_wide(
    const WeightProducts<T> w, const WeightEpilogue<Out> out) {
  typedef WideProduct<T, false, false, WM, WN> Product;
  constexpr int FM = Product::FM, FN = Product::FN;
  __shared__ __attribute__((aligned(16))) uint16_t lds[kRing * kStageValues];
  WeightTile t;
  if (!find_weight_tile(w, block_index(), t)) return;
  const Group g = group_of(w.groups, t.expert);
  int64_t from, K;
  part_rows(g, w.parts, t.part, kWideK, from, K);
  const int64_t M = w.M[t.product], N = w.N[t.product];
  const int64_t m0 = (int64_t)t.rt * kWideO, n0 = (int64_t)t.ct * kWideO;
  typename Product::LoadsA a;
  typename Product::LoadsB b;
  a.init_oc(w.A[t.product] + (g.first + from) * M, M, m0, M, K);
  b.init_oc(w.B[t.product] + (g.first + from) * N, N, n0, N, K);
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const uint32_t wm = wave % WM * (kWideO / WM), wn = wave / WM * (kWideO / WN);
  f32x4 acc[FM][FN];
  Product::run(a, b, (int64_t)kWideK * 2 * M, (int64_t)kWideK * 2 * N,
               (int32_t)((K + kWideK - 1) / kWideK), Fragments<false, kWideO>(wm, lane),
               Fragments<false, kWideO>(wn, lane), [](int j) { return (uint32_t)(j * 16); }, lds, acc);
  const int64_t matrix = (int64_t)t.expert * w.parts + t.part;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m = m0 + wm + i * 16 + (lane & 15u);
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int64_t n = n0 + wn + j * 16 + (lane >> 4) * 4;
      if (n < N) out(t.product, matrix, M, N, m, n, acc[i][j]);
    }
  }
}

}  // namespace embtab
