// Grouped matrix products of 16-bit values in tiles of 256 x 256, for gfx950.
//
// Bound by the matrix instructions, which take three quarters of the time by
// themselves and keep the card at its power limit, and by what of the way from L2
// into LDS (10 TB/s in these kernels) they do not hide: the largest tile that eight
// waves hold in registers (128 x 64 results each) moves the fewest bytes, and both
// operands go from memory straight into LDS, in lines of 128 bytes.  (In stages of
// 32 k, with 64 bytes of a row at a time, L2 serves twice the requests for the same
// bytes: 32768 x 3328 x 3328, both with k innermost, 748 us against 718.)  16 experts
// of 3328 x 1664 with 32768 rows, bf16: forward 1.01 to 1.06 ms (1.0 PFLOP/s), backward
// 2.03 to 2.11 ms (1.0 PFLOP/s); a library's single products of the largest of these
// sizes run at 1.05, 0.98 and 0.69 PFLOP/s (both with k innermost, one, none).
// Without the loads the same kernels take 80% of the time, without the fragments'
// reads 85 to 95%, without either 75%.
//
// LDS holds two slots of 64 k.  Each half slot is a step of 32 matrix instructions
// a wave; the next step's fragments are read into a second set of registers between
// them.  One barrier a slot, between its halves: by then every wave has read the
// slot out and the other has landed, so the slot after the next is sent for.  (Two
// blocks a CU of 256 x 128, so that one's stores hide behind the other's products,
// move half as many bytes again: rows' products 5 to 20% slower.)
#pragma once

#include <utility>

#include "ffn_tiles.hpp"

namespace embtab {

constexpr int kWideO = 256, kWideK = 64, kHalfK = 32;
constexpr int kWideValues = kWideO * kWideK;  // of one operand's slot
constexpr int kSlotValues = 2 * kWideValues;

// Sixteen bytes of zeros that vectors past the end are taken from.
__device__ const uint32_t kZeroVector[4] = {0u, 0u, 0u, 0u};

__device__ inline uint32_t lds_address(const void* p) {
  typedef __attribute__((address_space(3))) const void lds_void;
  return (uint32_t)(uintptr_t)(lds_void*)p;
}

// A vector of 16 bytes to each lane's place behind the wave's `lds` (a byte
// address), from a lane's address or from a lane's offset behind a common one.  In
// assembly, which the compiler does not wait for: it would have every load land
// before each read of LDS.  No register is written.
__device__ inline void load_to_lds(const char* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds),
               "v"(p)
               : "m0");
}
__device__ inline void load_to_lds(const char* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds),
               "v"(offset), "s"(base)
               : "m0");
}
// The hardware wants five wait states between a vector instruction that writes a scalar
// register and a load that reads it, and the compiler, which keeps them between its own
// instructions, does not look into assembly.
template <class P>
__device__ inline const P* common_pointer(const P* p) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  asm volatile("s_nop 4" : "+s"(lo), "+s"(hi));
  return reinterpret_cast<const P*>((uintptr_t)(((uint64_t)hi << 32) | lo));
}

// All but the last LEFT loads of every wave have landed, and every wave has its
// fragments: what they were read from may be written.
template <int LEFT>
__device__ inline void stage_landed() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(LEFT) : "memory");
}

// The eight 16-byte pieces of a KC row of 128 bytes are turned by the row, so that
// the 16 lanes a read serves at once (ffn_tiles.hpp) meet no bank twice.
__device__ inline uint32_t wide_kc_turn(uint32_t row) { return (row >> 1) & 7u; }
// The same for the columns' operand, whose fragments take 4 of every 8 indexes.
__device__ inline uint32_t wide_kc_pair_turn(uint32_t row) {
  return ((row >> 1) & 1u) | ((row >> 2) & 6u);
}

// Loads of one operand straight into LDS: THREADS threads, kVecs vectors each a
// slot.  The place of a vector in LDS is the thread's own (the hardware puts a
// wave's 64 vectors one after another), so the turning is in the address read from;
// it is the same for all of a thread's vectors.
template <bool KC, bool PAIRS, int THREADS>
struct WideLoads {
  static constexpr int kVecs = kWideValues / 8 / THREADS;
  static constexpr int kRows = THREADS / (KC ? 8 : kWideO / 8);  // from a vector to the next
  const char* base;        // of the next slot, the same in every lane
  uint32_t offset[kVecs];  // bytes from there
  int64_t left;            // k values from the slot on

  // k of the thread's first vector in a slot; formed where it is needed, a register
  // less in the loop
  static __device__ inline uint32_t first_k() {
    uint32_t t = threadIdx.x;
    asm volatile("" : "+v"(t));
    if (!KC) return t / (kWideO / 8);
    return ((t & 7u) ^ (PAIRS ? wide_kc_pair_turn(t >> 3) : wide_kc_turn(t >> 3))) * 8;
  }

  // row(i): offset in values of the operand's index i, below 2^31 (KC)
  template <class T, class Row>
  __device__ inline void init_kc(const T* p, int64_t K, Row row) {
    base = reinterpret_cast<const char*>(common_pointer(p));
    left = K;
    const uint32_t k = first_k();
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      offset[i] = (uint32_t)(row((threadIdx.x >> 3) + i * kRows) + k) * 2;
  }
  // columns o0 on of `limit`, rows of ld values; one past the end takes the first
  template <class T>
  __device__ inline void init_oc(const T* p, int64_t ld, int64_t o0, int64_t limit, int64_t K) {
    base = reinterpret_cast<const char*>(common_pointer(p + o0));
    left = K;
    const uint32_t k = first_k();
    const uint32_t c = (threadIdx.x % (kWideO / 8) ^ oc_turn(k)) * 8;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      offset[i] = (uint32_t)((k + i * kRows) * ld + (o0 + c < limit ? c : 0)) * 2;
  }
  // Vector i of the next slot.  A slot past the end is not loaded, a vector past it
  // is zeros.
  __device__ inline void issue(int i, uint32_t lds) const {
    const uint32_t to = lds + i * THREADS * 16;
    if (left >= kWideK) {
      load_to_lds(base, offset[i], to);
    } else if (left > 0) {
      const int64_t k = first_k() + (KC ? 0 : i * kRows);
      load_to_lds(k < left ? base + offset[i] : reinterpret_cast<const char*>(kZeroVector), to);
    }
  }
  // step: bytes from one slot to the next
  __device__ inline void advance(int64_t step) {
    base += step;
    left -= kWideK;
  }
};

// A lane's fragments: 16 indexes from o0 + delta on, with delta a multiple of 16
// in the bits below o0's, and half 0 or 1 of a slot's k.  Bytes from the operand's
// slot on.
template <bool KC>
struct WideFragments {
  uint32_t base[2], turn;
  __device__ inline WideFragments(uint32_t o0, uint32_t lane) {
    const uint32_t i = lane & 15u, q = lane >> 4;
    if (KC) {
#pragma unroll
      for (uint32_t h = 0; h < 2; ++h)
        base[h] = (o0 + i) * (kWideK * 2) + (((h * 4 + q) ^ wide_kc_turn(i)) << 4);
      turn = 0;
    } else {
      const uint32_t k = q * 8 + (i >> 2);
      base[0] = k * kWideO * 2 + (i & 3u) * 8;
      base[1] = base[0] + kHalfK * kWideO * 2;
      turn = (o0 * 2) ^ (oc_turn(k) << 4);
    }
  }
  __device__ inline i16x8 read(uint32_t slot, int half, uint32_t delta) const {
    typedef __attribute__((address_space(3))) i16x8 lds_i16x8;
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
    if (KC) return *(const lds_i16x8*)(uintptr_t)(base[half] + slot + delta * (kWideK * 2));
    const uint32_t at = (turn ^ (delta * 2)) + (base[half] + slot);
    const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(uintptr_t)at);
    const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_i16x4*)(uintptr_t)(at + 4 * kWideO * 2));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

// The columns' fragments go in pairs that share 32 columns: the first takes columns
// 8 q to 8 q + 3 of them and the second the next four, so that a lane's results of
// both are eight neighbouring columns of a row.  (The reads of OC pairs meet two
// lanes in a bank.)
template <bool KC>
struct WidePairs {
  uint32_t base[2], turn;
  __device__ inline WidePairs(uint32_t o0, uint32_t lane) {
    const uint32_t i = lane & 15u, q = lane >> 4;
    if (KC) {
      const uint32_t r = (i >> 2) * 8 + (i & 3u);
#pragma unroll
      for (uint32_t h = 0; h < 2; ++h)
        base[h] = (o0 + r) * (kWideK * 2) + (((h * 4 + q) ^ wide_kc_pair_turn(r)) << 4);
      turn = 0;
    } else {
      const uint32_t k = q * 8 + (i >> 2);
      base[0] = k * kWideO * 2;
      base[1] = base[0] + kHalfK * kWideO * 2;
      turn = (o0 * 2 + (i & 3u) * 16) ^ (oc_turn(k) << 4);
    }
  }
  // fragment `second` of the pair that begins at o0 + delta
  __device__ inline i16x8 read(uint32_t slot, int half, uint32_t delta, int second) const {
    typedef __attribute__((address_space(3))) i16x8 lds_i16x8;
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
    if (KC)
      return *(const lds_i16x8*)(uintptr_t)(base[half] + slot +
                                             (delta + second * 4) * (kWideK * 2));
    const uint32_t at = (turn ^ (delta * 2)) + (base[half] + slot) + second * 8;
    const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(uintptr_t)at);
    const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_i16x4*)(uintptr_t)(at + 4 * kWideO * 2));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

template <class T, bool A_KC, bool B_KC, int WM, int WN>
struct WideProduct {
  static constexpr int kThreads = 64 * WM * WN;
  static constexpr int FM = kWideO / WM / 16, FN = kWideO / WN / 16;
  typedef WideLoads<A_KC, false, kThreads> LoadsA;
  typedef WideLoads<B_KC, true, kThreads> LoadsB;
  static constexpr int kLoads = LoadsA::kVecs + LoadsB::kVecs;

  // acc[fm][fn] over K; step_a, step_b: bytes from one slot to the next;
  // delta_b(p): of the wave's pair p of column fragments
  template <class Delta>
  __device__ static inline void run(LoadsA& a, LoadsB& b, int64_t step_a, int64_t step_b,
                                    int64_t K, const WideFragments<A_KC>& at_a,
                                    const WidePairs<B_KC>& at_b, Delta delta_b,
                                    uint16_t* lds, f32x4 (&acc)[FM][FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int32_t steps = (int32_t)((K + kHalfK - 1) / kHalfK);
    if (steps <= 0) return;
    constexpr uint32_t kSlot = kSlotValues * 2, kOperand = kWideValues * 2;
    const uint32_t first = lds_address(lds);
    const uint32_t mine = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
    const auto issue = [&](int load, uint32_t slot) {
      if (load < LoadsA::kVecs) a.issue(load, slot + mine);
      else b.issue(load - LoadsA::kVecs, slot + mine + kOperand);
    };
    const auto advance = [&] {
      a.advance(step_a);
      b.advance(step_b);
    };
    i16x8 fa[2][FM], fb[2][FN];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int l = 0; l < kLoads; ++l) issue(l, first + s * kSlot);
      advance();
    }
    if (steps > 2) stage_landed<kLoads>();
    else stage_landed<0>();
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[0][j] = at_b.read(first + kOperand, 0, delta_b(j / 2), j & 1);
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[0][i] = at_a.read(first, 0, i * 16);
    // A step's matrix instructions, and between them the reads of the next step's
    // fragments and, in a slot's second step, the loads of the slot after the next.
    constexpr int kReads = (FM + FN + FM - 3) / (FM - 2);  // a row, none in the last two
    const auto step = [&](auto place, uint32_t from, uint32_t in) {
      constexpr int now = decltype(place)::value, next = now ^ 1;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int r = i * kReads; r < (i + 1) * kReads; ++r) {
          if (r < FN) fb[next][r] = at_b.read(from + kOperand, next, delta_b(r / 2), r & 1);
          else if (r < FN + FM) fa[next][r - FN] = at_a.read(from, next, (r - FN) * 16);
        }
        if (now == 1)
#pragma unroll
          for (int l = i * kLoads / FM; l < (i + 1) * kLoads / FM; ++l) issue(l, in);
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = mfma_16x16x32<T>(fb[now][j], fa[now][i], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    uint32_t slot = first;
    for (int32_t t = 0; t < steps; t += 2) {
      step(std::integral_constant<int, 0>{}, slot, 0u);
      if (t + 1 == steps) break;
      stage_landed<0>();
      const uint32_t other = slot == first ? first + kSlot : first;
      step(std::integral_constant<int, 1>{}, other, slot);
      advance();
      slot = other;
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
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * kSlotValues];
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
  const WideFragments<true> at_a(wm, lane);
  const WidePairs<B_KC> at_b(wn, lane);
  f32x4 acc[FM][FN];
  Product::run(a, b, kWideK * 2, B_KC ? kWideK * 2 : (int64_t)kWideK * 2 * N,
               K, at_a, at_b,
               [](int p) { return (uint32_t)(p * (Epilogue::kDual ? kCols : 32)); }, lds, acc);
  // What the epilogue reads for a row is on its way while the row before is
  // stored; rows and columns past the end read inside the matrix.
  constexpr int kPairs = Epilogue::kDual ? FN / 4 : FN / 2;
  typename Epilogue::template Held<8> held[2][kPairs];
  const auto row_of = [&](int i) { return m0 + wm + i * 16 + (lane & 15u); };
  const auto col_of = [&](int p) { return n0 + wn + p * 32 + (lane >> 4) * 8; };
  const auto hold = [&](int i) {
    const int64_t m = row_of(i) < t.count ? row_of(i) : t.count - 1;
    const typename Epilogue::Row row = epilogue.row(first + m);
#pragma unroll
    for (int p = 0; p < kPairs; ++p)
      held[i & 1][p] = epilogue.template held<8>(row, col_of(p) < N ? col_of(p) : N - 1);
  };
  hold(0);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    if (i + 1 < FM) hold(i + 1);
    const int64_t m = row_of(i);
    if (m >= t.count) continue;
    const typename Epilogue::Row row = epilogue.row(first + m);
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      const int64_t n = col_of(p);
      if (n >= N) continue;
      float v[8], u[8];
      put4(v, acc[i][2 * p]);
      put4(v + 4, acc[i][2 * p + 1]);
      if constexpr (Epilogue::kDual) {
        put4(u, acc[i][2 * p + FN / 2]);
        put4(u + 4, acc[i][2 * p + FN / 2 + 1]);
        epilogue.store(row, n, v, u, held[i & 1][p]);
      } else {
        epilogue.store(row, n, v, held[i & 1][p]);
      }
    }
  }
}

template <class T, class Out, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void k_ffn_weights_wide(
    const WeightProducts<T> w, const WeightEpilogue<Out> out) {
  typedef WideProduct<T, false, false, WM, WN> Product;
  constexpr int FM = Product::FM, FN = Product::FN;
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * kSlotValues];
  WeightTile t;
  if (!find_weight_tile(w, block_index(), t)) return;
  const Group g = group_of(w.groups, t.expert);
  int64_t from, K;
  part_rows(g, w.parts, t.part, kHalfK, from, K);
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
               K, WideFragments<false>(wm, lane),
               WidePairs<false>(wn, lane), [](int p) { return (uint32_t)(p * 32); }, lds, acc);
  Out* to = out.out[t.product] + ((int64_t)t.expert * w.parts + t.part) * M * N;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m = m0 + wm + i * 16 + (lane & 15u);
    if (m >= M) continue;
#pragma unroll
    for (int p = 0; p < FN / 2; ++p) {
      const int64_t n = n0 + wn + p * 32 + (lane >> 4) * 8;
      float v[8];
      put4(v, acc[i][2 * p]);
      put4(v + 4, acc[i][2 * p + 1]);
      if (n < N) store_span(to + m * N + n, v, N - n);
    }
  }
}

}  // namespace embtab
