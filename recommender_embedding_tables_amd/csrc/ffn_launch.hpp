// Launches of the experts' gated feed-forward for one element type (included by
// one source per type).
#pragma once

#include "ffn_few.hpp"
#include "ffn_planes.hpp"

namespace embtab {

namespace {

// Weight gradients with fewer blocks than this cut the experts' rows into parts,
// whose sums a second kernel adds in order.
constexpr int64_t kWeightBlocks = 512;
constexpr int64_t kMaxParts = 16, kPartRows = 256;

int64_t tiles_of(int64_t m, int64_t n, int64_t tile) {
  return ((m + tile - 1) / tile) * ((n + tile - 1) / tile);
}

// dw_in and dw_out of every expert; 128 x 128 tiles count for the rule in both
// kernels (the workspace does not depend on alignment).
int64_t weight_parts(int64_t rows, int32_t experts, int64_t dim, int64_t hidden) {
  const int64_t blocks =
      (tiles_of(2 * hidden, dim, kTileO) + tiles_of(dim, hidden, kTileO)) * experts;
  int64_t parts = kWeightBlocks / blocks;
  const int64_t most = rows / experts / kPartRows;
  parts = parts < most ? parts : most;
  parts = parts < kMaxParts ? parts : kMaxParts;
  return parts > 1 ? parts : 1;
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Workspace: the pre-activations' gradients, then the weights' partial sums.
size_t dgu_bytes(int64_t rows, int64_t hidden, size_t size) {
  return align256((size_t)rows * 2 * hidden * size);
}
size_t parts_bytes(int64_t rows, int32_t experts, int64_t dim, int64_t hidden) {
  const int64_t p = weight_parts(rows, experts, dim, hidden);
  return p > 1 ? align256((size_t)p * experts * 3 * hidden * dim * 4) : 0;
}

// out[e] = the sum of the expert's parts, in order.
template <class T>
__global__ __launch_bounds__(256) void k_ffn_add_parts(const float* __restrict__ sums,
                                                       uint32_t parts, int64_t size,
                                                       int32_t experts, T* __restrict__ out) {
  const int64_t per = (size + 3) / 4;
  const int64_t v = (int64_t)block_index() * 256 + threadIdx.x;
  const int64_t e = v / per, i = (v - e * per) * 4;
  if (e >= experts) return;
  const float* p = sums + e * parts * size + i;
  float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (uint32_t k = 0; k < parts; ++k) {
    const Span<float, 4> v4 = load_span<4>(p + k * size, size - i);
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] += v4.get(j);
  }
  store_span(out + e * size + i, t, size - i);
}

// Whether a product of the groups' rows goes by tiles of 256 x 256 (ffn_wide.hpp): they
// hold offsets of 32 bits (256 rows of one operand, 64 of the other, a projection behind
// the other), take long to start and need enough blocks to fill the card (us of a
// forward, against tiles of 128 x 128):
//   8 experts, 512 x 1024: 512 rows each (128 blocks) 47, 44; 1024 (256 blocks) 52, 55
//   1 expert, 3328 x 1664: 1024 rows (52 blocks) 110, 101; 4096 (208 blocks) 140, 238
//   64 experts, 128 x 256: 4096 rows each 168, 144: two slots of k are too few
constexpr int64_t kWideBlocks = 160, kWideLeastK = 256;
bool wide_fits(int64_t K, int64_t N) {
  return K >= kWideLeastK && K * N < (1ll << 30) && K + N < (1ll << 20);
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether the forward's products go by ffn_few.hpp: each of its passes over the
// weights serves 64 rows of an expert, and keeps up with the tiles while few blocks of
// 128 columns would be at work (`tiles`), or few rows use what is read (us of a
// forward, this kernel against tiles):
//   bf16  1 expert, 3328 x 1664: 256 rows 77, 99; 512 rows 149, 98
//         8 experts, 512 x 1024: 64 rows each 19, 35; 128 34, 36; 256 59, 37
//         32 experts, 1664 x 1024: 8 rows each 76, 88; 16 85, 88; 32 107, 91
//         24 experts, 3328 x 1664: 16 rows each 194, 269; 32 255, 272; 48 326, 276
//   fp32  1 expert, 3328 x 1664: 128 rows 80, 130; 256 189, 131
//         32 experts, 1664 x 1024: 16 rows each 174, 241; 32 231, 251; 64 402, 245
template <class T>
bool by_few_rows(int64_t rows, int32_t experts, int64_t hidden) {
  const int64_t passes = (rows + kFewRows * experts - 1) / (kFewRows * experts);
  const int64_t tiles = experts * ((hidden + 127) / 128);
  return rows <= (sizeof(T) == 2 ? 16 : 32) * (int64_t)experts ||
         passes * tiles <= (passes == 1 ? 128 : sizeof(T) == 2 ? 64 : 40);
}

// C = A B' over groups of few rows
template <class T, class Epilogue>
hipError_t few_rows_product(const Groups& g, const void* a, const void* b, int64_t K, int64_t N,
                            int64_t b_stride, const Epilogue& epilogue, hipStream_t s) {
  const int64_t col_tiles = (N + kFewCols - 1) / kFewCols;
  const int64_t blocks = blocks_of(row_tiles_bound(g, kFewRows) * col_tiles, kRowChunk);
  hipLaunchKernelGGL((k_ffn_few_rows<T, Epilogue>), tile_grid(blocks, 64 * kFewWaves),
                     dim3(64 * kFewWaves), 0, s, g, static_cast<const T*>(a),
                     static_cast<const T*>(b), (int32_t)K, N, b_stride, (uint32_t)col_tiles,
                     epilogue);
  return hipGetLastError();
}

// C = A B' or A B (B_KC) over the groups' rows
template <class T, bool B_KC, class Epilogue>
hipError_t rows_product(const Groups& g, const void* a, const void* b, int64_t K, int64_t N,
                        int64_t b_stride, const Epilogue& epilogue, hipStream_t s) {
  if (g.rows == 0) return hipSuccess;
  if constexpr (sizeof(T) == 2) {
    constexpr int WM = 2, WN = 4;
    const int64_t cols = Epilogue::kDual ? kWideO / 2 : kWideO;
    const int64_t col_tiles = (N + cols - 1) / cols;
    const int64_t blocks = blocks_of(row_tiles_bound(g, kWideO) * col_tiles, kRowChunk);
    if (K % 8 == 0 && (B_KC || N % 8 == 0) && on16(a) && on16(b) && wide_fits(K, N) &&
        blocks >= kWideBlocks) {
      hipLaunchKernelGGL((k_ffn_rows_wide<T, B_KC, Epilogue, WM, WN>),
                         tile_grid(blocks, 64 * WM * WN), dim3(64 * WM * WN), 0, s, g,
                         static_cast<const T*>(a), static_cast<const T*>(b), K, N, b_stride,
                         (uint32_t)col_tiles, epilogue);
      return hipGetLastError();
    }
  }
  const int64_t cols = Epilogue::kDual ? kTileO / 2 : kTileO;
  const int64_t col_tiles = (N + cols - 1) / cols;
  const int64_t blocks = blocks_of(row_tiles_bound(g, kTileO) * col_tiles, kRowChunk);
  hipLaunchKernelGGL((k_ffn_rows<T, B_KC, Epilogue>), tile_grid(blocks, kTileThreads),
                     dim3(kTileThreads), 0, s, g, static_cast<const T*>(a),
                     static_cast<const T*>(b), K, N, b_stride, (uint32_t)col_tiles, epilogue);
  return hipGetLastError();
}

// Whether fp32 goes through planes.  Planes save waits along k: a product of tiles that
// cut their own values takes 0.8 (forward) to 1.3 us for every 32 k while one block
// is alone on its CU, and several blocks hide each other's.  Planes cost the cutting of
// every weight, of experts without rows too, and its reading with 6 bytes for 4: 2.6 to
// 2.9 us for a million.  So they are taken while the weights are few for the k that the
// products walk along, and their tiles too few to hide the waits (us, planes against tiles):
//   forward   8 experts, 1664 x 640: 128 rows each 111, 130 (3700 weights a k); 1664 x
//             1024 201, 151 (5070)
//             1 expert, 479 x 1000: 2048 rows (320 tiles) 70, 95; 4096 (640) 101, 115;
//             8192 (1280) 174, 167; 1664 x 640: 2048 rows (368) 126, 133; 4096 (736)
//             211, 202; 4 experts, 1664 x 640: 1024 rows each (805) 231, 203
//             4 experts, 128 x 256 (384 k): 1024 rows each (175) 29, 34; 2048 (335) 36, 35
//   backward  8 experts, 1664 x 1024: 8 rows each 221, 275 (3670 weights a k); 3327 x 1663
//             679, 594 (6650); 32 experts, 479 x 640: 8 rows each 175, 163 (5580); 1664 x
//             640 532, 359 (11600)
//             4 experts, 479 x 1000: 1024 rows each (280 blocks) 197, 307; 8 experts, 479 x
//             640: 1024 (355) 251, 274; 16 experts (2790 weights a k): 256 (235) 192, 207;
//             512 (395) 297, 286
//             4 experts, 128 x 256 (640 k): 2048 rows each (134) 72, 94; 4096 (262) 115, 113
int64_t row_tiles_128(int64_t rows, int32_t experts) {  // whatever the capacity
  const int64_t used = rows < experts ? rows : experts;
  return (rows + used * 127) / 128;
}
bool forward_by_planes(int64_t rows, int32_t experts, int64_t dim, int64_t hidden) {
  const int64_t k = dim + hidden;
  const int64_t tiles = row_tiles_128(rows, experts) * ((hidden + 63) / 64 + (dim + 127) / 128);
  return rows > 0 && experts * dim * hidden <= 4000 * k && tiles <= 780 && 10 * tiles <= 7 * k;
}
bool backward_by_planes(int64_t rows, int32_t experts, int64_t dim, int64_t hidden) {
  const int64_t k = dim + 2 * hidden, weights = experts * dim * hidden;
  const int64_t blocks = row_tiles_128(rows, experts) * ((hidden + 127) / 128);  // of the middle
  return rows > 0 && weights <= 4500 * k &&
         (blocks <= 256 || (blocks <= 512 && weights <= 2500 * k && k >= 1500));
}

// Hands out the workspace from its start.
struct Space {
  char* at;
  Planes planes(int64_t rows, int64_t width) {
    const Planes p{reinterpret_cast<bf16_t*>(at), padded(width), rows * padded(width)};
    at += align256((size_t)p.size * 6);
    return p;
  }
};
size_t planes_bytes(int64_t rows, int64_t width) {
  return align256((size_t)rows * padded(width) * 6);
}
// Planes of x, a and the weights, which both directions hold first.
size_t forward_planes_bytes(int64_t rows, int32_t experts, int64_t dim, int64_t hidden) {
  return planes_bytes(rows, dim) + planes_bytes(rows, hidden) +
         planes_bytes(experts * 2 * hidden, dim) + planes_bytes(experts * dim, hidden);
}

struct Cutter {
  Cuts c{};
  void add(const void* src, const Planes& dst, int64_t width) {
    const int i = c.count++;
    c.src[i] = static_cast<const float*>(src);
    c.dst[i] = dst;
    c.width[i] = width;
    c.first[i + 1] = c.first[i] + dst.size / 8;
  }
  template <class T>
  hipError_t launch(hipStream_t s) const {
    hipLaunchKernelGGL(k_ffn_cut<T>, row_grid((c.first[c.count] + 255) / 256), dim3(256), 0, s, c);
    return hipGetLastError();
  }
};

template <bool B_KC, class Epilogue>
hipError_t rows_product_planes(const Groups& g, const Planes& a, const Planes& b, int64_t N,
                               int64_t b_rows, const Epilogue& epilogue, hipStream_t s) {
  const int64_t cols = Epilogue::kDual ? kTileO / 2 : kTileO;
  const int64_t col_tiles = (epilogue.columns() + cols - 1) / cols;
  const int64_t blocks = blocks_of(row_tiles_bound(g, 128) * col_tiles, kRowChunk);
  // 64 rows a block where 128 leave CUs without one (4096 x 479 from 1000: 36 us
  // against 49), and two such blocks a CU where the epilogue reads what it stores with,
  // so that one's waits and stores hide behind the other (backward of 8 experts, 479 x
  // 640, 1024 rows each, 262 us with 128 rows, 253; 1 expert, 479 x 1000, 4096 rows 207,
  // 200; 3327 x 1663 1454, 1466)
  const int64_t half = blocks_of(row_tiles_bound(g, 64) * col_tiles, kRowChunk);
  if (blocks <= 192) {
    hipLaunchKernelGGL((k_ffn_rows_planes<B_KC, Epilogue, 64, 4>), tile_grid(half, 256),
                       dim3(256), 0, s, g, a, b, N, b_rows, (uint32_t)col_tiles, epilogue);
  } else if constexpr (Epilogue::kReads) {
    hipLaunchKernelGGL((k_ffn_rows_planes<B_KC, Epilogue, 64, 2>), tile_grid(half, 256),
                       dim3(256), 0, s, g, a, b, N, b_rows, (uint32_t)col_tiles, epilogue);
  } else {
    hipLaunchKernelGGL((k_ffn_rows_planes<B_KC, Epilogue, 128, 3>), tile_grid(blocks, 512), dim3(512),
                       0, s, g, a, b, N, b_rows, (uint32_t)col_tiles, epilogue);
  }
  return hipGetLastError();
}

template <class T, class Out>
hipError_t launch_weights(WeightProducts<T>& w, const WeightPlanes* planes,
                          const WeightEpilogue<Out>& out, hipStream_t s) {
  constexpr int WM = 2, WN = 4;
  bool wide = sizeof(T) == 2;
  for (int p = 0; p < 2; ++p)
    wide = wide && w.M[p] % 8 == 0 && w.N[p] % 8 == 0 && on16(w.A[p]) && on16(w.B[p]);
  // (1 expert, 512 x 1024, 24 tiles: the backward of 512 rows 106 us with these tiles,
  // 94 with 128 x 128; 8 experts, 480 x 640, 128 tiles: 85 and 101)
  wide = wide && w.groups.experts * (tiles_of(w.M[0], w.N[0], kWideO) +
                                     tiles_of(w.M[1], w.N[1], kWideO)) >= 100;
  const int64_t tile = wide ? kWideO : kTileO;
  int64_t tiles = 0;
  for (int p = 0; p < 2; ++p) {
    w.row_tiles[p] = (uint32_t)((w.M[p] + tile - 1) / tile);
    w.col_tiles[p] = (uint32_t)((w.N[p] + tile - 1) / tile);
    tiles += (int64_t)w.row_tiles[p] * w.col_tiles[p];
  }
  const int64_t blocks = blocks_of(tiles * w.parts * w.groups.experts, kWeightChunk);
  if constexpr (sizeof(T) == 2) {
    if (wide) {
      hipLaunchKernelGGL((k_ffn_weights_wide<T, Out, WM, WN>), tile_grid(blocks, 64 * WM * WN),
                         dim3(64 * WM * WN), 0, s, w, out);
      return hipGetLastError();
    }
  } else if (planes) {
    hipLaunchKernelGGL((k_ffn_weights_planes<Out, 128>), tile_grid(blocks, 512), dim3(512), 0, s,
                       w, *planes, out);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((k_ffn_weights<T, Out>), tile_grid(blocks, kTileThreads), dim3(kTileThreads),
                     0, s, w, out);
  return hipGetLastError();
}

// dw_in[e] = dgu' x and dw_out[e] = dy' a over expert e's rows
template <class T>
hipError_t weight_gradients(const Groups& g, const T* dgu, const void* x, const void* dy,
                            const void* a, const WeightPlanes* planes, int64_t D, int64_t F,
                            void* dw_in, void* dw_out, float* sums, hipStream_t s) {
  const int64_t parts = weight_parts(g.rows, g.experts, D, F);
  WeightProducts<T> w{g, {dgu, static_cast<const T*>(dy)},
                      {static_cast<const T*>(x), static_cast<const T*>(a)},
                      {2 * F, D}, {D, F}, {}, {}, (uint32_t)parts};
  T* const out[2] = {static_cast<T*>(dw_in), static_cast<T*>(dw_out)};
  if (parts == 1) return launch_weights(w, planes, WeightEpilogue<T>{{out[0], out[1]}}, s);
  float* const part[2] = {sums, sums + parts * g.experts * 2 * F * D};
  hipError_t e = launch_weights(w, planes, WeightEpilogue<float>{{part[0], part[1]}}, s);
  for (int p = 0; p < 2 && e == hipSuccess; ++p) {
    const int64_t vecs = (w.M[p] * w.N[p] + 3) / 4 * g.experts;
    hipLaunchKernelGGL((k_ffn_add_parts<T>), row_grid((vecs + 255) / 256), dim3(256), 0, s,
                       part[p], (uint32_t)parts, w.M[p] * w.N[p], g.experts, out[p]);
    e = hipGetLastError();
  }
  return e;
}

// The forward and backward of fp32 through planes.
template <class T>
hipError_t forward_planes(const GatedFfn& f, void* gu, void* a, void* y, char* ws,
                          hipStream_t s) {
  const int64_t D = f.dim, F = f.hidden;
  const Groups g{f.offsets, f.rows, f.capacity, f.experts};
  Space space{ws};
  const Planes px = space.planes(f.rows, D), pa = space.planes(f.rows, F);
  const Planes pin = space.planes(f.experts * 2 * F, D), pout = space.planes(f.experts * D, F);
  Cutter cut;
  cut.add(f.x, px, D);
  cut.add(f.w_in, pin, D);
  cut.add(f.w_out, pout, F);
  hipError_t e = cut.launch<T>(s);
  if (e != hipSuccess) return e;
  e = rows_product_planes<true>(
      g, px, pin, F, 2 * F,
      ActPlanesEpilogue{{static_cast<float*>(gu), static_cast<float*>(a), F, f.act}, pa}, s);
  if (e != hipSuccess) return e;
  return rows_product_planes<true>(g, pa, pout, D, D,
                                   StorePlanesEpilogue{{static_cast<float*>(y), D}}, s);
}

template <class T>
hipError_t backward_planes(const GatedFfn& f, const void* gu, const void* a, const void* dy,
                           void* dx, void* dw_in, void* dw_out, char* ws, hipStream_t s) {
  const int64_t D = f.dim, F = f.hidden;
  const Groups g{f.offsets, f.rows, f.capacity, f.experts};
  Space space{ws};
  const Planes px = space.planes(f.rows, D), pa = space.planes(f.rows, F);
  const Planes pin = space.planes(f.experts * 2 * F, D), pout = space.planes(f.experts * D, F);
  const Planes pdy = space.planes(f.rows, D), pdgu = space.planes(f.rows, 2 * F);
  Cutter cut;
  cut.add(f.x, px, D);
  cut.add(a, pa, F);
  cut.add(f.w_in, pin, D);
  cut.add(f.w_out, pout, F);
  cut.add(dy, pdy, D);
  hipError_t e = cut.launch<T>(s);
  if (e != hipSuccess) return e;
  e = rows_product_planes<false>(
      g, pdy, pout, F, D,
      ActGradPlanesEpilogue{{static_cast<const float*>(gu), nullptr, F, f.act}, pdgu}, s);
  if (e != hipSuccess) return e;
  e = rows_product_planes<false>(g, pdgu, pin, D, 2 * F,
                                 StorePlanesEpilogue{{static_cast<float*>(dx), D}}, s);
  if (e != hipSuccess) return e;
  const WeightPlanes planes{{pdgu, pdy}, {px, pa}};
  return weight_gradients<T>(g, nullptr, f.x, dy, a, &planes, D, F, dw_in, dw_out,
                                 reinterpret_cast<float*>(space.at), s);
}

}  // namespace

template <class T>
size_t ffn_forward_workspace_bytes_t(int64_t rows, int32_t experts, int64_t dim,
                                     int64_t hidden) {
  const bool planes = sizeof(T) == 4 && !by_few_rows<T>(rows, experts, hidden) &&
                      forward_by_planes(rows, experts, dim, hidden);
  return (planes ? forward_planes_bytes(rows, experts, dim, hidden) : 0) + 256;
}

template <class T>
size_t ffn_workspace_bytes_t(int64_t rows, int32_t experts, int64_t dim, int64_t hidden) {
  const size_t forward = ffn_forward_workspace_bytes_t<T>(rows, experts, dim, hidden);
  size_t backward = dgu_bytes(rows, hidden, sizeof(T));
  if (sizeof(T) == 4 && backward_by_planes(rows, experts, dim, hidden))
    backward = forward_planes_bytes(rows, experts, dim, hidden) + planes_bytes(rows, dim) +
               planes_bytes(rows, 2 * hidden);
  backward += parts_bytes(rows, experts, dim, hidden) + 256;
  return forward > backward ? forward : backward;
}

template <class T>
hipError_t ffn_forward_t(const GatedFfn& f, void* gu, void* a, void* y, char* ws, hipStream_t s) {
  const int64_t D = f.dim, F = f.hidden;
  const Groups g{f.offsets, f.rows, f.capacity, f.experts};
  const ActEpilogue<T> middle{static_cast<T*>(gu), static_cast<T*>(a), F, f.act};
  const StoreEpilogue<T> end{static_cast<T*>(y), D};
  if (g.rows == 0) return hipSuccess;
  if (by_few_rows<T>(f.rows, f.experts, F)) {
    const hipError_t e = few_rows_product<T>(g, f.x, f.w_in, D, F, 2 * F * D, middle, s);
    if (e != hipSuccess) return e;
    return few_rows_product<T>(g, a, f.w_out, F, D, D * F, end, s);
  }
  if constexpr (sizeof(T) == 4)
    if (forward_by_planes(f.rows, f.experts, D, F))
      return forward_planes<T>(f, gu, a, y, ws, s);
  const hipError_t e = rows_product<T, true>(g, f.x, f.w_in, D, F, 2 * F * D, middle, s);
  if (e != hipSuccess) return e;
  return rows_product<T, true>(g, a, f.w_out, F, D, D * F, end, s);
}

template <class T>
hipError_t ffn_backward_t(const GatedFfn& f, const void* gu, const void* a, const void* dy,
                          void* dx, void* dw_in, void* dw_out, char* ws, hipStream_t s) {
  if constexpr (sizeof(T) == 4)
    if (backward_by_planes(f.rows, f.experts, f.dim, f.hidden))
      return backward_planes<T>(f, gu, a, dy, dx, dw_in, dw_out, ws, s);
  const int64_t D = f.dim, F = f.hidden;
  const Groups g{f.offsets, f.rows, f.capacity, f.experts};
  T* dgu = reinterpret_cast<T*>(ws);
  float* sums = reinterpret_cast<float*>(ws + dgu_bytes(f.rows, F, sizeof(T)));
  hipError_t e = rows_product<T, false>(
      g, dy, f.w_out, D, F, D * F,
      ActGradEpilogue<T>{static_cast<const T*>(gu), dgu, F, f.act}, s);
  if (e != hipSuccess) return e;
  e = rows_product<T, false>(g, dgu, f.w_in, 2 * F, D, 2 * F * D,
                             StoreEpilogue<T>{static_cast<T*>(dx), D}, s);
  if (e != hipSuccess) return e;
  return weight_gradients<T>(g, dgu, f.x, dy, a, nullptr, D, F, dw_in, dw_out, sums, s);
}

#define EMBTAB_FFN_TYPE(T)                                                                     \
  template size_t ffn_forward_workspace_bytes_t<T>(int64_t, int32_t, int64_t, int64_t);        \
  template size_t ffn_workspace_bytes_t<T>(int64_t, int32_t, int64_t, int64_t);                \
  template hipError_t ffn_forward_t<T>(const GatedFfn&, void*, void*, void*, char*,            \
                                       hipStream_t);                                           \
  template hipError_t ffn_backward_t<T>(const GatedFfn&, const void*, const void*, const void*, \
                                        void*, void*, void*, char*, hipStream_t);

}  // namespace embtab
