// Launches of the experts' gated feed-forward for one element type (included by
// one source per type).
#pragma once

#include "ffn_tiles.hpp"

namespace embtab {

namespace {

// Weight gradients with fewer tiles than this cut the rows into parts, whose
// sums a second kernel adds in order.
constexpr int64_t kWeightBlocks = 512;
constexpr int64_t kMaxParts = 16, kPartRows = 256;

int64_t weight_tiles(int64_t m, int64_t n) {
  return ((m + kTileO - 1) / kTileO) * ((n + kTileO - 1) / kTileO);
}

int64_t weight_parts(int64_t rows, int32_t experts, int64_t m, int64_t n) {
  const int64_t blocks = weight_tiles(m, n) * experts;
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
size_t parts_bytes(int64_t rows, int32_t experts, int64_t m, int64_t n) {
  const int64_t p = weight_parts(rows, experts, m, n);
  return p > 1 ? align256((size_t)p * experts * m * n * 4) : 0;
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
  f32x4 t = load4(p, size - i);
  for (uint32_t k = 1; k < parts; ++k) t += load4(p + k * size, size - i);
  store4(out + e * size + i, t, size - i);
}

int64_t blocks_of(int64_t tiles) { return (tiles + kXcds - 1) / kXcds * kXcds; }

// C = A B' or A B (B_KC) over the groups' rows
template <class T, bool B_KC, class Epilogue>
hipError_t rows_product(const Groups& g, const void* a, const void* b, int64_t K, int64_t N,
                        int64_t b_stride, const Epilogue& epilogue, hipStream_t s) {
  const int64_t cols = Epilogue::kDual ? kTileO / 2 : kTileO;
  const int64_t col_tiles = (N + cols - 1) / cols;
  const int64_t blocks = blocks_of(row_tiles_bound(g, kTileO) * col_tiles);
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL((k_ffn_rows<T, B_KC, Epilogue>), tile_grid(blocks, kTileThreads),
                     dim3(kTileThreads), 0, s, g, static_cast<const T*>(a),
                     static_cast<const T*>(b), K, N, b_stride, (uint32_t)col_tiles, epilogue);
  return hipGetLastError();
}

// out[e] = A' B over expert e's rows
template <class T>
hipError_t weights_product(const Groups& g, const void* a, const void* b, int64_t M, int64_t N,
                           void* out, float* sums, hipStream_t s) {
  const int64_t parts = weight_parts(g.rows, g.experts, M, N);
  const uint32_t rt = (uint32_t)((M + kTileO - 1) / kTileO);
  const uint32_t ct = (uint32_t)((N + kTileO - 1) / kTileO);
  const dim3 grid =
      tile_grid(blocks_of((int64_t)rt * ct * parts * g.experts), kTileThreads);
  if (parts == 1) {
    const StoreEpilogue<T> epilogue{static_cast<T*>(out), N, M * N};
    hipLaunchKernelGGL((k_ffn_weights<T, StoreEpilogue<T>>), grid, dim3(kTileThreads), 0, s, g,
                       static_cast<const T*>(a), static_cast<const T*>(b), M, N, rt, ct, 1u,
                       epilogue);
    return hipGetLastError();
  }
  const PartEpilogue epilogue{sums, N, M * N};
  hipLaunchKernelGGL((k_ffn_weights<T, PartEpilogue>), grid, dim3(kTileThreads), 0, s, g,
                     static_cast<const T*>(a), static_cast<const T*>(b), M, N, rt, ct,
                     (uint32_t)parts, epilogue);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t vecs = (M * N + 3) / 4 * g.experts;
  hipLaunchKernelGGL((k_ffn_add_parts<T>), row_grid((vecs + 255) / 256), dim3(256), 0, s, sums,
                     (uint32_t)parts, M * N, g.experts, static_cast<T*>(out));
  return hipGetLastError();
}

}  // namespace

template <class T>
size_t ffn_workspace_bytes_t(int64_t rows, int32_t experts, int64_t dim, int64_t hidden) {
  const size_t in = parts_bytes(rows, experts, 2 * hidden, dim);
  const size_t out = parts_bytes(rows, experts, dim, hidden);
  return dgu_bytes(rows, hidden, sizeof(T)) + (in > out ? in : out) + 256;
}

template <class T>
hipError_t ffn_forward_t(const GatedFfn& f, void* gu, void* a, void* y, char*, hipStream_t s) {
  const int64_t D = f.dim, F = f.hidden;
  const Groups g{f.offsets, f.rows, f.capacity, f.experts};
  const hipError_t e = rows_product<T, true>(
      g, f.x, f.w_in, D, F, 2 * F * D,
      ActEpilogue<T>{static_cast<T*>(gu), static_cast<T*>(a), F, f.act}, s);
  if (e != hipSuccess) return e;
  return rows_product<T, true>(g, a, f.w_out, F, D, D * F,
                               StoreEpilogue<T>{static_cast<T*>(y), D, 0}, s);
}

template <class T>
hipError_t ffn_backward_t(const GatedFfn& f, const void* gu, const void* a, const void* dy,
                          void* dx, void* dw_in, void* dw_out, char* ws, hipStream_t s) {
  const int64_t D = f.dim, F = f.hidden;
  const Groups g{f.offsets, f.rows, f.capacity, f.experts};
  T* dgu = reinterpret_cast<T*>(ws);
  float* sums = reinterpret_cast<float*>(ws + dgu_bytes(f.rows, F, sizeof(T)));
  hipError_t e = rows_product<T, false>(
      g, dy, f.w_out, D, F, D * F,
      ActGradEpilogue<T>{static_cast<const T*>(gu), dgu, F, f.act}, s);
  if (e != hipSuccess) return e;
  e = rows_product<T, false>(g, dgu, f.w_in, 2 * F, D, 2 * F * D,
                             StoreEpilogue<T>{static_cast<T*>(dx), D, 0}, s);
  if (e != hipSuccess) return e;
  e = weights_product<T>(g, dgu, f.x, 2 * F, D, dw_in, sums, s);
  if (e != hipSuccess) return e;
  return weights_product<T>(g, dy, a, D, F, dw_out, sums, s);
}

#define EMBTAB_FFN_TYPE(T)                                                                     \
  template size_t ffn_workspace_bytes_t<T>(int64_t, int32_t, int64_t, int64_t);                \
  template hipError_t ffn_forward_t<T>(const GatedFfn&, void*, void*, void*, char*,            \
                                       hipStream_t);                                           \
  template hipError_t ffn_backward_t<T>(const GatedFfn&, const void*, const void*, const void*, \
                                        void*, void*, void*, char*, hipStream_t);

}  // namespace embtab
