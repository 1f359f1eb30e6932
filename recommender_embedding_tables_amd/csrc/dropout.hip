// Dropout whose mask is never stored, with the residual added, for gfx950.
//
// Element i of the call takes 16 bits of a counter-based random word:
//   h = SM(SM(seed) ^ (counter + floor(i / 4))),  bits = 16 bits of h at 16 (i mod 4)
// with SM one SplitMix64 step (Steele, Lea and Flood, OOPSLA 2014), as the
// tables' initial values are drawn.  It is kept where bits < keep, with
// keep = round((1 - p) 2^16), and scaled by 2^16 / keep, the reciprocal of the
// share that is in fact kept:
//   y = residual + x * (2^16 / keep)   or   residual,  rounded once
// The backward pass is the same call on dy without a residual: the words depend
// on the seed, the counter and the element alone.  Seed and counter are read on
// the device, so that a captured graph draws new words where the program moves
// its counter on.
//
// Bound by memory: x and the residual read, y written; one 16-byte vector a
// thread, one-shot blocks.  A word serves four elements (two products of 64 bits
// in about 50 issue slots of a wave): with a word of its own for every element
// the arithmetic would take longer than the memory does.  218 million bf16 values
// with a residual: 200 us, 6.5 TB/s, the rate of a copy.
#include "dense.hpp"

namespace embtab {

namespace {

template <class T>
__global__ __launch_bounds__(256) void k_dropout(const T* x, const T* residual, int64_t numel,
                                                 const int64_t* __restrict__ rng, uint32_t keep,
                                                 float scale, T* y) {
  constexpr int N = kVec<T>;
  const int64_t i = ((int64_t)block_index() * 256 + threadIdx.x) * N;
  if (i >= numel) return;
  const uint64_t key = sm64((uint64_t)rng[0]);
  const uint64_t group = (uint64_t)rng[1] + (uint64_t)(i >> 2);
  uint64_t words[N / 4];
#pragma unroll
  for (int k = 0; k < N / 4; ++k) words[k] = sm64(key ^ (group + k));
  const auto value = [&](int e, float v, float r) {
    const bool kept = ((uint32_t)(words[e >> 2] >> (16 * (e & 3))) & 0xFFFFu) < keep;
    return kept ? __builtin_fmaf(v, scale, r) : r;
  };
  if (i + N <= numel) {
    const Raw<T> in = load_raw<T, N, true>(x + i);
    Raw<T> res{};
    if (residual) res = load_raw<T, N, true>(residual + i);
    float v[N];
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = value(e, in.get(e), res.get(e));
    Raw<T> out;
    out.set_all(v);
    store_raw<T, N, true>(y + i, out);
    return;
  }
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (i + e < numel)
      y[i + e] = from_f32<T>(
          value(e, to_f32(x[i + e]), residual ? to_f32(residual[i + e]) : 0.0f));
}

template <class T>
hipError_t dropout_t(const void* x, const void* residual, int64_t numel, const int64_t* rng,
                     uint32_t keep, void* y, hipStream_t s) {
  const int64_t per = 256 * kVec<T>;
  const int64_t blocks = (numel + per - 1) / per;
  if (blocks == 0) return hipSuccess;
  const float scale = keep ? (float)(65536.0 / keep) : 0.0f;
  hipLaunchKernelGGL((k_dropout<T>), row_grid(blocks), dim3(256), 0, s,
                     static_cast<const T*>(x), static_cast<const T*>(residual), numel, rng, keep,
                     scale, static_cast<T*>(y));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const void* x, const void* residual, int64_t numel, int32_t dtype,
                          uint32_t keep, const int64_t* rng, void* y, hipStream_t s) {
  switch (dtype) {
    case EMB_F32: return dropout_t<float>(x, residual, numel, rng, keep, y, s);
    case EMB_BF16: return dropout_t<bf16_t>(x, residual, numel, rng, keep, y, s);
    default: return dropout_t<f16_t>(x, residual, numel, rng, keep, y, s);
  }
}

}  // namespace embtab
