// Global norm of a list of gradients and the list scaled by it, for gfx950.
//
//   norm = sqrt(sum_i sum_k g_i[k]^2 + sum_e extra[e])
//   coef = min(1, max_norm / (norm + 1e-6)), 0 when the norm is not finite
//   out_i = g_i * coef (0 when coef is 0, whatever the gradient holds)
//
// The squares are formed and summed in 64 bits, so a gradient of 1e-30 or 1e30
// neither vanishes nor overflows, and a list of any length keeps its small
// members.
//
// Bound by memory: the sum reads every gradient, the scale reads it again and
// writes it, since no element can be scaled before the last one is summed.  60
// tensors of 256 million bf16 and fp32 elements: 111 us for the sum (6.2 TB/s)
// and 284 us for the scale (6.0 TB/s); 12 small tensors: 4 us each, the latency
// of a launch and of the dependent loads in it.
//
// The list is cut into chunks of kClipChunk elements of one tensor; the tensor
// table travels as a kernel argument (kClipItems tensors to a launch), so no
// copy to the device is made and the calls can be captured into a graph.  The
// partial sums are combined in a fixed order: the result does not depend on
// the order in which blocks run.
#include "dense.hpp"

namespace embtab {

namespace {

constexpr int kClipThreads = 256;
constexpr int kClipChunk = 8192;
constexpr int kClipItems = 104;     // 36 bytes each: the arguments stay under 4 KiB
constexpr int kClipParts = 1024;    // blocks (and partial sums) of one sum launch
constexpr int kScaleBlocks = 2048;  // blocks of one scale launch: what the chip holds

// The sums (partial ones and the caller's) are added by every block of every
// scale launch up to this many times the launches; beyond, one block adds them
// first, or the work would grow with the square of the list's length.  10000
// tensors of 81920 fp32 elements, 97 launches and 97 thousand sums: 2.26 ms,
// and 7.1 added by every block; 2500 tensors 0.56 and 0.82; 200 tensors (4
// thousand sums times launches) 43 us either way; 12 small tensors and 3000
// sums of the caller's 17 and 14.
constexpr int64_t kClipDirect = 4 * kClipParts;

struct ClipItem {
  const void* in;
  void* out;
  int64_t n;
  uint32_t types;  // input type | output type << 8
};
struct ClipList {
  ClipItem item[kClipItems];
  uint32_t first[kClipItems];  // chunks of the items before
  uint32_t count, chunks;
};
static_assert(kClipItems <= 128, "two per lane");

// The last item with first <= chunk (no item is empty).  Every lane compares
// two of the starts and the wave counts them: two loads in parallel, where a
// binary search waits for seven.
struct ClipFinder {
  uint32_t a, b;
  __device__ ClipFinder(const ClipList& l) {
    const uint32_t lane = threadIdx.x & 63u;
    a = lane < l.count ? l.first[lane] : ~0u;
    b = lane + 64u < l.count ? l.first[lane + 64u < kClipItems ? lane + 64u : 0u] : ~0u;
  }
  __device__ uint32_t operator()(uint32_t chunk) const {
    return (uint32_t)(__popcll(__ballot(a <= chunk)) + __popcll(__ballot(b <= chunk))) - 1u;
  }
};

__device__ inline double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Sum over the block, valid in every thread.
__device__ inline double block_sum(double v, double* lds4) {
  v = wave_sum(v);
  if ((threadIdx.x & 63u) == 0u) lds4[threadIdx.x >> 6] = v;
  __syncthreads();
  return (lds4[0] + lds4[1]) + (lds4[2] + lds4[3]);
}

template <class T>
__device__ inline double chunk_square_sum(const T* p, int64_t len) {
  constexpr int N = kVec<T>;
  constexpr int U = kClipChunk / (kClipThreads * N);
  double acc = 0.0;
  if (len == kClipChunk) {
    Raw<T> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = load_raw<T>(p + (u * kClipThreads + threadIdx.x) * N);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const double g = (double)r[u].get(i);
        acc = __builtin_fma(g, g, acc);
      }
    return acc;
  }
  const int n = (int)len;
  for (int k = threadIdx.x * N; k + N <= n; k += kClipThreads * N) {
    const Raw<T> r = load_raw<T>(p + k);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const double g = (double)r.get(i);
      acc = __builtin_fma(g, g, acc);
    }
  }
  const int k = n / N * N + (int)threadIdx.x;  // the last n % N elements
  if (k < n) {
    const double g = (double)to_f32(p[k]);
    acc = __builtin_fma(g, g, acc);
  }
  return acc;
}

__global__ __launch_bounds__(kClipThreads) void k_grad_square_sum(const ClipList l,
                                                                  double* __restrict__ parts) {
  __shared__ double lds4[4];
  const ClipFinder find(l);
  double acc = 0.0;
  for (uint32_t c = blockIdx.x; c < l.chunks; c += gridDim.x) {
    const uint32_t i = find(c);
    const ClipItem& it = l.item[i];
    const int64_t at = (int64_t)(c - l.first[i]) * kClipChunk;
    const int64_t len = it.n - at < kClipChunk ? it.n - at : kClipChunk;
    switch (it.types & 0xFFu) {
      case EMB_F32: acc += chunk_square_sum(static_cast<const float*>(it.in) + at, len); break;
      case EMB_BF16: acc += chunk_square_sum(static_cast<const bf16_t*>(it.in) + at, len); break;
      default: acc += chunk_square_sum(static_cast<const f16_t*>(it.in) + at, len); break;
    }
  }
  acc = block_sum(acc, lds4);
  if (threadIdx.x == 0) parts[blockIdx.x] = acc;
}

// This thread's share of n values, added one after another with eight loads in
// flight.
__device__ inline double strided_sum(double acc, const double* __restrict__ v, uint32_t n) {
  for (uint32_t i = threadIdx.x; i < n; i += 8u * kClipThreads) {
    double x[8];
#pragma unroll
    for (uint32_t k = 0; k < 8u; ++k)
      x[k] = n - i > k * kClipThreads ? v[i + k * kClipThreads] : 0.0;
#pragma unroll
    for (uint32_t k = 0; k < 8u; ++k) acc += x[k];
  }
  return acc;
}

// The norm and the coefficient from the partial sums, the same in every thread
// of every block that forms them.
__device__ inline float2 norm_and_coef(const double* __restrict__ parts, uint32_t num_parts,
                                       const double* __restrict__ extra, int32_t num_extra,
                                       float max_norm, double* lds4) {
  const double acc = strided_sum(strided_sum(0.0, parts, num_parts), extra, (uint32_t)num_extra);
  const double norm = sqrt(block_sum(acc, lds4));
  double c = (double)max_norm / (norm + 1e-6);
  c = c < 1.0 ? c : 1.0;
  return make_float2((float)norm, __builtin_isfinite(norm) ? (float)c : 0.0f);
}

// Elements of one access: 16 bytes of the wider of the two types.
template <class TI, class TO>
constexpr int kScaleVec = 16 / (int)(sizeof(TI) > sizeof(TO) ? sizeof(TI) : sizeof(TO));

template <class TI, class TO, int N>
__device__ inline Raw<TO, N> scaled(const Raw<TI, N>& r, float c) {
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = c == 0.0f ? 0.0f : r.get(i) * c;
  Raw<TO, N> o;
  o.set_all(v);
  return o;
}

template <class TI, class TO>
__device__ inline void chunk_scale(const TI* p, TO* q, int64_t len, float c) {
  constexpr int N = kScaleVec<TI, TO>;
  constexpr int U = kClipChunk / (kClipThreads * N);
  if (len == kClipChunk) {
    Raw<TI, N> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      r[u] = load_raw<TI, N, true>(p + (u * kClipThreads + threadIdx.x) * N);
#pragma unroll
    for (int u = 0; u < U; ++u)
      store_raw<TO, N, true>(q + (u * kClipThreads + threadIdx.x) * N,
                             scaled<TI, TO, N>(r[u], c));
    return;
  }
  const int n = (int)len;
  for (int k = threadIdx.x * N; k + N <= n; k += kClipThreads * N)
    store_raw<TO, N>(q + k, scaled<TI, TO, N>(load_raw<TI, N>(p + k), c));
  const int k = n / N * N + (int)threadIdx.x;
  if (k < n) q[k] = from_f32<TO>(c == 0.0f ? 0.0f : to_f32(p[k]) * c);
}

template <class TI>
__device__ inline void scale_item(const ClipItem& it, int64_t at, int64_t len, float c) {
  const TI* p = static_cast<const TI*>(it.in) + at;
  switch (it.types >> 8) {
    case EMB_F32: chunk_scale(p, static_cast<float*>(it.out) + at, len, c); break;
    case EMB_BF16: chunk_scale(p, static_cast<bf16_t*>(it.out) + at, len, c); break;
    default: chunk_scale(p, static_cast<f16_t*>(it.out) + at, len, c); break;
  }
}

__global__ __launch_bounds__(kClipThreads) void k_clip_norm(const double* __restrict__ parts,
                                                            uint32_t num_parts,
                                                            const double* __restrict__ extra,
                                                            int32_t num_extra, float max_norm,
                                                            float* __restrict__ norm_out) {
  __shared__ double lds4[4];
  const float2 nc = norm_and_coef(parts, num_parts, extra, num_extra, max_norm, lds4);
  if (threadIdx.x == 0) {
    norm_out[0] = nc.x;
    norm_out[1] = nc.y;
  }
}

// Every block forms the coefficient itself (at most kClipDirect sums, which its
// L2 holds), so no launch stands between the sum and the scale, and the first
// block of the first launch stores it; for longer lists it is `ready`.  The
// chunks go from the last one back: what the sum read last is still in the
// cache.
__global__ __launch_bounds__(kClipThreads) void k_clip_scale(
    const ClipList l, const double* __restrict__ parts, uint32_t num_parts,
    const double* __restrict__ extra, int32_t num_extra, float max_norm,
    const float* __restrict__ ready, float* __restrict__ norm_out) {
  __shared__ double lds4[4];
  const ClipFinder find(l);
  float2 nc = make_float2(0.0f, 0.0f);
  if (ready) nc.y = *ready;
  else nc = norm_and_coef(parts, num_parts, extra, num_extra, max_norm, lds4);
  const float c = nc.y;
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) {
    norm_out[0] = nc.x;
    norm_out[1] = c;
  }
  for (uint32_t k = blockIdx.x; k < l.chunks; k += gridDim.x) {
    const uint32_t chunk = l.chunks - 1u - k, i = find(chunk);
    const ClipItem& it = l.item[i];
    if (it.in == it.out && c == 1.0f) continue;  // in place and not clipped: already there
    const int64_t at = (int64_t)(chunk - l.first[i]) * kClipChunk;
    const int64_t len = it.n - at < kClipChunk ? it.n - at : kClipChunk;
    switch (it.types & 0xFFu) {
      case EMB_F32: scale_item<float>(it, at, len, c); break;
      case EMB_BF16: scale_item<bf16_t>(it, at, len, c); break;
      default: scale_item<f16_t>(it, at, len, c); break;
    }
  }
}

// Fills `l` from the list's tensors at `*at` on; advances *at past them.
bool next_list(const emb_tensor_t* grads, const emb_tensor_t* out, int32_t n, int32_t* at,
               ClipList* l) {
  l->count = l->chunks = 0;
  for (; *at < n && l->count < (uint32_t)kClipItems; ++*at) {
    const emb_tensor_t& g = grads[*at];
    if (g.numel == 0) continue;
    const int64_t chunks = (g.numel + kClipChunk - 1) / kClipChunk;
    if ((int64_t)l->chunks + chunks > 0x7FFFFFFF) break;  // the next launch takes it
    ClipItem& it = l->item[l->count];
    l->first[l->count++] = l->chunks;
    it.in = g.data;
    it.out = out ? out[*at].data : nullptr;
    it.n = g.numel;
    it.types = (uint32_t)g.dtype | (uint32_t)(out ? out[*at].dtype : 0) << 8;
    l->chunks += (uint32_t)chunks;
  }
  return l->count != 0;
}

unsigned sum_blocks(const ClipList& l) {
  return l.chunks < (unsigned)kClipParts ? l.chunks : (unsigned)kClipParts;
}

}  // namespace

size_t grad_workspace_bytes(const emb_tensor_t* grads, int32_t n) {
  ClipList l;
  int32_t at = 0;
  size_t parts = 0;
  while (next_list(grads, nullptr, n, &at, &l)) parts += sum_blocks(l);
  return (parts * sizeof(double) + 256) & ~(size_t)255;
}

hipError_t launch_clip_grad_norm(const emb_tensor_t* grads, const emb_tensor_t* out, int32_t n,
                                 const double* extra, int32_t num_extra, float max_norm,
                                 float* norm_out, char* ws, hipStream_t s) {
  double* parts = reinterpret_cast<double*>(ws);
  ClipList l;
  int32_t at = 0;
  uint32_t num_parts = 0, launches = 0;
  while (next_list(grads, out, n, &at, &l)) {
    const unsigned grid = sum_blocks(l);
    hipLaunchKernelGGL(k_grad_square_sum, dim3(grid), dim3(kClipThreads), 0, s, l,
                       parts + num_parts);
    num_parts += grid;
    ++launches;
  }
  // (without an output one block forms the coefficient in any case)
  const bool direct = !out || ((int64_t)num_parts + num_extra) * launches <= kClipDirect;
  if (!direct)
    hipLaunchKernelGGL(k_clip_norm, dim3(1), dim3(kClipThreads), 0, s, parts, num_parts, extra,
                       num_extra, max_norm, norm_out);
  // the coefficient is wanted without an output too: then of an empty list
  at = out ? 0 : n;
  bool more = next_list(grads, out, n, &at, &l);
  const float* ready = direct ? nullptr : norm_out + 1;
  float* store = direct ? norm_out : nullptr;
  do {
    const unsigned grid = l.chunks < (unsigned)kScaleBlocks ? l.chunks : (unsigned)kScaleBlocks;
    hipLaunchKernelGGL(k_clip_scale, dim3(grid ? grid : 1u), dim3(kClipThreads), 0, s, l, parts,
                       num_parts, extra, num_extra, max_norm, ready, store);
    store = nullptr;
    more = more && next_list(grads, out, n, &at, &l);
  } while (more);
  return hipGetLastError();
}

}  // namespace embtab
