// C ABI of the dense operators (declared in include/embtab.h): host-side
// checks, then the launches on the caller's stream.
#include <cmath>

#include "dense.hpp"

using namespace embtab;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

emb_status_t hip_status(hipError_t e) { return e == hipSuccess ? EMB_OK : EMB_ERR_HIP; }

bool workspace_ok(const void* ws, size_t have, size_t need) {
  return ws && have >= need && aligned(ws, 256);
}

bool tensor_ok(const emb_tensor_t& t) {
  return t.numel >= 0 && t.numel < (1ll << 40) && dtype_ok(t.dtype) &&
         (t.numel == 0 || (t.data && aligned(t.data, dtype_size(t.dtype))));
}

bool list_ok(const emb_tensor_t* l, int32_t n) {
  if (n < 0 || (n > 0 && !l)) return false;
  for (int32_t i = 0; i < n; ++i)
    if (!tensor_ok(l[i])) return false;
  return true;
}

constexpr int64_t kMaxRows = 0x7FFFFFFF;  // rows and choices are int32 in src and pos

bool expert_shape_ok(int64_t tokens, int32_t topk) {
  return tokens >= 0 && topk >= 1 && topk <= 64 && tokens <= kMaxRows / topk;
}

bool rows_ok(int64_t tokens, int32_t topk, int64_t rows, int32_t dim, int32_t dtype) {
  return expert_shape_ok(tokens, topk) && rows >= 0 && rows <= kMaxRows && dim >= 8 &&
         dim <= (1 << 20) && dtype_ok(dtype);
}

bool data_ok(const void* p, int64_t count, size_t align) {
  return count == 0 || (p && aligned(p, align));
}

// Shape, types and the inputs both directions share.
bool gated_norm_ok(const GatedNorm& a, int32_t dtype, int32_t gate_kind) {
  if (a.rows < 0 || a.rows > kMaxRows || a.dim < 8 || a.dim > 8192 || !dtype_ok(dtype))
    return false;
  if (gate_kind < 0 || (gate_kind & ~(EMB_GATE_SIGMOID | 3)) != 0 || a.gate_kind == 3) return false;
  if (a.gate_kind == EMB_GATE_NONE && (a.sigmoid || a.gate)) return false;
  if (!(a.eps >= 0.0f) || !std::isfinite(a.eps)) return false;
  const size_t al = dtype_size(dtype);
  return data_ok(a.x, a.rows, al) && data_ok(a.block, a.rows, al) &&
         (a.gate_kind == EMB_GATE_NONE || data_ok(a.gate, a.rows, al)) && aligned(a.w_post, 4) &&
         a.scale && aligned(a.scale, 4) && a.w_pre && aligned(a.w_pre, 4);
}

// Sizes of the feed-forward.  rows * dim and rows * hidden stay below 2^40, so
// every launch has fewer than 2^31 blocks.
bool ffn_shape_ok(int64_t rows, int32_t experts, int32_t dim, int32_t hidden, int32_t dtype) {
  return rows >= 0 && rows <= kMaxRows && experts >= 1 && experts <= 1024 && dim >= 8 &&
         dim <= 65536 && hidden >= 8 && hidden <= 65536 && dtype_ok(dtype) &&
         rows * dim < (1ll << 40) && rows * hidden < (1ll << 40);
}

bool ffn_ok(const GatedFfn& f, int32_t dtype) {
  if (!ffn_shape_ok(f.rows, f.experts, f.dim, f.hidden, dtype)) return false;
  if (f.act < EMB_ACT_SILU || f.act > EMB_ACT_SIGMOID) return false;
  if (f.offsets ? !aligned(f.offsets, 4) : f.experts != 1 || f.capacity != 0) return false;
  if (f.capacity < 0 || f.capacity > kMaxRows ||
      (f.capacity > 0 && f.rows != f.capacity * f.experts))
    return false;
  const size_t a = dtype_size(dtype);
  return data_ok(f.x, f.rows, a) && f.w_in && aligned(f.w_in, a) && f.w_out &&
         aligned(f.w_out, a);
}

size_t ffn_workspace(int64_t rows, int32_t experts, int32_t dim, int32_t hidden, int32_t dtype) {
  switch (dtype) {
    case EMB_F32: return ffn_workspace_bytes_t<float>(rows, experts, dim, hidden);
    case EMB_BF16: return ffn_workspace_bytes_t<bf16_t>(rows, experts, dim, hidden);
    default: return ffn_workspace_bytes_t<f16_t>(rows, experts, dim, hidden);
  }
}

size_t ffn_forward_workspace(int64_t rows, int32_t experts, int32_t dim, int32_t hidden,
                             int32_t dtype) {
  switch (dtype) {
    case EMB_F32: return ffn_forward_workspace_bytes_t<float>(rows, experts, dim, hidden);
    case EMB_BF16: return ffn_forward_workspace_bytes_t<bf16_t>(rows, experts, dim, hidden);
    default: return ffn_forward_workspace_bytes_t<f16_t>(rows, experts, dim, hidden);
  }
}

}  // namespace

extern "C" {

size_t emb_grad_workspace_bytes(const emb_tensor_t* grads, int32_t n) {
  if (!list_ok(grads, n)) return 0;
  return grad_workspace_bytes(grads, n);
}

emb_status_t emb_clip_grad_norm(const emb_tensor_t* grads, const emb_tensor_t* out, int32_t n,
                                const double* extra_sq, int32_t num_extra, float max_norm,
                                float* norm_out, void* ws, size_t ws_bytes, void* stream) {
  if (!list_ok(grads, n) || (out && !list_ok(out, n))) return EMB_ERR_INVALID_ARG;
  for (int32_t i = 0; out && i < n; ++i)
    if (out[i].numel != grads[i].numel ||
        (out[i].dtype != EMB_F32 && out[i].dtype != grads[i].dtype) ||
        (out[i].data == grads[i].data && out[i].dtype != grads[i].dtype && grads[i].numel > 0))
      return EMB_ERR_INVALID_ARG;
  if (num_extra < 0 || (num_extra > 0 && !extra_sq) || !aligned(extra_sq, 8))
    return EMB_ERR_INVALID_ARG;
  if (!(max_norm >= 0.0f) || !norm_out || !aligned(norm_out, 4)) return EMB_ERR_INVALID_ARG;
  if (!workspace_ok(ws, ws_bytes, grad_workspace_bytes(grads, n))) return EMB_ERR_WORKSPACE;
  return hip_status(launch_clip_grad_norm(grads, out, n, extra_sq, num_extra, max_norm, norm_out,
                                          static_cast<char*>(ws),
                                          static_cast<hipStream_t>(stream)));
}

size_t emb_expert_workspace_bytes(int64_t tokens, int32_t topk, int32_t experts) {
  if (!expert_shape_ok(tokens, topk) || experts < 1 || experts > 1024) return 0;
  return expert_workspace_bytes(tokens, topk, experts);
}

emb_status_t emb_expert_sort(const int64_t* ids, int64_t tokens, int32_t topk, int32_t experts,
                             int64_t capacity, int32_t* offsets, int32_t* src, int32_t* pos,
                             void* ws, size_t ws_bytes, void* stream) {
  if (!expert_shape_ok(tokens, topk) || experts < 1 || experts > 1024 || capacity < 0 ||
      capacity > kMaxRows / experts)
    return EMB_ERR_INVALID_ARG;
  const int64_t rows = capacity ? capacity * experts : tokens * topk;
  if (!data_ok(ids, tokens, 8) || !data_ok(pos, tokens, 4) || !data_ok(src, rows, 4) ||
      !offsets || !aligned(offsets, 4))
    return EMB_ERR_INVALID_ARG;
  if (!workspace_ok(ws, ws_bytes, expert_workspace_bytes(tokens, topk, experts)))
    return EMB_ERR_WORKSPACE;
  return hip_status(launch_expert_sort(ids, tokens, topk, experts, capacity, offsets, src, pos,
                                       static_cast<char*>(ws),
                                       static_cast<hipStream_t>(stream)));
}

emb_status_t emb_expert_dispatch(const void* x, const int32_t* pos, const int32_t* src,
                                 int64_t tokens, int32_t topk, int64_t rows, int32_t dim,
                                 int32_t dtype, void* xs, void* stream) {
  if (!rows_ok(tokens, topk, rows, dim, dtype)) return EMB_ERR_INVALID_ARG;
  const size_t a = dtype_size(dtype);
  if (!data_ok(x, tokens, a) || !data_ok(pos, tokens, 4) || !data_ok(src, rows, 4) ||
      !data_ok(xs, rows, a))
    return EMB_ERR_INVALID_ARG;
  return hip_status(launch_expert_dispatch(x, pos, src, tokens, topk, rows, dim, dtype, xs,
                                           static_cast<hipStream_t>(stream)));
}

emb_status_t emb_expert_combine(const void* ys, const int32_t* pos, const float* weights,
                                int64_t tokens, int32_t topk, int64_t rows, int32_t dim,
                                int32_t dtype, void* y, void* stream) {
  if (!rows_ok(tokens, topk, rows, dim, dtype)) return EMB_ERR_INVALID_ARG;
  const size_t a = dtype_size(dtype);
  if (!data_ok(ys, tokens ? rows : 0, a) || !data_ok(pos, tokens, 4) || !aligned(weights, 4) ||
      !data_ok(y, tokens, a))
    return EMB_ERR_INVALID_ARG;
  return hip_status(launch_expert_combine(ys, pos, weights, tokens, topk, rows, dim, dtype, y,
                                          static_cast<hipStream_t>(stream)));
}

emb_status_t emb_expert_combine_backward(const void* dy, const void* ys, const int32_t* pos,
                                         const int32_t* src, const float* weights,
                                         int64_t tokens, int32_t topk, int64_t rows, int32_t dim,
                                         int32_t dtype, void* dys, float* dweights,
                                         void* stream) {
  if (!rows_ok(tokens, topk, rows, dim, dtype)) return EMB_ERR_INVALID_ARG;
  const size_t a = dtype_size(dtype);
  if (!data_ok(dy, tokens, a) || !data_ok(ys, tokens ? rows : 0, a) || !data_ok(pos, tokens, 4) ||
      !data_ok(src, rows, 4) || !data_ok(weights, tokens, 4) || !data_ok(dys, rows, a) ||
      !data_ok(dweights, tokens, 4))
    return EMB_ERR_INVALID_ARG;
  return hip_status(launch_expert_combine_backward(dy, ys, pos, src, weights, tokens, topk, rows,
                                                   dim, dtype, dys, dweights,
                                                   static_cast<hipStream_t>(stream)));
}

emb_status_t emb_expert_dispatch_backward(const void* dxs, const int32_t* pos, int64_t tokens,
                                          int32_t topk, int64_t rows, int32_t dim, int32_t dtype,
                                          void* dx, void* stream) {
  return emb_expert_combine(dxs, pos, nullptr, tokens, topk, rows, dim, dtype, dx, stream);
}

size_t emb_gated_norm_workspace_bytes(int64_t rows, int32_t dim) {
  if (rows < 0 || rows > kMaxRows || dim < 8 || dim > 8192) return 0;
  return gated_norm_workspace_bytes(rows, dim);
}

emb_status_t emb_gated_norm_forward(const void* x, const void* block, const void* gate,
                                    const float* w_post, const float* scale, const float* w_pre,
                                    int64_t rows, int32_t dim, int32_t dtype, int32_t gate_kind,
                                    float eps, void* y, void* h, void* stream) {
  const GatedNorm a{x, block, gate, w_post, scale, w_pre, rows, dim, gate_kind & 3,
                    (gate_kind & EMB_GATE_SIGMOID) != 0, eps};
  if (!gated_norm_ok(a, dtype, gate_kind)) return EMB_ERR_INVALID_ARG;
  if (!data_ok(y, rows, dtype_size(dtype)) || !data_ok(h, rows, dtype_size(dtype)))
    return EMB_ERR_INVALID_ARG;
  return hip_status(
      launch_gated_norm_forward(a, dtype, y, h, static_cast<hipStream_t>(stream)));
}

emb_status_t emb_gated_norm_backward(const void* y, const void* block, const void* gate,
                                     const float* w_post, const float* scale, const float* w_pre,
                                     const void* dy, const void* dh, int64_t rows, int32_t dim,
                                     int32_t dtype, int32_t gate_kind, float eps, void* dx,
                                     void* dblock, void* dgate, float* dw_post, float* dscale,
                                     float* dw_pre, void* ws, size_t ws_bytes, void* stream) {
  const GatedNorm a{y, block, gate, w_post, scale, w_pre, rows, dim, gate_kind & 3,
                    (gate_kind & EMB_GATE_SIGMOID) != 0, eps};
  if (!gated_norm_ok(a, dtype, gate_kind)) return EMB_ERR_INVALID_ARG;
  const size_t al = dtype_size(dtype);
  if (!data_ok(dy, rows, al) || !data_ok(dh, rows, al) || !data_ok(dx, rows, al) ||
      !data_ok(dblock, rows, al) || !dscale || !aligned(dscale, 4) || !dw_pre ||
      !aligned(dw_pre, 4) || !aligned(dw_post, 4))
    return EMB_ERR_INVALID_ARG;
  // a gradient is wanted for exactly what the forward took
  if ((w_post != nullptr) != (dw_post != nullptr)) return EMB_ERR_INVALID_ARG;
  if (a.gate_kind == EMB_GATE_NONE ? dgate != nullptr : !data_ok(dgate, rows, al))
    return EMB_ERR_INVALID_ARG;
  if (!workspace_ok(ws, ws_bytes, gated_norm_workspace_bytes(rows, dim))) return EMB_ERR_WORKSPACE;
  return hip_status(launch_gated_norm_backward(a, dtype, dy, dh, dx, dblock, dgate, dw_post,
                                               dscale, dw_pre, static_cast<char*>(ws),
                                               static_cast<hipStream_t>(stream)));
}

size_t emb_gated_ffn_workspace_bytes(int64_t rows, int32_t experts, int32_t dim, int32_t hidden,
                                     int32_t dtype) {
  if (!ffn_shape_ok(rows, experts, dim, hidden, dtype)) return 0;
  return ffn_workspace(rows, experts, dim, hidden, dtype);
}

size_t emb_gated_ffn_forward_workspace_bytes(int64_t rows, int32_t experts, int32_t dim,
                                             int32_t hidden, int32_t dtype) {
  if (!ffn_shape_ok(rows, experts, dim, hidden, dtype)) return 0;
  return ffn_forward_workspace(rows, experts, dim, hidden, dtype);
}

emb_status_t emb_gated_ffn_forward(const void* x, const void* w_in, const void* w_out,
                                   const int32_t* offsets, int64_t rows, int32_t experts,
                                   int64_t capacity, int32_t dim, int32_t hidden, int32_t dtype,
                                   int32_t act, void* gu, void* a, void* y, void* ws,
                                   size_t ws_bytes, void* stream) {
  const GatedFfn f{x, w_in, w_out, offsets, rows, capacity, experts, dim, hidden, act};
  if (!ffn_ok(f, dtype)) return EMB_ERR_INVALID_ARG;
  const size_t al = dtype_size(dtype);
  if (!aligned(gu, al) || !data_ok(a, rows, al) || !data_ok(y, rows, al))
    return EMB_ERR_INVALID_ARG;
  const size_t need = gu ? ffn_workspace(rows, experts, dim, hidden, dtype)
                         : ffn_forward_workspace(rows, experts, dim, hidden, dtype);
  if (!workspace_ok(ws, ws_bytes, need)) return EMB_ERR_WORKSPACE;
  char* w = static_cast<char*>(ws);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  switch (dtype) {
    case EMB_F32: return hip_status(ffn_forward_t<float>(f, gu, a, y, w, s));
    case EMB_BF16: return hip_status(ffn_forward_t<bf16_t>(f, gu, a, y, w, s));
    default: return hip_status(ffn_forward_t<f16_t>(f, gu, a, y, w, s));
  }
}

emb_status_t emb_gated_ffn_backward(const void* x, const void* gu, const void* a,
                                    const void* w_in, const void* w_out, const void* dy,
                                    const int32_t* offsets, int64_t rows, int32_t experts,
                                    int64_t capacity, int32_t dim, int32_t hidden, int32_t dtype,
                                    int32_t act, void* dx, void* dw_in, void* dw_out, void* ws,
                                    size_t ws_bytes, void* stream) {
  const GatedFfn f{x, w_in, w_out, offsets, rows, capacity, experts, dim, hidden, act};
  if (!ffn_ok(f, dtype)) return EMB_ERR_INVALID_ARG;
  const size_t al = dtype_size(dtype);
  if (!data_ok(gu, rows, al) || !data_ok(a, rows, al) || !data_ok(dy, rows, al) ||
      !data_ok(dx, rows, al) || !dw_in || !aligned(dw_in, al) || !dw_out || !aligned(dw_out, al))
    return EMB_ERR_INVALID_ARG;
  if (!workspace_ok(ws, ws_bytes, ffn_workspace(rows, experts, dim, hidden, dtype)))
    return EMB_ERR_WORKSPACE;
  char* w = static_cast<char*>(ws);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  switch (dtype) {
    case EMB_F32: return hip_status(ffn_backward_t<float>(f, gu, a, dy, dx, dw_in, dw_out, w, s));
    case EMB_BF16:
      return hip_status(ffn_backward_t<bf16_t>(f, gu, a, dy, dx, dw_in, dw_out, w, s));
    default: return hip_status(ffn_backward_t<f16_t>(f, gu, a, dy, dx, dw_in, dw_out, w, s));
  }
}

emb_status_t emb_add_norm_int8(const void* x, const void* block, const float* w, int64_t rows,
                               int32_t dim, int32_t dtype, float eps, void* y, int8_t* codes,
                               float* scales, void* stream) {
  if (rows < 0 || rows > kMaxRows || dim < 8 || dim > 8192 || !dtype_ok(dtype) ||
      !(eps >= 0.0f) || !std::isfinite(eps))
    return EMB_ERR_INVALID_ARG;
  const size_t a = dtype_size(dtype);
  if (!data_ok(x, rows, a) || !data_ok(block, rows, a) || !w || !aligned(w, 4) ||
      !data_ok(y, rows, a) || !data_ok(codes, rows, 1) || !data_ok(scales, rows, 4))
    return EMB_ERR_INVALID_ARG;
  return hip_status(launch_add_norm_int8({x, block, w, rows, dim, eps}, dtype, y, codes, scales,
                                         static_cast<hipStream_t>(stream)));
}

emb_status_t emb_expert_dispatch_int8(const int8_t* codes, const float* scales,
                                      const int32_t* pos, const int32_t* src, int64_t tokens,
                                      int32_t topk, int64_t rows, int32_t dim, int32_t dtype,
                                      void* xs, void* stream) {
  if (!rows_ok(tokens, topk, rows, dim, dtype)) return EMB_ERR_INVALID_ARG;
  if (!data_ok(codes, tokens, 1) || !data_ok(scales, tokens, 4) || !data_ok(pos, tokens, 4) ||
      !data_ok(src, rows, 4) || !data_ok(xs, rows, dtype_size(dtype)))
    return EMB_ERR_INVALID_ARG;
  return hip_status(launch_expert_dispatch_int8(codes, scales, pos, src, tokens, topk, rows, dim,
                                                dtype, xs, static_cast<hipStream_t>(stream)));
}

emb_status_t emb_dropout(const void* x, const void* residual, int64_t numel, int32_t dtype,
                         double p, const int64_t* rng, void* y, void* stream) {
  if (numel < 0 || numel >= (1ll << 40) || !dtype_ok(dtype) || !(p >= 0.0 && p <= 1.0))
    return EMB_ERR_INVALID_ARG;
  const size_t a = dtype_size(dtype);
  if (!data_ok(x, numel, a) || !aligned(residual, a) || !rng || !aligned(rng, 8) ||
      !data_ok(y, numel, a))
    return EMB_ERR_INVALID_ARG;
  const uint32_t keep = (uint32_t)std::floor((1.0 - p) * 65536.0 + 0.5);
  return hip_status(launch_dropout(x, residual, numel, dtype, keep, rng, y,
                                   static_cast<hipStream_t>(stream)));
}

}  // extern "C"
