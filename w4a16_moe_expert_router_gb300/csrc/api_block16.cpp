// api_block16.cpp -- the C ABI of the operators around the layer (the whole layer for a few
// tokens, the norms around a block with their gradient, the gradients' norm and clipping):
// host-side validation and the launches.  Nothing here reads device data, allocates device
// memory or synchronises the host.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "internal.h"
#include "moe_w4a16.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <typename... P>
bool all_aligned(const P*... p) {  // NULL counts as aligned
  return (... && aligned16(p));
}
moe_w4a16_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_W4A16_OK : MOE_W4A16_ERR_CUDA; }

moe_w4a16_status check_few(const moe_w4a16_shape* shape, moe::Dims* out) {
  const moe_w4a16_status st = moe::check_shape(shape, out);
  if (st != MOE_W4A16_OK) return st;
  return out->T > moe::kFewTokens ? MOE_W4A16_ERR_SHAPE : MOE_W4A16_OK;
}

moe_w4a16_status check_norm(const moe_w4a16_norm_cfg* c, moe::NormDims* out) {
  if (!c) return MOE_W4A16_ERR_NULL;
  if (c->rows < 0 || c->rows > moe::kMaxPairs || c->hidden < 8 || c->hidden % 8 != 0 || c->hidden > moe::kMaxHidden ||
      c->type < 0 || c->type > 2 || c->gate_rows < 0 || c->gate_rows > moe::kMaxPairs)
    return MOE_W4A16_ERR_SHAPE;
  if (!std::isfinite(c->residual_scale) || !std::isfinite(c->eps) || c->eps < 0.f) return MOE_W4A16_ERR_VALUE;
  *out = moe::NormDims{c->rows, c->hidden, c->type, c->gate_rows, c->residual_scale, c->eps};
  return MOE_W4A16_OK;
}

}  // namespace

extern "C" {

size_t moe_w4a16_few_workspace_bytes(const moe_w4a16_shape* shape) {
  moe::Dims s;
  return check_few(shape, &s) == MOE_W4A16_OK ? moe::few_ws_bytes(s) : 0;
}

moe_w4a16_status moe_w4a16_few(const moe_w4a16_shape* shape, int32_t type, const void* x, const float* logits,
                               const moe_w4a16_weights* weights, const void* residual, int32_t* topk_idx,
                               float* topk_w, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  moe::Dims s;
  moe_w4a16_status st = check_few(shape, &s);
  if (st != MOE_W4A16_OK) return st;
  if (type != MOE_W4A16_FP16 && type != MOE_W4A16_BF16) return MOE_W4A16_ERR_SHAPE;
  if (s.T == 0) return MOE_W4A16_OK;
  if (!x || !logits || !weights || !weights->gate_up || !weights->down || !out || !workspace) return MOE_W4A16_ERR_NULL;
  if (!all_aligned(x, residual, static_cast<const void*>(out), static_cast<const void*>(workspace)) ||
      !all_aligned(logits, topk_w) || !all_aligned(weights->gate_up, weights->down) || !aligned16(topk_idx))
    return MOE_W4A16_ERR_ALIGN;
  if (workspace_bytes < moe::few_ws_bytes(s)) return MOE_W4A16_ERR_WORKSPACE;
  int sms = 0;
  const moe::FewClusters* clusters = nullptr;
  if ((st = moe::current_device(&sms, &clusters)) != MOE_W4A16_OK) return st;
  return cuda_status(moe::launch_few(s, type, x, logits, weights->gate_up, weights->down, residual, topk_idx, topk_w,
                                     out, workspace, sms, *clusters, static_cast<cudaStream_t>(stream)));
}

moe_w4a16_status moe_w4a16_norm(const moe_w4a16_norm_cfg* cfg, const void* x, const void* y, const float* gamma_post,
                                const float* gate, const float* gamma_pre, void* out, void* u, void* stream) {
  moe::NormDims s;
  moe_w4a16_status st = check_norm(cfg, &s);
  if (st != MOE_W4A16_OK) return st;
  if (gate && s.gate_rows == 0) return MOE_W4A16_ERR_SHAPE;
  if (s.R == 0) return MOE_W4A16_OK;
  if ((!x && !y) || (!out && !u) || ((gamma_post || gate) && !y) || ((u != nullptr) != (gamma_pre != nullptr)))
    return MOE_W4A16_ERR_NULL;
  if (!all_aligned(x, y, static_cast<const void*>(out), static_cast<const void*>(u)) ||
      !all_aligned(gamma_post, gate, gamma_pre))
    return MOE_W4A16_ERR_ALIGN;
  int sms = 0;
  if ((st = moe::current_device(&sms)) != MOE_W4A16_OK) return st;
  return cuda_status(
      moe::launch_norm(s, x, y, gamma_post, gate, gamma_pre, out, u, static_cast<cudaStream_t>(stream)));
}

size_t moe_w4a16_norm_backward_workspace_bytes(const moe_w4a16_norm_cfg* cfg) {
  moe::NormDims s;
  return check_norm(cfg, &s) == MOE_W4A16_OK ? moe::norm_backward_ws_bytes(s) : 0;
}

moe_w4a16_status moe_w4a16_norm_backward(const moe_w4a16_norm_cfg* cfg, const void* y, const float* gamma_post,
                                         const float* gate, const void* out, const float* gamma_pre,
                                         const void* grad_out, const void* grad_u, void* grad_x, void* grad_y,
                                         float* grad_gamma_post, float* grad_gate, float* grad_gamma_pre,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  moe::NormDims s;
  moe_w4a16_status st = check_norm(cfg, &s);
  if (st != MOE_W4A16_OK) return st;
  if ((gate || grad_gate) && s.gate_rows == 0) return MOE_W4A16_ERR_SHAPE;
  if (!grad_x && !grad_y && !grad_gamma_post && !grad_gate && !grad_gamma_pre) return MOE_W4A16_ERR_NULL;
  if (s.R > 0) {
    const bool sums = grad_gamma_post || grad_gate || grad_gamma_pre;
    if ((!grad_out && !grad_u) || (grad_u && (!out || !gamma_pre)) || (grad_gamma_pre && !grad_u) ||
        (grad_gamma_post && !gamma_post) || (grad_gate && !gate) || (sums && !workspace))
      return MOE_W4A16_ERR_NULL;
    if (!y && ((grad_y && gamma_post) || grad_gamma_post || grad_gate)) return MOE_W4A16_ERR_NULL;
  }
  if (!all_aligned(y, out, grad_out, grad_u, static_cast<const void*>(grad_x), static_cast<const void*>(grad_y),
                   static_cast<const void*>(workspace)) ||
      !all_aligned(gamma_post, gate, gamma_pre, static_cast<const float*>(grad_gamma_post),
                   static_cast<const float*>(grad_gate), static_cast<const float*>(grad_gamma_pre)))
    return MOE_W4A16_ERR_ALIGN;
  if (s.R > 0 && workspace && workspace_bytes < moe::norm_backward_ws_bytes(s)) return MOE_W4A16_ERR_WORKSPACE;
  int sms = 0;
  if ((st = moe::current_device(&sms)) != MOE_W4A16_OK) return st;
  const auto cs = static_cast<cudaStream_t>(stream);
  if (s.R == 0) {  // no rows: the sums are zero (a gate has no rows then)
    for (float* p : {grad_gamma_post, grad_gamma_pre})
      if (p && cudaMemsetAsync(p, 0, size_t(s.d) * 4, cs) != cudaSuccess) return MOE_W4A16_ERR_CUDA;
    return MOE_W4A16_OK;
  }
  return cuda_status(moe::launch_norm_backward(s, y, gamma_post, gate, out, gamma_pre, grad_out, grad_u, grad_x, grad_y,
                                               grad_gamma_post, grad_gate, grad_gamma_pre, workspace, cs));
}

size_t moe_w4a16_clip_workspace_bytes(int32_t count) {
  return count < 0 || count > moe::kClipMaxTensors ? 0 : moe::clip_ws_bytes(count);
}

moe_w4a16_status moe_w4a16_clip(const moe_w4a16_tensor* tensors, int32_t count, double max_norm, float* norm,
                                void* workspace, size_t workspace_bytes, void* stream) {
  if (count < 0 || count > moe::kClipMaxTensors) return MOE_W4A16_ERR_SHAPE;
  if ((!tensors && count > 0) || !norm || !workspace) return MOE_W4A16_ERR_NULL;
  if (!(max_norm >= 0.0)) return MOE_W4A16_ERR_VALUE;
  if ((reinterpret_cast<uintptr_t>(norm) & 3u) != 0 || !aligned16(workspace)) return MOE_W4A16_ERR_ALIGN;
  for (int32_t i = 0; i < count; ++i) {
    const moe_w4a16_tensor& t = tensors[i];
    if (t.type < 0 || t.type > 2 || t.count < 0 || t.count > moe::kClipMaxCount) return MOE_W4A16_ERR_SHAPE;
    if (!t.data && t.count > 0) return MOE_W4A16_ERR_NULL;
    const uintptr_t low = t.type == 2 ? 3u : 1u;
    if (((reinterpret_cast<uintptr_t>(t.data) | reinterpret_cast<uintptr_t>(t.out)) & low) != 0)
      return MOE_W4A16_ERR_ALIGN;
  }
  if (workspace_bytes < moe::clip_ws_bytes(count)) return MOE_W4A16_ERR_WORKSPACE;
  int sms = 0;
  const moe_w4a16_status st = moe::current_device(&sms);
  if (st != MOE_W4A16_OK) return st;
  return cuda_status(
      moe::launch_clip(tensors, count, max_norm, norm, workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
