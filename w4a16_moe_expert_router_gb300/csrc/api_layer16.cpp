// api_layer16.cpp -- the C ABI of the 16-bit layer's operators (rows sorted by
// expert and back, products with an epilogue, and their gradients): host-side
// validation and the launches.  Nothing here reads device data, allocates device
// memory or synchronises the host.
#include <cstdint>

#include <cuda_runtime.h>

#include "internal.h"
#include "moe_w4a16.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
moe_w4a16_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_W4A16_OK : MOE_W4A16_ERR_CUDA; }

template <typename... P>
bool any_null(const P*... p) {
  return (... || (p == nullptr));
}
template <typename... P>
bool all_aligned(const P*... p) {  // NULL counts as aligned
  return (... && aligned16(p));
}

moe_w4a16_status check_rows(const moe_w4a16_rows* c, moe::RowDims* out) {
  if (!c) return MOE_W4A16_ERR_NULL;
  const moe::RowDims s{c->tokens, c->experts, c->top_k, c->hidden, c->type};
  if (s.T < 0 || s.E < 1 || s.E > moe::kMaxExperts || s.k < 1 || s.k > moe::kMaxTopK || s.k > s.E ||
      s.d < 8 || s.d % 8 != 0 || s.d > moe::kMaxRowCols || s.type < 0 || s.type > 2 || s.pairs() > moe::kMaxPairs)
    return MOE_W4A16_ERR_SHAPE;
  *out = s;
  return MOE_W4A16_OK;
}

moe_w4a16_status check_linear(const moe_w4a16_linear_cfg* c, moe::LinearDims* out) {
  if (!c) return MOE_W4A16_ERR_NULL;
  const auto cols_ok = [](int n) { return n >= 8 && n % 8 == 0 && n <= moe::kMaxRowCols; };
  if (c->rows < 0 || c->rows > moe::kMaxPairs || !cols_ok(c->in) || !cols_ok(c->out) || c->groups < 1 ||
      c->groups > moe::kMaxExperts || c->activation < 0 || c->activation > 3 || c->gated < 0 || c->gated > 1 ||
      c->type < 0 || c->type > 1)
    return MOE_W4A16_ERR_SHAPE;
  *out = moe::LinearDims{c->rows, c->in, c->out, c->groups, c->activation, c->gated, c->type, false};
  return MOE_W4A16_OK;
}

// Workspace of the gradient: header | dz | partial sums of the bias gradient (sized for
// rows sorted by expert, which have the most row blocks).
struct GradWorkspace {
  size_t dz, partial, total;
};
GradWorkspace grad_workspace(moe::LinearDims s) {
  GradWorkspace w;
  s.grouped = true;
  w.dz = sizeof(moe::WsHeader);
  w.partial = w.dz + (size_t(s.R) * s.Nw() * 2 + 255) / 256 * 256;
  w.total = w.partial + size_t(moe::linear_row_blocks(s)) * s.Nw() * 4;
  return w;
}

}  // namespace

extern "C" {

size_t moe_w4a16_dispatch_workspace_bytes(const moe_w4a16_rows* cfg) {
  moe::RowDims s;
  return check_rows(cfg, &s) == MOE_W4A16_OK ? moe::dispatch_ws_bytes(s) : 0;
}

moe_w4a16_status moe_w4a16_dispatch(const moe_w4a16_rows* cfg, const int32_t* topk_idx, const void* x,
                                    int32_t* expert_offsets, int32_t* pair_list, int32_t* pair_pos, void* rows,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  moe::RowDims s;
  moe_w4a16_status st = check_rows(cfg, &s);
  if (st != MOE_W4A16_OK) return st;
  const auto cs = static_cast<cudaStream_t>(stream);
  int sms = 0;
  if (s.T == 0) {  // no pairs: every expert is empty
    if (!expert_offsets) return MOE_W4A16_ERR_NULL;
    if (!aligned16(expert_offsets)) return MOE_W4A16_ERR_ALIGN;
    if ((st = moe::current_device(&sms)) != MOE_W4A16_OK) return st;
    return cuda_status(cudaMemsetAsync(expert_offsets, 0, (size_t(s.E) + 1) * 4, cs));
  }
  if (any_null(topk_idx, expert_offsets, pair_list, pair_pos) || any_null(x, rows, workspace)) return MOE_W4A16_ERR_NULL;
  if (!all_aligned(topk_idx, expert_offsets, pair_list, pair_pos) || !all_aligned(x, rows, workspace))
    return MOE_W4A16_ERR_ALIGN;
  if (workspace_bytes < moe::dispatch_ws_bytes(s)) return MOE_W4A16_ERR_WORKSPACE;
  if ((st = moe::current_device(&sms)) != MOE_W4A16_OK) return st;
  return cuda_status(
      moe::launch_dispatch(s, topk_idx, x, expert_offsets, pair_list, pair_pos, rows, workspace, cs));
}

moe_w4a16_status moe_w4a16_dispatch_backward(const moe_w4a16_rows* cfg, const int32_t* pair_pos, const void* grad_rows,
                                             void* grad_x, void* stream) {
  moe::RowDims s;
  moe_w4a16_status st = check_rows(cfg, &s);
  if (st != MOE_W4A16_OK) return st;
  if (s.T == 0) return MOE_W4A16_OK;
  if (!pair_pos || !grad_rows || !grad_x) return MOE_W4A16_ERR_NULL;
  if (!aligned16(pair_pos) || !all_aligned(grad_rows, grad_x)) return MOE_W4A16_ERR_ALIGN;
  int sms = 0;
  if ((st = moe::current_device(&sms)) != MOE_W4A16_OK) return st;
  return cuda_status(moe::launch_combine_rows(s, pair_pos, nullptr, grad_rows, nullptr, grad_x,
                                              static_cast<cudaStream_t>(stream)));
}

moe_w4a16_status moe_w4a16_combine_rows(const moe_w4a16_rows* cfg, const int32_t* pair_pos, const float* topk_w,
                                        const void* rows, const void* residual, void* out, void* stream) {
  moe::RowDims s;
  moe_w4a16_status st = check_rows(cfg, &s);
  if (st != MOE_W4A16_OK) return st;
  if (s.T == 0) return MOE_W4A16_OK;
  if (!pair_pos || !rows || !out) return MOE_W4A16_ERR_NULL;
  if (!aligned16(pair_pos) || !aligned16(topk_w) || !all_aligned(rows, residual, out)) return MOE_W4A16_ERR_ALIGN;
  int sms = 0;
  if ((st = moe::current_device(&sms)) != MOE_W4A16_OK) return st;
  return cuda_status(
      moe::launch_combine_rows(s, pair_pos, topk_w, rows, residual, out, static_cast<cudaStream_t>(stream)));
}

moe_w4a16_status moe_w4a16_combine_rows_backward(const moe_w4a16_rows* cfg, const int32_t* topk_idx,
                                                 const int32_t* pair_pos, const float* topk_w, const void* rows,
                                                 const void* grad_out, void* grad_rows, float* grad_topk_w,
                                                 float* grad_logits, void* stream) {
  moe::RowDims s;
  moe_w4a16_status st = check_rows(cfg, &s);
  if (st != MOE_W4A16_OK) return st;
  if (s.T == 0) return MOE_W4A16_OK;
  if (!pair_pos || !topk_w || !rows || !grad_out || (grad_logits && !topk_idx)) return MOE_W4A16_ERR_NULL;
  if (!grad_rows && !grad_topk_w && !grad_logits) return MOE_W4A16_ERR_NULL;
  if (!all_aligned(topk_idx, pair_pos) || !all_aligned(topk_w, grad_topk_w, grad_logits) ||
      !all_aligned(rows, grad_out, grad_rows))
    return MOE_W4A16_ERR_ALIGN;
  int sms = 0;
  if ((st = moe::current_device(&sms)) != MOE_W4A16_OK) return st;
  return cuda_status(moe::launch_combine_rows_backward(s, topk_idx, pair_pos, topk_w, rows, grad_out, grad_rows,
                                                       grad_topk_w, grad_logits, static_cast<cudaStream_t>(stream)));
}

size_t moe_w4a16_linear_workspace_bytes(const moe_w4a16_linear_cfg* cfg) {
  moe::LinearDims s;
  return check_linear(cfg, &s) == MOE_W4A16_OK ? sizeof(moe::WsHeader) : 0;
}

size_t moe_w4a16_linear_backward_workspace_bytes(const moe_w4a16_linear_cfg* cfg) {
  moe::LinearDims s;
  return check_linear(cfg, &s) == MOE_W4A16_OK ? grad_workspace(s).total : 0;
}

moe_w4a16_status moe_w4a16_linear(const moe_w4a16_linear_cfg* cfg, const void* x, const int32_t* expert_offsets,
                                  const void* weight, const float* bias, const void* residual, void* out, void* preact,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  moe::LinearDims s;
  moe_w4a16_status st = check_linear(cfg, &s);
  if (st != MOE_W4A16_OK) return st;
  if (s.R == 0) return MOE_W4A16_OK;
  s.grouped = expert_offsets != nullptr;
  if (!s.grouped && s.E != 1) return MOE_W4A16_ERR_NULL;
  if (any_null(x, weight, out, workspace)) return MOE_W4A16_ERR_NULL;
  if (!all_aligned(x, weight, residual, out, preact, workspace) || !aligned16(expert_offsets) || !aligned16(bias))
    return MOE_W4A16_ERR_ALIGN;
  if (workspace_bytes < sizeof(moe::WsHeader)) return MOE_W4A16_ERR_WORKSPACE;
  int sms = 0;
  if ((st = moe::current_device(&sms)) != MOE_W4A16_OK) return st;
  const auto cs = static_cast<cudaStream_t>(stream);
  int32_t* const err = &static_cast<moe::WsHeader*>(workspace)->error;
  if (moe::is_small_linear(s))
    return cuda_status(
        moe::launch_linear_small(s, expert_offsets, x, weight, bias, residual, out, preact, err, sms, cs));
  return cuda_status(moe::launch_linear(s, expert_offsets, x, weight, bias, residual, out, preact, err, sms, cs));
}

moe_w4a16_status moe_w4a16_linear_backward(const moe_w4a16_linear_cfg* cfg, const void* x,
                                           const int32_t* expert_offsets, const void* weight, const void* preact,
                                           const void* grad_out, void* grad_x, void* grad_weight, float* grad_bias,
                                           void* workspace, size_t workspace_bytes, void* stream) {
  moe::LinearDims s;
  moe_w4a16_status st = check_linear(cfg, &s);
  if (st != MOE_W4A16_OK) return st;
  s.grouped = expert_offsets != nullptr;
  if (!s.grouped && s.E != 1) return MOE_W4A16_ERR_NULL;
  if (!grad_x && !grad_weight && !grad_bias) return MOE_W4A16_ERR_NULL;
  const bool needs_z = s.gated || s.act != 3;
  if (s.R > 0) {
    if (!grad_out || !workspace || (needs_z && !preact) || (grad_weight && !x) || (grad_x && !weight))
      return MOE_W4A16_ERR_NULL;
  }
  if (!all_aligned(x, weight, preact, grad_out, grad_x, grad_weight, workspace) || !aligned16(expert_offsets) ||
      !aligned16(grad_bias))
    return MOE_W4A16_ERR_ALIGN;
  const GradWorkspace w = grad_workspace(s);
  if (s.R > 0 && workspace_bytes < w.total) return MOE_W4A16_ERR_WORKSPACE;
  int sms = 0;
  if ((st = moe::current_device(&sms)) != MOE_W4A16_OK) return st;
  const auto cs = static_cast<cudaStream_t>(stream);
  if (s.R == 0) {
    if (grad_weight && cudaMemsetAsync(grad_weight, 0, size_t(s.E) * s.Nw() * s.K * 2, cs) != cudaSuccess)
      return MOE_W4A16_ERR_CUDA;
    if (grad_bias && cudaMemsetAsync(grad_bias, 0, size_t(s.E) * s.Nw() * 4, cs) != cudaSuccess)
      return MOE_W4A16_ERR_CUDA;
    return MOE_W4A16_OK;
  }
  auto* base = static_cast<uint8_t*>(workspace);
  int32_t* err = &static_cast<moe::WsHeader*>(workspace)->error;
  const void* dz = needs_z ? base + w.dz : grad_out;
  auto* const partial = grad_bias ? reinterpret_cast<float*>(base + w.partial) : nullptr;
  if ((needs_z || grad_bias) &&
      moe::launch_linear_dz(s, expert_offsets, needs_z ? preact : nullptr, grad_out, base + w.dz, partial, cs) !=
          cudaSuccess)
    return MOE_W4A16_ERR_CUDA;
  if (grad_x &&
      moe::launch_linear_input_grad(s, expert_offsets, weight, dz, grad_x, err, sms, cs) != cudaSuccess)
    return MOE_W4A16_ERR_CUDA;
  if (grad_weight && moe::launch_linear_weight_grad(s, expert_offsets, x, dz, grad_weight, partial, grad_bias, err, sms,
                                                    cs) != cudaSuccess)
    return MOE_W4A16_ERR_CUDA;
  if (grad_bias && !grad_weight &&
      moe::launch_linear_dbias(s, expert_offsets, partial, grad_bias, cs) != cudaSuccess)
    return MOE_W4A16_ERR_CUDA;
  return MOE_W4A16_OK;
}

}  // extern "C"
