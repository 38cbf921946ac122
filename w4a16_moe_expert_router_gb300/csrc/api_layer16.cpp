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
  if (!pair_pos || !topk_w || !rows || !out) return MOE_W4A16_ERR_NULL;
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

}  // extern "C"
