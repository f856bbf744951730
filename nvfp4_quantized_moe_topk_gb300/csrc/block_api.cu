// block_api.cu -- C entry points of the operators around the layer (declared
// in include/moe_nvfp4.h): argument checks, each before anything is enqueued,
// and the launches.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/moe_nvfp4.h"
#include "kernels.h"

namespace {

using namespace moe;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool is_dtype(int32_t d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F32; }
int64_t dtype_bytes(int32_t d) { return d == MOE_DTYPE_BF16 ? 2 : 4; }

// A row array whose data may be NULL: aligned, rows that do not overlap (and
// a stride below 2^31 vectors of 16 bytes, as the kernels address them).
bool rows_ok(const moe_rows& r, int64_t cols, int32_t dtype) {
  if (!r.data) return true;
  return aligned(r.data, 16) && (r.stride == 0 || (r.stride >= cols && r.stride <= (int64_t(1) << 31) &&
                                                   r.stride * dtype_bytes(dtype) % 16 == 0));
}

moe_status status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

moe_status check_norm(const moe_block_norm_args& a) {
  if (a.n < 0 || a.hidden <= 0) return MOE_ERR_INVALID_ARG;
  if (!is_dtype(a.residual_dtype) || !is_dtype(a.branch_dtype) || !is_dtype(a.param_dtype)) return MOE_ERR_INVALID_ARG;
  if (a.gate_kind < MOE_GATE_NONE || a.gate_kind > MOE_GATE_FULL || (a.gate_sigmoid != 0 && a.gate_sigmoid != 1))
    return MOE_ERR_INVALID_ARG;
  if (a.gate_sigmoid && a.gate_kind == MOE_GATE_NONE) return MOE_ERR_INVALID_ARG;
  if (!(a.eps > 0.f)) return MOE_ERR_INVALID_ARG;
  if (a.hidden % 8 || a.hidden > kNormMaxHidden) return MOE_ERR_UNSUPPORTED;
  if (!rows_ok(a.residual, a.hidden, a.residual_dtype) || !rows_ok(a.branch, a.hidden, a.branch_dtype) ||
      !rows_ok(a.residual_out, a.hidden, a.residual_dtype) || !rows_ok(a.x_out, a.hidden, MOE_DTYPE_BF16))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(a.post_weight, 16) || !aligned(a.pre_weight, 16) || !aligned(a.rstd_post, 4) || !aligned(a.rstd_pre, 4))
    return MOE_ERR_INVALID_ARG;
  if ((a.gate_kind != MOE_GATE_NONE) != (a.gate.data != nullptr) && a.n > 0) return MOE_ERR_INVALID_ARG;
  if (a.gate_kind == MOE_GATE_FULL ? !rows_ok(a.gate, a.hidden, a.branch_dtype)
                                   : !aligned(a.gate.data, a.gate_kind == MOE_GATE_TOKEN ? 4 : 16))
    return MOE_ERR_INVALID_ARG;
  if (a.n > 0 && !a.branch.data && (a.post_weight || a.gate_kind != MOE_GATE_NONE || a.rstd_post))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status check_router(const moe_router_args& a) {
  if (a.n < 0 || a.n_experts <= 0 || a.top_k < 1 || a.n_seqs < 1) return MOE_ERR_INVALID_ARG;
  if (a.top_k > 32 || a.n_experts > 1024) return MOE_ERR_UNSUPPORTED;
  if (!a.seq_offsets && a.n_seqs != 1) return MOE_ERR_INVALID_ARG;
  if (a.n > 0 && (!a.logits || !a.topk_ids)) return MOE_ERR_INVALID_ARG;
  if (!aligned(a.logits, 4) || !aligned(a.bias, 4) || !aligned(a.topk_ids, 4) || !aligned(a.seq_offsets, 4) ||
      !aligned(a.counts, 4) || !aligned(a.tokens, 4))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_block_norm(const moe_block_norm_args* args, moe_stream_t stream) {
  if (!args) return MOE_ERR_INVALID_ARG;
  const moe_block_norm_args& a = *args;
  const moe_status st = check_norm(a);
  if (st != MOE_OK) return st;
  if (a.n == 0) return MOE_OK;
  if (!a.residual.data || (!a.pre_weight && !a.residual_out.data)) return MOE_ERR_INVALID_ARG;
  if ((a.pre_weight != nullptr) != (a.x_out.data != nullptr) || (a.rstd_pre && !a.pre_weight) ||
      (a.rstd_post && !a.post_weight))
    return MOE_ERR_INVALID_ARG;
  return status_of(launch_block_norm(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_block_norm_workspace_bytes(int32_t n, int32_t hidden) {
  if (n < 0 || hidden <= 0) return 0;
  if (hidden > kNormMaxHidden) return 0;
  return (size_t)block_norm_backward_slots(n, hidden) * 2 * (size_t)hidden * sizeof(float);
}

moe_status moe_block_norm_backward(const moe_block_norm_args* args, const moe_block_norm_grads* grads, void* workspace,
                                   size_t workspace_bytes, moe_stream_t stream) {
  if (!args || !grads) return MOE_ERR_INVALID_ARG;
  const moe_block_norm_args& a = *args;
  const moe_block_norm_grads& d = *grads;
  const moe_status st = check_norm(a);
  if (st != MOE_OK) return st;
  if (!rows_ok(d.d_residual_out, a.hidden, a.residual_dtype) || !rows_ok(d.d_x, a.hidden, MOE_DTYPE_BF16) ||
      !rows_ok(d.d_residual, a.hidden, a.residual_dtype) || !rows_ok(d.d_branch, a.hidden, a.branch_dtype))
    return MOE_ERR_INVALID_ARG;
  if (a.gate_kind == MOE_GATE_FULL ? !rows_ok(d.d_gate, a.hidden, a.branch_dtype) : !aligned(d.d_gate.data, 4))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(d.d_post_weight, 4) || !aligned(d.d_pre_weight, 4)) return MOE_ERR_INVALID_ARG;
  if ((d.d_gate.data && a.gate_kind == MOE_GATE_NONE) || (d.d_post_weight && !a.post_weight) ||
      ((d.d_pre_weight || d.d_x.data) && !a.pre_weight))
    return MOE_ERR_INVALID_ARG;
  if (a.n > 0) {
    if (d.d_branch.data && !a.branch.data) return MOE_ERR_INVALID_ARG;
    if ((a.post_weight && !a.rstd_post) || (d.d_x.data && (!a.rstd_pre || !a.residual_out.data)))
      return MOE_ERR_INVALID_ARG;
  }
  if (!aligned(workspace, 16) || (!workspace && workspace_bytes)) return MOE_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < moe_block_norm_workspace_bytes(a.n, a.hidden)) return MOE_ERR_CAPACITY;
  return status_of(
      launch_block_norm_backward(a, d, static_cast<float*>(workspace), reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_router_workspace_bytes(int32_t n, int32_t n_experts, int32_t n_seqs) {
  if (n < 0 || n_experts <= 0 || n_seqs < 1) return 0;
  return router_loss_workspace(n, n_experts, n_seqs);
}

moe_status moe_balance_loss(const moe_router_args* args, float* prob_sums, float* loss, void* workspace,
                            size_t workspace_bytes, moe_stream_t stream) {
  if (!args) return MOE_ERR_INVALID_ARG;
  const moe_router_args& a = *args;
  const moe_status st = check_router(a);
  if (st != MOE_OK) return st;
  if (!a.counts || !a.tokens || !prob_sums || !loss) return MOE_ERR_INVALID_ARG;
  if (!aligned(prob_sums, 4) || !aligned(loss, 4) || !aligned(workspace, 16)) return MOE_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < router_loss_workspace(a.n, a.n_experts, a.n_seqs)) return MOE_ERR_CAPACITY;
  return status_of(launch_balance_loss(a, prob_sums, loss, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_router_backward(const moe_router_args* args, const float* topk_weights, const float* d_weights,
                               const float* d_loss, float* d_logits, float* d_bias, void* workspace,
                               size_t workspace_bytes, moe_stream_t stream) {
  if (!args) return MOE_ERR_INVALID_ARG;
  const moe_router_args& a = *args;
  const moe_status st = check_router(a);
  if (st != MOE_OK) return st;
  if ((a.counts != nullptr) != (a.tokens != nullptr) || (topk_weights != nullptr) != (d_weights != nullptr))
    return MOE_ERR_INVALID_ARG;
  if (a.n > 0 && !d_logits) return MOE_ERR_INVALID_ARG;
  if (!aligned(topk_weights, 4) || !aligned(d_weights, 4) || !aligned(d_loss, 4) || !aligned(d_logits, 4) ||
      !aligned(d_bias, 4) || !aligned(workspace, 16))
    return MOE_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < router_loss_workspace(a.n, a.n_experts, a.n_seqs)) return MOE_ERR_CAPACITY;
  if (a.n == 0 && !d_bias) return MOE_OK;
  return status_of(launch_router_backward(a, topk_weights, d_weights, d_loss, d_logits, d_bias, workspace,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_lora_workspace_bytes(int32_t n, int32_t n_adapters) {
  if (n < 0 || n_adapters <= 0) return 0;
  return lora_workspace(n, n_adapters);
}

moe_status moe_lora_apply(const moe_lora_args* args, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  if (!args) return MOE_ERR_INVALID_ARG;
  const moe_lora_args& a = *args;
  if (a.n < 0 || a.in_features <= 0 || a.out_features <= 0 || a.n_adapters <= 0 || a.max_rank <= 0)
    return MOE_ERR_INVALID_ARG;
  if (!is_dtype(a.y_dtype) || !is_dtype(a.out_dtype)) return MOE_ERR_INVALID_ARG;
  if (a.in_features % 8 || a.out_features % 8 || a.max_rank % 8 || a.max_rank > kLoraMaxRank || a.n_adapters > 1024 ||
      a.in_features > kLoraMaxFeatures || a.out_features > kLoraMaxFeatures)
    return MOE_ERR_UNSUPPORTED;
  if (!rows_ok(a.x, a.in_features, MOE_DTYPE_BF16) || !rows_ok(a.y, a.out_features, a.y_dtype) ||
      !rows_ok(a.out, a.out_features, a.out_dtype) || !aligned(a.a, 16) || !aligned(a.b, 16) || !aligned(a.scale, 4) ||
      !aligned(a.ranks, 4) || !aligned(a.adapter_ids, 4) || !aligned(workspace, 16))
    return MOE_ERR_INVALID_ARG;
  if (a.n == 0) return MOE_OK;
  if (!a.a || !a.b || !a.adapter_ids || !a.x.data || !a.out.data) return MOE_ERR_INVALID_ARG;
  if (a.y.data == a.out.data && (a.y_dtype != a.out_dtype || (a.y.stride ? a.y.stride : a.out_features) !=
                                                                 (a.out.stride ? a.out.stride : a.out_features)))
    return MOE_ERR_INVALID_ARG;
  const size_t need = lora_workspace(a.n, a.n_adapters);
  if (need && (!workspace || workspace_bytes < need)) return MOE_ERR_CAPACITY;
  return status_of(launch_lora(a, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_lora_get_device_error(int32_t* flags) {
  if (!flags) return MOE_ERR_INVALID_ARG;
  return status_of(lora_device_flags(flags));
}

}  // extern "C"
