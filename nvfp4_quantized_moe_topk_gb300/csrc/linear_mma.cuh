// linear_mma.cuh -- what the matrix products of linear_mma.cu are asked for.
#pragma once

#include "kernels.h"

namespace moe {

// out[r][f] = finish(sum over c of p[f][c] * q[r][c]): F features, R rows, C
// columns, bf16, sums in fp32.  An operand lies either with c contiguous
// ([f][c], c_inner) or with f (r) contiguous ([c][f]); its stride is in elements.
struct LinearOperand {
  const void* data;
  int64_t stride;
  bool c_inner;
};
// What happens to a sum on its way out: z = sum + bias, out = act(z) + scale * residual.
struct LinearFinish {
  void *out, *z;                     // z may be NULL
  const void *residual, *bias;       // may be NULL
  int64_t out_stride, z_stride, residual_stride;
  int32_t out_f32, z_f32, residual_f32, bias_f32, act;
  float scale;
};
// q may be a sum of terms of the same layout.
constexpr int kLinearTerms = 3;
struct LinearProduct {
  int32_t R, F, C, terms;
  LinearOperand p, q[kLinearTerms];
  LinearFinish finish;
  // Launched right after a product of the same call, whose operands it shares and whose results it does not take: it
  // begins where that one leaves SMs free.  (That one waits for what came before it before it lets this one begin, so
  // that the operands are there.)
  bool beside;
  int32_t share = 1;  // products that run beside one another
  int32_t* flags = nullptr;  // device memory that a wait that ran out is written to; nullptr: linear_mma_flags'
};
cudaError_t launch_linear_mma(const LinearProduct& a, cudaStream_t s);
// For a few rows (linear_rows.cu): one term, both operands with their columns contiguous, R <= 64.
cudaError_t launch_linear_rows(const LinearProduct& a, cudaStream_t s);
// d_weight of a few tokens (linear_outer.cu): C <= kLinearOuterTokens, neither operand with its columns contiguous, a plain
// finish.
constexpr int32_t kLinearOuterTokens = 128;
cudaError_t launch_linear_outer(const LinearProduct& a, cudaStream_t s);
cudaError_t linear_mma_flags(int32_t* flags);  // reads and clears; the device is idle

}  // namespace moe
