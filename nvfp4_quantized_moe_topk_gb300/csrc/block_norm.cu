// block_norm.cu -- the norms before and after a block, with the block's gate
// and the scaled residual (moe_block_norm, moe_block_norm_backward).
//
//   z = y rp (o + w_post)     rp = (mean y^2 + eps)^-1/2
//   u = alpha r + beta g z
//   x = u ru (o + w_pre)      ru = (mean u^2 + eps)^-1/2
//
// Each row is read once: a CTA holds one row in registers (8 consecutive
// channels a thread, one or two such groups), so the second norm's statistics
// come from the values that the first one left there.  Memory bounds it: per
// element the residual in and out, the branch and x.
#include <algorithm>

#include "block.cuh"
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kNormMaxThreads = 512;

// Threads of a row's CTA: every thread owns ITERS groups of 8 channels.
int norm_iters(int32_t hidden) { return hidden / 8 > kNormMaxThreads ? 2 : 1; }
int norm_threads(int32_t hidden) {
  const int it = norm_iters(hidden), vecs = hidden / 8;
  return ((vecs + it - 1) / it + 31) / 32 * 32;
}

__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + expf(-v)); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Sums of N values over the CTA, in a fixed order, by one barrier; red is
// this reduction's own [N][warps] floats of shared memory.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[i * warps + warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < warps ? red[i * warps + lane] : 0.f);
}

template <typename RT, typename YT, int ITERS>
__global__ void __launch_bounds__(kNormMaxThreads) block_norm_kernel(const moe_block_norm_args a) {
  __shared__ float red[2][kNormMaxThreads / 32];
  const int64_t t = blockIdx.x;
  const int H = a.hidden;
  const float inv_h = 1.f / (float)H;
  const bool branch = a.branch.data != nullptr;
  float u[ITERS][8];
  int32_t col[ITERS];
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    col[i] = (int32_t)(threadIdx.x + i * blockDim.x) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) u[i][j] = 0.f;
    if (col[i] < H) load8(row_ptr<const RT>(a.residual, t, H) + col[i], u[i]);
  }
  if (branch) {
    float z[ITERS][8];
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) z[i][j] = 0.f;
      if (col[i] < H) load8(row_ptr<const YT>(a.branch, t, H) + col[i], z[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss[0] = fmaf(z[i][j], z[i][j], ss[0]);
    }
    float rp = 1.f;
    if (a.post_weight) {
      block_sums<1>(ss, red[0]);
      rp = 1.f / sqrtf(ss[0] * inv_h + a.eps);
      if (a.rstd_post && threadIdx.x == 0) a.rstd_post[t] = rp;
    }
    float gt = 1.f;
    if (a.gate_kind == MOE_GATE_TOKEN) {
      gt = static_cast<const float*>(a.gate.data)[t];
      if (a.gate_sigmoid) gt = sigmoid(gt);
    }
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
      if (col[i] >= H) continue;
      float w[8], g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w[j] = rp;
        g[j] = gt;
      }
      if (a.post_weight) {
        load8_param(a.post_weight, a.param_dtype, col[i], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = rp * (a.weight_offset + w[j]);
      }
      if (a.gate_kind == MOE_GATE_CHANNEL) load8_param(a.gate.data, a.param_dtype, col[i], g);
      if (a.gate_kind == MOE_GATE_FULL) load8(row_ptr<const YT>(a.gate, t, H) + col[i], g);
      if (a.gate_sigmoid && a.gate_kind != MOE_GATE_TOKEN) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = sigmoid(g[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        u[i][j] = fmaf(a.residual_scale, u[i][j], a.branch_scale * (g[j] * (z[i][j] * w[j])));
    }
  } else {
#pragma unroll
    for (int i = 0; i < ITERS; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) u[i][j] *= a.residual_scale;
  }
  if (a.residual_out.data) {
#pragma unroll
    for (int i = 0; i < ITERS; ++i)
      if (col[i] < H) store8(row_ptr<RT>(a.residual_out, t, H) + col[i], u[i]);
  }
  if (!a.pre_weight) return;
  float ss[1] = {0.f};
#pragma unroll
  for (int i = 0; i < ITERS; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss[0] = fmaf(u[i][j], u[i][j], ss[0]);
  block_sums<1>(ss, red[1]);
  const float ru = 1.f / sqrtf(ss[0] * inv_h + a.eps);
  if (a.rstd_pre && threadIdx.x == 0) a.rstd_pre[t] = ru;
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    if (col[i] >= H) continue;
    float w[8];
    load8_param(a.pre_weight, a.param_dtype, col[i], w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = u[i][j] * ru * (a.weight_offset + w[j]);
    store8(row_ptr<uint16_t>(a.x_out, t, H) + col[i], w);
  }
}

// Backward.  G needs s1 = sum(w dx h), and the branch's gradient needs
// s2 = sum(beta g w' yhat G); G is linear in s1, so s2 = A - s1 B with A and B
// sums that do not wait for s1, and one reduction of three values serves the
// row (for a gate per token the factor g is left out of A and B, and the same
// sum is that gate's gradient).  Row b, b + gridDim.x, ... belong to CTA b,
// whose threads keep the column sums (the weights' and the channel gate's
// gradients) of their channels in registers; the CTAs' sums are joined by
// column_sum_kernel in CTA order.
template <typename RT, typename YT, int ITERS>
__global__ void __launch_bounds__(kNormMaxThreads)
    block_norm_backward_kernel(const moe_block_norm_args a, const moe_block_norm_grads d, float* __restrict__ part) {
  __shared__ float red[2][3 * (kNormMaxThreads / 32)];
  const int H = a.hidden;
  const float inv_h = 1.f / (float)H;
  const bool branch = a.branch.data != nullptr;
  const bool pre = a.pre_weight && d.d_x.data;
  const bool channel = a.gate_kind == MOE_GATE_CHANNEL;
  float acc_pre[ITERS][8] = {}, acc_post[ITERS][8] = {}, acc_gate[ITERS][8] = {};
  int32_t col[ITERS];
#pragma unroll
  for (int i = 0; i < ITERS; ++i) col[i] = (int32_t)(threadIdx.x + i * blockDim.x) * 8;
  int buf = 0;
  for (int64_t t = blockIdx.x; t < a.n; t += gridDim.x, buf ^= 1) {
    const float ru = pre ? a.rstd_pre[t] : 0.f;
    const float rp = a.post_weight ? a.rstd_post[t] : 1.f;
    float gt = 1.f;
    if (a.gate_kind == MOE_GATE_TOKEN) {
      gt = static_cast<const float*>(a.gate.data)[t];
      if (a.gate_sigmoid) gt = sigmoid(gt);
    }
    // q: dr + ru w dx (G without its s1 term); h: u ru; yh: y rp; w: w'; g: gate
    float q[ITERS][8], h[ITERS][8], yh[ITERS][8], w[ITERS][8], g[ITERS][8];
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) q[i][j] = h[i][j] = yh[i][j] = w[i][j] = g[i][j] = 0.f;
      if (col[i] >= H) continue;
      if (d.d_residual_out.data) load8(row_ptr<const RT>(d.d_residual_out, t, H) + col[i], q[i]);
      if (pre) {
        float dx[8], wp[8];
        load8(row_ptr<const uint16_t>(d.d_x, t, H) + col[i], dx);
        load8(row_ptr<const RT>(a.residual_out, t, H) + col[i], h[i]);
        load8_param(a.pre_weight, a.param_dtype, col[i], wp);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[i][j] *= ru;
          acc_pre[i][j] = fmaf(dx[j], h[i][j], acc_pre[i][j]);
          const float dxw = dx[j] * (a.weight_offset + wp[j]);
          s[0] = fmaf(dxw, h[i][j], s[0]);
          q[i][j] = fmaf(ru, dxw, q[i][j]);
        }
      }
      if (branch) {
        load8(row_ptr<const YT>(a.branch, t, H) + col[i], yh[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          yh[i][j] *= rp;
          w[i][j] = 1.f;
          g[i][j] = 1.f;
        }
        if (a.post_weight) {
          load8_param(a.post_weight, a.param_dtype, col[i], w[i]);
#pragma unroll
          for (int j = 0; j < 8; ++j) w[i][j] += a.weight_offset;
        }
        if (channel) load8_param(a.gate.data, a.param_dtype, col[i], g[i]);
        if (a.gate_kind == MOE_GATE_FULL) load8(row_ptr<const YT>(a.gate, t, H) + col[i], g[i]);
        if (a.gate_sigmoid && a.gate_kind != MOE_GATE_TOKEN) {
#pragma unroll
          for (int j = 0; j < 8; ++j) g[i][j] = sigmoid(g[i][j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float c = a.branch_scale * g[i][j] * w[i][j] * yh[i][j];
          s[1] = fmaf(c, q[i][j], s[1]);
          s[2] = fmaf(c, h[i][j], s[2]);
        }
      }
    }
    block_sums<3>(s, red[buf]);
    const float m1 = ru * (s[0] * inv_h);      // G = q - h m1
    const float s2 = s[1] - s[2] * m1;         // sum(beta g w' yhat G), g = 1 for a gate per token
    const float m2 = gt * s2 * inv_h;
    if (a.gate_kind == MOE_GATE_TOKEN && d.d_gate.data && threadIdx.x == 0)
      static_cast<float*>(d.d_gate.data)[t] = a.gate_sigmoid ? s2 * gt * (1.f - gt) : s2;
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
      if (col[i] >= H) continue;
      float G[8], o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        G[j] = fmaf(-m1, h[i][j], q[i][j]);
        o[j] = a.residual_scale * G[j];
      }
      if (d.d_residual.data) store8(row_ptr<RT>(d.d_residual, t, H) + col[i], o);
      if (!branch) continue;
      float dg[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float bG = a.branch_scale * G[j];
        const float dz = gt * g[i][j] * bG;
        dg[j] = bG * (w[i][j] * yh[i][j]);
        acc_post[i][j] = fmaf(dz, yh[i][j], acc_post[i][j]);
        acc_gate[i][j] += dg[j];
        o[j] = a.post_weight ? rp * (w[i][j] * dz - yh[i][j] * m2) : dz;
        if (a.gate_sigmoid) dg[j] *= g[i][j] * (1.f - g[i][j]);
      }
      if (d.d_branch.data) store8(row_ptr<YT>(d.d_branch, t, H) + col[i], o);
      if (a.gate_kind == MOE_GATE_FULL && d.d_gate.data) store8(row_ptr<YT>(d.d_gate, t, H) + col[i], dg);
    }
  }
  // part[b][0..2][H]: d_pre_weight, d_post_weight, d_gate (channel)
  float* mine = part + (size_t)blockIdx.x * 3 * H;
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    if (col[i] >= H) continue;
    if (d.d_pre_weight) store8(mine + col[i], acc_pre[i]);
    if (d.d_post_weight) store8(mine + H + col[i], acc_post[i]);
    if (channel && d.d_gate.data) store8(mine + 2 * H + col[i], acc_gate[i]);
  }
}

// out[c] = sum over b of part[b][which][c], b in a fixed order: warp w of a
// 32-column CTA sums b = w, w + warps, ... and warp 0 joins the warps in order.
constexpr int kColWarps = 16;
__global__ void __launch_bounds__(32 * kColWarps)
    column_sum_kernel(const moe_block_norm_args a, const moe_block_norm_grads d, const float* __restrict__ part,
                      int32_t blocks) {
  __shared__ float sum[kColWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, which = blockIdx.y, H = a.hidden;
  float* out = which == 0 ? d.d_pre_weight
                          : which == 1 ? d.d_post_weight
                                       : a.gate_kind == MOE_GATE_CHANNEL ? static_cast<float*>(d.d_gate.data) : nullptr;
  if (!out) return;
  const int32_t c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < H)
    for (int32_t b = warp; b < blocks; b += kColWarps) v += part[((size_t)b * 3 + which) * H + c];
  sum[warp][lane] = v;
  __syncthreads();
  if (warp || c >= H) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < kColWarps; ++i) v += sum[i][lane];
  if (which == 2 && a.gate_sigmoid) {
    const float g = sigmoid(a.param_dtype == MOE_DTYPE_BF16
                                ? bf16lo(static_cast<const uint16_t*>(a.gate.data)[c])
                                : static_cast<const float*>(a.gate.data)[c]);
    v *= g * (1.f - g);
  }
  out[c] = v;
}

template <typename RT, typename YT>
cudaError_t norm_forward_t(const moe_block_norm_args& a, cudaStream_t s) {
  const int threads = norm_threads(a.hidden);
  if (norm_iters(a.hidden) == 1)
    block_norm_kernel<RT, YT, 1><<<(unsigned)a.n, threads, 0, s>>>(a);
  else
    block_norm_kernel<RT, YT, 2><<<(unsigned)a.n, threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename RT, typename YT>
cudaError_t norm_backward_t(const moe_block_norm_args& a, const moe_block_norm_grads& d, float* part, int blocks,
                            cudaStream_t s) {
  const int threads = norm_threads(a.hidden);
  if (norm_iters(a.hidden) == 1)
    block_norm_backward_kernel<RT, YT, 1><<<blocks, threads, 0, s>>>(a, d, part);
  else
    block_norm_backward_kernel<RT, YT, 2><<<blocks, threads, 0, s>>>(a, d, part);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_norm(const moe_block_norm_args& a, cudaStream_t s) {
  const bool rb = a.residual_dtype == MOE_DTYPE_BF16, yb = a.branch_dtype == MOE_DTYPE_BF16;
  if (rb) return yb ? norm_forward_t<uint16_t, uint16_t>(a, s) : norm_forward_t<uint16_t, float>(a, s);
  return yb ? norm_forward_t<float, uint16_t>(a, s) : norm_forward_t<float, float>(a, s);
}

int block_norm_backward_blocks(int32_t n) { return std::max(1, std::min<int32_t>(n, kNormBackwardBlocks)); }

cudaError_t launch_block_norm_backward(const moe_block_norm_args& a, const moe_block_norm_grads& d, float* part,
                                       cudaStream_t s) {
  const bool rb = a.residual_dtype == MOE_DTYPE_BF16, yb = a.branch_dtype == MOE_DTYPE_BF16;
  const int blocks = block_norm_backward_blocks(a.n);
  if (a.n > 0) {
    cudaError_t e;
    if (rb)
      e = yb ? norm_backward_t<uint16_t, uint16_t>(a, d, part, blocks, s)
             : norm_backward_t<uint16_t, float>(a, d, part, blocks, s);
    else
      e = yb ? norm_backward_t<float, uint16_t>(a, d, part, blocks, s)
             : norm_backward_t<float, float>(a, d, part, blocks, s);
    if (e != cudaSuccess) return e;
  }
  if (!d.d_pre_weight && !d.d_post_weight && !(a.gate_kind == MOE_GATE_CHANNEL && d.d_gate.data)) return cudaSuccess;
  column_sum_kernel<<<dim3((a.hidden + 31) / 32, 3), 32 * kColWarps, 0, s>>>(a, d, part, a.n > 0 ? blocks : 0);
  return cudaGetLastError();
}

}  // namespace moe
