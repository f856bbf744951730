// block_norm.cu -- the norms before and after a block, with the block's gate
// and the scaled residual (moe_block_norm).
//
//   z = y rp (o + w_post)     rp = (mean y^2 + eps)^-1/2
//   u = alpha r + beta g z
//   x = u ru (o + w_pre)      ru = (mean u^2 + eps)^-1/2
//
// Each row is read once: a group of threads holds one row in registers (8
// consecutive channels a thread, one or two such vectors), so the second
// norm's statistics come from the values that the first one left there.
// Memory bounds it: per element the residual in and out, the branch and x.
//
// Batches of several rows per CTA run persistent groups, each over rows
// b, b + groups, ...: a thread copies its own vectors of the next rows into
// shared memory by asynchronous copies while it works on the current one and
// reads back only what it copied itself, so the copies need no barrier and no
// registers; the weights stay in registers over all rows.
#include "block_norm.cuh"

namespace moe {

namespace {

// The channels' factors: cz = beta g (o + w_post) without the row's factors, wx = o + w_pre.
template <int MODE>
__device__ __forceinline__ void channel_factors(const NormParams& a, int32_t c, float (&cz)[8], float (&wx)[8]) {
  const bool channel = MODE == kNormAny ? a.gate_kind == MOE_GATE_CHANNEL : MODE == kNormChannel;
  float w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    cz[j] = a.beta;
    wx[j] = 0.f;
  }
  if (MODE != kNormAny || a.post) {
    load8_param(a.post, a.param_dtype, c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) cz[j] *= a.offset + w[j];
  }
  if (channel) {
    load8_param(a.gate.p, a.param_dtype, c, w);
    if (a.gate_sigmoid) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = sigmoid(w[j]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) cz[j] *= w[j];
  }
  if (MODE != kNormAny || a.pre) {
    load8_param(a.pre, a.param_dtype, c, wx);
#pragma unroll
    for (int j = 0; j < 8; ++j) wx[j] += a.offset;
  }
}

// One row per CTA: batches too small for the persistent groups.
template <typename RT, typename YT, int ITERS>
__global__ void __launch_bounds__(kNormMaxThreads) block_norm_kernel(const NormParams a) {
  __shared__ float red[2][kNormMaxThreads / 32];
  const int32_t t = blockIdx.x;
  const bool branch = a.branch.p != nullptr;
  constexpr int kR = Vec8<RT>::kVecs, kY = Vec8<YT>::kVecs;
  float u[ITERS][8], z[ITERS][8], cz[ITERS][8], wx[ITERS][8];
  int32_t vec[ITERS];  // index of the thread's group of 8 channels
  float ss[1] = {0.f};
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    vec[i] = threadIdx.x + i * blockDim.x;
#pragma unroll
    for (int j = 0; j < 8; ++j) u[i][j] = z[i][j] = 0.f;
    if (vec[i] * 8 >= a.H) continue;
    load8(reinterpret_cast<const RT*>(a.residual.at(t, vec[i] * kR)), u[i]);
    if (branch) load8(reinterpret_cast<const YT*>(a.branch.at(t, vec[i] * kY)), z[i]);
    channel_factors<kNormAny>(a, vec[i] * 8, cz[i], wx[i]);
    if (a.gate_kind == MOE_GATE_FULL) {
      float g[8];
      load8(reinterpret_cast<const YT*>(a.gate.at(t, vec[i] * kY)), g);
#pragma unroll
      for (int j = 0; j < 8; ++j) cz[i][j] *= a.gate_sigmoid ? sigmoid(g[j]) : g[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss[0] = fmaf(z[i][j], z[i][j], ss[0]);
  }
  float f = 1.f;
  if (a.gate_kind == MOE_GATE_TOKEN) {
    f = reinterpret_cast<const float*>(a.gate.p)[t];
    if (a.gate_sigmoid) f = sigmoid(f);
  }
  if (a.post) {
    group_sums<1>(ss, red[0]);
    const float rp = rsqrtf(fmaf(ss[0], a.inv_h, a.eps));
    if (a.rstd_post && threadIdx.x == 0) a.rstd_post[t] = rp;
    f *= rp;
  }
  ss[0] = 0.f;
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    if (vec[i] * 8 >= a.H) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      u[i][j] *= a.alpha;
      if (branch) u[i][j] = fmaf(cz[i][j], f * z[i][j], u[i][j]);
      ss[0] = fmaf(u[i][j], u[i][j], ss[0]);
    }
    if (a.residual_out.p) store8(reinterpret_cast<RT*>(a.residual_out.at(t, vec[i] * kR)), u[i]);
  }
  if (!a.pre) return;
  group_sums<1>(ss, red[1]);
  const float ru = rsqrtf(fmaf(ss[0], a.inv_h, a.eps));
  if (a.rstd_pre && threadIdx.x == 0) a.rstd_pre[t] = ru;
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    if (vec[i] * 8 >= a.H) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) u[i][j] *= ru * wx[i][j];
    store8(reinterpret_cast<uint16_t*>(a.x_out.at(t, vec[i])), u[i]);
  }
}

// The same for a persistent group of blockDim.x threads (threadIdx.y: which of
// the CTA's groups) over rows blockIdx.x * groups + threadIdx.y, + all groups, ...
template <typename RT, typename YT, int ITERS, int MODE>
__global__ void __launch_bounds__(kNormMaxThreads, 3 - ITERS)
    block_norm_rows_kernel(const NormParams a, int32_t stages, int32_t stage_vecs) {
  extern __shared__ __align__(16) char ring[];
  __shared__ float red[kNormMaxGroups][4][kNormMaxThreads / 32];
  constexpr int kR = Vec8<RT>::kVecs, kY = Vec8<YT>::kVecs;
  const bool branch = MODE != kNormAny || a.branch.p != nullptr;
  const bool post = MODE != kNormAny || a.post != nullptr, pre = MODE != kNormAny || a.pre != nullptr;
  const bool full = MODE == kNormAny ? a.gate_kind == MOE_GATE_FULL : MODE == kNormFull;
  const bool token = (MODE == kNormAny || MODE == kNormScalar) && a.gate_kind == MOE_GATE_TOKEN;
  const uint32_t pitch = blockDim.x * blockDim.y * 16;
  const uint32_t mine = smem_u32(ring) + (threadIdx.y * blockDim.x + threadIdx.x) * 16;
  const uint32_t iter_bytes = stage_vecs / ITERS * pitch, stage_bytes = stage_vecs * pitch;
  const int32_t step = gridDim.x * blockDim.y, t0 = blockIdx.x * blockDim.y + threadIdx.y;
  int32_t vec[ITERS];
  float cz[ITERS][8], wx[ITERS][8];
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    vec[i] = threadIdx.x + i * blockDim.x;
    if (vec[i] * 8 < a.H) channel_factors<MODE>(a, vec[i] * 8, cz[i], wx[i]);
  }
  auto fetch = [&](int64_t t, int stage) {
    if (t < a.n) {
#pragma unroll
      for (int i = 0; i < ITERS; ++i) {
        if (vec[i] * 8 >= a.H) continue;
        uint32_t at = mine + stage * stage_bytes + i * iter_bytes;
        ring_copy<RT>(at, pitch, a.residual.at((int32_t)t, vec[i] * kR));
        if (branch) ring_copy<YT>(at + kR * pitch, pitch, a.branch.at((int32_t)t, vec[i] * kY));
        if (full) ring_copy<YT>(at + (kR + kY) * pitch, pitch, a.gate.at((int32_t)t, vec[i] * kY));
      }
    }
    cp_async_commit();  // one group a row, empty past the end
  };
  for (int s = 0; s + 1 < stages; ++s) fetch((int64_t)t0 + (int64_t)s * step, s);
  int stage = 0, buf = 0;
  for (int64_t t64 = t0; t64 < a.n; t64 += step, stage = stage + 1 == stages ? 0 : stage + 1, buf ^= 2) {
    const int32_t t = (int32_t)t64;
    fetch(t64 + (int64_t)(stages - 1) * step, stage == 0 ? stages - 1 : stage - 1);
    float f = 1.f;
    if (token) {
      f = reinterpret_cast<const float*>(a.gate.p)[t];
      if (a.gate_sigmoid) f = sigmoid(f);
    }
    cp_async_wait(stages - 1);
    const uint32_t at = mine + stage * stage_bytes;
    float u[ITERS][8], z[ITERS][8];
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) u[i][j] = z[i][j] = 0.f;
      if (!branch || vec[i] * 8 >= a.H) continue;
      ring_read<YT>(at + i * iter_bytes + kR * pitch, pitch, z[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss[0] = fmaf(z[i][j], z[i][j], ss[0]);
    }
    if (post) {
      group_sums<1>(ss, red[threadIdx.y][buf]);
      const float rp = rsqrtf(fmaf(ss[0], a.inv_h, a.eps));
      if (a.rstd_post && threadIdx.x == 0) a.rstd_post[t] = rp;
      f *= rp;
    }
    ss[0] = 0.f;
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
      if (vec[i] * 8 >= a.H) continue;
      ring_read<RT>(at + i * iter_bytes, pitch, u[i]);
      if (full) {
        float g[8];
        ring_read<YT>(at + i * iter_bytes + (kR + kY) * pitch, pitch, g);
        if (a.gate_sigmoid) {
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] = sigmoid(g[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) z[i][j] *= g[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[i][j] *= a.alpha;
        if (branch) u[i][j] = fmaf(cz[i][j], f * z[i][j], u[i][j]);
        ss[0] = fmaf(u[i][j], u[i][j], ss[0]);
      }
      if (a.residual_out.p) store8(reinterpret_cast<RT*>(a.residual_out.at(t, vec[i] * kR)), u[i]);
    }
    if (!pre) continue;
    group_sums<1>(ss, red[threadIdx.y][buf + 1]);
    const float ru = rsqrtf(fmaf(ss[0], a.inv_h, a.eps));
    if (a.rstd_pre && threadIdx.x == 0) a.rstd_pre[t] = ru;
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
      if (vec[i] * 8 >= a.H) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) u[i][j] *= ru * wx[i][j];
      store8(reinterpret_cast<uint16_t*>(a.x_out.at(t, vec[i])), u[i]);
    }
  }
}

template <typename RT, typename YT, int ITERS, int MODE>
cudaError_t norm_rows(const NormParams& a, cudaStream_t s) {
  constexpr int y = Vec8<YT>::kVecs;
  const int vecs = ITERS * (Vec8<RT>::kVecs + (a.branch.p ? y : 0) + (a.gate_kind == MOE_GATE_FULL ? y : 0));
  const NormPlan p = norm_plan(a.n, a.H, vecs, 1024 / ITERS);
  static std::atomic<bool> configured[kMaxDevices];
  const cudaError_t e = raise_smem_limit(block_norm_rows_kernel<RT, YT, ITERS, MODE>, kNormSmem, configured);
  if (e != cudaSuccess) return e;
  block_norm_rows_kernel<RT, YT, ITERS, MODE><<<p.ctas, p.block, p.smem, s>>>(a, p.stages, vecs);
  return cudaGetLastError();
}

template <typename RT, typename YT, int ITERS>
cudaError_t norm_forward_i(const NormParams& a, cudaStream_t s) {
  if (a.n <= kNormDirectRows) {
    block_norm_kernel<RT, YT, ITERS><<<(unsigned)a.n, norm_threads(a.H), 0, s>>>(a);
    return cudaGetLastError();
  }
  if (!a.branch.p || !a.post || !a.pre) return norm_rows<RT, YT, ITERS, kNormAny>(a, s);
  if (a.gate_kind == MOE_GATE_CHANNEL) return norm_rows<RT, YT, ITERS, kNormChannel>(a, s);
  if (a.gate_kind == MOE_GATE_FULL) return norm_rows<RT, YT, ITERS, kNormFull>(a, s);
  return norm_rows<RT, YT, ITERS, kNormScalar>(a, s);
}

template <typename RT, typename YT>
cudaError_t norm_forward_t(const NormParams& a, cudaStream_t s) {
  return norm_iters(a.H) == 1 ? norm_forward_i<RT, YT, 1>(a, s) : norm_forward_i<RT, YT, 2>(a, s);
}

}  // namespace

cudaError_t launch_block_norm(const moe_block_norm_args& args, cudaStream_t s) {
  const NormParams a = norm_params(args);
  const bool rb = args.residual_dtype == MOE_DTYPE_BF16, yb = args.branch_dtype == MOE_DTYPE_BF16;
  if (rb) return yb ? norm_forward_t<uint16_t, uint16_t>(a, s) : norm_forward_t<uint16_t, float>(a, s);
  return yb ? norm_forward_t<float, uint16_t>(a, s) : norm_forward_t<float, float>(a, s);
}

}  // namespace moe
