// block_norm.cu -- the norms before and after a block, with the block's gate
// and the scaled residual (moe_block_norm).
//
//   z = y rp (o + w_post)     rp = (mean y^2 + eps)^-1/2
//   u = alpha r + beta g z
//   x = u ru (o + w_pre)      ru = (mean u^2 + eps)^-1/2
//
// Each row is read once: a CTA holds one row in registers (8
// consecutive channels a thread, one or two such vectors), so the second
// norm's statistics come from the values that the first one left there.
// Memory bounds it: per element the residual in and out, the branch and x.
//
// Persistent CTAs (one for every row of a small batch), each over rows b, b +
// CTAs, ...: a thread copies its part of the next rows into shared memory by
// asynchronous copies while it works on the current one and reads back only
// what its warp copied, so the copies need no barrier and no registers; the
// weights stay in registers over all rows.  Measured on a GB300: 16384 rows of
// 4096, fp32 residual, bf16 branch: 136 us, 5.9 TB/s (87 % of a copy's rate); 1536
// threads an SM or two vectors a thread gain nothing.  One row of 2688: 2.8 us,
// latency of a launch, one load and two sums over the CTA (a kernel without
// the ring, a CTA a row, takes as long, and with 304 rows of 8192 9.7 us
// instead of 7.6, so there is none).
#include "block_norm.cuh"

namespace moe {

namespace {

// The channels' factors: cz = beta g (o + w_post) without the row's factors, wx = o + w_pre.
template <int MODE, bool QUADS>
__device__ __forceinline__ void channel_factors(const NormParams& a, const Lane<QUADS>& l, F2 (&cz)[4], F2 (&wx)[4]) {
  const bool channel = MODE == kNormAny ? a.gate_kind == MOE_GATE_CHANNEL : MODE == kNormChannel;
  F2 w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    cz[j] = f2(a.beta);
    wx[j] = f2(0.f);
  }
  if (MODE != kNormAny || a.post) {
    load_param(a.post, a.param_dtype, l, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) cz[j] = mul2(cz[j], add2(f2(a.offset), w[j]));
  }
  if (channel) {
    load_param(a.gate.p, a.param_dtype, l, w);
    if (a.gate_sigmoid) sigmoid2(w);
#pragma unroll
    for (int j = 0; j < 4; ++j) cz[j] = mul2(cz[j], w[j]);
  }
  if (MODE != kNormAny || a.pre) {
    load_param(a.pre, a.param_dtype, l, wx);
#pragma unroll
    for (int j = 0; j < 4; ++j) wx[j] = add2(wx[j], f2(a.offset));
  }
}

// z <- gate * z
__device__ __forceinline__ void apply_gate(const NormParams& a, F2 (&z)[4], F2 (&g)[4]) {
  if (a.gate_sigmoid) sigmoid2(g);
#pragma unroll
  for (int j = 0; j < 4; ++j) z[j] = mul2(z[j], g[j]);
}

__device__ __forceinline__ float squares(const F2 (&v)[4]) {
  F2 s = mul2(v[0], v[0]);
#pragma unroll
  for (int j = 1; j < 4; ++j) s = fma2(v[j], v[j], s);
  return s.x + s.y;
}

// Persistent CTAs over rows blockIdx.x, + gridDim.x, ...
template <typename RT, typename YT, int ITERS, int MODE>
__global__ void __launch_bounds__(kNormMaxThreads, 3 - ITERS)
    block_norm_rows_kernel(const NormParams a, int32_t stages, int32_t stage_vecs) {
  extern __shared__ __align__(16) char ring[];
  __shared__ float red[4][16];
  constexpr int kR = Vec8<RT>::kVecs, kY = Vec8<YT>::kVecs;
  constexpr bool Q = kR + kY > 2;
  const bool branch = MODE != kNormAny || a.branch.p != nullptr;
  const bool post = MODE != kNormAny || a.post != nullptr, pre = MODE != kNormAny || a.pre != nullptr;
  const bool full = MODE == kNormAny ? a.gate_kind == MOE_GATE_FULL : MODE == kNormFull;
  const bool token = (MODE == kNormAny || MODE == kNormScalar) && a.gate_kind == MOE_GATE_TOKEN;
  const uint32_t pitch = blockDim.x * 16, mine = threadIdx.x * 16, ring_u32 = smem_u32(ring);
  const uint32_t iter_bytes = stage_vecs / ITERS * pitch, stage_bytes = stage_vecs * pitch;
  const uint32_t n = a.n, step = gridDim.x;
  F2 cz[ITERS][4], wx[ITERS][4];
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    const Lane<Q> l(i, a.H);
    if (l.ok0) channel_factors<MODE>(a, l, cz[i], wx[i]);
  }
  auto fetch = [&](uint32_t t, int stage) {
    if (t < n) {
#pragma unroll
      for (int i = 0; i < ITERS; ++i) {
        const uint32_t at = mine + stage * stage_bytes + i * iter_bytes;
        ring_copy<RT, Q>(ring_u32 + at, pitch, a.residual.at(t, 0), i, a.H);
        if (branch) ring_copy<YT, Q>(ring_u32 + at + kR * pitch, pitch, a.branch.at(t, 0), i, a.H);
        if (full) ring_copy<YT, Q>(ring_u32 + at + (kR + kY) * pitch, pitch, a.gate.at(t, 0), i, a.H);
      }
    }
    cp_async_commit();  // one group a row, empty past the end
  };
  // a token's gate is loaded one row ahead
  auto token_gate = [&](uint32_t t) {
    return token && t < n ? reinterpret_cast<const float*>(a.gate.p)[t] : 1.f;
  };
  for (int s = 0; s + 1 < stages; ++s) fetch(blockIdx.x + s * step, s);
  float next_gate = token_gate(blockIdx.x);
  int stage = 0, buf = 0;
  for (uint32_t t = blockIdx.x; t < n; t += step, stage = stage + 1 == stages ? 0 : stage + 1, buf ^= 2) {
    __syncwarp();  // the warp has read the slot that is filled next
    fetch(t + (stages - 1) * step, stage == 0 ? stages - 1 : stage - 1);
    float f = next_gate;
    next_gate = token_gate(t + step);
    if (token && a.gate_sigmoid) f = sigmoid(f);
    cp_async_wait(stages - 1);
    __syncwarp();
    const uint32_t at = mine + stage * stage_bytes;
    F2 u[ITERS][4], z[ITERS][4];
    float ss = 0.f;
    if (branch) {
#pragma unroll
      for (int i = 0; i < ITERS; ++i) {
        const Lane<Q> l(i, a.H);
        if (!l.ok0) continue;
        ring_read<YT>(ring, at + i * iter_bytes + kR * pitch, pitch, l, z[i]);
        ss += squares(z[i]);
      }
    }
    if (post) {
      ss = cta_sum(ss, red[buf]);
      const float rp = rsqrtf(fmaf(ss, a.inv_h, a.eps));
      if (a.rstd_post && threadIdx.x == 0) a.rstd_post[t] = rp;
      f *= rp;
    }
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
      const Lane<Q> l(i, a.H);
      if (!l.ok0) continue;
      ring_read<RT>(ring, at + i * iter_bytes, pitch, l, u[i]);
      if (full) {
        F2 g[4];
        ring_read<YT>(ring, at + i * iter_bytes + (kR + kY) * pitch, pitch, l, g);
        apply_gate(a, z[i], g);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u[i][j] = mul2(u[i][j], f2(a.alpha));
        if (branch) u[i][j] = fma2(cz[i][j], mul2(f2(f), z[i][j]), u[i][j]);
      }
      ss += squares(u[i]);
      if (a.residual_out.p) row_store<RT>(a.residual_out, t, l, u[i]);
    }
    if (!pre) continue;
    ss = cta_sum(ss, red[buf + 1]);
    const float ru = rsqrtf(fmaf(ss, a.inv_h, a.eps));
    if (a.rstd_pre && threadIdx.x == 0) a.rstd_pre[t] = ru;
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
      const Lane<Q> l(i, a.H);
      if (!l.ok0) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) u[i][j] = mul2(u[i][j], mul2(f2(ru), wx[i][j]));
      row_store<uint16_t>(a.x_out, t, l, u[i]);
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
  block_norm_rows_kernel<RT, YT, ITERS, MODE><<<p.ctas, p.threads, p.smem, s>>>(a, p.stages, vecs);
  return cudaGetLastError();
}

template <typename RT, typename YT, int ITERS>
cudaError_t norm_forward_i(const NormParams& a, cudaStream_t s) {
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
