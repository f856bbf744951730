// block_norm_bwd.cu -- backward pass of the norms around a block
// (moe_block_norm_backward).
//
// With p = w dx and c = beta g w' (w, w' the two norms' weights, g the gate):
//   q  = dr + ru p                       the gradient at u but for its mean term
//   G  = q - m1 u                        m1 = ru^3 mean(p u)
//   dy = rp (c G - m2 y)                 m2 = rp^2 mean(c y G)
// G is linear in m1, so sum(c y G) = sum(c y q) - m1 sum(c y u), and one
// reduction of three sums that do not wait for one another serves the row.
// For a gate per token its factor stays out of c, and sum(c y G) rp is that
// gate's gradient.  Of the sums over tokens two are kept, sum(dx u ru) and
// S = sum(gt G y rp g) (without the channel's factors, which the join applies):
//   d_pre_weight is the first, d_post_weight = beta g S, d_gate = beta w' S.
//
// Memory bounds it: two gradients, u and y in, two gradients out.  Persistent
// CTAs and rings in shared memory as in the forward pass.  A
// row's vectors are read twice from the ring, before and after the reduction,
// which is cheaper than holding them in registers beside the channels' sums.
// Each CTA writes its sums, and column_sum_kernel joins them in a fixed order.
// Measured on a GB300: 4314 rows of 2688, all bf16, gate per channel: 30.6 us with
// the join, 4.6 TB/s (67 % of a copy's rate; 40 us with one CTA an SM).  61 rows of
// 1000: 4.9 us, two launches' latency.
#include "block_norm.cuh"

namespace moe {

namespace {

constexpr int kNormBackwardPerSm = 8;

struct NormGrads {
  NormRows dr, dx, d_residual, d_branch, d_gate;
  float *d_post, *d_pre;
};

template <typename RT, typename YT, int ITERS, int MAXT, int MODE>
__global__ void __launch_bounds__(MAXT, 768 / MAXT)
    block_norm_backward_kernel(const NormParams a, const NormGrads d, float* __restrict__ part, int32_t stages,
                               int32_t stage_vecs) {
  extern __shared__ __align__(16) char ring[];
  __shared__ float red[2][64];
  const bool branch = MODE != kNormAny || a.branch.p != nullptr;
  const bool post = MODE != kNormAny || a.post != nullptr, pre = MODE != kNormAny || (a.pre && d.dx.p);
  const bool full = MODE == kNormAny ? a.gate_kind == MOE_GATE_FULL : MODE == kNormFull;
  const bool channel = MODE == kNormAny ? a.gate_kind == MOE_GATE_CHANNEL : MODE == kNormChannel;
  const bool token = (MODE == kNormAny || MODE == kNormScalar) && a.gate_kind == MOE_GATE_TOKEN;
  const uint32_t pitch = blockDim.x * 16, mine = threadIdx.x * 16, ring_u32 = smem_u32(ring);
  const uint32_t iter_bytes = stage_vecs / ITERS * pitch, stage_bytes = stage_vecs * pitch;
  const uint32_t n = a.n, step = gridDim.x;
  constexpr bool Q = Vec8<RT>::kVecs + Vec8<YT>::kVecs > 2;
  pdl_launch_dependents();
  F2 acc_pre[ITERS][4] = {}, acc_post[ITERS][4] = {};
  F2 wx[ITERS][4], c[ITERS][4];  // o + w_pre; beta g (o + w_post), without a full gate
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    const Lane<Q> l(i, a.H);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      wx[i][j] = f2(0.f);
      c[i][j] = f2(a.beta);
    }
    if (!l.ok0) continue;
    F2 w[4];
    if (pre) {
      load_param(a.pre, a.param_dtype, l, wx[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) wx[i][j] = add2(wx[i][j], f2(a.offset));
    }
    if (post) {
      load_param(a.post, a.param_dtype, l, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) c[i][j] = mul2(c[i][j], add2(f2(a.offset), w[j]));
    }
    if (channel) {
      load_param(a.gate.p, a.param_dtype, l, w);
      if (a.gate_sigmoid) sigmoid2(w);
#pragma unroll
      for (int j = 0; j < 4; ++j) c[i][j] = mul2(c[i][j], w[j]);
    }
  }
  // ring order: d_residual_out, residual_out, d_x, branch, full gate
  constexpr int kR = Vec8<RT>::kVecs, kY = Vec8<YT>::kVecs;
  constexpr uint32_t kU = kR, kDx = 2 * kR, kB = kDx + 1, kG = kB + kY;
  auto fetch = [&](uint32_t t, int stage) {
    if (t < n) {
#pragma unroll
      for (int i = 0; i < ITERS; ++i) {
        const uint32_t at = mine + stage * stage_bytes + i * iter_bytes;
        if (d.dr.p) ring_copy<RT, Q>(ring_u32 + at, pitch, d.dr.at(t, 0), i, a.H);
        if (pre) {
          ring_copy<RT, Q>(ring_u32 + at + kU * pitch, pitch, a.residual_out.at(t, 0), i, a.H);
          ring_copy<uint16_t, Q>(ring_u32 + at + kDx * pitch, pitch, d.dx.at(t, 0), i, a.H);
        }
        if (branch) ring_copy<YT, Q>(ring_u32 + at + kB * pitch, pitch, a.branch.at(t, 0), i, a.H);
        if (full) ring_copy<YT, Q>(ring_u32 + at + kG * pitch, pitch, a.gate.at(t, 0), i, a.H);
      }
    }
    cp_async_commit();
  };
  // the row's scalars are loaded one row ahead
  float next_ru = 0.f, next_rp = 1.f, next_gate = 1.f;
  auto scalars = [&](uint32_t t) {
    if (t >= n) return;
    if (pre) next_ru = a.rstd_pre[t];
    if (post) next_rp = a.rstd_post[t];
    if (token) next_gate = reinterpret_cast<const float*>(a.gate.p)[t];
  };
  for (int s = 0; s + 1 < stages; ++s) fetch(blockIdx.x + s * step, s);
  scalars(blockIdx.x);
  int stage = 0, buf = 0;
  for (uint32_t t = blockIdx.x; t < n; t += step, stage = stage + 1 == stages ? 0 : stage + 1, buf ^= 1) {
    __syncwarp();  // the warp has read the slot that is filled next
    fetch(t + (stages - 1) * step, stage == 0 ? stages - 1 : stage - 1);
    const float ru = next_ru, rp = next_rp;
    const float gt = token && a.gate_sigmoid ? sigmoid(next_gate) : next_gate;
    scalars(t + step);
    cp_async_wait(stages - 1);
    __syncwarp();
    const uint32_t at = mine + stage * stage_bytes;
    F2 q[4], u[4], dx[4], y[4], g[4];
    auto read = [&](int i, const Lane<Q>& l) {
      const uint32_t v = at + i * iter_bytes;
      if (MODE == kNormAny || !full) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (MODE == kNormAny) q[j] = u[j] = dx[j] = y[j] = f2(0.f);
          g[j] = f2(1.f);
        }
      }
      if (d.dr.p) {
        ring_read<RT>(ring, v, pitch, l, q);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = f2(0.f);
      }
      if (pre) {
        ring_read<RT>(ring, v + kU * pitch, pitch, l, u);
        ring_read<uint16_t>(ring, v + kDx * pitch, pitch, l, dx);
      }
      if (branch) ring_read<YT>(ring, v + kB * pitch, pitch, l, y);
      if (full) {
        ring_read<YT>(ring, v + kG * pitch, pitch, l, g);
        if (a.gate_sigmoid) sigmoid2(g);
      }
    };
    F2 s2[3] = {};
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
      const Lane<Q> l(i, a.H);
      if (!l.ok0) continue;
      read(i, l);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const F2 p = mul2(dx[j], wx[i][j]);
        const F2 e = mul2(full ? mul2(c[i][j], g[j]) : c[i][j], y[j]);
        s2[0] = fma2(p, u[j], s2[0]);
        s2[1] = fma2(e, fma2(f2(ru), p, q[j]), s2[1]);
        s2[2] = fma2(e, u[j], s2[2]);
      }
    }
    float s[3] = {s2[0].x + s2[0].y, s2[1].x + s2[1].y, s2[2].x + s2[2].y};
    cta_sums3(s[0], s[1], s[2], red[buf]);
    // (from the sum outward: with a small eps ru^3 of a row of zeros is more than fp32 holds, where its sum is 0)
    const float m1 = ru * (ru * (ru * (s[0] * a.inv_h)));
    const float T = rp * (s[1] - s[2] * m1);  // sum(c y rp G)
    if (token && d.d_gate.p && threadIdx.x == 0)
      reinterpret_cast<float*>(d.d_gate.p)[t] = a.gate_sigmoid ? T * gt * (1.f - gt) : T;
    const float kc = rp * gt, ky = post ? rp * (rp * (gt * (T * a.inv_h))) : 0.f;
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
      const Lane<Q> l(i, a.H);
      if (!l.ok0) continue;
      read(i, l);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const F2 rdx = mul2(f2(ru), dx[j]);
        q[j] = fma2(f2(-m1), u[j], fma2(rdx, wx[i][j], q[j]));  // G
        acc_pre[i][j] = fma2(rdx, u[j], acc_pre[i][j]);
        dx[j] = mul2(f2(a.alpha), q[j]);
      }
      if (d.d_residual.p) row_store<RT>(d.d_residual, t, l, dx);
      if (!branch) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const F2 kq = mul2(f2(kc), q[j]);
        const F2 yG = mul2(y[j], kq);
        acc_post[i][j] = full ? fma2(g[j], yG, acc_post[i][j]) : add2(acc_post[i][j], yG);
        if (full) {
          u[j] = mul2(c[i][j], yG);  // d_gate of this element
          if (a.gate_sigmoid) u[j] = mul2(u[j], fma2(mul2(f2(-1.f), g[j]), g[j], g[j]));
        }
        q[j] = fma2(f2(-ky), y[j], mul2(full ? mul2(c[i][j], g[j]) : c[i][j], kq));
      }
      if (d.d_branch.p) row_store<YT>(d.d_branch, t, l, q);
      if (full && d.d_gate.p) row_store<YT>(d.d_gate, t, l, u);
    }
  }
  // part[CTA][0..1][H]
  const NormRows own = {reinterpret_cast<char*>(part), a.H / 4};
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    const Lane<Q> l(i, a.H);
    if (!l.ok0) continue;
    if (d.d_pre) row_store<float>(own, 2 * blockIdx.x, l, acc_pre[i]);
    if (d.d_post || channel) row_store<float>(own, 2 * blockIdx.x + 1, l, acc_post[i]);
  }
}

// Joins the CTAs' sums, 32 columns a CTA (blockIdx.y: which of the two sums).
__global__ void __launch_bounds__(kJoinThreads)
    column_sum_kernel(const NormParams a, const NormGrads d, const float* __restrict__ part, int32_t ctas) {
  __shared__ float sum[kJoinWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, which = blockIdx.y, H = a.H;
  const bool channel = a.gate_kind == MOE_GATE_CHANNEL;
  float* d_gate = channel ? reinterpret_cast<float*>(d.d_gate.p) : nullptr;
  if (which == 0 ? !d.d_pre : !d.d_post && !d_gate) return;
  const int32_t c = blockIdx.x * 32 + lane, mine = blockIdx.x * 32 + warp;  // column loaded, column written
  auto param = [&](const void* p) {
    return a.param_dtype == MOE_DTYPE_BF16 ? bf16lo(static_cast<const uint16_t*>(p)[mine])
                                           : static_cast<const float*>(p)[mine];
  };
  float g = 1.f, w = 1.f;  // (no results of the kernel before)
  if (which && mine < H) {
    if (channel) g = param(a.gate.p);
    if (a.post) w = a.offset + param(a.post);
  }
  pdl_wait();
  sum[warp][lane] = join_part<10>(part + (size_t)which * H, 0, ctas - 1, 2 * H, c, c < H);
  __syncthreads();
  float v = join_parts(sum);
  if (lane || mine >= H) return;
  if (which == 0) {
    d.d_pre[mine] = v;
    return;
  }
  v *= a.beta;
  if (channel && a.gate_sigmoid) g = sigmoid(g);
  if (d_gate) d_gate[mine] = v * w * (a.gate_sigmoid ? g * (1.f - g) : 1.f);
  if (d.d_post) d.d_post[mine] = v * g;
}

template <typename RT, typename YT, int ITERS, int MAXT, int MODE>
cudaError_t norm_backward_m(const NormParams& a, const NormGrads& d, float* part, int* ctas, cudaStream_t s) {
  const int vecs = ITERS * (2 * Vec8<RT>::kVecs + 1 + Vec8<YT>::kVecs * (a.gate_kind == MOE_GATE_FULL ? 2 : 1));
  NormPlan p = norm_plan(a.n, a.H, vecs, 768);
  // Every CTA's sums cost the join a row: no more than eight CTAs an SM, and four rows a CTA where that leaves one an SM
  // (4470 rows of 128: 15.7 us without, 10.3 so; 16384 19.5 / 16.8; 1000 rows of 2048 12.9 / 11.7).
  const int sms = norm_sms();
  p.ctas = std::min({p.ctas, kNormBackwardPerSm * sms, std::max(sms, (int)(a.n / 4)), block_norm_backward_slots(a.n, a.H)});
  *ctas = p.ctas;
  static std::atomic<bool> configured[kMaxDevices];
  const cudaError_t e = raise_smem_limit(block_norm_backward_kernel<RT, YT, ITERS, MAXT, MODE>, kNormSmem, configured);
  if (e != cudaSuccess) return e;
  block_norm_backward_kernel<RT, YT, ITERS, MAXT, MODE><<<p.ctas, p.threads, p.smem, s>>>(a, d, part, p.stages, vecs);
  return cudaGetLastError();
}

template <typename RT, typename YT, int ITERS, int MAXT>
cudaError_t norm_backward_i(const NormParams& a, const NormGrads& d, float* part, int* ctas, cudaStream_t s) {
  if (!a.branch.p || !a.post || !a.pre || !d.dx.p)
    return norm_backward_m<RT, YT, ITERS, MAXT, kNormAny>(a, d, part, ctas, s);
  if (a.gate_kind == MOE_GATE_CHANNEL) return norm_backward_m<RT, YT, ITERS, MAXT, kNormChannel>(a, d, part, ctas, s);
  if (a.gate_kind == MOE_GATE_FULL) return norm_backward_m<RT, YT, ITERS, MAXT, kNormFull>(a, d, part, ctas, s);
  return norm_backward_m<RT, YT, ITERS, MAXT, kNormScalar>(a, d, part, ctas, s);
}

template <typename RT, typename YT>
cudaError_t norm_backward_t(const NormParams& a, const NormGrads& d, float* part, int* ctas, cudaStream_t s) {
  if (norm_iters(a.H) == 2) return norm_backward_i<RT, YT, 2, 512>(a, d, part, ctas, s);
  // rows of up to 384 threads: two CTAs an SM, at 85 registers a thread (2688 channels: 31 us, with one of 128 registers
  // 40); wider rows fill an SM alone
  if (norm_threads(a.H) <= 384) return norm_backward_i<RT, YT, 1, 384>(a, d, part, ctas, s);
  return norm_backward_i<RT, YT, 1, 512>(a, d, part, ctas, s);
}

}  // namespace

// CTAs that the workspace has room for: those of a GPU with up to 160 SMs.
int block_norm_backward_slots(int32_t n, int32_t hidden) {
  return std::max(1, std::min<int32_t>(n, 160 * std::max(1, std::min(768 / norm_threads(hidden), kNormBackwardPerSm))));
}

cudaError_t launch_block_norm_backward(const moe_block_norm_args& args, const moe_block_norm_grads& grads, float* part,
                                       cudaStream_t s) {
  const NormParams a = norm_params(args);
  const bool rb = args.residual_dtype == MOE_DTYPE_BF16, yb = args.branch_dtype == MOE_DTYPE_BF16;
  NormGrads d;
  d.dr = norm_rows(grads.d_residual_out, a.H, rb ? 2 : 4);
  d.dx = norm_rows(grads.d_x, a.H, 2);
  d.d_residual = norm_rows(grads.d_residual, a.H, rb ? 2 : 4);
  d.d_branch = norm_rows(grads.d_branch, a.H, yb ? 2 : 4);
  d.d_gate = norm_rows(grads.d_gate, a.H, yb ? 2 : 4);
  d.d_post = grads.d_post_weight;
  d.d_pre = grads.d_pre_weight;
  int ctas = 0;
  if (a.n > 0) {
    cudaError_t e;
    if (rb)
      e = yb ? norm_backward_t<uint16_t, uint16_t>(a, d, part, &ctas, s)
             : norm_backward_t<uint16_t, float>(a, d, part, &ctas, s);
    else
      e = yb ? norm_backward_t<float, uint16_t>(a, d, part, &ctas, s)
             : norm_backward_t<float, float>(a, d, part, &ctas, s);
    if (e != cudaSuccess) return e;
  }
  if (!d.d_pre && !d.d_post && !(a.gate_kind == MOE_GATE_CHANNEL && d.d_gate.p)) return cudaSuccess;
  return launch_ex(column_sum_kernel, dim3((a.H + 31) / 32, 2), dim3(kJoinThreads), 0, s, a.n > 0, a, d,
                   (const float*)part, ctas);
}

}  // namespace moe
