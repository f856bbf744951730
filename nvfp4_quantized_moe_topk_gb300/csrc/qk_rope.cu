// qk_rope.cu -- the norms of queries and keys for each head with the rotation
// of their positions, forward and backward, in one pass over the data.
//
// Moving the heads bounds it (16 flops a value).  A warp takes a token's heads,
// 32 / GROUP at a time, and computes the token's cosines and sines once; a few
// tokens are cut further, a warp a step, so that all SMs have work.
#include "qk_rope.cuh"

#include <algorithm>

namespace moe {

namespace {

template <typename T, int GROUP, bool INTERLEAVED>
__global__ void __launch_bounds__(kQkThreads) qk_rope_kernel(const QkParams a, int32_t slices) {
  __shared__ QkTable table;
  constexpr int kHeads = 32 / GROUP;  // heads a step
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / GROUP;
  fill_table(a, table);
  __syncthreads();
  const QkUnit u = unit_of<INTERLEAVED>(lane % GROUP, a.D, a.rot);
  const int32_t steps0 = (a.side[0].heads + kHeads - 1) / kHeads, steps1 = (a.side[1].heads + kHeads - 1) / kHeads;
  const int64_t items = (int64_t)a.n * slices, jump = (int64_t)gridDim.x * kQkWarps;
  for (int64_t item = (int64_t)blockIdx.x * kQkWarps + warp; item < items; item += jump) {
    const int32_t t = (int32_t)(item / slices), slice = (int32_t)(item % slices);
    const int32_t lo = (int32_t)((int64_t)(steps0 + steps1) * slice / slices);
    const int32_t hi = (int32_t)((int64_t)(steps0 + steps1) * (slice + 1) / slices);
    float c[8], s[8];
    if (u.rotated)
#pragma unroll
      for (int j = 0; j < 8; ++j) turn_of(a, table, 8 * (lane % GROUP) + j, t, c[j], s[j]);
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const QkSide& side = a.side[which];
      const int32_t first = which ? max(lo - steps0, 0) : lo, last = which ? hi - steps0 : min(hi, steps0);
      if (first >= last) continue;
      float w[2][8];
      if (side.weight) qk_weight(a, side.weight, u, w);
      const T* in = row_ptr<const T>(side.in, t, (int64_t)side.heads * a.D);
      T* out = row_ptr<T>(side.out, t, (int64_t)side.heads * a.D);
      for (int32_t st = first; st < last; ++st) {
        const int32_t head = st * kHeads + sub;
        const bool live = head < side.heads;
        float v[2][8];
        qk_values(qk_load(in + (int64_t)head * a.D, u, live), v);
        if (side.weight) {
          float ss = 0.f;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[h][j], v[h][j], ss);
          const float r = rsqrtf(group_sum<GROUP>(ss) * a.inv_D + a.eps);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[h][j] = v[h][j] * r * w[h][j];
        }
        if (u.rotated) qk_turn<INTERLEAVED>(v, c, s, 1.f);
        if (live) qk_store(out + (int64_t)head * a.D, u, v);
      }
    }
  }
}

// d_weight of one side: the lanes' sums over their heads and tokens, added over the CTA's warps and groups in order.
template <typename T, int GROUP, bool INTERLEAVED>
__global__ void __launch_bounds__(kQkThreads)
    qk_rope_backward_kernel(const QkParams a, int32_t ctas0, float* __restrict__ part) {
  __shared__ QkTable table;
  __shared__ float sums[kQkWarps][16][33];
  constexpr int kHeads = 32 / GROUP;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / GROUP;
  const int which = (int)blockIdx.x >= ctas0;
  const int32_t cta = which ? blockIdx.x - ctas0 : blockIdx.x, ctas = which ? gridDim.x - ctas0 : ctas0;
  const QkSide& side = a.side[which];
  fill_table(a, table);
  __syncthreads();
  const QkUnit u = unit_of<INTERLEAVED>(lane % GROUP, a.D, a.rot);
  const int32_t steps = (side.heads + kHeads - 1) / kHeads;
  const int64_t items = (int64_t)a.n * steps;
  float w[2][8], acc[2][8] = {};
  if (side.weight) qk_weight(a, side.weight, u, w);
  // every warp a run of (token, step) items, so that it computes a token's angles once
  const int64_t of = (int64_t)ctas * kQkWarps, me = (int64_t)cta * kQkWarps + warp;
  const int64_t begin = items * me / of, end = items * (me + 1) / of;
  float c[8], s[8];
  int32_t have = -1;
  for (int64_t item = begin; item < end; ++item) {
    const int32_t t = (int32_t)(item / steps), head = (int32_t)(item % steps) * kHeads + sub;
    if (t != have && u.rotated) {
#pragma unroll
      for (int j = 0; j < 8; ++j) turn_of(a, table, 8 * (lane % GROUP) + j, t, c[j], s[j]);
    }
    have = t;
    const bool live = head < side.heads;
    const int64_t cols = (int64_t)side.heads * a.D, at = (int64_t)head * a.D;
    float g[2][8];
    qk_values(qk_load(row_ptr<const T>(side.grad, t, cols) + at, u, live), g);
    if (side.weight) {
      float v[2][8];
      qk_values(qk_load(row_ptr<const T>(side.in, t, cols) + at, u, live), v);
      if (u.rotated) qk_turn<INTERLEAVED>(g, c, s, -1.f);
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ss = fmaf(v[h][j], v[h][j], ss);
          dot = fmaf(g[h][j] * w[h][j], v[h][j], dot);
        }
      ss = group_sum<GROUP>(ss);
      dot = group_sum<GROUP>(dot);
      const float r = rsqrtf(ss * a.inv_D + a.eps), m = r * dot * a.inv_D;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float y = v[h][j] * r;
          acc[h][j] = fmaf(g[h][j], y, acc[h][j]);
          g[h][j] = r * (g[h][j] * w[h][j] - y * m);
        }
    } else if (u.rotated) {
      qk_turn<INTERLEAVED>(g, c, s, -1.f);
    }
    if (live && side.out.data) qk_store(row_ptr<T>(side.out, t, cols) + at, u, g);
  }
  if (!side.weight || !part) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) sums[warp][i][lane] = acc[i / 8][i % 8];
  __syncthreads();
  // part[CTA][D]: thread i of the unit's 16 elements adds the warps and their groups
  for (int32_t e = threadIdx.x; e < 16 * GROUP; e += kQkThreads) {
    const QkUnit v = unit_of<INTERLEAVED>(e / 16, a.D, a.rot);
    const int32_t at = v.at[(e % 16) / 8];
    if (at < 0) continue;
    float x = 0.f;
    for (int k = 0; k < kQkWarps; ++k)
      for (int q = 0; q < kHeads; ++q) x += sums[k][e % 16][q * GROUP + e / 16];
    part[(int64_t)blockIdx.x * a.D + at + e % 8] = x;
  }
}

// Joins the CTAs' sums, 32 columns a CTA (blockIdx.y: the queries' or the keys').
__global__ void __launch_bounds__(kJoinThreads)
    qk_weight_sum_kernel(const float* __restrict__ part, int32_t ctas0, int32_t ctas, int32_t D, float* d_q, float* d_k) {
  __shared__ float sum[kJoinWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, which = blockIdx.y;
  float* to = which ? d_k : d_q;
  if (!to) return;
  const int32_t c = blockIdx.x * 32 + lane, mine = blockIdx.x * 32 + warp;
  pdl_wait();
  sum[warp][lane] = join_part<10>(part, which ? ctas0 : 0, (which ? ctas : ctas0) - 1, D, c, c < D);
  __syncthreads();
  const float v = join_parts(sum);
  if (lane == 0 && mine < D) to[mine] = v;
}

int qk_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return std::max(sms, 1);
}

QkParams qk_params(const moe_qk_args& a) {
  QkParams p = {};
  p.n = a.n;
  p.D = a.head_dim;
  p.rot = a.rotary_dim;
  p.axes = std::max(a.n_axes, 1);
  p.pairs_interleaved = a.pairs_interleaved;
  p.sections_interleaved = a.sections_interleaved;
  p.param_dtype = a.param_dtype;
  for (int i = 0; i < MOE_MAX_AXES; ++i) p.sections[i] = a.sections[i];
  if (p.axes == 1) p.sections[0] = p.rot / 2;
  p.eps = a.eps;
  p.offset = a.weight_offset;
  p.scale = a.rotary_scale;
  p.inv_D = 1.f / (float)a.head_dim;
  p.positions = a.positions;
  p.inv_freq = a.inv_freq;
  p.side[0] = {a.q, a.q_out, {}, a.q_weight, a.q_heads};
  p.side[1] = {a.k, a.k_out, {}, a.k_weight, a.k_heads};
  return p;
}

template <typename T, int GROUP, bool INTERLEAVED>
cudaError_t qk_forward(const QkParams& p, cudaStream_t s) {
  constexpr int kHeads = 32 / GROUP;
  const int32_t steps = (p.side[0].heads + kHeads - 1) / kHeads + (p.side[1].heads + kHeads - 1) / kHeads;
  const int64_t wave = (int64_t)qk_sms() * 4 * kQkWarps;
  const int32_t slices = (int32_t)std::max<int64_t>(1, std::min<int64_t>(steps, wave / p.n));
  const int64_t ctas = ((int64_t)p.n * slices + kQkWarps - 1) / kQkWarps;
  qk_rope_kernel<T, GROUP, INTERLEAVED><<<(unsigned)std::min<int64_t>(ctas, qk_sms() * 8), kQkThreads, 0, s>>>(p, slices);
  return cudaGetLastError();
}

template <typename T, int GROUP, bool INTERLEAVED>
cudaError_t qk_backward(const QkParams& p, float* d_q_weight, float* d_k_weight, float* part, cudaStream_t s) {
  constexpr int kHeads = 32 / GROUP;
  int32_t ctas[2];
  const int64_t all = (int64_t)p.side[0].heads + p.side[1].heads;
  for (int i = 0; i < 2; ++i) {
    const int64_t items = (int64_t)p.n * ((p.side[i].heads + kHeads - 1) / kHeads);
    const int64_t share = std::max<int64_t>(1, (int64_t)kQkBackwardCtas * p.side[i].heads / all);
    ctas[i] = (int32_t)std::min((items + kQkWarps - 1) / kQkWarps, share);
  }
  const bool sums = d_q_weight || d_k_weight;
  qk_rope_backward_kernel<T, GROUP, INTERLEAVED>
      <<<(unsigned)(ctas[0] + ctas[1]), kQkThreads, 0, s>>>(p, ctas[0], sums ? part : nullptr);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !sums) return e;
  return launch_ex(qk_weight_sum_kernel, dim3((p.D + 31) / 32, 2), dim3(kJoinThreads), 0, s, true, (const float*)part,
                   ctas[0], ctas[0] + ctas[1], p.D, d_q_weight, d_k_weight);
}

// Calls f<T, GROUP, INTERLEAVED>.
#define QK_GROUP(f, T, G, ...) (p.pairs_interleaved ? f<T, G, true>(p, __VA_ARGS__) : f<T, G, false>(p, __VA_ARGS__))
#define QK_TYPE(f, T, ...)                                                                           \
  (units <= 1 ? QK_GROUP(f, T, 1, __VA_ARGS__) : units <= 2 ? QK_GROUP(f, T, 2, __VA_ARGS__)        \
   : units <= 4 ? QK_GROUP(f, T, 4, __VA_ARGS__) : units <= 8 ? QK_GROUP(f, T, 8, __VA_ARGS__)      \
                : QK_GROUP(f, T, 16, __VA_ARGS__))

}  // namespace

cudaError_t launch_qk_norm_rope(const moe_qk_args& a, cudaStream_t s) {
  const QkParams p = qk_params(a);
  const int units = (p.D + 15) / 16;
  return a.dtype == MOE_DTYPE_BF16 ? QK_TYPE(qk_forward, uint16_t, s) : QK_TYPE(qk_forward, float, s);
}

cudaError_t launch_qk_norm_rope_backward(const moe_qk_args& a, const moe_qk_grads& d, float* part, cudaStream_t s) {
  if (a.n == 0) {
    for (float* w : {d.d_q_weight, d.d_k_weight}) {
      const cudaError_t e = w ? cudaMemsetAsync(w, 0, (size_t)a.head_dim * sizeof(float), s) : cudaSuccess;
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
  QkParams p = qk_params(a);
  p.side[0].grad = d.d_q_out;
  p.side[0].out = d.d_q;
  p.side[1].grad = d.d_k_out;
  p.side[1].out = d.d_k;
  const int units = (p.D + 15) / 16;
  return a.dtype == MOE_DTYPE_BF16 ? QK_TYPE(qk_backward, uint16_t, d.d_q_weight, d.d_k_weight, part, s)
                                   : QK_TYPE(qk_backward, float, d.d_q_weight, d.d_k_weight, part, s);
}

}  // namespace moe
