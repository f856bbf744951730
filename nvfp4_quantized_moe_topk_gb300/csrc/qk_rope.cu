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

// Slots of a warp's ring, for the forward's one array or the backward's two.
template <typename T>
constexpr int qk_stages(int arrays) {
  return sizeof(T) == 2 ? (arrays == 1 ? 6 : 4) : (arrays == 1 ? 4 : 3);
}

// A warp's way through its work: items of one token's steps (the queries', then the keys', kHeads heads a step), cut
// into slices, every jump-th item its own.
struct QkWalk {
  int64_t item;
  int32_t token, st, end;  // the steps of the token, in both sides' count
};
struct QkPlan {
  int64_t items, jump;
  int32_t slices, q_steps, steps;
};
template <int GROUP>
__device__ __forceinline__ QkPlan plan_of(const QkParams& a, int32_t slices) {
  constexpr int kHeads = 32 / GROUP;
  QkPlan p;
  p.slices = slices;
  p.items = (int64_t)a.n * slices;
  p.jump = (int64_t)gridDim.x * kQkWarps;
  p.q_steps = (a.side[0].heads + kHeads - 1) / kHeads;
  p.steps = p.q_steps + (a.side[1].heads + kHeads - 1) / kHeads;
  return p;
}
__device__ __forceinline__ void enter(const QkPlan& p, QkWalk& w) {
  if (w.item >= p.items) return;
  w.token = (int32_t)(w.item / p.slices);
  const int32_t slice = (int32_t)(w.item - (int64_t)w.token * p.slices);
  w.st = (int32_t)((int64_t)p.steps * slice / p.slices);
  w.end = (int32_t)((int64_t)p.steps * (slice + 1) / p.slices);
}
__device__ __forceinline__ void advance(const QkPlan& p, QkWalk& w) {
  if (++w.st < w.end) return;
  w.item += p.jump;
  enter(p, w);
}
// The lane's head at a step, where it starts in each array, and whether it is there.
struct QkHead {
  int32_t which, head;
  bool live;
};
template <int GROUP>
__device__ __forceinline__ QkHead head_at(const QkParams& a, const QkPlan& p, const QkWalk& w, int sub) {
  QkHead h;
  h.which = w.st >= p.q_steps;
  h.head = (w.st - (h.which ? p.q_steps : 0)) * (32 / GROUP) + sub;
  h.live = h.head < a.side[h.which].heads;
  return h;
}
template <typename T>
__device__ __forceinline__ T* head_ptr(const QkParams& a, const moe_rows& r, const QkHead& h, int32_t token) {
  return row_ptr<T>(r, token, (int64_t)a.side[h.which].heads * a.D) + (int64_t)h.head * a.D;
}

template <typename T, int GROUP, bool INTERLEAVED>
__global__ void __launch_bounds__(kQkThreads) qk_rope_kernel(const __grid_constant__ QkParams a, int32_t slices) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ QkTable table;
  __shared__ __align__(16) QkTurns turns[kQkWarps];
  constexpr int kStages = qk_stages<T>(1);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / GROUP, unit = lane % GROUP;
  const QkUnit u = unit_of<INTERLEAVED>(unit, a.D, a.rot);
  const QkPlan plan = plan_of<GROUP>(a, slices);
  const uint32_t slots = smem_u32(ring) + warp * kStages * kQkSlot<T>;
  pdl_wait();
  pdl_launch_dependents();
  QkWalk ahead = {(int64_t)blockIdx.x * kQkWarps + warp};
  enter(plan, ahead);
  QkWalk w = ahead;
  auto fetch = [&](int stage) {
    if (ahead.item < plan.items) {
      const QkHead h = head_at<GROUP>(a, plan, ahead, sub);
      qk_fetch(slots + stage * kQkSlot<T>, lane, head_ptr<const T>(a, a.side[h.which].in, h, ahead.token), u, h.live);
      advance(plan, ahead);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i + 1 < kStages; ++i) fetch(i);
  fill_table(a, table);
  __syncthreads();
  // a pair's members (a, b) become r (a k0 + b k1), r (b k2 + a k3): weight and turn in one
  float k[4][8];
  int32_t token = -1, which = -1;
  int stage = 0;
  while (w.item < plan.items) {
    const QkHead h = head_at<GROUP>(a, plan, w, sub);
    const QkSide& side = a.side[h.which];
    const bool norm = side.weight != nullptr;
    if (w.token != token && a.rot > 0) fill_turns(a, table, w.token, lane, turns[warp]);
    if (w.token != token || h.which != which) {
      float wt[2][8], c[8], s[8];
      if (norm) {
        qk_weight(a, side.weight, u, wt);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) wt[0][j] = wt[1][j] = 1.f;
      }
      if (u.rotated) {
        load8(turns[warp].c + 8 * unit, c);
        load8(turns[warp].s + 8 * unit, s);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float wa = member<INTERLEAVED>(wt, 0, j), wb = member<INTERLEAVED>(wt, 1, j);
        k[0][j] = u.rotated ? wa * c[j] : wa;
        k[1][j] = u.rotated ? -wb * s[j] : 0.f;
        k[2][j] = u.rotated ? wb * c[j] : wb;
        k[3][j] = u.rotated ? wa * s[j] : 0.f;
      }
      token = w.token;
      which = h.which;
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    float v[2][8];
    qk_values(qk_slot<T>(slots + stage * kQkSlot<T>, lane, u, h.live), v);
    fetch(stage == 0 ? kStages - 1 : stage - 1);  // into the slot of the step before
    stage = stage + 1 == kStages ? 0 : stage + 1;
    float r = 1.f;
    if (norm) {
      float ss = 0.f;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[m][j], v[m][j], ss);
      r = rsqrtf(group_sum<GROUP>(ss) * a.inv_D + a.eps);
    }
    if (u.rotated) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float &x = member<INTERLEAVED>(v, 0, j), &y = member<INTERLEAVED>(v, 1, j);
        const float t = r * fmaf(y, k[1][j], x * k[0][j]);
        y = r * fmaf(x, k[3][j], y * k[2][j]);
        x = t;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        member<INTERLEAVED>(v, 0, j) *= r * k[0][j];
        member<INTERLEAVED>(v, 1, j) *= r * k[2][j];
      }
    }
    if (h.live) qk_store(head_ptr<T>(a, side.out, h, w.token), u, v);
    advance(plan, w);
  }
}

// d_weight: the lanes' sums over a token's heads, kept in shared memory from one token to the next and added over the
// CTA's warps and groups in order at the end.
template <typename T, int GROUP, bool INTERLEAVED>
__global__ void __launch_bounds__(kQkThreads)
    qk_rope_backward_kernel(const __grid_constant__ QkParams a, int32_t slices, float* __restrict__ part) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ QkTable table;
  __shared__ __align__(16) QkTurns turns[kQkWarps];
  __shared__ float sums[2][kQkWarps][16][33];
  constexpr int kHeads = 32 / GROUP, kStages = qk_stages<T>(2);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / GROUP, unit = lane % GROUP;
  const QkUnit u = unit_of<INTERLEAVED>(unit, a.D, a.rot);
  const QkPlan plan = plan_of<GROUP>(a, slices);
  const uint32_t slots = smem_u32(ring) + warp * kStages * 2 * kQkSlot<T>;
#pragma unroll
  for (int i = 0; i < 16; ++i) sums[0][warp][i][lane] = sums[1][warp][i][lane] = 0.f;
  pdl_wait();
  pdl_launch_dependents();
  QkWalk ahead = {(int64_t)blockIdx.x * kQkWarps + warp};
  enter(plan, ahead);
  QkWalk w = ahead;
  auto fetch = [&](int stage) {
    if (ahead.item < plan.items) {
      const QkHead h = head_at<GROUP>(a, plan, ahead, sub);
      const QkSide& side = a.side[h.which];
      const uint32_t slot = slots + stage * 2 * kQkSlot<T>;
      qk_fetch(slot, lane, head_ptr<const T>(a, side.grad, h, ahead.token), u, h.live);
      if (side.weight)
        qk_fetch(slot + kQkSlot<T>, lane, head_ptr<const T>(a, side.in, h, ahead.token), u, h.live);
      advance(plan, ahead);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i + 1 < kStages; ++i) fetch(i);
  fill_table(a, table);
  __syncthreads();
  float wt[2][8], c[8], s[8], acc[2][8] = {};
  int32_t token = -1, which = 0;
  auto keep = [&]() {  // the sums of the side that ends
    if (!part || !a.side[which].weight) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      sums[which][warp][i][lane] += acc[i / 8][i % 8];
      acc[i / 8][i % 8] = 0.f;
    }
  };
  int stage = 0;
  while (w.item < plan.items) {
    const QkHead h = head_at<GROUP>(a, plan, w, sub);
    const QkSide& side = a.side[h.which];
    const bool norm = side.weight != nullptr;
    if (w.token != token || h.which != which) {
      if (token >= 0) keep();
      if (w.token != token && a.rot > 0) {
        fill_turns(a, table, w.token, lane, turns[warp]);
        if (u.rotated) {
          load8(turns[warp].c + 8 * unit, c);
          load8(turns[warp].s + 8 * unit, s);
        }
      }
      if (norm) qk_weight(a, side.weight, u, wt);
      token = w.token;
      which = h.which;
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    float g[2][8], v[2][8];
    const uint32_t slot = slots + stage * 2 * kQkSlot<T>;
    qk_values(qk_slot<T>(slot, lane, u, h.live), g);
    qk_values(qk_slot<T>(slot + kQkSlot<T>, lane, u, h.live && norm), v);
    fetch(stage == 0 ? kStages - 1 : stage - 1);  // into the slot of the step before
    stage = stage + 1 == kStages ? 0 : stage + 1;
    if (u.rotated) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float &x = member<INTERLEAVED>(g, 0, j), &y = member<INTERLEAVED>(g, 1, j);
        const float t = fmaf(y, s[j], x * c[j]);
        y = fmaf(-x, s[j], y * c[j]);
        x = t;
      }
    }
    if (norm) {
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ss = fmaf(v[m][j], v[m][j], ss);
          dot = fmaf(g[m][j] * wt[m][j], v[m][j], dot);
        }
      ss = group_sum<GROUP>(ss);
      dot = group_sum<GROUP>(dot);
      const float r = rsqrtf(ss * a.inv_D + a.eps), mean = r * dot * a.inv_D;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float y = v[m][j] * r;
          acc[m][j] = fmaf(g[m][j], y, acc[m][j]);
          g[m][j] = r * fmaf(-y, mean, g[m][j] * wt[m][j]);
        }
    }
    if (h.live && side.out.data) qk_store(head_ptr<T>(a, side.out, h, w.token), u, g);
    advance(plan, w);
  }
  if (token >= 0) keep();
  if (!part) return;
  __syncthreads();
  // part[CTA][side][D]: a thread a side's element
  for (int32_t e = threadIdx.x; e < 2 * 16 * GROUP; e += kQkThreads) {
    const int32_t side = e / (16 * GROUP), in = e % (16 * GROUP);
    const QkUnit v = unit_of<INTERLEAVED>(in / 16, a.D, a.rot);
    const int32_t at = v.at[(in % 16) / 8];
    if (at < 0) continue;
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < kQkWarps; ++k)
#pragma unroll
      for (int q = 0; q < kHeads; ++q) x += sums[side][k][in % 16][q * GROUP + in / 16];
    part[((int64_t)blockIdx.x * 2 + side) * a.D + at + in % 8] = x;
  }
}

// Joins the CTAs' sums, 32 columns a CTA (blockIdx.y: the queries' or the keys').
__global__ void __launch_bounds__(kJoinThreads)
    qk_weight_sum_kernel(const float* __restrict__ part, int32_t ctas, int32_t D, float* d_q, float* d_k) {
  __shared__ float sum[kJoinWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, which = blockIdx.y;
  float* to = which ? d_k : d_q;
  if (!to) return;
  const int32_t c = blockIdx.x * 32 + lane, mine = blockIdx.x * 32 + warp;
  pdl_wait();
  sum[warp][lane] = join_part<10>(part + (int64_t)which * D, 0, ctas - 1, 2 * D, c, c < D);
  __syncthreads();
  const float v = join_parts(sum);
  if (lane == 0 && mine < D) to[mine] = v;
}

constexpr int64_t kQkItems = 4;

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

// CTAs that an SM holds, asked for once a device.
template <typename Kernel>
cudaError_t resident(Kernel* kernel, size_t smem, std::atomic<int32_t> (&known)[kMaxDevices], int32_t* ctas) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
  int32_t v = known[dev].load(std::memory_order_acquire);
  if (!v) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, kernel, kQkThreads, smem);
    if (e != cudaSuccess) return e;
    v = std::max(v, 1) * qk_sms();
    known[dev].store(v, std::memory_order_release);
  }
  *ctas = v;
  return cudaSuccess;
}

// Slices of a token's steps: enough that each warp has a few items, so that they come out even.
int32_t qk_slices(const QkParams& p, int32_t heads, int64_t warps) {
  const int32_t steps = (p.side[0].heads + heads - 1) / heads + (p.side[1].heads + heads - 1) / heads;
  return (int32_t)std::max<int64_t>(1, std::min<int64_t>(steps, kQkItems * warps / p.n));
}

template <typename T, int GROUP, bool INTERLEAVED>
cudaError_t qk_forward(const QkParams& p, cudaStream_t s) {
  static std::atomic<bool> configured[kMaxDevices];
  static std::atomic<int32_t> known[kMaxDevices];
  const size_t smem = (size_t)kQkWarps * qk_stages<T>(1) * kQkSlot<T>;
  cudaError_t e = raise_smem_limit(qk_rope_kernel<T, GROUP, INTERLEAVED>, (int)smem, configured);
  int32_t most = 0;
  if (e == cudaSuccess) e = resident(qk_rope_kernel<T, GROUP, INTERLEAVED>, smem, known, &most);
  if (e != cudaSuccess) return e;
  const int32_t slices = qk_slices(p, 32 / GROUP, (int64_t)most * kQkWarps);
  const int64_t ctas = std::min<int64_t>(((int64_t)p.n * slices + kQkWarps - 1) / kQkWarps, most);
  return launch_ex(qk_rope_kernel<T, GROUP, INTERLEAVED>, dim3((unsigned)ctas), dim3(kQkThreads), smem, s, true, p, slices);
}

template <typename T, int GROUP, bool INTERLEAVED>
cudaError_t qk_backward(const QkParams& p, float* d_q_weight, float* d_k_weight, float* part, cudaStream_t s) {
  static std::atomic<bool> configured[kMaxDevices];
  static std::atomic<int32_t> known[kMaxDevices];
  const size_t smem = (size_t)kQkWarps * qk_stages<T>(2) * 2 * kQkSlot<T>;
  cudaError_t e = raise_smem_limit(qk_rope_backward_kernel<T, GROUP, INTERLEAVED>, (int)smem, configured);
  int32_t most = 0;
  if (e == cudaSuccess) e = resident(qk_rope_backward_kernel<T, GROUP, INTERLEAVED>, smem, known, &most);
  if (e != cudaSuccess) return e;
  most = std::min(most, kQkBackwardCtas);
  const int32_t slices = qk_slices(p, 32 / GROUP, (int64_t)most * kQkWarps);
  const int32_t ctas = (int32_t)std::min<int64_t>(((int64_t)p.n * slices + kQkWarps - 1) / kQkWarps, most);
  const bool sums = d_q_weight || d_k_weight;
  e = launch_ex(qk_rope_backward_kernel<T, GROUP, INTERLEAVED>, dim3((unsigned)ctas), dim3(kQkThreads), smem, s, true, p,
                slices, sums ? part : nullptr);
  if (e != cudaSuccess || !sums) return e;
  return launch_ex(qk_weight_sum_kernel, dim3((p.D + 31) / 32, 2), dim3(kJoinThreads), 0, s, true, (const float*)part, ctas,
                   p.D, d_q_weight, d_k_weight);
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
