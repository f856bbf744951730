// qk_rope.cu -- the norms of queries and keys for each head with the rotation
// of their positions, forward and backward, in one pass over the data.
//
// Moving the heads bounds it.  A warp takes a token's heads, 32 / GROUP at a time,
// through a ring of asynchronous copies, and computes the token's cosines and
// sines once; every warp has the same number of steps, which may begin and end
// inside a token.  With loads of its own instead of the ring and a token a turn:
// 80 us for 16384 tokens of 32 + 8 heads of 128 (70 with the ring, 64 with values
// in pairs), their backward pass at 4314 tokens of 32 + 2 66 (35, then 27).
//
//   y = h r (offset + w),  r = (mean h^2 + eps)^-1/2
//   out_a = scale (y_a cos - y_b sin),  out_b = scale (y_b cos + y_a sin)
// and backward, dy the gradient turned back, v = dy (offset + w):
//   d_h = r (v - h r mean(v h r)),  d_w = sum over tokens and heads of dy h r
#include "qk_rope.cuh"

#include <algorithm>

namespace moe {

namespace {

// Slots of a warp's ring, for the forward's one array or the backward's two.
// (16384 tokens, bf16: 64.4 us for 335 MB, 5.2 TB/s; the backward pass at 4314 tokens 26.8 us for 113 MB, 4.2 TB/s, whose
// arithmetic, four turns and two sums a value, takes as long as its bytes.)
template <typename T>
constexpr int qk_stages(int arrays) {
  return sizeof(T) == 2 ? (arrays == 1 ? 6 : 4) : (arrays == 1 ? 4 : 3);
}

// A warp's way through its work: a run of all tokens' steps (a token's queries, then its keys, kHeads heads a step), as
// many as any other warp's; a segment is the run's part on one side of one token.
struct QkPlan {
  int32_t q_steps, steps;
};
struct QkSegment {
  int64_t at, end;                    // the run's next step and its end
  int32_t token, which, first, left;  // the side's steps: the first, and how many (0: no work left)
};
__device__ __forceinline__ void next(const QkPlan& p, QkSegment& g) {
  g.left = 0;
  if (g.at >= g.end) return;
  g.token = (int32_t)(g.at / p.steps);
  const int32_t st = (int32_t)(g.at - (int64_t)g.token * p.steps);
  g.which = st >= p.q_steps;
  g.first = g.which ? st - p.q_steps : st;
  g.left = (int32_t)min((int64_t)((g.which ? p.steps : p.q_steps) - st), g.end - g.at);
  g.at += g.left;
}
template <int GROUP>
__device__ __forceinline__ QkSegment run_of(const QkParams& a, int warp, QkPlan& p) {
  constexpr int kHeads = 32 / GROUP;
  p.q_steps = (a.side[0].heads + kHeads - 1) / kHeads;
  p.steps = p.q_steps + (a.side[1].heads + kHeads - 1) / kHeads;
  const int64_t all = (int64_t)a.n * p.steps, warps = (int64_t)gridDim.x * kQkWarps;
  const int64_t me = (int64_t)blockIdx.x * kQkWarps + warp, each = all / warps, more = all % warps;
  QkSegment g;
  g.at = me * each + min(me, more);
  g.end = g.at + each + (me < more);
  next(p, g);
  return g;
}
// A lane's place in an array over a segment's steps.
template <typename T, int GROUP>
__device__ __forceinline__ T* place(const QkParams& a, const moe_rows& r, const QkSegment& g, int sub) {
  return row_ptr<T>(r, g.token, (int64_t)a.side[g.which].heads * a.D) + (int64_t)(g.first * (32 / GROUP) + sub) * a.D;
}

template <typename T, int GROUP, bool INTERLEAVED>
__global__ void __launch_bounds__(kQkThreads) qk_rope_kernel(const __grid_constant__ QkParams a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ QkTable table;
  __shared__ __align__(16) QkTurns turns[kQkWarps];
  __shared__ __align__(16) float weights[2][kQkMaxDim];
  constexpr int kStages = qk_stages<T>(1), kHeads = 32 / GROUP;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / GROUP, unit = lane % GROUP;
  const QkUnit u = unit_of<INTERLEAVED>(unit, a.D, a.rot);
  QkPlan plan;
  const uint32_t slots = smem_u32(ring) + warp * kStages * kQkSlot<T>;
  const int32_t jump_head = kHeads * a.D;
  pdl_wait();
  pdl_launch_dependents();
  QkSegment ahead = run_of<GROUP>(a, warp, plan), g = ahead;
  const T* src = nullptr;
  int32_t src_head = 0, src_left = 0;
  auto start = [&]() {
    src_left = ahead.left;
    if (!src_left) return;
    src = place<const T, GROUP>(a, a.side[ahead.which].in, ahead, sub);
    src_head = a.side[ahead.which].heads - ahead.first * kHeads - sub;  // heads from the lane's on
  };
  start();
  auto fetch = [&](int stage) {
    if (src_left) {
      qk_fetch(slots + stage * kQkSlot<T>, lane, src, u, src_head > 0);
      src += jump_head;
      src_head -= kHeads;
      if (--src_left == 0) {
        next(plan, ahead);
        start();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i + 1 < kStages; ++i) fetch(i);
  fill_table(a, table);
  fill_weights(a, weights);
  __syncthreads();
  int32_t token = -1;
  int stage = 0;
  for (; g.left > 0; next(plan, g)) {
    const QkSide& side = a.side[g.which];
    const bool norm = side.weight != nullptr;
    if (g.token != token && a.rot > 0) fill_turns(a, table, g.token, lane, turns[warp]);
    token = g.token;
    QkTurn k = turn_of<INTERLEAVED>(turns[warp], u, unit);  // and the weights: of a value, and of its partner
    {
      const QkVals w = qk_floats(weights[g.which], u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        k.own.v[i] = mul2(k.own.v[i], w.v[i]);
        k.other.v[i] = mul2(k.other.v[i], partner<INTERLEAVED>(w, i));
      }
    }
    T* out = place<T, GROUP>(a, side.out, g, sub);
    int32_t heads = side.heads - g.first * kHeads - sub;
    for (int32_t left = g.left; left > 0; --left) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      QkVals v = qk_values(qk_slot<T>(slots + stage * kQkSlot<T>, lane, u, heads > 0));
      fetch(stage == 0 ? kStages - 1 : stage - 1);  // into the slot of the step before
      stage = stage + 1 == kStages ? 0 : stage + 1;
      float r = 1.f;
      if (norm) {
        F2 ss = mul2(v.v[0], v.v[0]), st = mul2(v.v[4], v.v[4]);
#pragma unroll
        for (int i = 1; i < 4; ++i) {
          ss = fma2(v.v[i], v.v[i], ss);
          st = fma2(v.v[4 + i], v.v[4 + i], st);
        }
        r = rsqrtf(group_sum<GROUP>(ss.x + ss.y + (st.x + st.y)) * a.inv_D + a.eps);
      }
      QkVals o;
      if (u.rotated) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o.v[i] = mul2(f2(r), fma2(partner<INTERLEAVED>(v, i), k.other.v[i], mul2(v.v[i], k.own.v[i])));
      } else {  // (a partner would bring its infinities along)
#pragma unroll
        for (int i = 0; i < 8; ++i) o.v[i] = mul2(f2(r), mul2(v.v[i], k.own.v[i]));
      }
      if (heads > 0) qk_store(out, u, o);
      out += jump_head;
      heads -= kHeads;
    }
  }
}

// d_weight: the lanes' sums over a token's heads, kept in shared memory from one token to the next and added over the
// CTA's warps and groups in order at the end.
template <typename T, int GROUP, bool INTERLEAVED>
__global__ void __launch_bounds__(kQkThreads, 3)
    qk_rope_backward_kernel(const __grid_constant__ QkParams a, float* __restrict__ part) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ QkTable table;
  __shared__ __align__(16) QkTurns turns[kQkWarps];
  __shared__ __align__(16) float weights[2][kQkMaxDim];
  __shared__ float sums[2][kQkWarps][16][33];
  constexpr int kHeads = 32 / GROUP, kStages = qk_stages<T>(2);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / GROUP, unit = lane % GROUP;
  const QkUnit u = unit_of<INTERLEAVED>(unit, a.D, a.rot);
  QkPlan plan;
  const uint32_t slots = smem_u32(ring) + warp * kStages * 2 * kQkSlot<T>;
  const int32_t jump_head = kHeads * a.D;
#pragma unroll
  for (int i = 0; i < 16; ++i) sums[0][warp][i][lane] = sums[1][warp][i][lane] = 0.f;
  pdl_wait();
  pdl_launch_dependents();
  QkSegment ahead = run_of<GROUP>(a, warp, plan), g = ahead;
  const T *src = nullptr, *src_in = nullptr;
  int32_t src_head = 0, src_left = 0;
  auto start = [&]() {
    src_left = ahead.left;
    if (!src_left) return;
    const QkSide& side = a.side[ahead.which];
    src = place<const T, GROUP>(a, side.grad, ahead, sub);
    src_in = side.weight ? place<const T, GROUP>(a, side.in, ahead, sub) : nullptr;
    src_head = side.heads - ahead.first * kHeads - sub;
  };
  start();
  auto fetch = [&](int stage) {
    if (src_left) {
      const uint32_t slot = slots + stage * 2 * kQkSlot<T>;
      qk_fetch(slot, lane, src, u, src_head > 0);
      src += jump_head;
      if (src_in) {
        qk_fetch(slot + kQkSlot<T>, lane, src_in, u, src_head > 0);
        src_in += jump_head;
      }
      src_head -= kHeads;
      if (--src_left == 0) {
        next(plan, ahead);
        start();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i + 1 < kStages; ++i) fetch(i);
  fill_table(a, table);
  fill_weights(a, weights);
  __syncthreads();
  int32_t token = -1;
  int stage = 0;
  for (; g.left > 0; next(plan, g)) {
    const QkSide& side = a.side[g.which];
    const bool norm = side.weight != nullptr;
    if (g.token != token && a.rot > 0) fill_turns(a, table, g.token, lane, turns[warp]);
    token = g.token;
    const QkTurn k = turn_of<INTERLEAVED>(turns[warp], u, unit);
    const QkVals w = qk_floats(weights[g.which], u);
    QkVals acc;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc.v[i] = f2(0.f);
    T* out = side.out.data ? place<T, GROUP>(a, side.out, g, sub) : nullptr;
    int32_t heads = side.heads - g.first * kHeads - sub;
    for (int32_t left = g.left; left > 0; --left) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      const uint32_t slot = slots + stage * 2 * kQkSlot<T>;
      QkVals d = qk_values(qk_slot<T>(slot, lane, u, heads > 0));
      QkVals v = qk_values(qk_slot<T>(slot + kQkSlot<T>, lane, u, heads > 0 && norm));
      fetch(stage == 0 ? kStages - 1 : stage - 1);  // into the slot of the step before
      stage = stage + 1 == kStages ? 0 : stage + 1;
      if (u.rotated) {  // turned back: the partner's part with the other sign
        QkVals t;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          t.v[i] = fma2(partner<INTERLEAVED>(d, i), mul2(f2(-1.f), k.other.v[i]), mul2(d.v[i], k.own.v[i]));
        d = t;
      }
      if (norm) {
        F2 ss = f2(0.f), dot = f2(0.f);
        QkVals dw;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw.v[i] = mul2(d.v[i], w.v[i]);
          ss = fma2(v.v[i], v.v[i], ss);
          dot = fma2(dw.v[i], v.v[i], dot);
        }
        const float sq = group_sum<GROUP>(ss.x + ss.y), dt = group_sum<GROUP>(dot.x + dot.y);
        const float r = rsqrtf(sq * a.inv_D + a.eps), mean = r * dt * a.inv_D;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const F2 y = mul2(v.v[i], f2(r));
          acc.v[i] = fma2(d.v[i], y, acc.v[i]);
          d.v[i] = mul2(f2(r), fma2(y, f2(-mean), dw.v[i]));
        }
      }
      if (out) {
        if (heads > 0) qk_store(out, u, d);
        out += jump_head;
      }
      heads -= kHeads;
    }
    if (norm && part) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sums[g.which][warp][2 * i][lane] += acc.v[i].x;
        sums[g.which][warp][2 * i + 1][lane] += acc.v[i].y;
      }
    }
  }
  if (!part) return;
  __syncthreads();
  // part[CTA][side][D]: a thread a side's element
  for (int32_t e = threadIdx.x; e < 2 * 16 * GROUP; e += kQkThreads) {
    const int32_t which = e / (16 * GROUP), in = e % (16 * GROUP);
    const QkUnit v = unit_of<INTERLEAVED>(in / 16, a.D, a.rot);
    const int32_t at = v.at[(in % 16) / 8];
    if (at < 0) continue;
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < kQkWarps; ++k)
#pragma unroll
      for (int q = 0; q < kHeads; ++q) x += sums[which][k][in % 16][q * GROUP + in / 16];
    part[((int64_t)blockIdx.x * 2 + which) * a.D + at + in % 8] = x;
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

// CTAs for the steps there are, a warp a step at least.
int32_t qk_ctas(const QkParams& p, int32_t heads, int32_t most) {
  const int64_t steps = (p.side[0].heads + heads - 1) / heads + (p.side[1].heads + heads - 1) / heads;
  return (int32_t)std::min<int64_t>((p.n * steps + kQkWarps - 1) / kQkWarps, most);
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
  return launch_ex(qk_rope_kernel<T, GROUP, INTERLEAVED>, dim3((unsigned)qk_ctas(p, 32 / GROUP, most)), dim3(kQkThreads),
                   smem, s, true, p);
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
  const int32_t ctas = qk_ctas(p, 32 / GROUP, most);
  const bool sums = d_q_weight || d_k_weight;
  e = launch_ex(qk_rope_backward_kernel<T, GROUP, INTERLEAVED>, dim3((unsigned)ctas), dim3(kQkThreads), smem, s, true, p,
                sums ? part : nullptr);
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
