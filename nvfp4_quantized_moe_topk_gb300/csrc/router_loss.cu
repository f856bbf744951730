// router_loss.cu -- the router's balance loss with its per-expert counts, and
// the router's backward pass (moe_balance_loss, moe_router_backward).
//
//   p = softmax(logits + bias);  per sequence s, over tokens that take part:
//   c[s][e] picks, P[s][e] = sum of p, N_s tokens, N = sum of N_s
//   loss = coef E / (N k) sum_s (1 / N_s) sum_e c[s][e] P[s][e]
//   d_logits = p (g - sum g p) + the top-k weights' own softmax gradient
//
// One warp takes one token, its logits in registers.  A block owns a
// contiguous range of tokens and walks the sequences that meet it; the column
// sums of its tokens stay in registers until the sequence or the range ends
// and are then written to slot block + sequence of the workspace (both only
// grow along the walk, so each pair has a slot of its own).  The join adds the
// slots of a sequence in block order: no atomics on floats, the same bits on
// every run.
#include <algorithm>

#include "block.cuh"
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kLossWarps = 8;

// The workspace of both calls.
struct LossSpace {
  float* sums;     // [blocks + n_seqs][E]
  int32_t* picks;  // [blocks + n_seqs][E]
  int32_t* toks;   // [blocks + n_seqs]
  float* dots;     // [n_seqs]: (1 / N_s) sum_e c P
};

__host__ __device__ inline int64_t round4(int64_t v) { return (v + 3) & ~int64_t(3); }

LossSpace loss_space(void* ws, int32_t n, int32_t E, int32_t S) {
  const int64_t slots = router_loss_blocks(n) + (int64_t)S;
  LossSpace p;
  p.sums = static_cast<float*>(ws);
  p.picks = reinterpret_cast<int32_t*>(p.sums + round4(slots * E));
  p.toks = p.picks + round4(slots * E);
  p.dots = reinterpret_cast<float*>(p.toks + round4(slots));
  return p;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}
__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Token range [lo, hi) of sequence s, inside [0, n).
__device__ __forceinline__ int32_t seq_bound(const moe_router_args& a, int32_t s) {
  if (!a.seq_offsets) return s <= 0 ? 0 : a.n;
  const int32_t v = a.seq_offsets[s];
  return v < 0 ? 0 : v > a.n ? a.n : v;
}
// First sequence that ends after token t (n_seqs if none does).
__device__ __forceinline__ int32_t first_seq(const moe_router_args& a, int32_t t) {
  int32_t lo = 0, hi = a.n_seqs;
  while (lo < hi) {
    const int32_t mid = (lo + hi) >> 1;
    if (seq_bound(a, mid + 1) > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// A token's softmax: lane l holds experts l + 32 i.  A row without any logit
// above -inf gives p = 0.
template <int SLOTS>
__device__ __forceinline__ void token_softmax(const moe_router_args& a, int64_t t, int lane, float (&p)[SLOTS]) {
  const float* row = a.logits + t * a.n_experts;
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    const int32_t e = lane + 32 * i;
    p[i] = -INFINITY;
    if (e < a.n_experts) p[i] = a.bias ? row[e] + __ldg(a.bias + e) : row[e];
    m = fmaxf(m, p[i]);
  }
  m = warp_max(m);
  if (m == -INFINITY) m = 0.f;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    p[i] = expf(p[i] - m);
    sum += p[i];
  }
  sum = warp_add(sum);
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) p[i] *= inv;
}

template <int SLOTS>
__global__ void __launch_bounds__(kLossWarps * 32)
    balance_partial_kernel(const moe_router_args a, const LossSpace ws, int32_t per_block) {
  extern __shared__ float sm[];  // [kLossWarps][E] sums, then [E] picks
  __shared__ int32_t s_toks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.n_experts;
  int32_t* s_picks = reinterpret_cast<int32_t*>(sm + kLossWarps * E);
  const int32_t lo = (int32_t)min((int64_t)blockIdx.x * per_block, (int64_t)a.n);
  const int32_t hi = (int32_t)min((int64_t)lo + per_block, (int64_t)a.n);
  for (int32_t s = first_seq(a, lo); s < a.n_seqs; ++s) {
    const int32_t beg = max(lo, seq_bound(a, s)), end = min(hi, seq_bound(a, s + 1));
    if (seq_bound(a, s) >= hi) break;
    if (beg >= end) continue;
    for (int32_t e = threadIdx.x; e < E; e += blockDim.x) s_picks[e] = 0;
    if (threadIdx.x == 0) s_toks = 0;
    __syncthreads();
    float acc[SLOTS] = {};
    int32_t toks = 0;
    for (int64_t t = (int64_t)beg + warp; t < end; t += kLossWarps) {
      if (a.token_mask && !a.token_mask[t]) continue;
      ++toks;
      float p[SLOTS];
      token_softmax<SLOTS>(a, t, lane, p);
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) acc[i] += p[i];
      if (lane < a.top_k) {
        const int32_t e = a.topk_ids[t * a.top_k + lane];
        if (e >= 0 && e < E) atomicAdd(&s_picks[e], 1);
      }
    }
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
      if (lane + 32 * i < E) sm[warp * E + lane + 32 * i] = acc[i];
    if (lane == 0) atomicAdd(&s_toks, toks);
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + s;
    for (int32_t e = threadIdx.x; e < E; e += blockDim.x) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kLossWarps; ++w) v += sm[w * E + e];
      ws.sums[slot * E + e] = v;
      ws.picks[slot * E + e] = s_picks[e];
    }
    if (threadIdx.x == 0) ws.toks[slot] = s_toks;
    __syncthreads();
  }
}

// One block per sequence: joins its slots in block order.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads)
    balance_join_kernel(const moe_router_args a, const LossSpace ws, int32_t per_block, float* __restrict__ prob_sums) {
  __shared__ float s_dot[kJoinThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.n_experts;
  const int32_t s = blockIdx.x, beg = seq_bound(a, s), end = seq_bound(a, s + 1);
  const int32_t b0 = beg / per_block, b1 = end > beg ? (end - 1) / per_block : b0 - 1;
  int32_t toks = 0;
  for (int32_t b = b0; b <= b1; ++b) toks += ws.toks[(int64_t)b + s];
  float dot = 0.f;
  for (int32_t e = threadIdx.x; e < E; e += kJoinThreads) {
    float v = 0.f;
    int32_t c = 0;
    for (int32_t b = b0; b <= b1; ++b) {
      v += ws.sums[((int64_t)b + s) * E + e];
      c += ws.picks[((int64_t)b + s) * E + e];
    }
    prob_sums[(int64_t)s * E + e] = v;
    a.counts[(int64_t)s * E + e] = c;
    dot = fmaf((float)c, v, dot);
  }
  dot = warp_add(dot);
  if (lane == 0) s_dot[warp] = dot;
  __syncthreads();
  if (threadIdx.x) return;
  dot = 0.f;
  for (int w = 0; w < kJoinThreads / 32; ++w) dot += s_dot[w];
  a.tokens[s] = toks;
  ws.dots[s] = toks > 0 ? dot / (float)toks : 0.f;
}

// One warp: the loss over the sequences.
__global__ void balance_loss_kernel(const moe_router_args a, const LossSpace ws, float* __restrict__ loss) {
  float v = 0.f;
  int32_t n = 0;
  for (int32_t s = threadIdx.x; s < a.n_seqs; s += 32) {
    v += ws.dots[s];
    n += a.tokens[s];
  }
  v = warp_add(v);
  n = __reduce_add_sync(0xffffffffu, n);
  if (threadIdx.x) return;
  a.tokens[a.n_seqs] = n;
  loss[0] = n > 0 ? a.coef * ((float)a.n_experts / ((float)n * (float)a.top_k)) * v : 0.f;
}

// d_logits of a block's tokens and, where d_bias is wanted, their column sums
// (slot = block).
template <int SLOTS>
__global__ void __launch_bounds__(kLossWarps * 32)
    router_backward_kernel(const moe_router_args a, const float* __restrict__ w, const float* __restrict__ dw,
                           const float* __restrict__ d_loss, float* __restrict__ d_logits, float* __restrict__ sums,
                           int32_t per_block) {
  extern __shared__ float sm[];  // [kLossWarps][E] where sums are wanted
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.n_experts, k = a.top_k;
  const int32_t lo = (int32_t)min((int64_t)blockIdx.x * per_block, (int64_t)a.n);
  const int32_t hi = (int32_t)min((int64_t)lo + per_block, (int64_t)a.n);
  float acc[SLOTS] = {}, g[SLOTS] = {};
  float scale = 0.f;
  if (a.counts) {
    const int32_t total = a.tokens[a.n_seqs];
    if (total > 0) scale = a.coef * (d_loss ? d_loss[0] : 1.f) * ((float)E / ((float)total * (float)k));
  }
  int32_t s = a.counts ? first_seq(a, lo) : 0, s_end = -1;  // g holds sequence s once s_end is its end
  for (int64_t t = (int64_t)lo + warp; t < hi; t += kLossWarps) {
    float d[SLOTS] = {};
    if (a.counts && (!a.token_mask || a.token_mask[t])) {
      if (t >= s_end) {
        while (s < a.n_seqs && seq_bound(a, s + 1) <= t) ++s;
        s_end = a.n;
        float f = 0.f;
        if (s < a.n_seqs && seq_bound(a, s) <= t) {
          s_end = seq_bound(a, s + 1);
          const int32_t mine = a.tokens[s];
          if (mine > 0) f = scale / (float)mine;
        }
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
          const int32_t e = lane + 32 * i;
          g[i] = e < E && f != 0.f ? f * (float)a.counts[(int64_t)s * E + e] : 0.f;
        }
      }
      token_softmax<SLOTS>(a, t, lane, d);
      float mean = 0.f;
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) mean = fmaf(g[i], d[i], mean);
      mean = warp_add(mean);
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) d[i] *= g[i] - mean;
    }
    if (w) {
      int32_t id = -1;
      float dz = 0.f, wj = 0.f, dj = 0.f;
      if (lane < k) {
        id = a.topk_ids[t * k + lane];
        wj = w[t * k + lane];
        dj = dw[t * k + lane];
      }
      dz = wj * (dj - warp_add(wj * dj));
      for (int j = 0; j < k; ++j) {
        const int32_t e = __shfl_sync(0xffffffffu, id, j);
        const float z = __shfl_sync(0xffffffffu, dz, j);
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
          if (e == lane + 32 * i) d[i] += z;
      }
    }
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int32_t e = lane + 32 * i;
      if (e < E) d_logits[t * E + e] = d[i];
      acc[i] += d[i];
    }
  }
  if (!sums) return;
#pragma unroll
  for (int i = 0; i < SLOTS; ++i)
    if (lane + 32 * i < E) sm[warp * E + lane + 32 * i] = acc[i];
  __syncthreads();
  for (int32_t e = threadIdx.x; e < E; e += blockDim.x) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kLossWarps; ++i) v += sm[i * E + e];
    sums[(int64_t)blockIdx.x * E + e] = v;
  }
}

// out[e] = sum of sums[b][e], b in order within each of 8 warps, warps in order.
__global__ void __launch_bounds__(256)
    router_bias_kernel(const float* __restrict__ sums, int32_t blocks, int32_t E, float* __restrict__ out) {
  __shared__ float part[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t e = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (e < E)
    for (int32_t b = warp; b < blocks; b += 8) v += sums[(int64_t)b * E + e];
  part[warp][lane] = v;
  __syncthreads();
  if (warp || e >= E) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v += part[i][lane];
  out[e] = v;
}

// Tokens of a block.
int32_t loss_per_block(int32_t n) {
  const int32_t blocks = router_loss_blocks(n);
  return std::max(1, (int32_t)(((int64_t)n + blocks - 1) / blocks));
}

template <int SLOTS>
cudaError_t balance_t(const moe_router_args& a, const LossSpace& ws, cudaStream_t s) {
  const size_t smem = (size_t)(kLossWarps + 1) * a.n_experts * sizeof(float);
  balance_partial_kernel<SLOTS><<<router_loss_blocks(a.n), kLossWarps * 32, smem, s>>>(a, ws, loss_per_block(a.n));
  return cudaGetLastError();
}

template <int SLOTS>
cudaError_t router_backward_t(const moe_router_args& a, const float* w, const float* dw, const float* d_loss,
                              float* d_logits, float* sums, cudaStream_t s) {
  const size_t smem = sums ? (size_t)kLossWarps * a.n_experts * sizeof(float) : 0;
  router_backward_kernel<SLOTS><<<router_loss_blocks(a.n), kLossWarps * 32, smem, s>>>(a, w, dw, d_loss, d_logits, sums,
                                                                                       loss_per_block(a.n));
  return cudaGetLastError();
}

}  // namespace

int32_t router_loss_blocks(int32_t n) {
  return std::max(1, (int32_t)std::min<int64_t>(kRouterLossBlocks, ((int64_t)n + kLossWarps - 1) / kLossWarps));
}

size_t router_loss_workspace(int32_t n, int32_t E, int32_t S) {
  const int64_t slots = router_loss_blocks(n) + (int64_t)S;
  return (size_t)(2 * round4(slots * E) + round4(slots) + round4(S)) * 4;
}

cudaError_t launch_balance_loss(const moe_router_args& a, float* prob_sums, float* loss, void* workspace,
                                cudaStream_t s) {
  const LossSpace ws = loss_space(workspace, a.n, a.n_experts, a.n_seqs);
  const int32_t E = a.n_experts;
  if (a.n > 0) {
    cudaError_t e;
    if (E <= 32)
      e = balance_t<1>(a, ws, s);
    else if (E <= 64)
      e = balance_t<2>(a, ws, s);
    else if (E <= 128)
      e = balance_t<4>(a, ws, s);
    else if (E <= 256)
      e = balance_t<8>(a, ws, s);
    else if (E <= 512)
      e = balance_t<16>(a, ws, s);
    else
      e = balance_t<32>(a, ws, s);
    if (e != cudaSuccess) return e;
  }
  balance_join_kernel<<<(unsigned)a.n_seqs, kJoinThreads, 0, s>>>(a, ws, loss_per_block(a.n), prob_sums);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  balance_loss_kernel<<<1, 32, 0, s>>>(a, ws, loss);
  return cudaGetLastError();
}

cudaError_t launch_router_backward(const moe_router_args& a, const float* w, const float* dw, const float* d_loss,
                                   float* d_logits, float* d_bias, void* workspace, cudaStream_t s) {
  float* sums = d_bias ? static_cast<float*>(workspace) : nullptr;
  const int32_t E = a.n_experts;
  if (a.n > 0) {
    cudaError_t e;
    if (E <= 32)
      e = router_backward_t<1>(a, w, dw, d_loss, d_logits, sums, s);
    else if (E <= 64)
      e = router_backward_t<2>(a, w, dw, d_loss, d_logits, sums, s);
    else if (E <= 128)
      e = router_backward_t<4>(a, w, dw, d_loss, d_logits, sums, s);
    else if (E <= 256)
      e = router_backward_t<8>(a, w, dw, d_loss, d_logits, sums, s);
    else if (E <= 512)
      e = router_backward_t<16>(a, w, dw, d_loss, d_logits, sums, s);
    else
      e = router_backward_t<32>(a, w, dw, d_loss, d_logits, sums, s);
    if (e != cudaSuccess) return e;
  }
  if (!d_bias) return cudaSuccess;
  router_bias_kernel<<<(unsigned)((E + 31) / 32), 256, 0, s>>>(sums, a.n > 0 ? router_loss_blocks(a.n) : 0, E, d_bias);
  return cudaGetLastError();
}

}  // namespace moe
