// router_loss.cu -- the router's balance loss with its per-expert counts, and
// the router's backward pass (moe_balance_loss, moe_router_backward).
//
//   p = softmax(logits + bias);  per sequence s, over tokens that take part:
//   c[s][e] picks, P[s][e] = sum of p, N_s tokens, N = sum of N_s
//   loss = coef E / (N k) sum_s (1 / N_s) sum_e c[s][e] P[s][e]
//   d_logits = p (g - sum g p) + the top-k weights' own softmax gradient
//
// One warp takes one token, its logits in registers (for few experts several
// tokens at a time, so that enough loads are in flight).  A block owns a
// contiguous range of tokens and walks the sequences that meet it; the column
// sums of its tokens stay in registers until the sequence or the range ends
// and are then written to slot block + sequence of the workspace (both only
// grow along the walk, so each pair has a slot of its own).  The join adds the
// slots of a sequence in block order: no atomics on floats, the same bits on
// every run.  Batches that one block holds need no join: one launch.
//
// Measured on a GB300: loss of 16384 tokens, 128 experts, 7 sequences, two
// launches 13.8 us (what it reads takes 1.3 at a copy's rate: a warp's chain of
// maximum, exponentials, sum, and then the join; 4.2 to 4.5 us for 33 tokens in one
// launch); backward of 16384 tokens, 512 experts 22.4 us, 3 TB/s, of 4314 tokens,
// 128 experts 8.5.
//
// The top-k weights' gradient touches k of a row's experts: each warp adds it
// to its row through its own row of shared memory, zero but for those.
#include <algorithm>

#include "block.cuh"
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kLossThreads = 512, kLossWarps = kLossThreads / 32;

// Blocks of a call: 16 tokens a block, one a warp, or fewer where there are
// more sequences than that (each costs a walk of the block some 1.5 us), up to
// two blocks an SM (with four, 16384 tokens of 64 experts take 17.6 instead of
// 13.7 us in the loss, 27 instead of 23 in the backward pass).  The loss of one
// block needs no join, so there one block takes up to 96 tokens of up to 4
// sequences.  One block against several, measured on a GB300, loss with 64
// experts: 64 tokens 4.6 / 7.1 us, 96 6.0 / 7.2, 128 6.5 / 7.2, with 256 experts
// 128 7.5 / 7.4; 64 tokens of 4 sequences 9.9 / 10.8, of 16 30 / 11.4.  (Backward,
// whose join only adds d_bias up: 32 tokens 5.0 / 4.8, 64 7.3 / 4.8.)
int32_t loss_blocks(int32_t n, int32_t S) {
  const int32_t by_tokens = (int32_t)(((int64_t)n + kLossWarps - 1) / kLossWarps);
  return std::max(1, std::min(kRouterLossBlocks, std::max(by_tokens, std::min(n, S))));
}
int32_t balance_blocks(int32_t n, int32_t S) { return n <= 6 * kLossWarps && S <= 4 ? 1 : loss_blocks(n, S); }

// The workspace of both calls.
struct LossSpace {
  float* sums;      // [blocks + n_seqs][E]
  int32_t* picks;   // [blocks + n_seqs][E]
  int32_t* toks;    // [blocks + n_seqs]
  float* dots;      // [n_seqs]: (1 / N_s) sum_e c P
  int32_t* ticket;  // blocks of the join that are done
};

__host__ __device__ inline int64_t round4(int64_t v) { return (v + 3) & ~int64_t(3); }

LossSpace loss_space(void* ws, int32_t n, int32_t E, int32_t S) {
  const int64_t slots = loss_blocks(n, S) + (int64_t)S;
  LossSpace p;
  p.sums = static_cast<float*>(ws);
  p.picks = reinterpret_cast<int32_t*>(p.sums + round4(slots * E));
  p.toks = p.picks + round4(slots * E);
  p.dots = reinterpret_cast<float*>(p.toks + round4(slots));
  p.ticket = reinterpret_cast<int32_t*>(p.dots + round4(S));
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

// The same for a block, by all its threads at once where there are not too
// many sequences (a binary search is a chain of dependent loads).
__device__ __forceinline__ int32_t block_first_seq(const moe_router_args& a, int32_t t, int32_t* s_min) {
  if (!a.seq_offsets || a.n_seqs > 4096) return first_seq(a, t);
  if (threadIdx.x == 0) *s_min = a.n_seqs;
  __syncthreads();
  for (int32_t i = threadIdx.x; i < a.n_seqs; i += blockDim.x)
    if (seq_bound(a, i + 1) > t) {
      atomicMin(s_min, i);
      break;
    }
  __syncthreads();
  return *s_min;
}

// A lane's N experts of a row.  VEC: groups of 4 (rows aligned to 16 bytes),
// else one by one.
template <bool VEC, int N>
struct Row {
  static_assert(N % 4 == 0, "");
  static __device__ __forceinline__ int32_t expert(int i, int lane) {
    return VEC ? 128 * (i >> 2) + 4 * lane + (i & 3) : 32 * i + lane;
  }
  static __device__ __forceinline__ void load(const float* row, int32_t E, int lane, float (&v)[N], float fill) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        float4 d = make_float4(fill, fill, fill, fill);
        if (expert(i, lane) < E) d = *reinterpret_cast<const float4*>(row + expert(i, lane));
        v[i] = d.x;
        v[i + 1] = d.y;
        v[i + 2] = d.z;
        v[i + 3] = d.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = expert(i, lane) < E ? row[expert(i, lane)] : fill;
    }
  }
  static __device__ __forceinline__ void store(float* row, int32_t E, int lane, const float (&v)[N]) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        if (expert(i, lane) < E)
          *reinterpret_cast<float4*>(row + expert(i, lane)) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (expert(i, lane) < E) row[expert(i, lane)] = v[i];
    }
  }
};

// A token's softmax from its logits (-inf past the last expert), in place; a
// row without any logit above -inf gives p = 0.  s_bias: the bias in shared
// memory, or nullptr.  The exponential is that of 2 in hardware (2 units in the
// last place, and the rounding of (z - max) log2 e: 1e-7 to 1e-6 of p); p below
// 2^-126 counts as 0.
template <bool VEC, int N>
__device__ __forceinline__ void softmax_row(const float* s_bias, int32_t E, int lane, float (&z)[N]) {
  if (s_bias) {
    float b[N];
    Row<VEC, N>::load(s_bias, E, lane, b, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] += b[i];
  }
  float m = z[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, z[i]);
  m = warp_max(m);
  if (m == -INFINITY) m = 0.f;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    z[i] = __expf(z[i] - m);
    sum += z[i];
  }
  sum = warp_add(sum);
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) z[i] *= inv;
}

// The block's sum over its warps of a column of s_acc [kLossWarps][pitch].
__device__ __forceinline__ float column(const float* s_acc, int32_t pitch, int32_t e) {
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < kLossWarps; ++w) v += s_acc[w * pitch + e];
  return v;
}

// Floats of a row in shared memory: the last lanes' groups of 4 included.
__host__ __device__ inline int32_t row_pitch(int32_t E) { return (E + 3) & ~3; }

__device__ __forceinline__ float block_sum(float v, float* s_warp) {
  v = warp_add(v);
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) v += s_warp[w];
  __syncthreads();
  return v;
}

// A warp's tokens in a block's range [lo, hi): group j holds tokens lo + warp +
// kLossWarps (TOK j + u), u < TOK.  A group's loads do not depend on the
// sequences, so the first group is on its way while those are looked up.
template <bool VEC, int N>
struct Group {
  static constexpr int TOK = N >= 16 ? 1 : 16 / N;
  static constexpr int kSpan = kLossWarps * TOK;
  int32_t j;  // which group is loaded (-1: none)
  float z[TOK][N];
  int32_t id[TOK];
  bool on[TOK];  // the token takes part in the loss

  static __device__ __forceinline__ int64_t token(int32_t lo, int32_t j, int u) {
    return (int64_t)lo + (threadIdx.x >> 5) + kLossWarps * ((int64_t)TOK * j + u);
  }
  __device__ __forceinline__ void load(const moe_router_args& a, int32_t lo, int32_t hi, int32_t group, bool logits,
                                       bool ids) {
    const int lane = threadIdx.x & 31;
    j = group;
#pragma unroll
    for (int u = 0; u < TOK; ++u) {
      const int64_t t = token(lo, j, u);
      id[u] = -1;
      on[u] = t < hi;
      if (t >= hi) continue;
      if (logits) Row<VEC, N>::load(a.logits + t * a.n_experts, a.n_experts, lane, z[u], -INFINITY);
      if (ids && lane < a.top_k) id[u] = a.topk_ids[t * a.top_k + lane];
      if (a.token_mask) on[u] = a.token_mask[t];
    }
  }
};

template <bool VEC, int N>
__global__ void __launch_bounds__(kLossThreads, N > 16 ? 1 : 2)
    balance_kernel(const moe_router_args a, const LossSpace ws, int32_t per_block, float* __restrict__ prob_sums,
                   float* __restrict__ loss) {
  constexpr int TOK = Group<VEC, N>::TOK, kSpan = Group<VEC, N>::kSpan;
  extern __shared__ __align__(16) float sm[];  // [kLossWarps][pitch] sums, bias, picks
  __shared__ int32_t s_toks, s_first;
  __shared__ float s_warp[kLossWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.n_experts, k = a.top_k;
  const int32_t pitch = row_pitch(E);
  float* s_bias = sm + kLossWarps * pitch;
  int32_t* s_picks = reinterpret_cast<int32_t*>(s_bias + pitch);
  const bool alone = gridDim.x == 1;
  pdl_launch_dependents();
  const int32_t lo = (int32_t)min((int64_t)blockIdx.x * per_block, (int64_t)a.n);
  const int32_t hi = (int32_t)min((int64_t)lo + per_block, (int64_t)a.n);
  Group<VEC, N> gr;
  gr.load(a, lo, hi, 0, true, true);
  if (blockIdx.x == 0 && threadIdx.x == 0 && !alone) *ws.ticket = 0;
  for (int32_t e = threadIdx.x; e < E; e += kLossThreads) {
    if (a.bias) s_bias[e] = a.bias[e];
    s_picks[e] = 0;
  }
  if (threadIdx.x == 0) s_toks = 0;
  const int32_t s0 = alone ? 0 : block_first_seq(a, lo, &s_first);
  __syncthreads();
  float total_dot = 0.f;
  int32_t total = 0;
  for (int32_t s = s0; s < a.n_seqs; ++s) {
    const int32_t at = seq_bound(a, s);
    if (!alone && at >= hi) break;
    const int32_t beg = max(lo, at), end = min(hi, seq_bound(a, s + 1));
    if (beg >= end) {
      if (alone) {
        for (int32_t e = threadIdx.x; e < E; e += kLossThreads) {
          prob_sums[(int64_t)s * E + e] = 0.f;
          a.counts[(int64_t)s * E + e] = 0;
        }
        if (threadIdx.x == 0) a.tokens[s] = 0;
      }
      continue;
    }
    float acc[N] = {};
    int32_t toks = 0;
    for (int32_t j = (beg - lo) / kSpan; j <= (end - 1 - lo) / kSpan; ++j) {
      if (gr.j != j) gr.load(a, lo, hi, j, true, true);
      gr.j = -1;
#pragma unroll
      for (int u = 0; u < TOK; ++u) {
        const int64_t t = Group<VEC, N>::token(lo, j, u);
        if (t < beg || t >= end || !gr.on[u]) continue;
        ++toks;
        if (gr.id[u] >= 0 && gr.id[u] < E) atomicAdd(&s_picks[gr.id[u]], 1);
        __syncwarp();
        softmax_row<VEC, N>(a.bias ? s_bias : nullptr, E, lane, gr.z[u]);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += gr.z[u][i];
      }
    }
    Row<VEC, N>::store(sm + warp * pitch, E, lane, acc);
    if (lane == 0 && toks) atomicAdd(&s_toks, toks);
    __syncthreads();
    const int32_t all = s_toks;
    if (alone) {
      float dot = 0.f;
      for (int32_t e = threadIdx.x; e < E; e += kLossThreads) {
        const float v = column(sm, pitch, e);
        const int32_t c = s_picks[e];
        prob_sums[(int64_t)s * E + e] = v;
        a.counts[(int64_t)s * E + e] = c;
        s_picks[e] = 0;
        dot = fmaf((float)c, v, dot);
      }
      dot = block_sum(dot, s_warp);
      if (threadIdx.x == 0) a.tokens[s] = all;
      if (all > 0) total_dot += dot / (float)all;
      total += all;
    } else {
      const int64_t slot = (int64_t)blockIdx.x + s;
      for (int32_t e = threadIdx.x; e < E; e += kLossThreads) {
        ws.sums[slot * E + e] = column(sm, pitch, e);
        ws.picks[slot * E + e] = s_picks[e];
        s_picks[e] = 0;
      }
      if (threadIdx.x == 0) ws.toks[slot] = all;
    }
    __syncthreads();
    if (threadIdx.x == 0) s_toks = 0;
    __syncthreads();
  }
  if (alone && threadIdx.x == 0) {
    a.tokens[a.n_seqs] = total;
    loss[0] = total > 0 ? a.coef * ((float)E / ((float)total * (float)k)) * total_dot : 0.f;
  }
}

// One block per sequence joins its slots in block order: thread (column, part
// of the slots); the parts meet in shared memory in order.  The last block to
// finish adds up the loss over the sequences, in their order.
constexpr int kJoinThreads = 1024;
__global__ void __launch_bounds__(kJoinThreads)
    balance_join_kernel(const moe_router_args a, const LossSpace ws, int32_t per_block, int32_t cols,
                        float* __restrict__ prob_sums, float* __restrict__ loss) {
  __shared__ float s_sum[kJoinThreads];
  __shared__ int32_t s_pick[kJoinThreads];
  __shared__ float s_warp[kJoinThreads / 32];
  __shared__ int32_t s_last;
  const int E = a.n_experts, tid = threadIdx.x;
  const int32_t s = blockIdx.x, beg = seq_bound(a, s), end = seq_bound(a, s + 1);
  const int32_t b0 = beg / per_block, b1 = end > beg ? (end - 1) / per_block : b0 - 1;
  const int32_t parts = kJoinThreads / cols, part = tid / cols, col = tid % cols;  // cols: a power of two
  pdl_wait();
  int32_t toks = 0;
  for (int32_t b = b0 + tid; b <= b1; b += kJoinThreads) toks += ws.toks[(int64_t)b + s];
  float dot = 0.f;
  for (int32_t e0 = 0; e0 < E; e0 += cols) {
    const int32_t e = e0 + col;
    float v = 0.f;
    int32_t c = 0;
    if (e < E) {
#pragma unroll 4
      for (int32_t b = b0 + part; b <= b1; b += parts) {
        v += ws.sums[((int64_t)b + s) * E + e];
        c += ws.picks[((int64_t)b + s) * E + e];
      }
    }
    s_sum[tid] = v;
    s_pick[tid] = c;
    __syncthreads();
    if (part == 0 && e < E) {
      for (int32_t i = 1; i < parts; ++i) {
        v += s_sum[i * cols + col];
        c += s_pick[i * cols + col];
      }
      prob_sums[(int64_t)s * E + e] = v;
      a.counts[(int64_t)s * E + e] = c;
      dot = fmaf((float)c, v, dot);
    }
    __syncthreads();
  }
  s_pick[tid] = toks;
  dot = block_sum(dot, s_warp);
  if (tid < 32) {
    toks = 0;
    for (int i = tid; i < kJoinThreads; i += 32) toks += s_pick[i];
    toks = __reduce_add_sync(0xffffffffu, toks);
  }
  if (tid == 0) {
    a.tokens[s] = toks;
    ws.dots[s] = toks > 0 ? dot / (float)toks : 0.f;
    __threadfence();
    s_last = atomicAdd(ws.ticket, 1) == (int32_t)gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last || tid >= 32) return;
  __threadfence();
  float v = 0.f;
  int32_t n = 0;
  for (int32_t i = tid; i < a.n_seqs; i += 32) {
    v += __ldcg(ws.dots + i);
    n += __ldcg(a.tokens + i);
  }
  v = warp_add(v);
  n = __reduce_add_sync(0xffffffffu, n);
  if (tid) return;
  a.tokens[a.n_seqs] = n;
  loss[0] = n > 0 ? a.coef * ((float)E / ((float)n * (float)a.top_k)) * v : 0.f;
}

// d_logits of a block's tokens and, where d_bias is wanted, their column sums
// (slot = block; straight into d_bias where there is one block).
template <bool VEC, int N>
__global__ void __launch_bounds__(kLossThreads, N > 16 ? 1 : 2)
    router_backward_kernel(const moe_router_args a, const float* __restrict__ w, const float* __restrict__ dw,
                           const float* __restrict__ d_loss, float* __restrict__ d_logits, float* __restrict__ sums,
                           int32_t per_block) {
  constexpr int TOK = N >= 16 ? 1 : 8 / N;
  extern __shared__ __align__(16) float sm[];  // [kLossWarps][pitch] the warps' rows, bias, g
  __shared__ int32_t s_first;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.n_experts, k = a.top_k;
  const int32_t pitch = row_pitch(E);
  float* pick = sm + warp * pitch;  // zero between tokens
  float* s_bias = sm + kLossWarps * pitch;
  float* s_g = s_bias + pitch;
  pdl_launch_dependents();
  for (int32_t i = threadIdx.x; i < kLossWarps * pitch; i += kLossThreads) sm[i] = 0.f;
  if (a.bias)
    for (int32_t e = threadIdx.x; e < E; e += kLossThreads) s_bias[e] = a.bias[e];
  const int32_t lo = (int32_t)min((int64_t)blockIdx.x * per_block, (int64_t)a.n);
  const int32_t hi = (int32_t)min((int64_t)lo + per_block, (int64_t)a.n);
  float acc[N] = {};
  const int32_t total = a.counts ? a.tokens[a.n_seqs] : 0;
  const float up = d_loss ? d_loss[0] : 1.f;
  int32_t s = a.counts ? block_first_seq(a, lo, &s_first) : 0;
  const float scale = total > 0 ? a.coef * up * ((float)E / ((float)total * (float)k)) : 0.f;
  // the sequences that meet the block (without a loss term: all its tokens at once)
  for (int32_t at = lo; at < hi;) {
    int32_t end = hi;
    bool lossy = false;
    if (a.counts && s < a.n_seqs) {
      const int32_t beg = seq_bound(a, s);
      if (beg > at) {
        end = min(hi, beg);  // tokens of no sequence
      } else {
        end = max(at, min(hi, seq_bound(a, s + 1)));
        lossy = true;
        __syncthreads();  // the last sequence's g has been read
        const int32_t mine = a.tokens[s];
        const float f = mine > 0 ? scale / (float)mine : 0.f;
        for (int32_t e = threadIdx.x; e < E; e += kLossThreads) s_g[e] = f * (float)a.counts[(int64_t)s * E + e];
        ++s;
      }
    }
    __syncthreads();
    for (int64_t t = (int64_t)at + warp; t < end; t += kLossWarps * TOK) {
      float d[TOK][N];
      bool on[TOK];
      int32_t id[TOK];
      float wj[TOK], dj[TOK];
#pragma unroll
      for (int u = 0; u < TOK; ++u) {
        const int64_t tu = t + u * kLossWarps;
        const bool there = tu < end;
        on[u] = there && lossy && (!a.token_mask || a.token_mask[tu]);
        if (on[u]) Row<VEC, N>::load(a.logits + tu * E, E, lane, d[u], -INFINITY);
        id[u] = -1;
        wj[u] = dj[u] = 0.f;
        if (w && there && lane < k) {
          id[u] = a.topk_ids[tu * k + lane];
          wj[u] = w[tu * k + lane];
          dj[u] = dw[tu * k + lane];
        }
      }
#pragma unroll
      for (int u = 0; u < TOK; ++u) {
        const int64_t tu = t + u * kLossWarps;
        if (tu >= end) break;
        if (on[u]) {
          float g[N];
          softmax_row<VEC, N>(a.bias ? s_bias : nullptr, E, lane, d[u]);
          Row<VEC, N>::load(s_g, E, lane, g, 0.f);
          float mean = 0.f;
#pragma unroll
          for (int i = 0; i < N; ++i) mean = fmaf(g[i], d[u][i], mean);
          mean = warp_add(mean);
#pragma unroll
          for (int i = 0; i < N; ++i) d[u][i] *= g[i] - mean;
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) d[u][i] = 0.f;
        }
        if (w) {
          const float dz = wj[u] * (dj[u] - warp_add(wj[u] * dj[u]));
          const bool in = id[u] >= 0 && id[u] < E;
          const uint32_t same = __match_any_sync(0xffffffffu, in ? id[u] : -1 - lane);
          if (__any_sync(0xffffffffu, __popc(same) > 1)) {  // an expert picked twice: one lane after the other
            for (int j = 0; j < k; ++j) {
              if (lane == j && in) pick[id[u]] += dz;
              __syncwarp();
            }
          } else if (in) {
            pick[id[u]] = dz;
          }
          __syncwarp();
          float v[N];
          Row<VEC, N>::load(pick, E, lane, v, 0.f);
#pragma unroll
          for (int i = 0; i < N; ++i) d[u][i] += v[i];
          __syncwarp();
          if (in) pick[id[u]] = 0.f;
          __syncwarp();
        }
        Row<VEC, N>::store(d_logits + tu * E, E, lane, d[u]);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += d[u][i];
      }
    }
    at = end;
  }
  if (!sums) return;
  __syncthreads();
  Row<VEC, N>::store(pick, E, lane, acc);
  __syncthreads();
  for (int32_t e = threadIdx.x; e < E; e += kLossThreads) sums[(int64_t)blockIdx.x * E + e] = column(sm, pitch, e);
}

// out[e] = sum of sums[b][e], b in order within each of 32 warps, warps in order.
constexpr int kBiasWarps = 32;
__global__ void __launch_bounds__(32 * kBiasWarps)
    router_bias_kernel(const float* __restrict__ sums, int32_t blocks, int32_t E, float* __restrict__ out) {
  __shared__ float part[kBiasWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t e = blockIdx.x * 32 + lane;
  pdl_wait();
  float v = 0.f;
  if (e < E) {
#pragma unroll 8
    for (int32_t b = warp; b < blocks; b += kBiasWarps) v += sums[(int64_t)b * E + e];
  }
  part[warp][lane] = v;
  __syncthreads();
  if (warp || e >= E) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < kBiasWarps; ++i) v += part[i][lane];
  out[e] = v;
}

// Tokens of a block.
int32_t loss_per_block(int32_t n, int32_t blocks) {
  return std::max(1, (int32_t)(((int64_t)n + blocks - 1) / blocks));
}

size_t loss_smem(int32_t E) { return (size_t)(kLossWarps + 2) * row_pitch(E) * sizeof(float); }

template <bool VEC, int N>
cudaError_t balance_t(const moe_router_args& a, const LossSpace& ws, float* prob_sums, float* loss, cudaStream_t s) {
  static std::atomic<bool> configured[kMaxDevices];
  const cudaError_t e = raise_smem_limit(balance_kernel<VEC, N>, 80 * 1024, configured);
  if (e != cudaSuccess) return e;
  const int32_t blocks = balance_blocks(a.n, a.n_seqs);
  balance_kernel<VEC, N><<<blocks, kLossThreads, loss_smem(a.n_experts), s>>>(
      a, ws, loss_per_block(a.n, blocks), prob_sums, loss);
  return cudaGetLastError();
}

template <bool VEC, int N>
cudaError_t router_backward_t(const moe_router_args& a, const float* w, const float* dw, const float* d_loss,
                              float* d_logits, float* sums, cudaStream_t s) {
  static std::atomic<bool> configured[kMaxDevices];
  const cudaError_t e = raise_smem_limit(router_backward_kernel<VEC, N>, 80 * 1024, configured);
  if (e != cudaSuccess) return e;
  const int32_t blocks = loss_blocks(a.n, a.n_seqs);
  router_backward_kernel<VEC, N><<<blocks, kLossThreads, loss_smem(a.n_experts), s>>>(
      a, w, dw, d_loss, d_logits, sums, loss_per_block(a.n, blocks));
  return cudaGetLastError();
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

size_t router_loss_workspace(int32_t n, int32_t E, int32_t S) {
  const int64_t slots = loss_blocks(n, S) + (int64_t)S;
  return (size_t)(2 * round4(slots * E) + round4(slots) + round4(S) + 4) * 4;
}

cudaError_t launch_balance_loss(const moe_router_args& a, float* prob_sums, float* loss, void* workspace,
                                cudaStream_t s) {
  const LossSpace ws = loss_space(workspace, a.n, a.n_experts, a.n_seqs);
  const int32_t E = a.n_experts;
  const bool vec = E % 4 == 0 && aligned16(a.logits);
  cudaError_t e;
  if (E <= 128)
    e = vec ? balance_t<true, 4>(a, ws, prob_sums, loss, s) : balance_t<false, 4>(a, ws, prob_sums, loss, s);
  else if (E <= 256)
    e = vec ? balance_t<true, 8>(a, ws, prob_sums, loss, s) : balance_t<false, 8>(a, ws, prob_sums, loss, s);
  else if (E <= 512)
    e = vec ? balance_t<true, 16>(a, ws, prob_sums, loss, s) : balance_t<false, 16>(a, ws, prob_sums, loss, s);
  else
    e = vec ? balance_t<true, 32>(a, ws, prob_sums, loss, s) : balance_t<false, 32>(a, ws, prob_sums, loss, s);
  const int32_t blocks = balance_blocks(a.n, a.n_seqs);
  if (e != cudaSuccess || blocks == 1) return e;
  int32_t cols = 32;
  while (cols < E && cols < kJoinThreads) cols *= 2;
  return launch_ex(balance_join_kernel, dim3((unsigned)a.n_seqs), dim3(kJoinThreads), 0, s, true, a, ws,
                   loss_per_block(a.n, blocks), cols, prob_sums, loss);
}

cudaError_t launch_router_backward(const moe_router_args& a, const float* w, const float* dw, const float* d_loss,
                                   float* d_logits, float* d_bias, void* workspace, cudaStream_t s) {
  const int32_t E = a.n_experts, blocks = loss_blocks(a.n, a.n_seqs);
  float* sums = !d_bias ? nullptr : blocks == 1 ? d_bias : static_cast<float*>(workspace);
  const bool vec = E % 4 == 0 && aligned16(a.logits) && aligned16(d_logits);
  cudaError_t e;
  if (E <= 128)
    e = vec ? router_backward_t<true, 4>(a, w, dw, d_loss, d_logits, sums, s)
            : router_backward_t<false, 4>(a, w, dw, d_loss, d_logits, sums, s);
  else if (E <= 256)
    e = vec ? router_backward_t<true, 8>(a, w, dw, d_loss, d_logits, sums, s)
            : router_backward_t<false, 8>(a, w, dw, d_loss, d_logits, sums, s);
  else if (E <= 512)
    e = vec ? router_backward_t<true, 16>(a, w, dw, d_loss, d_logits, sums, s)
            : router_backward_t<false, 16>(a, w, dw, d_loss, d_logits, sums, s);
  else
    e = vec ? router_backward_t<true, 32>(a, w, dw, d_loss, d_logits, sums, s)
            : router_backward_t<false, 32>(a, w, dw, d_loss, d_logits, sums, s);
  if (e != cudaSuccess || !d_bias || blocks == 1) return e;
  return launch_ex(router_bias_kernel, dim3((unsigned)((E + 31) / 32)), dim3(32 * kBiasWarps), 0, s, true,
                   (const float*)sums, blocks, E, d_bias);
}

}  // namespace moe
