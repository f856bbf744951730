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
// launches 11.4 us (what it reads takes 1.3 at a copy's rate; latency: two
// launches, sequence lookup, a group's loads and softmax, the join; 4.2 us for 33
// tokens in one launch); backward of 16384 tokens, 512 experts 21.2 us, of which 11
// at 5.9 TB/s and the rest before the first logits and after the last; of 4314
// tokens, 128 experts 7.9.
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
// more sequences than that (each costs a walk of the block about a microsecond),
// up to two blocks an SM (with four, 16384 tokens take 15.5 instead of 11.6 us in
// the loss, 24 instead of 20 in the backward pass).  The loss of one block needs
// no join, so there one block takes up to 128 tokens of up to 4 sequences.  One
// block against several, measured on a GB300, us: 64 tokens, 64 experts 4.2 / 7.9,
// 128 tokens 5.6 / 7.9, 256 8.5 / 8.1; 128 tokens, 256 experts 6.7 / 7.9, 256 10.8
// / 8.0; 128 experts, 128 tokens of 4 sequences 9.2 / 9.8, of 16 22 / 11.5.
// (Backward, whose join only adds d_bias up, one block: 32 tokens 5.0 / 4.8, 64
// 7.3 / 4.8.)
int32_t loss_blocks(int32_t n, int32_t S) {
  const int32_t by_tokens = (int32_t)(((int64_t)n + kLossWarps - 1) / kLossWarps);
  return std::max(1, std::min(kRouterLossBlocks, std::max(by_tokens, std::min(n, S))));
}
int32_t balance_blocks(int32_t n, int32_t S) { return n <= 8 * kLossWarps && S <= 4 ? 1 : loss_blocks(n, S); }

// The workspace of both calls.
struct LossSpace {
  float* sums;      // [blocks + n_seqs][E]
  int32_t* picks;   // [blocks + n_seqs][E]
  int32_t* toks;    // [blocks + n_seqs]
  float* dots;      // [n_seqs][ceil(E / 32)]: (1 / N_s) sum of c P over 32 experts
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
  p.ticket = reinterpret_cast<int32_t*>(p.dots + round4((int64_t)S * ((E + 31) / 32)));
  return p;
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
  // Experts expert(i), expert(i + 1) of a row, i even.
  static __device__ __forceinline__ void load4(const float* row, int32_t E, int lane, int i, F2 (&v)[2], float fill) {
    v[0] = v[1] = f2(fill);
    if constexpr (VEC) {
      if (expert(i, lane) < E) {
        const float4 d = *reinterpret_cast<const float4*>(row + expert(i, lane));
        v[0] = {d.x, d.y};
        v[1] = {d.z, d.w};
      }
    } else {
      if (expert(i, lane) < E) v[0].x = row[expert(i, lane)];
      if (expert(i + 1, lane) < E) v[0].y = row[expert(i + 1, lane)];
      if (expert(i + 2, lane) < E) v[1].x = row[expert(i + 2, lane)];
      if (expert(i + 3, lane) < E) v[1].y = row[expert(i + 3, lane)];
    }
  }
  static __device__ __forceinline__ void load(const float* row, int32_t E, int lane, F2 (&v)[N / 2], float fill) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      F2 d[2];
      load4(row, E, lane, i, d, fill);
      v[i / 2] = d[0];
      v[i / 2 + 1] = d[1];
    }
  }
  static __device__ __forceinline__ void store(float* row, int32_t E, int lane, const F2 (&v)[N / 2]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const F2 p = v[i / 2], q = v[i / 2 + 1];
      if constexpr (VEC) {
        if (expert(i, lane) < E) *reinterpret_cast<float4*>(row + expert(i, lane)) = make_float4(p.x, p.y, q.x, q.y);
      } else {
        if (expert(i, lane) < E) row[expert(i, lane)] = p.x;
        if (expert(i + 1, lane) < E) row[expert(i + 1, lane)] = p.y;
        if (expert(i + 2, lane) < E) row[expert(i + 2, lane)] = q.x;
        if (expert(i + 3, lane) < E) row[expert(i + 3, lane)] = q.y;
      }
    }
  }
};

// Warp sums of M values, side by side.
template <int M>
__device__ __forceinline__ void warp_sums(float (&v)[M]) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int i = 0; i < M; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
}

// 2^x in hardware (2 units in the last place; results below 2^-126 are 0).
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// From the logits of TOK tokens (-inf past the last expert) the numerators of
// their softmax, z <- e^(z - max) in place, and the lane's part of their sums; a
// row without any logit above -inf gives 0.  s_bias: the bias in shared memory,
// or nullptr.  e^(z - max) is 2^((z - max) log2 e): the largest logit's is exactly
// 1, and differences count alone, whatever the logits' size (with max log2 e
// taken from z log2 e in one fma, its rounding is an exponent of 100 and more
// from |max| 2e9 on, and no time is gained).  A p is good to 2.3 |z - max| 2^-24
// of itself and a few units in the last place.
template <bool VEC, int N, int TOK>
__device__ __forceinline__ void softmax_parts(const float* s_bias, int32_t E, int lane, F2 (&z)[TOK][N / 2],
                                              float (&sum)[TOK]) {
  constexpr float kLog2e = 1.4426950408889634f;
  if (s_bias) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      F2 b[2];
      Row<VEC, N>::load4(s_bias, E, lane, i, b, 0.f);
#pragma unroll
      for (int u = 0; u < TOK; ++u) {
        z[u][i / 2] = add2(z[u][i / 2], b[0]);
        z[u][i / 2 + 1] = add2(z[u][i / 2 + 1], b[1]);
      }
    }
  }
  float m[TOK];
#pragma unroll
  for (int u = 0; u < TOK; ++u) {
    m[u] = fmaxf(z[u][0].x, z[u][0].y);
#pragma unroll
    for (int i = 1; i < N / 2; ++i) m[u] = fmaxf(m[u], fmaxf(z[u][i].x, z[u][i].y));
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int u = 0; u < TOK; ++u) m[u] = fmaxf(m[u], __shfl_xor_sync(0xffffffffu, m[u], off));
#pragma unroll
  for (int u = 0; u < TOK; ++u) {
    const F2 c = f2(m[u] == -INFINITY ? 0.f : -m[u]);
    F2 s = f2(0.f);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const F2 x = mul2(add2(z[u][i], c), f2(kLog2e));
      z[u][i] = {exp2_fast(x.x), exp2_fast(x.y)};
      s = add2(s, z[u][i]);
    }
    sum[u] = s.x + s.y;
  }
}
__device__ __forceinline__ float inverse(float sum) { return sum > 0.f ? 1.f / sum : 0.f; }

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
// kLossWarps (TOK j + u), u < TOK.  A group's loads and softmax do not depend on
// the sequences, so the first group is on its way while those are looked up.
template <bool VEC, int N>
struct Group {
  static constexpr int TOK = N >= 16 ? 1 : 16 / N;
  static constexpr int kBackward = N >= 8 ? 1 : 2;  // of the backward pass
  static constexpr int kSpan = kLossWarps * TOK;
  int32_t j;            // which group this is
  F2 z[TOK][N / 2];     // the logits, then the numerators of their softmax
  float inv[TOK];       // 1 / the sum of those
  int32_t id[TOK];
  bool on[TOK];         // the token takes part in the loss

  static __device__ __forceinline__ int64_t token(int32_t lo, int32_t j, int u) {
    return (int64_t)lo + (threadIdx.x >> 5) + kLossWarps * ((int64_t)TOK * j + u);
  }
  __device__ __forceinline__ void load(const moe_router_args& a, int32_t lo, int32_t hi, int32_t group) {
    const int lane = threadIdx.x & 31;
    j = group;
#pragma unroll
    for (int u = 0; u < TOK; ++u) {
      const int64_t t = token(lo, j, u);
      id[u] = -1;
      on[u] = t < hi;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) z[u][i] = f2(-INFINITY);
      if (t >= hi) continue;
      Row<VEC, N>::load(a.logits + t * a.n_experts, a.n_experts, lane, z[u], -INFINITY);
      if (lane < a.top_k) id[u] = a.topk_ids[t * a.top_k + lane];
      if (a.token_mask) on[u] = a.token_mask[t];
    }
  }
  // (a masked token's logits may be anything: its numerators become 0)
  __device__ __forceinline__ void softmax(const float* s_bias, int32_t E) {
#pragma unroll
    for (int u = 0; u < TOK; ++u)
      if (!on[u]) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) z[u][i] = f2(-INFINITY);
      }
    softmax_parts<VEC, N, TOK>(s_bias, E, threadIdx.x & 31, z, inv);
    warp_sums(inv);
#pragma unroll
    for (int u = 0; u < TOK; ++u) inv[u] = inverse(inv[u]);
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
  gr.load(a, lo, hi, 0);
  if (blockIdx.x == 0 && threadIdx.x == 0 && !alone) *ws.ticket = 0;
  for (int32_t e = threadIdx.x; e < E; e += kLossThreads) {
    if (a.bias) s_bias[e] = a.bias[e];
    s_picks[e] = 0;
  }
  if (threadIdx.x == 0) s_toks = 0;
  const int32_t s0 = alone ? 0 : block_first_seq(a, lo, &s_first);
  __syncthreads();
  gr.softmax(a.bias ? s_bias : nullptr, E);
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
    F2 acc[N / 2] = {};
    int32_t toks = 0;
    for (int32_t j = (beg - lo) / kSpan; j <= (end - 1 - lo) / kSpan; ++j) {
      if (gr.j != j) {  // (a group that meets two sequences is not loaded again)
        gr.load(a, lo, hi, j);
        gr.softmax(a.bias ? s_bias : nullptr, E);
      }
#pragma unroll
      for (int u = 0; u < TOK; ++u) {
        const int64_t t = Group<VEC, N>::token(lo, j, u);
        const bool in = t >= beg && t < end && gr.on[u];
        toks += in;
        if (in && gr.id[u] >= 0 && gr.id[u] < E) atomicAdd(&s_picks[gr.id[u]], 1);
        const F2 inv = f2(in ? gr.inv[u] : 0.f);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) acc[i] = fma2(gr.z[u][i], inv, acc[i]);
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

// Block (s, y) joins 32 columns of the slots of sequence s; the last block to
// finish adds up the loss over the sequences' parts, in a fixed order.
__global__ void __launch_bounds__(kJoinThreads)
    balance_join_kernel(const moe_router_args a, const LossSpace ws, int32_t per_block, float* __restrict__ prob_sums,
                        float* __restrict__ loss) {
  __shared__ float s_sum[32][33];
  __shared__ int32_t s_pick[32][33];
  __shared__ float s_dot[32];
  __shared__ int32_t s_toks[32], s_last;
  const int E = a.n_experts, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t s = blockIdx.x, beg = seq_bound(a, s), end = seq_bound(a, s + 1);
  const int32_t b0 = beg / per_block, b1 = end > beg ? (end - 1) / per_block : b0 - 1;
  const int32_t e = blockIdx.y * 32 + lane, mine = blockIdx.y * 32 + warp;
  pdl_wait();
  int32_t toks = 0;
  for (int32_t b = b0 + tid; b <= b1; b += kJoinThreads) toks += ws.toks[(int64_t)b + s];
  const float part = join_part<6>(ws.sums + (int64_t)s * E, b0, b1, E, e, e < E);
  const int32_t picks = join_part<6>(ws.picks + (int64_t)s * E, b0, b1, E, e, e < E);
  s_sum[warp][lane] = part;
  s_pick[warp][lane] = picks;
  __syncthreads();
  const float v = join_parts(s_sum);
  const int32_t c = join_parts(s_pick);
  toks = __reduce_add_sync(0xffffffffu, toks);
  if (lane == 0) {
    if (mine < E) {
      prob_sums[(int64_t)s * E + mine] = v;
      a.counts[(int64_t)s * E + mine] = c;
    }
    s_dot[warp] = (float)c * v;  // (0 past the last expert)
    s_toks[warp] = toks;
  }
  __syncthreads();
  if (warp) return;
  const float dot = warp_add(s_dot[lane]);
  toks = __reduce_add_sync(0xffffffffu, s_toks[lane]);
  if (lane == 0) {
    if (blockIdx.y == 0) a.tokens[s] = toks;
    ws.dots[(int64_t)s * gridDim.y + blockIdx.y] = toks > 0 ? dot / (float)toks : 0.f;
    __threadfence();
    s_last = atomicAdd(ws.ticket, 1) == (int32_t)(gridDim.x * gridDim.y) - 1;
  }
  __syncwarp();
  if (!s_last) return;
  __threadfence();
  float sum = 0.f;
  int32_t n = 0;
  const int64_t parts = (int64_t)a.n_seqs * gridDim.y;
#pragma unroll 4
  for (int64_t i = lane; i < parts; i += 32) sum += __ldcg(ws.dots + i);
  for (int32_t i = lane; i < a.n_seqs; i += 32) n += __ldcg(a.tokens + i);
  sum = warp_add(sum);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane) return;
  a.tokens[a.n_seqs] = n;
  loss[0] = n > 0 ? a.coef * ((float)E / ((float)n * (float)a.top_k)) * sum : 0.f;
}

// d_logits of a block's tokens and, where d_bias is wanted, their column sums
// (slot = block; straight into d_bias where there is one block).
template <bool VEC, int N>
__global__ void __launch_bounds__(kLossThreads, N > 16 ? 1 : 2)
    router_backward_kernel(const moe_router_args a, const float* __restrict__ w, const float* __restrict__ dw,
                           const float* __restrict__ d_loss, float* __restrict__ d_logits, float* __restrict__ sums,
                           int32_t per_block) {
  constexpr int TOK = Group<VEC, N>::kBackward;
  extern __shared__ __align__(16) float sm[];  // [TOK][kLossWarps][pitch] the warps' rows, bias, g
  __shared__ int32_t s_first;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.n_experts, k = a.top_k;
  const int32_t pitch = row_pitch(E);
  float* pick = sm + warp * pitch;  // zero between tokens; the next row of the warp kLossWarps rows further
  float* s_bias = sm + TOK * kLossWarps * pitch;
  float* s_g = s_bias + pitch;
  pdl_launch_dependents();
  for (int32_t i = threadIdx.x; i < TOK * kLossWarps * pitch; i += kLossThreads) sm[i] = 0.f;
  if (a.bias)
    for (int32_t e = threadIdx.x; e < E; e += kLossThreads) s_bias[e] = a.bias[e];
  const int32_t lo = (int32_t)min((int64_t)blockIdx.x * per_block, (int64_t)a.n);
  const int32_t hi = (int32_t)min((int64_t)lo + per_block, (int64_t)a.n);
  F2 acc[N / 2] = {};
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
      F2 d[TOK][N / 2];
      int32_t id[TOK];
      float wj[TOK], dj[TOK];
      bool any = false;
#pragma unroll
      for (int u = 0; u < TOK; ++u) {
        const int64_t tu = t + u * kLossWarps;
        const bool there = tu < end, on = there && lossy && (!a.token_mask || a.token_mask[tu]);
        any = any || on;
        if (on) {
          Row<VEC, N>::load(a.logits + tu * E, E, lane, d[u], -INFINITY);
        } else {
#pragma unroll
          for (int i = 0; i < N / 2; ++i) d[u][i] = f2(-INFINITY);
        }
        id[u] = -1;
        wj[u] = dj[u] = 0.f;
        if (w && there && lane < k) {
          id[u] = a.topk_ids[tu * k + lane];
          wj[u] = w[tu * k + lane];
          dj[u] = dw[tu * k + lane];
        }
      }
      // sums over the experts of e^z and g e^z, over the picks of w dw
      float part[3][TOK] = {};
      if (any) {
        softmax_parts<VEC, N, TOK>(a.bias ? s_bias : nullptr, E, lane, d, part[0]);
        F2 m[TOK] = {};
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          F2 g[2];
          Row<VEC, N>::load4(s_g, E, lane, i, g, 0.f);
#pragma unroll
          for (int u = 0; u < TOK; ++u) m[u] = fma2(g[1], d[u][i / 2 + 1], fma2(g[0], d[u][i / 2], m[u]));
        }
#pragma unroll
        for (int u = 0; u < TOK; ++u) part[1][u] = m[u].x + m[u].y;
      }
#pragma unroll
      for (int u = 0; u < TOK; ++u) part[2][u] = wj[u] * dj[u];
      warp_sums(reinterpret_cast<float(&)[3 * TOK]>(part));
      if (w) {
#pragma unroll
        for (int u = 0; u < TOK; ++u) {
          float* p = pick + u * kLossWarps * pitch;
          const float dz = wj[u] * (dj[u] - part[2][u]);
          if (id[u] >= E) id[u] = -1;
          // each lane leaves its number at its expert: where another is found, an expert was picked twice
          int32_t* tag = reinterpret_cast<int32_t*>(p);
          if (id[u] >= 0) tag[id[u]] = lane;
          __syncwarp();
          if (__any_sync(0xffffffffu, id[u] >= 0 && tag[id[u]] != lane)) {
            if (id[u] >= 0) p[id[u]] = 0.f;
            __syncwarp();
            for (int j = 0; j < k; ++j) {  // one lane after the other
              if (lane == j && id[u] >= 0) p[id[u]] += dz;
              __syncwarp();
            }
          } else if (id[u] >= 0) {
            p[id[u]] = dz;
          }
        }
        __syncwarp();
      }
#pragma unroll
      for (int u = 0; u < TOK; ++u) {
        const int64_t tu = t + u * kLossWarps;
        if (tu >= end) break;
        const float inv = inverse(part[0][u]);
        const F2 mean = f2(-part[1][u] * inv);
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          F2 g[2], v[2] = {f2(0.f), f2(0.f)};
          if (any) Row<VEC, N>::load4(s_g, E, lane, i, g, 0.f);
          if (w) Row<VEC, N>::load4(pick + u * kLossWarps * pitch, E, lane, i, v, 0.f);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            F2& e = d[u][i / 2 + q];
            e = any ? fma2(mul2(e, f2(inv)), add2(g[q], mean), v[q]) : v[q];
            acc[i / 2 + q] = add2(acc[i / 2 + q], e);
          }
        }
        Row<VEC, N>::store(d_logits + tu * E, E, lane, d[u]);
      }
      if (w) {
        __syncwarp();
#pragma unroll
        for (int u = 0; u < TOK; ++u)
          if (id[u] >= 0) pick[u * kLossWarps * pitch + id[u]] = 0.f;
        __syncwarp();
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

// out[e] = sum of sums[b][e] over the blocks.
__global__ void __launch_bounds__(kJoinThreads)
    router_bias_kernel(const float* __restrict__ sums, int32_t blocks, int32_t E, float* __restrict__ out) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t e = blockIdx.x * 32 + lane, mine = blockIdx.x * 32 + warp;
  pdl_wait();
  s[warp][lane] = join_part<10>(sums, 0, blocks - 1, E, e, e < E);
  __syncthreads();
  const float v = join_parts(s);
  if (lane == 0 && mine < E) out[mine] = v;
}

// Tokens of a block.
int32_t loss_per_block(int32_t n, int32_t blocks) {
  return std::max(1, (int32_t)(((int64_t)n + blocks - 1) / blocks));
}

size_t loss_smem(int32_t E, int rows) { return (size_t)(rows * kLossWarps + 2) * row_pitch(E) * sizeof(float); }

template <bool VEC, int N>
cudaError_t balance_t(const moe_router_args& a, const LossSpace& ws, float* prob_sums, float* loss, cudaStream_t s) {
  static std::atomic<bool> configured[kMaxDevices];
  const cudaError_t e = raise_smem_limit(balance_kernel<VEC, N>, 80 * 1024, configured);
  if (e != cudaSuccess) return e;
  const int32_t blocks = balance_blocks(a.n, a.n_seqs);
  balance_kernel<VEC, N><<<blocks, kLossThreads, loss_smem(a.n_experts, 1), s>>>(
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
  router_backward_kernel<VEC, N><<<blocks, kLossThreads, loss_smem(a.n_experts, Group<VEC, N>::kBackward), s>>>(
      a, w, dw, d_loss, d_logits, sums, loss_per_block(a.n, blocks));
  return cudaGetLastError();
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

size_t router_loss_workspace(int32_t n, int32_t E, int32_t S) {
  const int64_t slots = loss_blocks(n, S) + (int64_t)S;
  return (size_t)(2 * round4(slots * E) + round4(slots) + round4((int64_t)S * ((E + 31) / 32)) + 4) * 4;
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
  return launch_ex(balance_join_kernel, dim3((unsigned)a.n_seqs, (unsigned)((E + 31) / 32)), dim3(kJoinThreads), 0, s,
                   true, a, ws, loss_per_block(a.n, blocks), prob_sums, loss);
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
  return launch_ex(router_bias_kernel, dim3((unsigned)((E + 31) / 32)), dim3(kJoinThreads), 0, s, true,
                   (const float*)sums, blocks, E, d_bias);
}

}  // namespace moe
