// layer_few.cu -- the experts of the whole-layer call for a few tokens, both
// products and the sum in one launch.
//
// Reading the picked experts' weights bounds it (one token, 6 + 1 experts of 2688
// x 1856: 39 MB), and whatever keeps those reads from being in flight.  Work comes
// in items of 16 rows, whose weights are one run of memory that a bulk copy brings
// to one of a block's three slots while the block works on another.  Eight warps
// multiply, each an eighth of the item's columns; a ninth draws the items and asks
// for their weights and a down item's rows, and one more a slot finishes its sums,
// which the others would spend most of their time waiting for.  The whole call for
// one token: 43 us with the eight doing all, 35 with a drawing and a finishing
// warp, 31.5 with one a slot and the rows by bulk copies (by the drawing warp's own
// loads, a down item every 3 us though multiplying it takes 1.5: 35).
// First come the up product's items (an expert's 16 rows; gated: its gate and up
// tiles), then the down product's (16 columns of the output over a part of the
// experts' rows, so that there are a few items an SM).
//
// A block draws its items' numbers in order.  Its first down item's weights
// are on their way before the block waits, once, for the up items of all experts;
// those have lower numbers, so their blocks are under way, and a block
// waits only when it has finished its own up items: every wait ends (and is
// bounded all the same).  The last part to finish 16 columns adds the parts in
// order, so that the bits do not depend on timing.
//
// The tokens are the matrix instruction's columns: token t is column t of every
// expert's product, its activations zero where it does not take the expert.
#include <algorithm>

#include "layer_pick.cuh"
#include "tile.cuh"

namespace moe {

namespace {

constexpr int kFewWarps = 8, kFewMath = 32 * kFewWarps, kFewSlots = 3;
constexpr int kFewThreads = kFewMath + 32 + 32 * kFewSlots;

// Shared memory after the slots of weights: x [n][H], slots of rows [n][part's tiles x 64], rows padded by 16 bytes.
struct FewLayout {
  uint32_t slot, x_row, a_row, x_at, a_at, total;
};
__host__ __device__ inline FewLayout few_layout(int32_t n, int32_t H, int32_t I, int32_t up_tiles, int32_t part_tiles) {
  FewLayout l;
  const int32_t up = up_tiles * (H / 64), most = up > part_tiles ? up : part_tiles;
  l.slot = ((uint32_t)most * kTileBytes + 127) / 128 * 128;
  l.x_row = 2 * H + 16;
  l.a_row = part_tiles * 128 + 16;
  l.x_at = kFewSlots * l.slot;
  l.a_at = l.x_at + n * l.x_row;
  l.total = l.a_at + kFewSlots * n * l.a_row;
  return l;
}

template <bool GATED>
struct FewSums {  // gated: the gate's, then the up's
  float v[GATED ? 2 : 1][kFewWarps][16][kDecPassTok + 1];
};
// The experts that any token takes, in the order of their first pair, and each token's pair with them.
struct FewWork {
  int32_t expert[kFewPairs];
  int16_t pair[kFewPairs][kDecPassTok];  // or -1
  float weight[kFewPairs][kDecPassTok];
  float up_g[kFewPairs], dn_g[kFewPairs], gate_g[kFewPairs];  // times 2^8: the tiles carry 2^-8
  int32_t tokens[kFewPairs];  // that take the expert
  int32_t experts;
  float up_part, columns_part, tiles_part;  // reciprocals of I / 16, H / 16 and I / 64
};
struct FewPicks {
  int32_t id[kFewPairs], first[1024];
  float w[kFewPairs];
  int32_t at[1024], count[(kFewPairs + 31) / 32];
};
// Named barriers, one of each for a slot: the next item from the drawing warp, its sums' place free from the finishing
// one; the sums to the finishing warp; the slot back to the drawing one.
__device__ __forceinline__ void bar_sync(int id, int count) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id, int count) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}
constexpr int kBarItem = 1, kBarSums = kBarItem + kFewSlots, kBarFree = kBarSums + kFewSlots;
static_assert(kBarFree + kFewSlots <= 16, "named barriers");
constexpr int kBarItemCount = kFewMath + 64;  // the multiplying, the drawing and the slot's finishing warps
__device__ __forceinline__ void red_release(int32_t* p) {
  asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(p) : "memory");
}

__device__ __forceinline__ int32_t ld_acquire(const int32_t* p) {
  int32_t v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// Every block's own: the tokens' picks from the logits, a warp a token, and the experts among them (one token, 128
// experts: 2 us; by the router's last block, for all, it took as long, and 3 more until they all had it).
template <bool GATED>
__device__ __forceinline__ void pick_work(const LayerFewArgs& a, FewWork& work, FewPicks& picks) {
  const int32_t pairs = a.n * a.slots, p = threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  static_assert(kFewThreads / 32 >= kFewTokens && kFewThreads >= kFewPairs, "a warp a token, a thread a pair");
  if (warp < a.n)
    pick_any(a.pick, warp, lane, picks.id + warp * a.slots, picks.w + warp * a.slots, blockIdx.x == 0);
  __syncthreads();
  const int32_t e = p < pairs ? picks.id[p] : 0;
  if (p < pairs) picks.first[e] = pairs;
  __syncthreads();
  if (p < pairs) atomicMin(&picks.first[e], p);
  __syncthreads();
  const bool first = p < pairs && picks.first[e] == p;
  const uint32_t who = __ballot_sync(0xffffffffu, first);
  if (lane == 0 && warp < (kFewPairs + 31) / 32) picks.count[warp] = __popc(who);
  __syncthreads();
  int32_t at = __popc(who & ((1u << lane) - 1)), all = 0;
  for (int32_t w = 0; w < (kFewPairs + 31) / 32; ++w) {
    if (w < warp) at += picks.count[w];
    all += picks.count[w];
  }
  if (first) {
    work.expert[at] = e;
    picks.at[e] = at;
    work.up_g[at] = 256.f * a.up_g[e];
    work.dn_g[at] = 256.f * a.dn_g[e];
    if (GATED) work.gate_g[at] = 256.f * a.gate_g[e];
  }
  if (p == 0) work.experts = all;
  __syncthreads();
  if (p < pairs) {
    work.pair[picks.at[e]][p / a.slots] = (int16_t)p;
    work.weight[picks.at[e]][p / a.slots] = picks.w[p];
    atomicAdd(&work.tokens[picks.at[e]], 1);
  }
  __syncthreads();
}
template <bool GATED>
__device__ __forceinline__ void keep(FewSums<GATED>& sums, int which, int warp, int lane, const float (&acc)[4]) {
  const int g = lane >> 2, t = lane & 3;
  sums.v[which][warp][g][2 * t] = acc[0];
  sums.v[which][warp][g][2 * t + 1] = acc[1];
  sums.v[which][warp][g + 8][2 * t] = acc[2];
  sums.v[which][warp][g + 8][2 * t + 1] = acc[3];
}
template <bool GATED>
__device__ __forceinline__ float sum_of(const FewSums<GATED>& sums, int which, int row, int col) {
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < kFewWarps; ++w) v += sums.v[which][w][row][col];
  return v;
}
// The lane's 16 values of a k-tile of its token's row.
struct FewX {
  uint4 x0, x1;
};
__device__ __forceinline__ FewX load_x(const uint8_t* row, int32_t tile, bool live) {
  FewX x = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if (live) {
    x.x0 = *reinterpret_cast<const uint4*>(row + tile * 128);
    x.x1 = *reinterpret_cast<const uint4*>(row + tile * 128 + 16);
  }
  return x;
}

// x / d of whole numbers below 2^20, r = 1 / d: exact, and shorter than a division for a warp that everyone waits for.
__device__ __forceinline__ int32_t quotient(int32_t x, float r) { return (int32_t)(((float)x + 0.5f) * r); }

// A part's tiles: [first, last) of all experts' (expert by expert).
__device__ __forceinline__ int32_t part_begin(const LayerFewArgs& a, int32_t tiles, int32_t part) {
  return (int32_t)((uint32_t)tiles * (uint32_t)part / (uint32_t)a.parts);  // (tiles < 2^13, parts < 2^6)
}

// One thread: asks for an item's weights, and announces a down item's rows with them.
template <bool GATED>
__device__ __forceinline__ void issue(const LayerFewArgs& a, const FewWork& p, int32_t item, int32_t up, uint8_t* slot,
                                      uint64_t* bar) {
  fence_proxy_async_smem();
  if (item < up) {
    const int32_t KT = (GATED ? 2 : 1) * (a.H / 64), NT = a.I / 16, ai = quotient(item, p.up_part);
    const uint32_t bytes = (uint32_t)KT * kTileBytes;
    mbar_arrive_expect_tx(bar, bytes);
    bulk_g2s(slot, a.up_tiles + ((int64_t)p.expert[ai] * NT + (item - ai * NT)) * bytes, bytes, bar);
    return;
  }
  const int32_t KT = a.I / 64, NT = a.H / 16, part = quotient(item - up, p.columns_part), ct = item - up - part * NT;
  const int32_t all = p.experts * KT, p0 = part_begin(a, all, part), p1 = part_begin(a, all, part + 1);
  uint32_t bytes = (uint32_t)(p1 - p0) * kTileBytes;
  for (int32_t i = p0, ai = quotient(p0, p.tiles_part); i < p1; ++ai) {
    const int32_t run = min((ai + 1) * KT, p1) - i;
    bytes += (uint32_t)run * 128u * p.tokens[ai];
    i += run;
  }
  mbar_arrive_expect_tx(bar, bytes);
  for (int32_t i = p0, ai = quotient(p0, p.tiles_part); i < p1; ++ai) {
    const int32_t run = min((ai + 1) * KT, p1) - i;
    bulk_g2s(slot + (i - p0) * kTileBytes, a.dn_tiles + (((int64_t)p.expert[ai] * NT + ct) * KT + (i - ai * KT)) * kTileBytes,
             (uint32_t)run * kTileBytes, bar);
    i += run;
  }
}
// The rows that a down item multiplies (they are there).
__device__ __forceinline__ void issue_rows(const LayerFewArgs& a, const FewWork& p, int32_t item, int32_t up, uint8_t* as,
                                           uint32_t a_row, uint64_t* bar) {
  // (written by ordinary stores, read by a bulk copy)
  asm volatile("fence.proxy.async;" ::: "memory");
  const int32_t KT = a.I / 64, part = quotient(item - up, p.columns_part);
  const int32_t all = p.experts * KT, p0 = part_begin(a, all, part), p1 = part_begin(a, all, part + 1);
  for (int32_t i = p0, ai = quotient(p0, p.tiles_part); i < p1; ++ai) {
    const int32_t run = min((ai + 1) * KT, p1) - i;
    for (int32_t col = 0; col < a.n; ++col) {
      const int32_t pair = p.pair[ai][col];
      if (pair >= 0)
        bulk_g2s(as + col * a_row + (i - p0) * 128, a.Ap + (int64_t)pair * a.I + 64 * (i - ai * KT), (uint32_t)run * 128u, bar);
    }
    i += run;
  }
}

// The warps' sums of an up item.
template <bool GATED>
__device__ __forceinline__ void up_sums(const LayerFewArgs& a, const FewWork& p, int32_t ai, const uint8_t* slot,
                                        const uint8_t* xs, uint32_t x_row, const uint32_t* lut, FewSums<GATED>& sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int32_t KT = a.H / 64, k0 = KT * warp / kFewWarps, k1 = KT * (warp + 1) / kFewWarps;
  constexpr int kTiles = GATED ? 2 : 1;  // the gate's, then the up's
  const bool mine = g < a.n && p.pair[ai][g] >= 0;
  const uint8_t* row = xs + g * x_row + 32 * t;
  float acc[kTiles][4] = {}, acc2[kTiles][4] = {};
#pragma unroll 2
  for (int32_t k = k0; k < k1; ++k) {
    const FewX x = load_x(row, k, mine);
#pragma unroll
    for (int h = 0; h < kTiles; ++h)
      tile_mma(slot + (h * KT + k) * kTileBytes, x.x0, x.x1, lane, lut, acc[h], acc2[h]);
  }
#pragma unroll
  for (int h = 0; h < kTiles; ++h) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[h][i] += acc2[h][i];
    keep(sums, h, warp, lane, acc[h]);
  }
}
// By the finishing warp: the expert's rows, and word that they are there.
template <bool GATED>
__device__ __forceinline__ void up_finish(const LayerFewArgs& a, const FewWork& p, int32_t ai, int32_t rt, const FewSums<GATED>& sums) {
  const int lane = threadIdx.x & 31;
  for (int32_t i = lane; i < 16 * a.n; i += 32) {
    const int32_t r = i & 15, col = i >> 4, pair = p.pair[ai][col];
    if (pair < 0) continue;
    const float h = sum_of(sums, GATED ? 1 : 0, r, col) * p.up_g[ai];
    float v;
    if (GATED) {
      const float q = sum_of(sums, 0, r, col) * p.gate_g[ai];
      v = q / (1.f + expf(-q)) * h;
    } else {
      const float m = h > 0.f ? h : 0.f;
      v = m * m;
    }
    a.Ap[(int64_t)pair * a.I + 16 * rt + r] = f2bf_rn(v);
  }
  __syncwarp();
  if (lane == 0) red_release(&a.plan->done[ai]);
}

// By the drawing warp, once: every expert's rows are there.
__device__ __forceinline__ void wait_rows(const LayerFewArgs& a, int32_t experts) {
  const uint64_t t0 = globaltimer_ns();
  for (int32_t ai = threadIdx.x & 31; ai < experts; ai += 32)
    while (ld_acquire(&a.plan->done[ai]) < a.I / 16) {
      __nanosleep(40);
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        atomicOr(a.err, kFlagTimeout);
        break;
      }
    }
  __syncwarp();
}
// The warps' sums of a down item.
template <bool GATED>
__device__ __forceinline__ void down_sums(const LayerFewArgs& a, const FewWork& p, int32_t part, const uint8_t* slot,
                                          const uint8_t* as, uint32_t a_row, const uint32_t* lut, FewSums<GATED>& sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int32_t KT = a.I / 64, all = p.experts * KT;
  const int32_t p0 = part_begin(a, all, part), tiles = part_begin(a, all, part + 1) - p0;
  const int32_t i0 = tiles * warp / kFewWarps, i1 = tiles * (warp + 1) / kFewWarps;
  const uint8_t* row = as + g * a_row + 32 * t;
  float total[4] = {}, acc[4] = {}, acc2[4] = {};
  for (int32_t i = i0; i < i1;) {  // expert by expert
    const int32_t ai = quotient(p0 + i, p.tiles_part), end = min(i1, (ai + 1) * KT - p0);
    const bool mine = g < a.n && p.pair[ai][g] >= 0;
#pragma unroll 2
    for (; i < end; ++i) {
      const FewX x = load_x(row, i, mine);
      tile_mma(slot + i * kTileBytes, x.x0, x.x1, lane, lut, acc, acc2);
    }
    const float dg = p.dn_g[ai];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int32_t col = 2 * t + (k & 1);
      if (col < a.n && p.pair[ai][col] >= 0) total[k] = fmaf(p.weight[ai][col] * dg, acc[k] + acc2[k], total[k]);
      acc[k] = acc2[k] = 0.f;
    }
  }
  keep(sums, 0, warp, lane, total);
}
// By the finishing warp: the part's sums, and from the last part of its columns the output.
template <bool GATED>
__device__ __forceinline__ void down_finish(const LayerFewArgs& a, int32_t ct, int32_t part, const FewSums<GATED>& sums) {
  const int lane = threadIdx.x & 31;
  for (int32_t i = lane; i < 16 * a.n; i += 32) {
    const int64_t at = (int64_t)(i >> 4) * a.H + 16 * ct + (i & 15);
    a.part[(int64_t)part * a.n * a.H + at] = sum_of(sums, 0, i & 15, i >> 4);
  }
  __syncwarp();
  int32_t last = 0;
  if (lane == 0) {
    last = atom_add_acq_rel_gpu(&a.col_done[ct], 1) == a.parts - 1;
    if (last) a.col_done[ct] = 0;
  }
  if (!__shfl_sync(0xffffffffu, last, 0)) return;
  __syncwarp();
  for (int32_t i = lane; i < 16 * a.n; i += 32) {
    const int64_t at = (int64_t)(i >> 4) * a.H + 16 * ct + (i & 15);
    float v = 0.f;
#pragma unroll 8
    for (int32_t q = 0; q < a.parts; ++q) v += ld_cg_f32(a.part + (int64_t)q * a.n * a.H + at);
    if (a.residual) v += __uint_as_float((uint32_t)a.residual[at] << 16);
    a.dst[at] = f2bf_rn(v);
  }
}

template <bool GATED>
__global__ void __launch_bounds__(kFewThreads, 2) layer_few_kernel(const __grid_constant__ LayerFewArgs a, const FewLayout l) {
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ uint32_t lut[256];
  __shared__ FewSums<GATED> sums[kFewSlots];
  __shared__ FewWork work;
  __shared__ __align__(8) uint64_t full[kFewSlots];
  __shared__ int32_t item[kFewSlots], summed[kFewSlots];  // drawn; whose sums lie there
  __shared__ int32_t finished;  // up items that the block has finished
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < 256; i += kFewThreads) lut[i] = scale_bf16_2p118((uint32_t)i) * 0x10001u;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kFewSlots; ++s) mbar_init(&full[s], 1);
    finished = 0;
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < kFewPairs * kDecPassTok; i += kFewThreads) work.pair[i / kDecPassTok][i % kDecPassTok] = -1;
  for (int i = threadIdx.x; i < kFewPairs; i += kFewThreads) work.tokens[i] = 0;
  if (threadIdx.x == 0) {
    work.up_part = 16.f / (float)a.I;
    work.columns_part = 16.f / (float)a.H;
    work.tiles_part = 64.f / (float)a.I;
  }
  // x is there: the router, which lets this kernel begin, does so when all before it has finished
  for (int32_t i = threadIdx.x; i < a.n * (a.H / 8); i += kFewThreads) {
    const int32_t col = i / (a.H / 8), at = i - col * (a.H / 8);
    *reinterpret_cast<uint4*>(sm + l.x_at + col * l.x_row + 16 * at) =
        __ldcg(reinterpret_cast<const uint4*>(a.x + (int64_t)col * a.H) + at);
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  int32_t ticket = 0;
  if (threadIdx.x == kFewMath) ticket = atomicAdd(&a.plan->ticket, 1);
  static_assert(sizeof(FewPicks) <= sizeof(sums), "the picks lie where the sums will");
  pick_work<GATED>(a, work, *reinterpret_cast<FewPicks*>(sums));
  const int32_t experts = work.experts;
  const int32_t NT = a.I / 16, CT = a.H / 16, up = experts * NT, items = up + a.parts * CT;

  if (threadIdx.x >= kFewMath + 32) {  // a slot's finishing warp
    const int s = (threadIdx.x - kFewMath - 32) / 32;
    bar_arrive(kBarItem + s, kBarItemCount);
    while (true) {
      bar_sync(kBarSums + s, kFewMath + 32);
      const int32_t now = summed[s];  // (item[s] may be the next already)
      if (now >= items) break;
      if (now < up) {
        const int32_t ai = quotient(now, work.up_part);
        up_finish<GATED>(a, work, ai, now - ai * NT, sums[s]);
        if (lane == 0) atomicAdd(&finished, 1);
      } else {
        const int32_t part = quotient(now - up, work.columns_part);
        down_finish<GATED>(a, now - up - part * CT, part, sums[s]);
      }
      __syncwarp();
      bar_arrive(kBarItem + s, kBarItemCount);
    }
    return;
  }
  if (threadIdx.x >= kFewMath) {  // the drawing warp
    int32_t drawn = 0;  // up items
    bool waited = false;
    // The next item into slot s: its weights asked for, then a down item's rows, for which it waits only when the block
    // has no up item of its own left to finish.
    auto draw = [&](int s) {
      const int32_t now = __shfl_sync(0xffffffffu, ticket, 0);
      if (lane == 0) {
        item[s] = now;
        if (now < items) issue<GATED>(a, work, now, up, sm + s * l.slot, &full[s]);
        ticket = atomicAdd(&a.plan->ticket, 1);
      }
      if (now < up) {
        ++drawn;
      } else if (now < items) {
        if (!waited) {
          const uint64_t t0 = globaltimer_ns();
          while (*(volatile int32_t*)&finished < drawn && globaltimer_ns() - t0 < kWaitLimitNs) __nanosleep(20);
          wait_rows(a, experts);
          waited = true;
        }
        if (lane == 0) issue_rows(a, work, now, up, sm + l.a_at + s * a.n * l.a_row, l.a_row, &full[s]);
      }
      __syncwarp();
      bar_arrive(kBarItem + s, kBarItemCount);
      return now;
    };
    int32_t held[kFewSlots];
#pragma unroll
    for (int s = 0; s < kFewSlots; ++s) held[s] = draw(s);
    for (bool more = true; more;) {
#pragma unroll
      for (int s = 0; s < kFewSlots; ++s) {
        if (held[s] >= items) {
          more = false;
          break;
        }
        bar_sync(kBarFree + s, kFewMath + 32);
        held[s] = draw(s);
      }
    }
    return;
  }

  uint32_t parity = 0;
  for (int s = 0;;) {
    bar_sync(kBarItem + s, kBarItemCount);
    const int32_t now = item[s];
    if (now >= items) {
      // no further item: each slot's finishing warp, this one's first, learns it when it is through with its last
      for (int k = 0; k < kFewSlots; ++k) {
        if (k > 0) bar_sync(kBarItem + s, kBarItemCount);
        if (threadIdx.x == 0) summed[s] = items;
        bar_arrive(kBarSums + s, kFewMath + 32);
        s = s + 1 == kFewSlots ? 0 : s + 1;
      }
      break;
    }
    if (threadIdx.x == 0) summed[s] = now;
    mbar_wait(&full[s], parity, a.err);
    const uint8_t* slot = sm + s * l.slot;
    if (now < up)
      up_sums<GATED>(a, work, quotient(now, work.up_part), slot, sm + l.x_at, l.x_row, lut, sums[s]);
    else
      down_sums<GATED>(a, work, quotient(now - up, work.columns_part), slot, sm + l.a_at + s * a.n * l.a_row, l.a_row, lut, sums[s]);
    bar_arrive(kBarSums + s, kFewMath + 32);
    bar_arrive(kBarFree + s, kFewMath + 32);
    if (++s == kFewSlots) {
      s = 0;
      parity ^= 1u;
    }
  }
}

template <bool GATED>
cudaError_t few_launch(const LayerFewArgs& a, const FewLayout& l, int sms, cudaStream_t s) {
  static std::atomic<bool> configured[kMaxDevices];
  cudaError_t e = raise_smem_limit(layer_few_kernel<GATED>, kFewSmem, configured);
  int per = 0;
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, layer_few_kernel<GATED>, kFewThreads, l.total);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)a.n * a.slots * (a.I / 16) + (int64_t)a.parts * (a.H / 16);
  return launch_ex(layer_few_kernel<GATED>, dim3((unsigned)std::min<int64_t>(items, (int64_t)std::max(per, 1) * sms)),
                   dim3(kFewThreads), l.total, s, true, a, l);
}

int32_t part_tiles(int32_t n, int32_t slots, int32_t I, int32_t parts) { return (n * slots * (I / 64) + parts - 1) / parts; }

}  // namespace

// Parts of about 40 tiles where every pair takes an expert of its own.
int32_t layer_few_parts(int32_t n, int32_t slots, int32_t I) {
  return std::max(1, std::min((n * slots * (I / 64) + 39) / 40, kFewParts));
}

// One token, and a few where two blocks fit an SM.  Against the streaming kernel (decode.cu), whole calls of 6 + 1
// experts: of 2688 x 1856, one token 28.0 us and 35.5 (gated 37.6 and 38.3), but two tokens, a block an SM, 49.8 and
// 40.1 (gated 61.7 and 47.1); of 1024 x 512, two blocks, one token 14.1 and 22.4, two 18.2 and 27.7, six 28.5 and 35.7.
bool layer_few_takes(int32_t n, int32_t slots, int32_t H, int32_t I, bool gated) {
  if (n > kFewTokens || n * slots > kFewPairs) return false;
  const int32_t parts = layer_few_parts(n, slots, I);
  if ((int64_t)n * slots * (I / 16) + (int64_t)parts * (H / 16) >= 1 << 20) return false;  // quotient's range
  const size_t total = few_layout(n, H, I, gated ? 2 : 1, part_tiles(n, slots, I, parts)).total;
  const size_t fixed = sizeof(FewWork) + kFewSlots * (gated ? sizeof(FewSums<true>) : sizeof(FewSums<false>)) + 2048;
  return total <= kFewSmem && (n == 1 || 2 * (total + fixed) <= 227 * 1024);
}

cudaError_t launch_layer_few(const LayerFewArgs& a, bool gated, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const FewLayout l = few_layout(a.n, a.H, a.I, gated ? 2 : 1, part_tiles(a.n, a.slots, a.I, a.parts));
  return gated ? few_launch<true>(a, l, sms, s) : few_launch<false>(a, l, sms, s);
}

}  // namespace moe
