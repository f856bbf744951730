// lora.cu -- low-rank adapters of many requests at once, added to a shared
// projection's result (moe_lora_apply).
//
//   v = A[l] x (over the adapter's rank),  out = y + B[l] (scale[l] v)
//
// Tokens are grouped by adapter into tiles, and one CTA (or a cluster of CTAs,
// where there are few tiles) takes a tile through both products: v never
// leaves the SM.  Larger batches take tiles of 128 (lora_mma.cu) or 64
// (lora_rows.cu); here tiles are 16 tokens.  Both products are bf16 warp matrix
// instructions with tokens as rows.  What bounds a call of few tokens is
// latency: finding the tile, two chains of copies and a meeting of the cluster
// between them (32 tokens, 2688 to 1856, ranks to 32: 6.4 us on a GB300, of which
// the bytes are 0.5), so what counts is how many bytes are in flight at once.
// Every thread
// copies the 16-byte pieces of the operands that its own fragments are made of
// into its own slots of a shared-memory ring, some steps ahead, by
// asynchronous copies, and reads back only those: no barrier stands in the
// loops.  A lane's 16 bytes of a row are the k elements of two matrix
// instructions (the order of k inside a window of 32 is free as long as both
// operands use it).
//
//   first product:  the warps (and the cluster's CTAs) split in_features in
//     windows of 32; their partial sums meet in shared memory (and in the
//     cluster's shared memories, each store counted on the receiver's
//     mbarrier: half a microsecond less than a barrier of the cluster after
//     them), added in a fixed order.
//   second product: the warps split out_features in blocks of 32 columns.  The
//     columns of a block are dealt to the four 8-column instructions so that
//     a lane ends up with 8 neighbouring columns of a token (two runs of 4
//     where y or out is fp32): y comes in and out goes out in whole memory
//     sectors.  v enters as the sum of three bf16 terms (24 bits of mantissa).
//
// Grouping: up to kRankedTokens tokens every CTA compares each id with those
// before it (ranked_tile), up to small_tokens every CTA counts the adapters'
// tokens (counted_tile); for larger batches a one-CTA kernel (two kernels past
// kPlanSlice tokens) sorts the tokens by adapter into the workspace, which the
// next launch's start overlaps.  A token's row of the products depends on no
// other token, so the order inside a group does not matter to the result.
#include "lora.cuh"

namespace moe {

namespace {

__global__ void __launch_bounds__(kPlanThreads)
    lora_hist_kernel(const int32_t* __restrict__ ids, int32_t n, int32_t L, int32_t* __restrict__ hist) {
  extern __shared__ int32_t sm_hist[];  // [L + 1]
  for (int32_t l = threadIdx.x; l <= L; l += kPlanThreads) sm_hist[l] = 0;
  __syncthreads();
  const int64_t beg = (int64_t)blockIdx.x * kPlanSlice;
#pragma unroll 4
  for (int j = 0; j < kPlanPer; ++j) {
    const int64_t i = beg + threadIdx.x + j * kPlanThreads;
    const int32_t key = i < n ? bucket_of(ids[i], L) : -1;
    const bool one = __all_sync(0xffffffffu, key == __shfl_sync(0xffffffffu, key, 0));
    if (key >= 0 && (!one || (threadIdx.x & 31) == 0)) atomicAdd(&sm_hist[key], one ? 32 : 1);
  }
  __syncthreads();
  for (int32_t l = threadIdx.x; l <= L; l += kPlanThreads) hist[(int64_t)blockIdx.x * (L + 1) + l] = sm_hist[l];
}

// Sorts slice blockIdx.x (hist: the slices' histograms, nullptr for one slice).
__global__ void __launch_bounds__(kPlanThreads)
    lora_plan_kernel(const int32_t* __restrict__ ids, int32_t n, int32_t L, int32_t tile, LoraPlan p,
                     const int32_t* __restrict__ hist) {
  extern __shared__ int32_t sm_plan[];  // count, then first position, of each of this slice's buckets: [L + 1]
  __shared__ int32_t warp_cnt[32], warp_tiles[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
  const int64_t beg = (int64_t)blockIdx.x * kPlanSlice;
  pdl_launch_dependents();
  int32_t key[kPlanPer], rank[kPlanPer];
#pragma unroll
  for (int j = 0; j < kPlanPer; ++j) {
    const int64_t i = beg + tid + j * kPlanThreads;
    key[j] = i < n ? ids[i] : 0;
  }
  for (int32_t l = tid; l <= L; l += kPlanThreads) sm_plan[l] = 0;
  __syncthreads();
  const int steps = (int)min((int64_t)kPlanPer, ((int64_t)n - beg + kPlanThreads - 1) / kPlanThreads);
  // A token's place in its bucket: by one addition for a warp whose tokens share it (the rule in runs of a request's
  // tokens), else one a token.  (Matching the lanes of a warp instead takes a round for every bucket in it: 16384
  // tokens of 16 adapters in random order 22 us against 16, in runs 13.2 / 12.4; only random order over one or two
  // adapters is slower this way, 13.3 / 18.7.)
  constexpr int kBatch = 4;  // side by side
#pragma unroll
  for (int j0 = 0; j0 < kPlanPer; j0 += kBatch) {
    if (j0 >= steps) break;
    bool one[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int j = j0 + i;
      key[j] = beg + tid + j * kPlanThreads < n ? bucket_of(key[j], L) : -1;
      one[i] = __all_sync(0xffffffffu, key[j] == __shfl_sync(0xffffffffu, key[j], 0));
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int j = j0 + i;
      rank[j] = 0;
      if (key[j] >= 0 && (!one[i] || lane == 0)) rank[j] = atomicAdd(&sm_plan[key[j]], one[i] ? 32 : 1);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int j = j0 + i;
      const int32_t first = __shfl_sync(0xffffffffu, rank[j], 0);
      if (one[i]) rank[j] = first + lane;
    }
  }
  __syncthreads();
  // adapter tid: its tokens in all slices and in those before this one
  int32_t total = 0, before = 0, none_before = 0;
  if (tid < L) total = sm_plan[tid];
  if (hist) {
    if (tid < L) {
      total = 0;
      for (int32_t b = 0; b < (int32_t)gridDim.x; ++b) {
        const int32_t v = hist[(int64_t)b * (L + 1) + tid];
        total += v;
        before += b < (int32_t)blockIdx.x ? v : 0;
      }
    }
    for (int32_t b = 0; b < (int32_t)blockIdx.x; ++b) none_before += hist[(int64_t)b * (L + 1) + L];
  }
  const int32_t tiles = (total + tile - 1) / tile;
  int32_t ic = total, it = tiles;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t vc = __shfl_up_sync(0xffffffffu, ic, d), vt = __shfl_up_sync(0xffffffffu, it, d);
    if (lane >= d) {
      ic += vc;
      it += vt;
    }
  }
  if (lane == 31) {
    warp_cnt[warp] = ic;
    warp_tiles[warp] = it;
  }
  __syncthreads();
  if (warp == 0) {
    int32_t c = warp_cnt[lane], t = warp_tiles[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t vc = __shfl_up_sync(0xffffffffu, c, d), vt = __shfl_up_sync(0xffffffffu, t, d);
      if (lane >= d) {
        c += vc;
        t += vt;
      }
    }
    warp_cnt[lane] = c;
    warp_tiles[lane] = t;
  }
  __syncthreads();
  const int32_t start = ic - total + (warp ? warp_cnt[warp - 1] : 0);
  const int32_t tbase = it - tiles + (warp ? warp_tiles[warp - 1] : 0);
  if (tid < L) sm_plan[tid] = start + before;
  if (tid == 0) sm_plan[L] = warp_cnt[31] + none_before;
  if (blockIdx.x == 0) {
    if (tid < L) {
      p.starts[tid] = start;
      p.tile_base[tid] = tbase;
    }
    if (tid == 0) {
      p.starts[L] = warp_cnt[31];
      p.starts[L + 1] = n;
      p.tile_base[L] = warp_tiles[31];
      p.tile_base[L + 1] = warp_tiles[31] + (n - warp_cnt[31] + tile - 1) / tile;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPlanPer; ++j) {
    if (j >= steps) break;
    if (key[j] >= 0) p.order[sm_plan[key[j]] + rank[j]] = (int32_t)(beg + tid + j * kPlanThreads);
  }
}

// More tokens than these take the larger tiles of lora_mma.cu or lora_rows.cu:
// there the adapter's matrices are read less often, which counts the more the
// larger the rank, but fewer CTAs share a small batch.  Tiles of 16 against
// 128, us on a GB300:
//   4096 to 4096, rank 16: 1024 tokens 13.4 / 24.5, 2048 21.6 / 28.6, 3000 33.9 / 31.9
//   4096 to 1024, rank 32: 1024 10.8 / 19.3, 2048 15.0 / 19.7, 3000 23.4 / 21.1
//   4096 to 4096, rank 64: 300 22.4 / 31.5, 512 25.1 / 31.6, 640 34.1 / 32.3, 1536 49.5 / 34.3
//   the same, rank 128: 300 30.9 / 43.3, 512 40.8 / 43.9, 768 50.7 / 45.7
constexpr int32_t kSmallTokens = 2048, kSmallTokensWide = 512;  // max_rank up to 32, above
// Comparing against counting: 64 tokens 7.3 / 8.0 us, 128 8.1 / 8.1, 256 10.2 / 8.9; counting against a sorting
// kernel before: 384 9.6 / 12.1, 1024 13.4 / 16.1 (4096 to 4096, rank 16, 16 adapters); in lora_mma.cu, with up to
// 16384 tokens, counting gains nothing (4314 32.8 / 31.7, 16384 75.5 / 74.5).
constexpr int32_t kRankedTokens = 128;
static_assert(kRankedTokens <= kLoraThreads, "one token a thread");
// Batches without a workspace never reach a kernel that reads a plan from one (its pointers would be null).
static_assert(kSmallTokensWide <= kSmallTokens, "lora_workspace is 0 bytes up to kSmallTokensWide");
inline int32_t small_tokens(int32_t max_rank) { return max_rank <= 32 ? kSmallTokens : kSmallTokensWide; }

// Set where a bounded wait ran out.
__device__ int32_t g_lora_small_flags;

// Tiles of 16 tokens; NT groups of 8 ranks a pass of the first product.
template <int NT>
__global__ void __launch_bounds__(kLoraThreads, 2)
    lora_kernel(const moe_lora_args a, uint32_t ring_bytes) {
  constexpr int MT = 16, KG = kLoraWarps;
  constexpr int RPASS = 8 * NT, RP = RPASS + 8;  // ranks of a pass; row pitch of the partial sums
  extern __shared__ __align__(16) char sm[];
  __shared__ int32_t row[MT];
  __shared__ __align__(8) uint64_t met;  // the CTAs' sums of a pass have arrived
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const uint32_t C = cluster_size(), cr = cluster_rank();
  if (C > 1 && tid == 0) {
    mbar_init(&met, 1);
    fence_mbar_init();
  }
  Tile t;
  // ring; the warps' sums [KG][MT][RP]; in a cluster the CTAs' sums [C][MT][RP]; v [kLoraTerms][MT][VP] bf16
  float* part = reinterpret_cast<float*>(sm + ring_bytes);
  float* recv = part + KG * MT * RP;
  uint16_t* v = reinterpret_cast<uint16_t*>(recv + (C > 1 ? C * MT * RP : 0));
  const int32_t tile = (int32_t)(blockIdx.x / C);
  if (!(a.n <= kRankedTokens ? ranked_tile<MT>(a, tile, row, reinterpret_cast<int32_t*>(part), t)
                            : counted_tile<MT, kSmallTokens / kLoraThreads>(a, tile, row, reinterpret_cast<int32_t*>(sm), t)))
    return;
  if (C > 1) cluster_arrive();  // (waited for before the first store into a peer: its mbarrier is ready by then)
  const uint32_t slot = tid * 16, sm_u32 = smem_u32(sm);  // offsets in sm; cp.async takes addresses
  const int32_t VP = a.max_rank <= 32 ? 32 : ((a.max_rank + 63) & ~63) + 32;  // pitch of v: rows 64 bytes apart mod 128
  // places past the tile's count take its first token: their rows of the products are never looked at
  int32_t tok[2];
  int64_t at_tok[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    tok[h] = row[h * 8 + g];
    at_tok[h] = tok[h] >= 0 ? tok[h] : row[0];
  }

  // The first product's steps: a window of 32 columns of x and A.  A warp takes pairs of windows, 128 bytes of a row:
  // first the even, then the odd one.
  const uint32_t row_bytes = (uint32_t)a.in_features * 2, lane_a = g * row_bytes + 16 * q;
  const uint32_t pair0 = ((uint32_t)cr * KG + warp) * 128, jump = (uint32_t)C * KG * 128 - 64;
  const char* xr[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    xr[h] = static_cast<const char*>(a.x.data) + 16 * q + at_tok[h] * (a.x.stride ? a.x.stride : a.in_features) * 2;
  const char* A = reinterpret_cast<const char*>(a.a) + (int64_t)t.adapter * a.max_rank * (int64_t)row_bytes;
  uint32_t fetch_off = pair0;  // byte offset in a row of the window to fetch next
  bool fetch_odd = false;
  auto fetch = [&](int stage, uint32_t step, int32_t nt) {
    if (fetch_off < row_bytes && fetch_off + 16 * q < row_bytes) {  // else past the row's end, and read as 0
      const uint32_t at = slot + stage * step;
#pragma unroll
      for (int h = 0; h < 2; ++h) ring16(sm_u32 + at + h * kSlotVec, xr[h] + fetch_off);
      // rows from the rank on are in the bank and reach only entries of v that are set to zero
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (j >= nt) break;
        ring16(sm_u32 + at + (2 + j) * kSlotVec, A + ((uint64_t)(8 * j) * row_bytes + fetch_off) + lane_a);
      }
    }
    fetch_off += fetch_odd ? jump : 64;
    fetch_odd = !fetch_odd;
    ring_commit();
  };
  // (the first steps are on their way before the adapter's rank is here: as many rows as any has)
  int32_t nt = min(NT, a.max_rank / 8);
  uint32_t step = (2 + nt) * kSlotVec;
  int stages = ring_stages(ring_bytes, step);
  if (t.adapter < a.n_adapters)
    for (int s = 0; s + 1 < stages; ++s) fetch(s, step, nt);
  const int32_t rank = t.rank;
  const int32_t R32 = (rank + 31) & ~31;

  // The second product's steps: a block of 32 columns of y and B.  A lane's columns: 4 at c0 and 4 at c0 + next.
  const bool quads = a.y_dtype == MOE_DTYPE_F32 || a.out_dtype == MOE_DTYPE_F32;
  const bool yf = a.y_dtype == MOE_DTYPE_F32, has_y = a.y.data != nullptr;
  const int32_t lc = quads ? 4 : 8, next = quads ? 16 : 4;
  const uint32_t y_vecs = !has_y ? 0 : yf ? 2 : 1, y_size = yf ? 4 : 2;
  const char* B = reinterpret_cast<const char*>(a.b) +
                  (rank > 0 ? (int64_t)t.adapter * a.out_features * a.max_rank * 2 : 0);
  const int32_t blocks = (a.out_features + 31) / 32, kwins = R32 / 32;
  const uint32_t y_step = max(1u, 4 * kwins + 2 * y_vecs) * kSlotVec;
  const int y_stages = ring_stages(ring_bytes, y_step);
  const char* yr[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    yr[h] = static_cast<const char*>(a.y.data) +
            (at_tok[h] * (a.y.stride ? a.y.stride : a.out_features) + lc * q) * y_size;
  const int32_t b0 = (int32_t)cr * kLoraWarps + warp, bstep = (int32_t)C * kLoraWarps;
  const int32_t lane_o = (g >> 1) * lc + (g & 1);    // the lane's row of B in a block, without j's part
  const uint32_t b_bytes = (uint32_t)a.max_rank * 2;  // of a row of B
  const uint32_t lane_b = (uint32_t)lane_o * b_bytes + 16 * q;
  auto fetch_y = [&](int32_t ob, int stage) {
    if (ob < blocks) {
      uint32_t at = slot + stage * y_step;
      if (has_y) {
        const bool in0 = ob * 32 + lc * q < a.out_features, in1 = ob * 32 + lc * q + next < a.out_features;
        const uint32_t e = (uint32_t)ob * 32 * y_size;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (yf) {
            if (in0) ring16(sm_u32 + at, yr[h] + e);
            if (in1) ring16(sm_u32 + at + kSlotVec, yr[h] + e + 64);
            at += 2 * kSlotVec;
          } else {
            if (quads) {
              if (in0) ring8(sm_u32 + at, yr[h] + e);
              if (in1) ring8(sm_u32 + at + 8, yr[h] + e + 32);
            } else if (in0) {
              ring16(sm_u32 + at, yr[h] + e);
            }
            at += kSlotVec;
          }
        }
      }
      const char* Bo = B + (uint64_t)((uint32_t)ob * 32) * b_bytes;
      const int32_t left_o = a.out_features - ob * 32 - lane_o;
      for (int32_t k = 0; k < kwins; ++k) {
        const bool in = k * 32 + 8 * q < rank;
#pragma unroll
        for (int j = 0; j < 4; ++j, at += kSlotVec) {
          const int32_t jo = (j >> 1) * next + 2 * (j & 1);
          if (in && jo < left_o) ring16(sm_u32 + at, Bo + ((uint64_t)(uint32_t)jo * b_bytes + k * 64) + lane_b);
        }
      }
    }
    ring_commit();
  };
  auto fetch_first_y = [&] {
    for (int s = 0; s + 1 < y_stages; ++s) fetch_y(b0 + s * bstep, s);
  };

  if (rank == 0) {
    ring_wait(0);  // (what was fetched for the first product)
    fetch_first_y();
  }
  if (rank > 0) {
    for (int32_t r0 = 0; r0 < rank; r0 += RPASS) {
      nt = min(NT, (rank - r0 + 7) / 8);
      if (r0 > 0) {
        A += (uint64_t)RPASS * row_bytes;
        step = (2 + nt) * kSlotVec;
        stages = ring_stages(ring_bytes, step);
        fetch_off = pair0;
        fetch_odd = false;
        for (int s = 0; s + 1 < stages; ++s) fetch(s, step, nt);
      }
      float acc[NT][4] = {};
      int stage = 0;
      bool odd = false;
      for (uint32_t off = pair0; off < row_bytes;
           off += odd ? jump : 64, odd = !odd, stage = stage + 1 == stages ? 0 : stage + 1) {
        fetch(stage == 0 ? stages - 1 : stage - 1, step, nt);
        ring_wait(stages - 1);
        __syncwarp();
        const uint32_t at = slot + stage * step;
        const bool past = off + 16 * q >= row_bytes;
        uint4 xa[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          xa[h] = slot16(sm, at + h * kSlotVec);
          if (past) xa[h] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (j >= nt) break;
          uint4 av = slot16(sm, at + (2 + j) * kSlotVec);
          if (past) av = make_uint4(0, 0, 0, 0);
          mma_bf16(acc[j], xa[0].x, xa[1].x, xa[0].y, xa[1].y, av.x, av.y);
          mma_bf16(acc[j], xa[0].z, xa[1].z, xa[0].w, xa[1].w, av.z, av.w);
        }
      }
      // the thread's slots are free: the second product's first steps, while the sums meet
      if (r0 + RPASS >= rank) fetch_first_y();
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(part + (warp * MT + h * 8 + g) * RP + 8 * j + 2 * q) =
              make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
      __syncthreads();
      // a thread: M neighbouring ranks of a token
      constexpr int M = MT * RPASS / kLoraThreads;
      const int m = tid * M / RPASS, r = tid * M % RPASS;
      float sum[M] = {};
#pragma unroll
      for (int k = 0; k < KG; ++k)
#pragma unroll
        for (int i = 0; i < M; ++i) sum[i] += part[(k * MT + m) * RP + r + i];
      if (C > 1) {
        // Every CTA of the cluster gets all CTAs' sums, of the tokens and ranks that there are; each counts the bytes
        // that arrive (and the peers have read the last pass's).
        const int32_t ranks = min(RPASS, (rank - r0 + M - 1) / M * M);
        const bool used = m < t.count && r < ranks;
        if (tid == 0) mbar_arrive_expect_tx(&met, C * t.count * ranks * 4);
        cluster_wait();
        if (used)
          for (uint32_t k = 0; k < C; ++k) push_floats<M>(recv + (cr * MT + m) * RP + r, k, sum, &met);
        mbar_wait(&met, (uint32_t)(r0 / RPASS) & 1, &g_lora_small_flags);
#pragma unroll
        for (int i = 0; i < M; ++i) sum[i] = 0.f;
        if (used)
          for (uint32_t k = 0; k < C; ++k)
#pragma unroll
            for (int i = 0; i < M; ++i) sum[i] += recv[(k * MT + m) * RP + r + i];
      }
#pragma unroll
      for (int i = 0; i < M; ++i) {
        float s = r0 + r + i < rank ? sum[i] * t.scale : 0.f;
        if (r0 + r + i < R32)
          for (int k = 0; k < kLoraTerms; ++k) v[(k * MT + m) * VP + r0 + r + i] = (uint16_t)(take_term(s) >> 16);
      }
      if (NT == 2)  // the second half of the window of 32
        for (int k = 0; k < kLoraTerms; ++k) v[(k * MT + (tid >> 4)) * VP + 16 + (tid & 15)] = 0;
      if (C > 1 && r0 + RPASS < rank) cluster_arrive();
      __syncthreads();
    }
  }

  // out = y + B v
  int stage = 0;
  for (int32_t ob = b0; ob < blocks; ob += bstep, stage = stage + 1 == y_stages ? 0 : stage + 1) {
    fetch_y(ob + (y_stages - 1) * bstep, stage == 0 ? y_stages - 1 : stage - 1);
    ring_wait(y_stages - 1);
    __syncwarp();
    const uint32_t y_at = slot + stage * y_step;
    uint32_t at = y_at + 2 * y_vecs * kSlotVec;
    float acc[4][4] = {};
    for (int32_t k0 = 0; k0 < R32; k0 += 32) {
      uint4 bv[4];
      const int32_t left = rank - (k0 + 8 * q);
#pragma unroll
      for (int j = 0; j < 4; ++j, at += kSlotVec) {
        bv[j] = slot16(sm, at);
        if (left < 8) {  // what lies beyond the rank may hold anything
          bv[j].x &= left >= 2 ? 0xffffffffu : left == 1 ? 0xffffu : 0u;
          bv[j].y &= left >= 4 ? 0xffffffffu : left == 3 ? 0xffffu : 0u;
          bv[j].z &= left >= 6 ? 0xffffffffu : left == 5 ? 0xffffu : 0u;
          bv[j].w &= left == 7 ? 0xffffu : 0u;
        }
      }
      for (int k = 0; k < kLoraTerms; ++k) {
        const uint16_t* vr = v + (k * MT + g) * VP + k0 + 8 * q;
        const uint4 lo = *reinterpret_cast<const uint4*>(vr), hi = *reinterpret_cast<const uint4*>(vr + 8 * VP);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_bf16(acc[j], lo.x, hi.x, lo.y, hi.y, bv[j].x, bv[j].y);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_bf16(acc[j], lo.z, hi.z, lo.w, hi.w, bv[j].z, bv[j].w);
      }
    }
    const int32_t c = ob * 32 + lc * q;
    const bool in0 = c < a.out_features, in1 = c + next < a.out_features;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (tok[h] < 0 || !in0) continue;
      float r[8] = {};
      if (has_y) {
        const uint32_t ya = y_at + h * y_vecs * kSlotVec;
        const uint4 d = slot16(sm, ya);
        if (yf) {
          const uint4 e = slot16(sm, ya + kSlotVec);
          r[0] = __uint_as_float(d.x);
          r[1] = __uint_as_float(d.y);
          r[2] = __uint_as_float(d.z);
          r[3] = __uint_as_float(d.w);
          r[4] = __uint_as_float(e.x);
          r[5] = __uint_as_float(e.y);
          r[6] = __uint_as_float(e.z);
          r[7] = __uint_as_float(e.w);
        } else {
          unpack8(d, r);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[2 * j] += acc[j][2 * h];
        r[2 * j + 1] += acc[j][2 * h + 1];
      }
      if (a.out_dtype == MOE_DTYPE_F32) {
        float* p = row_ptr<float>(a.out, tok[h], a.out_features) + c;
        *reinterpret_cast<float4*>(p) = make_float4(r[0], r[1], r[2], r[3]);
        if (in1) *reinterpret_cast<float4*>(p + next) = make_float4(r[4], r[5], r[6], r[7]);
      } else {
        uint16_t* p = row_ptr<uint16_t>(a.out, tok[h], a.out_features) + c;
        if (!quads) {
          store8(p, r);
        } else {
          *reinterpret_cast<uint2*>(p) = make_uint2(pack2(r[0], r[1]), pack2(r[2], r[3]));
          if (in1) *reinterpret_cast<uint2*>(p + next) = make_uint2(pack2(r[4], r[5]), pack2(r[6], r[7]));
        }
      }
    }
  }
  if (C > 1 && rank == 0) cluster_wait();  // (the arrival at the start)
}

template <int NT>
cudaError_t lora_launch(const moe_lora_args& a, int32_t tiles, int32_t cluster, cudaStream_t s) {
  constexpr int MT = 16, RP = 8 * NT + 8;
  const int32_t VP = a.max_rank <= 32 ? 32 : ((a.max_rank + 63) & ~63) + 32;
  // up to four ring steps, as many as let two CTAs share an SM if those are two or more, else as fit one
  const uint32_t y_vecs = !a.y.data ? 0 : a.y_dtype == MOE_DTYPE_F32 ? 2 : 1;
  const uint32_t step = std::max<uint32_t>(2 + NT, 4 * ((a.max_rank + 31) / 32) + 2 * y_vecs) * kSlotVec;
  const uint32_t rest = (kLoraWarps + (cluster > 1 ? cluster : 0)) * MT * RP * 4 + kLoraTerms * MT * VP * 2;
  const uint32_t room = (rest + 2 * step <= 112 * 1024 ? 112 * 1024 : 220 * 1024) - rest;
  const uint32_t ring = std::min(4u, room / step) * step;
  static std::atomic<bool> configured[kMaxDevices];
  cudaError_t e = raise_smem_limit(lora_kernel<NT>, 220 * 1024, configured);
  if (e != cudaSuccess) return e;
  return lora_launch_cluster(lora_kernel<NT>, tiles, cluster, kLoraThreads, ring + rest, false, s, a, ring);
}

}  // namespace

cudaError_t lora_small_flags(int32_t* flags) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_lora_small_flags, sizeof(int32_t));
  const int32_t zero = 0;
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_lora_small_flags, &zero, sizeof(int32_t));
  return e;
}

size_t lora_workspace(int32_t n, int32_t n_adapters) {
  const int64_t L = n_adapters;
  if (n <= kSmallTokensWide) return 0;
  const int64_t slices = plan_slices(n);
  return (size_t)(up4(n) + 2 * up4(L + 2) + (slices > 1 ? slices * (L + 1) : 0)) * 4;
}

cudaError_t launch_lora(const moe_lora_args& a, void* workspace, cudaStream_t s) {
  const int32_t n = a.n, L = a.n_adapters;
  const bool small = n <= small_tokens(a.max_rank), mma = !small && lora_mma_takes(a);
  const int32_t mt = mma ? kMmaTokens : small ? 16 : kRowsTile;
  const LoraPlan p = small ? LoraPlan{} : lora_plan(workspace, n, L);
  if (!small) {
    const int32_t slices = plan_slices(n);
    const size_t smem = (size_t)(L + 1) * 4;
    if (slices > 1) {
      lora_hist_kernel<<<slices, kPlanThreads, smem, s>>>(a.adapter_ids, n, L, p.hist);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    lora_plan_kernel<<<slices, kPlanThreads, smem, s>>>(a.adapter_ids, n, L, mt, p, slices > 1 ? p.hist : nullptr);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  // Every group has at most one tile that is not full; an adapter has half of one on average, and three quarters are
  // allowed for (a tile too many for the clusters that fit at once waits for the first to finish).
  const int32_t tiles = n / mt + std::min(n, L + 1), expected = n / mt + (3 * std::min(n, L) + 3) / 4;
  if (mma) return launch_lora_mma(a, p, tiles, expected, s);
  if (!small) return launch_lora_rows(a, p, tiles, expected, s);
  // Up to 400 CTAs, of which two share an SM (`tiles` is a bound, so some have nothing to do).  With 608 a call of 768
  // tokens takes 20 us instead of 15, with 304 one of 1024 18 instead of 15.5; clusters of 4 or 2 for a single token
  // take 1.1 and 3.6 us more.
  int32_t cluster = 1;
  while (cluster < 8 && tiles * cluster * 2 <= 400) cluster *= 2;
  if (a.max_rank <= 16) return lora_launch<2>(a, tiles, cluster, s);
  if (a.max_rank <= 32) return lora_launch<4>(a, tiles, cluster, s);
  return lora_launch<8>(a, tiles, cluster, s);
}

}  // namespace moe
