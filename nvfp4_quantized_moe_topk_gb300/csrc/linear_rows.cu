// linear_rows.cu -- the projection of a few tokens: the weights stream through
// registers once.
//
// Reading the weights bounds it, and before that the way from launch to the first
// byte and from the last to the result, which the tensor memory's set-up, its
// barriers and a cluster's meeting make long.  Here a CTA takes 16 features, its
// warps an eighth of the columns each, all of a batch's loads in flight before
// the first product; warp-level matrix instructions take 16 features by 8
// tokens, and the warps' sums meet once in shared memory, in order.  One token of
// 2688 to 4608 (25 MB of weights, not in L2): 5.5 us, 4.5 TB/s; with weights in L2 3.6.
//
// A lane's 16 bytes of a row are 8 consecutive columns; which of them an
// instruction pairs with which only has to be the same for weights and x, so
// both sides take them as they lie.
#include <algorithm>

#include "block.cuh"
#include "linear_act.cuh"
#include "linear_mma.cuh"
#include "tile.cuh"

namespace moe {

namespace {

constexpr int kRowsThreads = 256, kRowsWarps = kRowsThreads / 32, kRowsFeatures = 16;
constexpr int kBatch = 6;  // steps of 32 columns in flight
// Batches that an instruction's sums run through before they move on: the tensor cores cut what they add to a sum where it
// would round, always towards zero (linear_mma.cu).  Shorter rows do without (16 tokens of 4096 to 4096: 7.7 us, with a
// second set of sums 8.1; of 16384 columns, which need it, 20.7 and 21.2).
constexpr int kChainBatches = 3, kChainColumns = kChainBatches * kBatch * 32 * kRowsWarps;

struct RowsPlan {
  int32_t n, in, out;
  const uint16_t *w, *x;
  int64_t x_stride;
  LinearFinish e;
};

__device__ __forceinline__ uint4 stream16(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// TILES: tiles of 8 tokens.  CHAIN: rows of more than kChainColumns.
template <int TILES, bool CHAIN>
__global__ void __launch_bounds__(kRowsThreads, TILES <= 2 ? 2 : 1) linear_rows_kernel(const __grid_constant__ RowsPlan p) {
  __shared__ float sums[kRowsWarps][8 * TILES][kRowsFeatures + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int32_t f0 = blockIdx.x * kRowsFeatures;
  const int32_t steps = (p.in + 31) / 32, s0 = steps * warp / kRowsWarps, s1 = steps * (warp + 1) / kRowsWarps;
  const uint16_t* wa = p.w + (int64_t)min(f0 + g, p.out - 1) * p.in + 8 * t;  // (rows past the last: not written)
  const uint16_t* wb = p.w + (int64_t)min(f0 + g + 8, p.out - 1) * p.in + 8 * t;
  const uint16_t* xr[TILES];
#pragma unroll
  for (int i = 0; i < TILES; ++i) xr[i] = p.x + (int64_t)min(8 * i + g, p.n - 1) * p.x_stride + 8 * t;
  float acc[TILES][4] = {}, total[TILES][4] = {};
  pdl_wait();
  pdl_launch_dependents();
  int chained = 0;
  for (int32_t s = s0; s < s1; s += kBatch) {
    uint4 a[kBatch], b[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      a[i] = b[i] = make_uint4(0, 0, 0, 0);
      if (s + i < s1 && 32 * (s + i) + 8 * t < p.in) {
        a[i] = stream16(wa + 32 * (s + i));
        b[i] = stream16(wb + 32 * (s + i));
      }
    }
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
      uint4 x[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        x[i] = make_uint4(0, 0, 0, 0);
        if (s + i < s1 && 32 * (s + i) + 8 * t < p.in && 8 * j + g < p.n)
          x[i] = __ldg(reinterpret_cast<const uint4*>(xr[j] + 32 * (s + i)));
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        mma_bf16_16816(acc[j], a[i].x, b[i].x, a[i].y, b[i].y, x[i].x, x[i].y);
        mma_bf16_16816(acc[j], a[i].z, b[i].z, a[i].w, b[i].w, x[i].z, x[i].w);
      }
    }
    if (CHAIN && ++chained == kChainBatches) {
      chained = 0;
#pragma unroll
      for (int j = 0; j < TILES; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          total[j][i] += acc[j][i];
          acc[j][i] = 0.f;
        }
    }
  }
  if (CHAIN) {
#pragma unroll
    for (int j = 0; j < TILES; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] += total[j][i];
  }
#pragma unroll
  for (int j = 0; j < TILES; ++j) {
    sums[warp][8 * j + 2 * t][g] = acc[j][0];
    sums[warp][8 * j + 2 * t + 1][g] = acc[j][1];
    sums[warp][8 * j + 2 * t][g + 8] = acc[j][2];
    sums[warp][8 * j + 2 * t + 1][g + 8] = acc[j][3];
  }
  __syncthreads();
  const LinearFinish& e = p.e;
  for (int32_t i = threadIdx.x; i < p.n * kRowsFeatures; i += kRowsThreads) {
    const int32_t r = i / kRowsFeatures, f = f0 + i % kRowsFeatures;
    if (f >= p.out) continue;
    float z = 0.f;
#pragma unroll
    for (int k = 0; k < kRowsWarps; ++k) z += sums[k][r][i % kRowsFeatures];
    if (e.bias) z += linear_read(e.bias, f, e.bias_f32);
    if (e.z) linear_write(e.z, r * e.z_stride + f, e.z_f32, z);
    float v = linear_act(z, e.act);
    if (e.residual) v = fmaf(e.scale, linear_read(e.residual, r * e.residual_stride + f, e.residual_f32), v);
    linear_write(e.out, r * e.out_stride + f, e.out_f32, v);
  }
}

}  // namespace

cudaError_t launch_linear_rows(const LinearProduct& a, cudaStream_t s) {
  const RowsPlan p = {a.R, a.C, a.F, static_cast<const uint16_t*>(a.p.data), static_cast<const uint16_t*>(a.q[0].data),
                      a.q[0].stride, a.finish};
  const dim3 grid((unsigned)((a.F + kRowsFeatures - 1) / kRowsFeatures)), block(kRowsThreads);
  const bool chain = a.C > kChainColumns;
  auto kernel = a.R <= 8    ? (chain ? linear_rows_kernel<1, true> : linear_rows_kernel<1, false>)
                : a.R <= 16 ? (chain ? linear_rows_kernel<2, true> : linear_rows_kernel<2, false>)
                : a.R <= 32 ? (chain ? linear_rows_kernel<4, true> : linear_rows_kernel<4, false>)
                            : (chain ? linear_rows_kernel<8, true> : linear_rows_kernel<8, false>);
  return launch_ex(kernel, grid, block, 0, s, true, p);
}

}  // namespace moe
