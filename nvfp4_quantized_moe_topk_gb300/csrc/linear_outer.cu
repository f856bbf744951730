// linear_outer.cu -- d_weight of a few tokens: a sum of few outer products.
//
//   d_weight[o][i] = sum over t of dz[t][o] x[t][i]
//
// Writing the result bounds it, so a CTA takes 64 rows by 128 columns of it, brings
// the tokens' parts of dz and x to shared memory once, and multiplies by warp-level
// matrix instructions whose operands turn on their way to registers.  Its start is
// short, where linear_mma.cu's tensor memory, barriers and descriptors take longer
// than the tokens' products.  A lane's sums of two instructions meet its neighbour's,
// so that it writes four values side by side and a row gets whole sectors.  One token
// of 2688 to 4608 in fp32 (50 MB): the backward pass 23.1 -> 17.8 us, half of it d_x.
#include <algorithm>

#include "block.cuh"
#include "linear_mma.cuh"
#include "tile.cuh"

namespace moe {

namespace {

constexpr int kOuterThreads = 256, kOuterRows = 64, kOuterCols = 128;
constexpr uint32_t kXRow = 2 * kOuterCols + 16, kDzRow = 2 * kOuterRows + 16;  // padded: 8 rows off each other's banks

struct OuterPlan {
  int32_t n, terms, steps;  // steps of 16 tokens
  int32_t R, F, tiles_f;
  const uint16_t *x, *dz[kLinearTerms];
  int64_t x_stride, dz_stride;
  void* out;
  int64_t out_stride;
  int32_t out_f32, beside;
};

__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void turned4(uint32_t (&v)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(at)
               : "memory");
}

// A matrix of tokens by `cols` columns from column c0 on, 8 of them a copy; zeros beyond the tokens and the last column.
__device__ __forceinline__ void fetch(uint32_t to, uint32_t row, const uint16_t* from, int64_t stride, int32_t n,
                                      int32_t tokens, int32_t c0, int32_t cols, int32_t all) {
  const int32_t chunks = cols / 8;
  for (int32_t i = threadIdx.x; i < tokens * chunks; i += kOuterThreads) {
    const int32_t t = i / chunks, c = 8 * (i - t * chunks);
    const bool live = t < n && c0 + c < all;
    copy16(to + t * row + 2 * c, live ? from + t * stride + c0 + c : from, live);
  }
}

__global__ void __launch_bounds__(kOuterThreads, 3) linear_outer_kernel(const __grid_constant__ OuterPlan p) {
  extern __shared__ __align__(16) uint8_t sm[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int32_t o0 = (int32_t)(blockIdx.x / p.tiles_f) * kOuterRows, i0 = (int32_t)(blockIdx.x % p.tiles_f) * kOuterCols;
  const int32_t tokens = 16 * p.steps;
  const uint32_t xs = smem_u32(sm), ds = xs + tokens * kXRow;
  if (!p.beside) pdl_wait();
  pdl_launch_dependents();
  fetch(xs, kXRow, p.x, p.x_stride, p.n, tokens, i0, kOuterCols, p.F);
  for (int32_t m = 0; m < p.terms; ++m)
    fetch(ds + m * tokens * kDzRow, kDzRow, p.dz[m], p.dz_stride, p.n, tokens, o0, kOuterRows, p.R);
  asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  // a warp: 16 rows and 64 columns
  const int32_t wo = 16 * (warp & 3), wi = 64 * (warp >> 2);
  const uint32_t ta = (lane >> 4) * 8 + (lane & 7), ca = wo + ((lane >> 3) & 1) * 8;
  const uint32_t tb = ((lane >> 3) & 1) * 8 + (lane & 7), cb = wi + (lane >> 4) * 8;
  float acc[8][4] = {};
  for (int32_t s = 0; s < p.steps; ++s) {
    uint32_t b[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) turned4(b[j], xs + (16 * s + tb) * kXRow + 2 * (cb + 16 * j));
    for (int32_t m = 0; m < p.terms; ++m) {
      uint32_t a[4];
      turned4(a, ds + (m * tokens + 16 * s + ta) * kDzRow + 2 * ca);
#pragma unroll
      for (int j = 0; j < 8; ++j) mma_bf16_16816(acc[j], a[0], a[1], a[2], a[3], b[j / 2][2 * (j & 1)], b[j / 2][2 * (j & 1) + 1]);
    }
  }
  const bool odd = q & 1;
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const int32_t i = i0 + wi + 8 * (j + odd) + 4 * (q >> 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int32_t o = o0 + wo + g + 8 * h;
      float v[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float lo = acc[j][2 * h + k], hi = acc[j + 1][2 * h + k];
        const float got = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1);
        v[k] = odd ? got : lo;
        v[2 + k] = odd ? hi : got;
      }
      if (o >= p.R || i >= p.F) continue;
      const int64_t at = o * p.out_stride + i;
      if (p.out_f32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
    }
  }
  if (p.beside) pdl_wait();
}

}  // namespace

cudaError_t launch_linear_outer(const LinearProduct& a, cudaStream_t s) {
  static std::atomic<bool> configured[kMaxDevices];
  constexpr int32_t kMost = (kLinearOuterTokens + 15) / 16 * 16;
  const cudaError_t e = raise_smem_limit(linear_outer_kernel, (int)(kMost * (kXRow + kLinearTerms * kDzRow)), configured);
  if (e != cudaSuccess) return e;
  OuterPlan p = {};
  p.n = a.C;
  p.terms = a.terms;
  p.steps = (a.C + 15) / 16;
  p.R = a.R;
  p.F = a.F;
  p.tiles_f = (a.F + kOuterCols - 1) / kOuterCols;
  p.x = static_cast<const uint16_t*>(a.p.data);
  p.x_stride = a.p.stride;
  for (int i = 0; i < a.terms; ++i) p.dz[i] = static_cast<const uint16_t*>(a.q[i].data);
  p.dz_stride = a.q[0].stride;
  p.out = a.finish.out;
  p.out_stride = a.finish.out_stride;
  p.out_f32 = a.finish.out_f32;
  p.beside = a.beside;
  const int64_t tiles = (int64_t)p.tiles_f * ((a.R + kOuterRows - 1) / kOuterRows);
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  const size_t smem = (size_t)16 * p.steps * (kXRow + p.terms * kDzRow);
  return launch_ex(linear_outer_kernel, dim3((unsigned)tiles), dim3(kOuterThreads), smem, s, true, p);
}

}  // namespace moe
