// linear.cu -- the projections: a matrix product with bias, activation and
// residual in its epilogue (linear_mma.cu), and its backward pass.
//
// Backward: dz = d_out * act'(z), then d_x = dz W and d_weight = dz^T x by the same
// products, their operands read as they lie in memory (no transposed copies).
// Where dz is not d_out itself it goes through the workspace: as one bf16 term for a
// gradient in bf16, whose own rounding (2^-8 of a value) hides what the terms' roundings,
// of either sign, leave in the sum; as three for a gradient in fp32, which keep dz's 24 bits.
// d_bias comes from dz in 32 bits, in the pass that makes it.
#include <algorithm>

#include "block.cuh"
#include "linear_act.cuh"
#include "linear_mma.cuh"

namespace moe {

namespace {

constexpr int kDzThreads = 256, kDzLanes = 32, kDzRows = kDzThreads / kDzLanes;  // 8 columns a lane
constexpr int kDzColumns = 8 * kDzLanes;
constexpr int kDzMostChunks = 64;

struct DzParams {
  int32_t n, out, act, chunks;
  int32_t d_f32, z_f32;
  moe_rows d_out, z;
  uint16_t* terms;    // [kLinearTerms][n][out] or NULL
  int32_t n_terms;
  float* part;        // [chunks][out] or NULL
};

__device__ __forceinline__ void load_row8(const moe_rows& r, int64_t t, int32_t cols, int32_t at, int32_t f32,
                                          float (&v)[8]) {
  if (f32) {
    const float4* p = reinterpret_cast<const float4*>(row_ptr<const float>(r, t, cols) + at);
    const float4 a = p[0], b = p[1];
    v[0] = a.x;
    v[1] = a.y;
    v[2] = a.z;
    v[3] = a.w;
    v[4] = b.x;
    v[5] = b.y;
    v[6] = b.z;
    v[7] = b.w;
  } else {
    unpack8(*reinterpret_cast<const uint4*>(row_ptr<const uint16_t>(r, t, cols) + at), v);
  }
}

// dz of 256 columns and a chunk of tokens, and its column sums.
__global__ void __launch_bounds__(kDzThreads) linear_dz_kernel(const DzParams a) {
  __shared__ float sums[kDzRows][kDzColumns];
  const int lane = threadIdx.x % kDzLanes, row = threadIdx.x / kDzLanes;
  const int32_t col = blockIdx.x * kDzColumns + 8 * lane;
  const int32_t begin = (int32_t)((int64_t)a.n * blockIdx.y / a.chunks), end = (int32_t)((int64_t)a.n * (blockIdx.y + 1) / a.chunks);
  float sum[8] = {};
  if (col < a.out) {
    for (int32_t t = begin + row; t < end; t += kDzRows) {
      float d[8];
      load_row8(a.d_out, t, a.out, col, a.d_f32, d);
      if (a.act != MOE_LINEAR_NONE) {
        float z[8];
        load_row8(a.z, t, a.out, col, a.z_f32, z);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] *= linear_slope(z[i], a.act);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += d[i];
      for (int k = 0; k < a.n_terms; ++k) {
        store8(a.terms + ((int64_t)k * a.n + t) * a.out + col, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float h = __bfloat162float(__float2bfloat16_rn(d[i]));
          d[i] = isfinite(h) ? d[i] - h : 0.f;  // (an infinity stays one)
        }
      }
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[row][8 * lane + i] = sum[i];
  __syncthreads();
  const int32_t c = blockIdx.x * kDzColumns + threadIdx.x;
  if (c >= a.out) return;
  float v = 0.f;
#pragma unroll
  for (int r = 0; r < kDzRows; ++r) v += sums[r][threadIdx.x];
  a.part[(int64_t)blockIdx.y * a.out + c] = v;
}

__global__ void __launch_bounds__(kDzThreads)
    linear_bias_kernel(const float* __restrict__ part, int32_t chunks, int32_t out, float* __restrict__ d_bias) {
  const int32_t c = blockIdx.x * kDzThreads + threadIdx.x;
  if (c >= out) return;
  float v = 0.f;
  for (int32_t k = 0; k < chunks; ++k) v += part[(int64_t)k * out + c];
  d_bias[c] = v;
}

int64_t stride_of(const moe_rows& r, int64_t cols) { return r.stride ? r.stride : cols; }
size_t term_bytes(int32_t n, int32_t out) { return (size_t)n * (size_t)out * 2; }

}  // namespace

size_t linear_workspace(int32_t n, int32_t in, int32_t out) {
  (void)in;
  return kLinearTerms * term_bytes(n, out) + (size_t)kDzMostChunks * (size_t)out * sizeof(float);
}

cudaError_t launch_linear(const moe_linear_args& a, cudaStream_t s) {
  LinearProduct p = {};
  p.R = a.n;
  p.F = a.out_features;
  p.C = a.in_features;
  p.p = {a.weight, a.in_features, true};
  p.terms = 1;
  p.q[0] = {a.x.data, stride_of(a.x, a.in_features), true};
  LinearFinish& e = p.finish;
  e.out = a.out.data;
  e.out_stride = stride_of(a.out, a.out_features);
  e.out_f32 = a.out_dtype == MOE_DTYPE_F32;
  e.z = a.z.data;
  e.z_stride = stride_of(a.z, a.out_features);
  e.z_f32 = a.z_dtype == MOE_DTYPE_F32;
  e.residual = a.residual.data;
  e.residual_stride = stride_of(a.residual, a.out_features);
  e.residual_f32 = a.residual_dtype == MOE_DTYPE_F32;
  e.bias = a.bias;
  e.bias_f32 = a.bias_dtype == MOE_DTYPE_F32;
  e.act = a.activation;
  e.scale = a.residual_scale;
  return launch_linear_mma(p, s);
}

cudaError_t launch_linear_backward(const moe_linear_args& a, const moe_linear_grads& d, void* workspace, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (a.n == 0) {
    if (d.d_weight)
      e = cudaMemsetAsync(d.d_weight, 0, (size_t)a.in_features * a.out_features * (d.d_weight_dtype == MOE_DTYPE_F32 ? 4 : 2), s);
    if (e == cudaSuccess && d.d_bias) e = cudaMemsetAsync(d.d_bias, 0, (size_t)a.out_features * 4, s);
    return e;
  }
  const bool same = a.activation == MOE_LINEAR_NONE && d.d_out_dtype == MOE_DTYPE_BF16;  // dz is d_out
  const bool products = d.d_x.data || d.d_weight;
  const int terms_x = !same && d.d_x_dtype == MOE_DTYPE_F32 ? kLinearTerms : 1;
  const int terms_w = !same && d.d_weight_dtype == MOE_DTYPE_F32 ? kLinearTerms : 1;
  uint16_t* terms = static_cast<uint16_t*>(workspace);
  const size_t term = (size_t)a.n * a.out_features;
  float* part = reinterpret_cast<float*>(terms + kLinearTerms * term);
  if ((!same && products) || d.d_bias) {
    DzParams z = {};
    z.n = a.n;
    z.out = a.out_features;
    z.act = a.activation;
    z.d_f32 = d.d_out_dtype == MOE_DTYPE_F32;
    z.z_f32 = a.z_dtype == MOE_DTYPE_F32;
    z.d_out = d.d_out;
    z.z = a.z;
    z.terms = terms;
    z.n_terms = same ? 0 : std::max(d.d_x.data ? terms_x : 0, d.d_weight ? terms_w : 0);
    if (d.d_bias) z.part = part;
    const int32_t strips = (a.out_features + kDzColumns - 1) / kDzColumns;
    z.chunks = std::max(1, std::min({kDzMostChunks, (a.n + 31) / 32, 1216 / strips}));
    linear_dz_kernel<<<dim3(strips, z.chunks), kDzThreads, 0, s>>>(z);
    e = cudaGetLastError();
    if (e == cudaSuccess && d.d_bias) {
      linear_bias_kernel<<<(a.out_features + kDzThreads - 1) / kDzThreads, kDzThreads, 0, s>>>(part, z.chunks,
                                                                                               a.out_features, d.d_bias);
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
  }
  auto operands = [&](LinearProduct& p, int count, bool c_inner) {
    p.terms = count;
    for (int i = 0; i < count; ++i)
      p.q[i] = same ? LinearOperand{d.d_out.data, stride_of(d.d_out, a.out_features), c_inner}
                    : LinearOperand{terms + i * term, a.out_features, c_inner};
  };
  if (d.d_x.data) {  // d_x[t][i] = sum over o of W[o][i] dz[t][o]
    LinearProduct p = {};
    p.R = a.n;
    p.F = a.in_features;
    p.C = a.out_features;
    p.p = {a.weight, a.in_features, false};
    operands(p, terms_x, true);
    p.finish.out = d.d_x.data;
    p.finish.out_stride = stride_of(d.d_x, a.in_features);
    p.finish.out_f32 = d.d_x_dtype == MOE_DTYPE_F32;
    e = launch_linear_mma(p, s);
    if (e != cudaSuccess) return e;
  }
  if (d.d_weight) {  // d_weight[o][i] = sum over t of x[t][i] dz[t][o]
    LinearProduct p = {};
    p.R = a.out_features;
    p.F = a.in_features;
    p.C = a.n;
    p.p = {a.x.data, stride_of(a.x, a.in_features), false};
    operands(p, terms_w, false);
    p.finish.out = d.d_weight;
    p.finish.out_stride = a.in_features;
    p.finish.out_f32 = d.d_weight_dtype == MOE_DTYPE_F32;
    e = launch_linear_mma(p, s);
  }
  return e;
}

cudaError_t linear_device_flags(int32_t* flags) {
  const cudaError_t e = cudaDeviceSynchronize();
  return e == cudaSuccess ? linear_mma_flags(flags) : e;
}

}  // namespace moe
