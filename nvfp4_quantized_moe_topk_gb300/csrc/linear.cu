// linear.cu -- the projections: a matrix product with bias, activation and
// residual in its epilogue (linear_mma.cu), and its backward pass.
//
// Backward: dz = d_out * act'(z), then d_x = dz W and d_weight = dz^T x by the same
// products, their operands read as they lie in memory (no transposed copies).
// Few tokens go other ways: forward linear_rows.cu, d_weight linear_outer.cu.
// Where dz is not d_out itself it goes through the workspace as a sum of bf16 terms: two
// for a gradient in bf16, within 2^-16 of each dz, which leaves in a sum of thousands of
// products what the tensor core's own cutting does (linear_mma.cu); three for a gradient
// in fp32, which keep dz's 24 bits.  (One term for a gradient in bf16, 2^-8 of each dz,
// halves the products' time, but a gradient's distance from 64 bits is 1.41 times that of
// rounding it alone, and small gradients among large ones are lost.)  d_bias comes from
// dz in 32 bits, in the pass that makes it.
#include <algorithm>

#include "block.cuh"
#include "linear_act.cuh"
#include "linear_mma.cuh"

namespace moe {

namespace {

constexpr int kDzThreads = 256;
constexpr int kDzMostChunks = 304, kDzOneChunk = 96;

struct DzParams {
  int32_t n, out, act, chunks;
  int32_t lanes;  // of 8 columns each, side by side in a CTA; the other threads take other rows
  moe_rows d_out, z;
  uint16_t* terms;    // [kLinearTerms][n][out] or NULL
  int32_t n_terms;    // none, two or three
  float* part;        // [chunks][out] or NULL
  int32_t beside;     // 1: launched after products whose results it does not take (LinearProduct::beside)
};

// 8 values of a row as they lie in memory.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> raw8(const moe_rows& r, int64_t t, int32_t cols, int32_t at) {
  const uint4* p = reinterpret_cast<const uint4*>(row_ptr<const T>(r, t, cols) + at);
  Raw8<T> o;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) o.v[i] = __ldg(p + i);
  return o;
}
__device__ __forceinline__ void values8(const Raw8<uint16_t>& r, float (&v)[8]) { unpack8(r.v[0], v); }
__device__ __forceinline__ void values8(const Raw8<float>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[4 * i] = __uint_as_float(r.v[i].x);
    v[4 * i + 1] = __uint_as_float(r.v[i].y);
    v[4 * i + 2] = __uint_as_float(r.v[i].z);
    v[4 * i + 3] = __uint_as_float(r.v[i].w);
  }
}

// The next bf16 term of 8 values, taken off them, rounded to nearest, cut to `most`: the first to bf16's range, so that a
// large finite value has finite terms.  (An infinity's second term is infinite; nothing is left of it then, or of a NaN,
// where a subtraction gives NaN.)
constexpr float kMostBf16 = 0x1.fep127f;
__device__ __forceinline__ float within(float v, float most) {
  asm("{\n .reg .f32 t;\n min.NaN.f32 t, %0, %1;\n neg.f32 %0, %1;\n max.NaN.f32 %0, t, %0;\n}\n" : "+f"(v) : "f"(most));
  return v;
}
__device__ __forceinline__ uint4 take_rounded(float (&v)[8], float most) {
  uint32_t t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float &a = v[2 * i], &b = v[2 * i + 1];
    t[i] = pack2(within(a, most), within(b, most));
    a -= bf16lo(t[i]);
    b -= bf16hi(t[i]);
    a = a == a ? a : 0.f;
    b = b == b ? b : 0.f;
  }
  return make_uint4(t[0], t[1], t[2], t[3]);
}

// dz of 8 lanes' columns and a chunk of tokens, and its column sums.
constexpr int kDzAhead = 4;  // rows of a thread on their way at once
constexpr int kDzRun = 16;   // such turns that are added one after another, so that a sum's error does not grow with n
template <bool ACT, typename DT, typename ZT>
__global__ void __launch_bounds__(kDzThreads) linear_dz_kernel(const DzParams a) {
  __shared__ float sums[8 * kDzThreads];
  const int lane = threadIdx.x % a.lanes, row = threadIdx.x / a.lanes, rows = kDzThreads / a.lanes;
  const int32_t columns = 8 * a.lanes, col = blockIdx.x * columns + 8 * lane;
  const int32_t begin = (int32_t)((int64_t)a.n * blockIdx.y / a.chunks), end = (int32_t)((int64_t)a.n * (blockIdx.y + 1) / a.chunks);
  float sum[8] = {};
  float* const total = sums + row * columns + 8 * lane;  // the thread's own until the CTA's sums meet
  bool runs = false;
  if (!a.beside) pdl_wait();
  pdl_launch_dependents();
  if (col < a.out) {
    int32_t t0 = begin + row;
    while (true) {
      const int32_t run = kDzRun * kDzAhead * rows, stop = end - t0 > run ? t0 + run : end;
      for (; t0 < stop; t0 += kDzAhead * rows) {
        Raw8<DT> rd[kDzAhead];
        Raw8<ZT> rz[kDzAhead];
#pragma unroll
        for (int k = 0; k < kDzAhead; ++k) {
          const int32_t t = min(t0 + k * rows, end - 1);
          rd[k] = raw8<DT>(a.d_out, t, a.out, col);
          if (ACT) rz[k] = raw8<ZT>(a.z, t, a.out, col);
        }
#pragma unroll
        for (int k = 0; k < kDzAhead; ++k) {
          const int32_t t = t0 + k * rows;
          if (t >= end) break;
          float d[8], z[8];
          values8(rd[k], d);
          if (ACT) values8(rz[k], z);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (ACT) d[i] *= linear_slope(z[i], a.act);
            sum[i] += d[i];
          }
          uint16_t* to = a.terms + (int64_t)t * a.out + col;
          for (int m = 0; m < a.n_terms; ++m, to += (int64_t)a.n * a.out)
            *reinterpret_cast<uint4*>(to) = take_rounded(d, m == 0 ? kMostBf16 : INFINITY);
        }
      }
      if (t0 >= end) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        total[i] = sum[i] + (runs ? total[i] : 0.f);
        sum[i] = 0.f;
      }
      runs = true;
    }
  }
  if (a.part) {
#pragma unroll
    for (int i = 0; i < 8; ++i) total[i] = sum[i] + (runs ? total[i] : 0.f);
    __syncthreads();
    for (int32_t i = threadIdx.x; i < columns; i += kDzThreads) {
      const int32_t c = blockIdx.x * columns + i;
      if (c >= a.out) break;
      float v = 0.f;
      for (int r = 0; r < rows; ++r) v += sums[r * columns + i];
      a.part[(int64_t)blockIdx.y * a.out + c] = v;
    }
  }
  if (a.beside) pdl_wait();
}

// d_bias: the chunks' sums, 32 columns a CTA.
__global__ void __launch_bounds__(kJoinThreads)
    linear_bias_kernel(const float* __restrict__ part, int32_t chunks, int32_t out, float* __restrict__ d_bias,
                       int32_t beside) {
  __shared__ float sum[kJoinWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t c = blockIdx.x * 32 + lane, mine = blockIdx.x * 32 + warp;
  if (!beside) pdl_wait();
  pdl_launch_dependents();
  sum[warp][lane] = join_part<2>(part, 0, chunks - 1, out, c, c < out);
  __syncthreads();
  const float v = join_parts(sum);
  if (lane == 0 && mine < out) d_bias[mine] = v;
  if (beside) pdl_wait();
}

int64_t stride_of(const moe_rows& r, int64_t cols) { return r.stride ? r.stride : cols; }
size_t term_bytes(int32_t n, int32_t out) { return (size_t)n * (size_t)out * 2; }

}  // namespace

size_t linear_workspace(int32_t n, int32_t in, int32_t out) {
  (void)in;
  return kLinearTerms * term_bytes(n, out) + (size_t)kDzMostChunks * (size_t)out * sizeof(float);
}

cudaError_t launch_linear(const moe_linear_args& a, cudaStream_t s, int32_t* flags) {
  LinearProduct p = {};
  p.flags = flags;
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
  // Few tokens: up to 16, and up to 64 where the features' CTAs leave half the SMs free (64 tokens of 2688 to 128: 6.3 us,
  // by launch_linear_mma 7.2; 24 of 4096 to 4096 13.4 / 11.6); not where rows are so short and many that a CTA's start
  // counts (16 tokens of 512 to 16384: 8.9 / 7.1; of 2688 to 4608 7.0 / 10.3, one 6.1 / 9.9).
  const bool few = a.n <= 16 ? a.out_features <= 16 * (int64_t)a.in_features : a.n <= 64 && a.out_features <= 16 * 76;
  return few ? launch_linear_rows(p, s) : launch_linear_mma(p, s);
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
  const int terms_x = same ? 1 : d.d_x_dtype == MOE_DTYPE_F32 ? kLinearTerms : 2;
  const int terms_w = same ? 1 : d.d_weight_dtype == MOE_DTYPE_F32 ? kLinearTerms : 2;
  uint16_t* terms = static_cast<uint16_t*>(workspace);
  const size_t term = (size_t)a.n * a.out_features;
  float* part = reinterpret_cast<float*>(terms + kLinearTerms * term);
  DzParams z = {};
  // A chunk of tokens a CTA, four CTAs an SM (16384 tokens of 8192: 42 us, with two 58, with eight 44); few tokens in one
  // chunk, whose sums are d_bias, and narrower CTAs.
  z.lanes = a.n <= kDzOneChunk ? 8 : 32;
  const int32_t strips = (a.out_features + 8 * z.lanes - 1) / (8 * z.lanes);
  z.chunks = a.n <= kDzOneChunk ? 1 : std::max(1, std::min({kDzMostChunks, (a.n + 15) / 16, 608 / strips}));
  auto make_dz = [&](bool beside) {
    z.n = a.n;
    z.out = a.out_features;
    z.act = a.activation;
    z.d_out = d.d_out;
    z.z = a.z;
    z.terms = terms;
    z.n_terms = same ? 0 : std::max(d.d_x.data ? terms_x : 0, d.d_weight ? terms_w : 0);
    z.beside = beside;
    if (d.d_bias) z.part = z.chunks == 1 ? d.d_bias : part;
    const bool d32 = d.d_out_dtype == MOE_DTYPE_F32, z32 = a.z_dtype == MOE_DTYPE_F32, act = a.activation != MOE_LINEAR_NONE;
    auto kernel = !act  ? (d32 ? linear_dz_kernel<false, float, float> : linear_dz_kernel<false, uint16_t, float>)
                  : z32 ? (d32 ? linear_dz_kernel<true, float, float> : linear_dz_kernel<true, uint16_t, float>)
                        : (d32 ? linear_dz_kernel<true, float, uint16_t> : linear_dz_kernel<true, uint16_t, uint16_t>);
    return launch_ex(kernel, dim3(strips, z.chunks), dim3(kDzThreads), 0, s, true, z);
  };
  auto join_bias = [&](bool beside) {
    if (!d.d_bias || z.chunks == 1) return cudaSuccess;
    return launch_ex(linear_bias_kernel, dim3((a.out_features + 31) / 32), dim3(kJoinThreads), 0, s, true, (const float*)part,
                     z.chunks, a.out_features, d.d_bias, (int32_t)beside);
  };
  if (!same && products) e = make_dz(false);
  if (e != cudaSuccess) return e;
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
    p.share = 2;  // (whichever outputs are asked for, so that their bits do not depend on it)
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
    p.beside = d.d_x.data != nullptr;
    p.share = 2;
    p.finish.out = d.d_weight;
    p.finish.out_stride = a.in_features;
    p.finish.out_f32 = d.d_weight_dtype == MOE_DTYPE_F32;
    // Few tokens, and more where the result is small (a backward pass in bf16 of one token, 2688 to 4608: 16.5 us, by
    // launch_linear_mma 20.2; of 33 20.2 / 20.5, of 64 22.0 / 21.0; 128 of 1000 to 520 6.3 / 7.0, of 3984 to 136 9.0 / 9.3).
    const bool outer = a.n <= 48 || (a.n <= kLinearOuterTokens && (int64_t)a.in_features * a.out_features <= 1 << 20);
    e = outer ? launch_linear_outer(p, s) : launch_linear_mma(p, s);
    if (e != cudaSuccess) return e;
  }
  // d_bias last, beside the products: their first one waited for dz where they take it, and for the caller's tensors
  // (55 tokens of 7992 to 2408: it adds 0.1 us to 28.6, before the products 1.7; 3631 of 784 to 240: 2.7, before 3.2).
  if (same || !products) {
    if (d.d_bias) e = make_dz(products);
    if (e == cudaSuccess) e = join_bias(false);
  } else {
    e = join_bias(true);
  }
  return e;
}

cudaError_t linear_device_flags(int32_t* flags) {
  const cudaError_t e = cudaDeviceSynchronize();
  return e == cudaSuccess ? linear_mma_flags(flags) : e;
}

}  // namespace moe
