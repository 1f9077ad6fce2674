// Layer norm over the last axis, forward and backward.
//   forward   mean = sum x / k, var = sum (x - mean)^2 / k, rstd = 1 / sqrt(var + eps),
//             y = (x - mean) rstd gamma + beta
//   backward  xh = (x - mean) rstd, a = dy gamma,
//             dx = rstd (a - sum a / k - xh sum(a xh) / k) [+ d_residual],
//             dgamma = sum over rows of dy xh, dbeta = sum over rows of dy
// All sums, means and products are fp32; each output is rounded once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "epilogue.cuh"
#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int LN_THREADS = 256;

// Sum of (a, b) over the block, the same on every thread.
__device__ __forceinline__ float2 block_sum2(float a, float b, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
  }
  __syncthreads();                       // the previous use of red is read
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  a = b = 0.0f;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
    a += red[w].x;
    b += red[w].y;
  }
  return make_float2(a, b);
}

__device__ __forceinline__ void publish_mag(uint32_t m, float* amax_dev) {
  if (!amax_dev) return;
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) atomicMax(reinterpret_cast<unsigned int*>(amax_dev), m);
}

struct LnParams {
  const void* x;
  int64_t ldx;
  const void* gamma;
  const void* beta;
  int param_f32;
  float eps;
  void* y;
  int64_t ldy;
  int y_f32;
  float* mean;
  float* rstd;
  float* amax;
  int64_t rows;
  int k;
};

// Rows of any length: one block per row at a time, three passes over the row
// (L2 holds it after the first).
template <typename TX>
__global__ void __launch_bounds__(LN_THREADS) ln_forward_long_kernel(const LnParams p) {
  __shared__ float2 red[LN_THREADS / 32];
  const float inv_k = 1.0f / static_cast<float>(p.k);
  uint32_t mag = 0;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const TX* x = static_cast<const TX*>(p.x) + r * p.ldx;
    float s = 0.0f;
    for (int i = threadIdx.x; i < p.k; i += LN_THREADS) s += to_f32(x[i]);
    const float mean = block_sum2(s, 0.0f, red).x * inv_k;
    s = 0.0f;
    for (int i = threadIdx.x; i < p.k; i += LN_THREADS) {
      const float d = to_f32(x[i]) - mean;
      s = fmaf(d, d, s);
    }
    const float rstd = __frsqrt_rn(fmaf(block_sum2(s, 0.0f, red).x, inv_k, p.eps));
    for (int i = threadIdx.x; i < p.k; i += LN_THREADS) {
      const float g = p.gamma ? load_param(p.gamma, p.param_f32, i) : 1.0f;
      const float b = p.beta ? load_param(p.beta, p.param_f32, i) : 0.0f;
      const float v = fmaf((to_f32(x[i]) - mean) * rstd, g, b);
      if (p.y_f32) {
        static_cast<float*>(p.y)[r * p.ldy + i] = v;
        mag = max(mag, mag_bits(v));
      } else {
        const __nv_bfloat16 h = __float2bfloat16_rn(v);
        static_cast<__nv_bfloat16*>(p.y)[r * p.ldy + i] = h;
        mag = max(mag, mag_bits(h));
      }
    }
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[r] = mean;
      if (p.rstd) p.rstd[r] = rstd;
    }
  }
  publish_mag(mag, p.amax);
}

struct LnBwdParams {
  const void* dy;
  int64_t lddy;
  int dy_f32;
  const void* x;
  int64_t ldx;
  const float* mean;
  const float* rstd;
  const void* gamma;
  int param_f32;
  const void* res;       // x's type, or null
  int64_t ldr;
  void* dx;              // x's type
  int64_t lddx;
  float* partial;        // [chunks][2][k]: dgamma and dbeta of a chunk of rows
  float* amax;
  int64_t rows;
  int k;
};

__device__ __forceinline__ float load_dy(const LnBwdParams& p, int64_t r, int i) {
  return p.dy_f32 ? static_cast<const float*>(p.dy)[r * p.lddy + i]
                  : to_f32(static_cast<const __nv_bfloat16*>(p.dy)[r * p.lddy + i]);
}

// dx of rows of any length: two passes over the row.
template <typename TX>
__global__ void __launch_bounds__(LN_THREADS) ln_backward_dx_long_kernel(const LnBwdParams p) {
  __shared__ float2 red[LN_THREADS / 32];
  const float inv_k = 1.0f / static_cast<float>(p.k);
  uint32_t mag = 0;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const TX* x = static_cast<const TX*>(p.x) + r * p.ldx;
    const float mean = p.mean[r], rstd = p.rstd[r];
    float s1 = 0.0f, s2 = 0.0f;
    for (int i = threadIdx.x; i < p.k; i += LN_THREADS) {
      const float a = load_dy(p, r, i) * (p.gamma ? load_param(p.gamma, p.param_f32, i) : 1.0f);
      s1 += a;
      s2 = fmaf(a, (to_f32(x[i]) - mean) * rstd, s2);
    }
    const float2 c = block_sum2(s1, s2, red);
    const float c1 = c.x * inv_k, c2 = c.y * inv_k;
    for (int i = threadIdx.x; i < p.k; i += LN_THREADS) {
      const float a = load_dy(p, r, i) * (p.gamma ? load_param(p.gamma, p.param_f32, i) : 1.0f);
      const float xh = (to_f32(x[i]) - mean) * rstd;
      float v = rstd * (a - fmaf(xh, c2, c1));
      if (p.res) v += to_f32(static_cast<const TX*>(p.res)[r * p.ldr + i]);
      const TX o = from_f32<TX>(v);
      static_cast<TX*>(p.dx)[r * p.lddx + i] = o;
      mag = max(mag, mag_bits(o));
    }
  }
  publish_mag(mag, p.amax);
}

// dgamma and dbeta of a chunk of rows: one thread per column.
template <typename TX>
__global__ void __launch_bounds__(LN_THREADS) ln_backward_params_long_kernel(const LnBwdParams p, int rows_per_chunk) {
  const int i = blockIdx.x * LN_THREADS + threadIdx.x;
  if (i >= p.k) return;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * rows_per_chunk;
  const int64_t r1 = min(p.rows, r0 + rows_per_chunk);
  float dg = 0.0f, db = 0.0f;
  for (int64_t r = r0; r < r1; ++r) {
    const float dy = load_dy(p, r, i);
    const float xh = (to_f32(static_cast<const TX*>(p.x)[r * p.ldx + i]) - p.mean[r]) * p.rstd[r];
    dg = fmaf(dy, xh, dg);
    db += dy;
  }
  float* out = p.partial + static_cast<int64_t>(blockIdx.y) * 2 * p.k;
  out[i] = dg;
  out[p.k + i] = db;
}

// out[i] = sum over chunks of partial[c][i]; each column's sum runs over the
// chunks in order, so the result does not depend on timing.
__global__ void __launch_bounds__(LN_THREADS) sum_chunks_kernel(const float* partial, int chunks, int64_t stride, int n,
                                                                 float* out) {
  const int i = blockIdx.x * LN_THREADS + threadIdx.x;
  if (i >= n) return;
  float s = 0.0f;
  for (int c = 0; c < chunks; ++c) s += partial[c * stride + i];
  out[i] = s;
}

constexpr int LN_CHUNKS = 64;

}  // namespace

size_t layernorm_backward_workspace_bytes(int64_t rows, int64_t k) {
  return rows > 0 ? static_cast<size_t>(LN_CHUNKS) * 2 * k * sizeof(float) : 256;
}

nvfp4_status launch_layernorm(const LayerNorm& a, cudaStream_t s) {
  if (a.amax) {
    const cudaError_t e = cudaMemsetAsync(a.amax, 0, sizeof(float), s);
    if (e != cudaSuccess) return launch_status(e);
  }
  if (a.rows == 0) return NVFP4_OK;
  const LnParams p{a.x, a.ldx, a.gamma, a.beta, a.param_dtype == NVFP4_DTYPE_F32, a.eps, a.y, a.ldy,
                   a.y_dtype == NVFP4_DTYPE_F32, a.mean, a.rstd, a.amax, a.rows, static_cast<int>(a.k)};
  const int grid = static_cast<int>(a.rows < 8 * device_sm_count() ? a.rows : 8 * device_sm_count());
  if (a.x_dtype == NVFP4_DTYPE_F32)
    ln_forward_long_kernel<float><<<grid, LN_THREADS, 0, s>>>(p);
  else
    ln_forward_long_kernel<__nv_bfloat16><<<grid, LN_THREADS, 0, s>>>(p);
  return launch_status(cudaGetLastError());
}

nvfp4_status launch_layernorm_backward(const LayerNormBackward& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (a.amax) e = cudaMemsetAsync(a.amax, 0, sizeof(float), s);
  if (a.rows == 0) {
    if (e == cudaSuccess && a.dgamma) e = cudaMemsetAsync(a.dgamma, 0, a.k * sizeof(float), s);
    if (e == cudaSuccess && a.dbeta) e = cudaMemsetAsync(a.dbeta, 0, a.k * sizeof(float), s);
    return launch_status(e);
  }
  if (e != cudaSuccess) return launch_status(e);
  const LnBwdParams p{a.dy, a.lddy, a.dy_dtype == NVFP4_DTYPE_F32, a.x, a.ldx, a.mean, a.rstd, a.gamma,
                      a.param_dtype == NVFP4_DTYPE_F32, a.residual, a.ldr, a.dx, a.lddx,
                      static_cast<float*>(a.workspace), a.amax, a.rows, static_cast<int>(a.k)};
  const bool f32 = a.x_dtype == NVFP4_DTYPE_F32;
  const int grid = static_cast<int>(a.rows < 8 * device_sm_count() ? a.rows : 8 * device_sm_count());
  if (f32)
    ln_backward_dx_long_kernel<float><<<grid, LN_THREADS, 0, s>>>(p);
  else
    ln_backward_dx_long_kernel<__nv_bfloat16><<<grid, LN_THREADS, 0, s>>>(p);
  if (!a.dgamma && !a.dbeta) return launch_status(cudaGetLastError());
  const int per = static_cast<int>((a.rows + LN_CHUNKS - 1) / LN_CHUNKS);
  const int chunks = static_cast<int>((a.rows + per - 1) / per);
  const int cols = static_cast<int>((a.k + LN_THREADS - 1) / LN_THREADS);
  if (f32)
    ln_backward_params_long_kernel<float><<<dim3(cols, chunks), LN_THREADS, 0, s>>>(p, per);
  else
    ln_backward_params_long_kernel<__nv_bfloat16><<<dim3(cols, chunks), LN_THREADS, 0, s>>>(p, per);
  if (a.dgamma) launch_sum_chunks(p.partial, chunks, 2 * a.k, a.k, a.dgamma, s);
  if (a.dbeta) launch_sum_chunks(p.partial + a.k, chunks, 2 * a.k, a.k, a.dbeta, s);
  return launch_status(cudaGetLastError());
}

void launch_sum_chunks(const float* partial, int chunks, int64_t stride, int64_t n, float* out, cudaStream_t s) {
  sum_chunks_kernel<<<static_cast<unsigned>((n + LN_THREADS - 1) / LN_THREADS), LN_THREADS, 0, s>>>(
      partial, chunks, stride, static_cast<int>(n), out);
}

}  // namespace nvfp4
