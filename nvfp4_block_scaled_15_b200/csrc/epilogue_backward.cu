// Gradient of the product epilogue D = act(pre) [+ residual], pre = alpha acc + bias:
//   dpre = dD act'(pre),  dbias = sum over rows of dpre  (dresidual = dD)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "epilogue.cuh"
#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int EB_THREADS = 256;
constexpr int EB_CHUNKS = 64;

struct EpiBwdParams {
  const void* dd;
  int64_t ldd;
  const void* pre;
  int64_t ldp;
  int act;
  void* dpre;            // null: only dbias
  int64_t lddp;
  float* partial;        // [chunks][N], null: no dbias
  float* amax;
  int64_t M;
  int N;
};

// A block takes EB_THREADS columns (one per thread) of a chunk of rows.
template <typename T>
__global__ void __launch_bounds__(EB_THREADS) epilogue_backward_kernel(const EpiBwdParams p, int rows_per_chunk) {
  const int i = blockIdx.x * EB_THREADS + threadIdx.x;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * rows_per_chunk;
  const int64_t r1 = min(p.M, r0 + rows_per_chunk);
  uint32_t mag = 0;
  if (i < p.N) {
    float s = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
      const float dd = to_f32(static_cast<const T*>(p.dd)[r * p.ldd + i]);
      const float v = p.act == NVFP4_ACT_NONE
                          ? dd
                          : dd * act_slope(to_f32(static_cast<const T*>(p.pre)[r * p.ldp + i]), p.act);
      s += v;
      const T o = from_f32<T>(v);
      if (p.dpre) static_cast<T*>(p.dpre)[r * p.lddp + i] = o;
      mag = max(mag, mag_bits(o));
    }
    if (p.partial) p.partial[static_cast<int64_t>(blockIdx.y) * p.N + i] = s;
  }
  if (p.amax) {
    mag = __reduce_max_sync(0xFFFFFFFFu, mag);
    if ((threadIdx.x & 31) == 0) atomicMax(reinterpret_cast<unsigned int*>(p.amax), mag);
  }
}

}  // namespace

size_t epilogue_backward_workspace_bytes(int64_t M, int64_t N) {
  return M > 0 ? static_cast<size_t>(EB_CHUNKS) * N * sizeof(float) : 256;
}

nvfp4_status launch_epilogue_backward(const EpilogueBackward& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (a.amax) e = cudaMemsetAsync(a.amax, 0, sizeof(float), s);
  if (a.M == 0) {
    if (e == cudaSuccess && a.dbias) e = cudaMemsetAsync(a.dbias, 0, a.N * sizeof(float), s);
    return launch_status(e);
  }
  if (e != cudaSuccess) return launch_status(e);
  const EpiBwdParams p{a.dd, a.ldd, a.pre, a.ldp, a.act, a.dpre, a.lddp,
                       a.dbias ? static_cast<float*>(a.workspace) : nullptr, a.amax, a.M, static_cast<int>(a.N)};
  const int per = static_cast<int>((a.M + EB_CHUNKS - 1) / EB_CHUNKS);
  const int chunks = static_cast<int>((a.M + per - 1) / per);
  const dim3 grid(static_cast<unsigned>((a.N + EB_THREADS - 1) / EB_THREADS), chunks);
  if (a.dtype == NVFP4_DTYPE_F32)
    epilogue_backward_kernel<float><<<grid, EB_THREADS, 0, s>>>(p, per);
  else
    epilogue_backward_kernel<__nv_bfloat16><<<grid, EB_THREADS, 0, s>>>(p, per);
  e = cudaGetLastError();
  if (e == cudaSuccess && a.dbias)
    e = launch_sum_partials(p.partial, chunks, a.N, static_cast<int>(a.N), 0, a.dbias, nullptr, nullptr, nullptr, s);
  return launch_status(e);
}

}  // namespace nvfp4
