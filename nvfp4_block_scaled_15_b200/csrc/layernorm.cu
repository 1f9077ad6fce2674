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
#include "ptx.cuh"

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

// Maximum of mag over the block, in warp 0.
__device__ __forceinline__ uint32_t block_max(uint32_t mag, uint32_t* mags) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  mag = __reduce_max_sync(0xFFFFFFFFu, mag);
  if (lane == 0) mags[warp] = mag;
  __syncthreads();
  return warp == 0 ? __reduce_max_sync(0xFFFFFFFFu, lane < static_cast<int>(blockDim.x >> 5) ? mags[lane] : 0u) : 0u;
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
  int joined;            // the grid is one cluster, which joins its blocks' maxima itself
};

// Few blocks: a single cluster, whose first block writes the maximum; clearing
// it first would take another launch, 8 x 8192 6.2 us against 4.4.
constexpr int LF_MAX_CLUSTER = 8;

__device__ __forceinline__ void publish_amax(const LnParams& p, uint32_t mag, uint32_t* mags) {
  __shared__ uint32_t blocks[LF_MAX_CLUSTER];
  if (!p.amax) return;
  uint32_t m = block_max(mag, mags);
  if (!p.joined) {
    if (threadIdx.x == 0) atomicMax(reinterpret_cast<unsigned int*>(p.amax), m);
    return;
  }
  if (threadIdx.x == 0) st_shared_cluster_u32(mapa_shared(smem_u32(&blocks[blockIdx.x]), 0), m);
  cluster_sync_all();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    for (int i = 1; i < static_cast<int>(gridDim.x); ++i) m = max(m, blocks[i]);
    *p.amax = __uint_as_float(m);
  }
}

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

// ---------------------------------------------------------------------------
// Rows held in registers
// ---------------------------------------------------------------------------
// Rows of whole 8-element chunks that all start on 16-byte boundaries: thread
// t of the nt threads that share a row holds chunks t, t + nt, ...  (Other rows
// have kernels of their own below: chunks cut by the row's end cost these
// kernels twice their instructions, as the compiler keeps the elementwise
// path's bounds in registers.)
__device__ __forceinline__ int chunk_col(int t, int nt, int j) { return 8 * (t + nt * j); }

// Columns c .. c+7 of gamma or beta (cached: every row reads them).
template <typename TP>
__device__ __forceinline__ Chunk load_param_chunk(const void* p, int c, float dflt) {
  Chunk x;
  if (!p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x.v[i] = both(dflt);
  } else if constexpr (sizeof(TP) == 4) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c));
    const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c + 4));
    x.v[0] = make_float2(a.x, a.y), x.v[1] = make_float2(a.z, a.w);
    x.v[2] = make_float2(b.x, b.y), x.v[3] = make_float2(b.z, b.w);
  } else {
    x = unpack_chunk(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + c)));
  }
  return x;
}

// cp.async copies into this thread's own slots of shared memory: nobody else
// reads them, so waiting for the own copies is all the ordering needed.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One operand's slots of one ring stage: 16 bytes each, slot (j, part) of
// thread t at [(j * parts + part) * nt + t] (conflict-free).
template <typename T, int NV>
__device__ __forceinline__ void stage_in(uint8_t* slots, const T* row, int t, int nt, int k) {
  constexpr int PARTS = sizeof(T) / 2, PER = 16 / sizeof(T);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = chunk_col(t, nt, j);
#pragma unroll
    for (int h = 0; h < PARTS; ++h) {
      uint8_t* slot = slots + ((j * PARTS + h) * nt + t) * 16;
      if (c < k)
        cp_async16(slot, row + c + h * PER);
      else
        *reinterpret_cast<uint4*>(slot) = make_uint4(0u, 0u, 0u, 0u);     // past the row's end: zeros
    }
  }
}

template <typename T>
__device__ __forceinline__ Chunk stage_out(const uint8_t* slots, int t, int nt, int j) {
  if constexpr (sizeof(T) == 2) {
    return unpack_chunk(*reinterpret_cast<const uint4*>(slots + (j * nt + t) * 16));
  } else {
    Chunk c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 v = *reinterpret_cast<const float4*>(slots + ((j * 2 + h) * nt + t) * 16);
      c.v[2 * h] = make_float2(v.x, v.y), c.v[2 * h + 1] = make_float2(v.z, v.w);
    }
    return c;
  }
}

// Sums of a and b over the warp at the price of one: after the first step the
// lower half-warp carries a's partial sums and the upper half b's.  The result
// (sum a, sum b) is on every lane.
__device__ __forceinline__ float2 warp_sum2(float a, float b) {
  const bool upper = threadIdx.x & 16;
  float v = (upper ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, upper ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return make_float2(__shfl_sync(0xFFFFFFFFu, v, 0), __shfl_sync(0xFFFFFFFFu, v, 16));
}

// Mean and squared deviations of a union, from each part's (n, mean, M): with
// a pivot c and d = mean - c, sum n d and sum (M + n d^2) give
//   mean = c + sum n d / N,   M = sum (M + n d^2) - (sum n d)^2 / N.
// The pivot is the first part's mean; then N d^2 is at most M N / n_first, so
// the last difference loses a factor of at most the number of parts (32),
// whatever the row's mean.  Parts are the lanes of a warp.
struct Stats {
  float mean, m2;
};
__device__ __forceinline__ Stats join_lanes(float n, float mean, float m2, float inv_total) {
  const float pivot = __shfl_sync(0xFFFFFFFFu, mean, 0);
  const float d = n > 0.0f ? mean - pivot : 0.0f;
  const float2 s = warp_sum2(n * d, n > 0.0f ? fmaf(n * d, d, m2) : 0.0f);
  return {fmaf(s.x, inv_total, pivot), fmaf(-s.x * inv_total, s.x, s.y)};
}

// Named barrier of the nt threads of group g (its warps only).
__device__ __forceinline__ void group_sync(int g, int nt) {
  asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(nt) : "memory");
}

// A group's barrier, whatever its size.
__device__ __forceinline__ void group_or_warp_sync(int g, int nt) {
  if (nt > 32)
    group_sync(g, nt);
  else
    __syncwarp();
}

// ---------------------------------------------------------------------------
// Rows that start anywhere (an odd pitch or width, a view into a buffer)
// ---------------------------------------------------------------------------
// Such a row comes into shared memory as it lies in memory, copied in 4-byte
// words (cp.async has no smaller ones): its element c is at slot c + shift,
// shift = 1 where a bf16 row starts in the middle of a word, and zeros follow
// the row's end.  Threads take the same 8-element chunks as above, out of five
// words and a funnel shift, and results go back through shared memory in the
// same way.  Any thread may have copied a thread's words, so a row takes two
// barriers more than an aligned one.
template <typename T>
__device__ __forceinline__ int row_shift(const T* row) {
  return sizeof(T) == 2 ? static_cast<int>((reinterpret_cast<uintptr_t>(row) >> 1) & 1) : 0;
}

// Bytes of a row's image: whole chunks, the word behind them and the shift.
__host__ __device__ constexpr int odd_bytes(int k, int size) { return (k + 7) / 8 * 8 * size + 16; }

template <typename T>
__device__ __forceinline__ void odd_in(uint8_t* image, const T* row, int t, int nt, int k) {
  T* dst = reinterpret_cast<T*>(image);
  if constexpr (sizeof(T) == 4) {
#pragma unroll 4
    for (int c = t; c < k; c += nt) cp_async4(dst + c, row + c);
  } else {
    const int shift = row_shift(row);
    const int words = (k + shift) >> 1;                  // up to the last whole one
#pragma unroll 4
    for (int w = t + shift; w < words; w += nt) cp_async4(dst + 2 * w, row + (2 * w - shift));
    // the ends, and zeros up to where a row with the other shift reaches
    if (t == 0 && shift) dst[1] = row[0];
    if (t == nt - 1) {
      if ((k + shift) & 1 && k > shift) dst[k + shift - 1] = row[k - 1];
      dst[k + shift] = from_f32<T>(0.0f);
      if (shift == 0) dst[k + 1] = from_f32<T>(0.0f);
    }
  }
}

// Zeros behind the rows of an image, which copies leave alone.
template <typename T>
__device__ __forceinline__ void odd_clear(uint8_t* image, int t, int nt, int k) {
  for (int c = k + t; c < odd_bytes(k, sizeof(T)) / static_cast<int>(sizeof(T)); c += nt)
    reinterpret_cast<T*>(image)[c] = from_f32<T>(0.0f);
}

template <typename T>
__device__ __forceinline__ Chunk odd_chunk(const uint8_t* image, int c, int shift) {
  if constexpr (sizeof(T) == 2) {
    const uint4 w = *reinterpret_cast<const uint4*>(image + 2 * c);
    const uint32_t next = *reinterpret_cast<const uint32_t*>(image + 2 * c + 16);
    const int bits = 16 * shift;
    return unpack_chunk(make_uint4(__funnelshift_r(w.x, w.y, bits), __funnelshift_r(w.y, w.z, bits),
                                   __funnelshift_r(w.z, w.w, bits), __funnelshift_r(w.w, next, bits)));
  } else {
    Chunk x;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 v = *reinterpret_cast<const float4*>(image + 4 * c + 16 * h);
      x.v[2 * h] = make_float2(v.x, v.y), x.v[2 * h + 1] = make_float2(v.z, v.w);
    }
    return x;
  }
}

// Elements of a chunk at or past the row's end become v.
__device__ __forceinline__ void cut_chunk(Chunk& x, int valid, float v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (2 * i >= valid) x.v[i].x = v;
    if (2 * i + 1 >= valid) x.v[i].y = v;
  }
}

// A result row in shared memory (element c at slot c) to a row that starts
// anywhere, in words where the row has whole ones.
template <typename T>
__device__ __forceinline__ void odd_out(const uint8_t* image, T* row, int t, int nt, int k) {
  const T* src = reinterpret_cast<const T*>(image);
  if constexpr (sizeof(T) == 4) {
#pragma unroll 4
    for (int c = t; c < k; c += nt) row[c] = src[c];
  } else {
    const int shift = row_shift(row);
    const int words = (k + shift) >> 1;
    const uint32_t* in = reinterpret_cast<const uint32_t*>(image);
#pragma unroll 4
    for (int w = t + shift; w < words; w += nt)          // columns 2 w - shift and the next
      *reinterpret_cast<uint32_t*>(row + (2 * w - shift)) = shift ? __funnelshift_r(in[w - 1], in[w], 16) : in[w];
    if (t == 0 && shift) row[0] = src[0];
    if (t == nt - 1 && ((k + shift) & 1) && k > shift) row[k - 1] = src[k - 1];
  }
}

// gamma and beta as fp32 in shared memory, whole chunks; a thread's loads of
// both are issued before the first is stored.
__device__ __forceinline__ void params_in(float* gamma, float* beta, const LnParams& p) {
  const int k8 = (p.k + 7) / 8 * 8;
  for (int c = threadIdx.x; c < k8; c += 4 * blockDim.x) {
    float g[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = min(c + i * static_cast<int>(blockDim.x), p.k - 1);
      g[i] = p.gamma ? load_param(p.gamma, p.param_f32, col) : 1.0f;
      b[i] = p.beta ? load_param(p.beta, p.param_f32, col) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = c + i * static_cast<int>(blockDim.x);
      if (col < k8) gamma[col] = g[i], beta[col] = b[i];
    }
  }
}
__device__ __forceinline__ Chunk param_chunk(const float* p, int c) {
  return odd_chunk<float>(reinterpret_cast<const uint8_t*>(p), c, 0);
}

// ---------------------------------------------------------------------------
// Forward in one pass
// ---------------------------------------------------------------------------
// A block has G groups of nt threads; a group takes one row at a time, held in
// registers as it lies in memory, NV chunks per thread.  A thread takes the
// mean and squared deviations of its own elements; lanes and then warps are
// joined (join_lanes), so a row needs one barrier and no sum of squares cancels
// against the mean.  A row's loads, its reductions and its stores alternate, so
// the memory is kept busy by the other blocks of the SM: registers are held to
// what allows LF_BLOCKS of them.
constexpr int LF_THREADS = 256;        // of a block, up to rows of LF_THREADS * 32; 512 beyond
template <typename TX, int NV>
constexpr int lf_blocks(int threads) {  // blocks per SM
  return (NV <= 4 ? (sizeof(TX) == 2 ? 1024 : 768) : 512) / threads;
}
template <int NV>
constexpr int lf_max_k() { return 512 * 8 * NV; }
constexpr int LF_MAX_K = lf_max_k<8>();

// A chunk as it lies in memory.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ Chunk get() const { return unpack_chunk(w); }
};
template <>
struct Raw<float> {
  Chunk c;
  __device__ __forceinline__ Chunk get() const { return c; }
};

// Streaming 16-byte load (read once, not kept in L1).
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void load_raw(Raw<__nv_bfloat16>& x, const __nv_bfloat16* row, int c, int k) {
  x.w = c < k ? ld_stream(row + c) : make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ void load_raw(Raw<float>& x, const float* row, int c, int k) {
  uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
  if (c < k) a = ld_stream(row + c), b = ld_stream(row + c + 4);
  x.c.v[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
  x.c.v[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
  x.c.v[2] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y));
  x.c.v[3] = make_float2(__uint_as_float(b.z), __uint_as_float(b.w));
}

template <typename TX, typename TY, typename TP, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS, lf_blocks<TX, NV>(THREADS)) ln_forward_rows_kernel(const LnParams p, int nt) {
  __shared__ float2 red[2][THREADS / 32];
  __shared__ uint32_t mags[THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = blockDim.x / nt, g = threadIdx.x / nt, t = threadIdx.x - g * nt;
  const int gw = nt >> 5, w0 = g * gw;                   // warps of a group, its first
  const float inv_k = 1.0f / static_cast<float>(p.k);
  // elements of this thread, of its warp, of warp `lane` of the group
  auto count = [&](int first, int lanes) {
    int n = 0;
    for (int j = 0; j < NV; ++j) n += min(max(p.k - 8 * (first + nt * j), 0), 8 * lanes);
    return static_cast<float>(n);
  };
  auto inverse = [](float n) { return n > 0.0f ? 1.0f / n : 0.0f; };
  const float n_thread = count(t, 1), inv_thread = inverse(n_thread);
  const float inv_warp = inverse(count(t - lane, 32));
  const float n_lane = lane < gw ? count(32 * lane, 32) : 0.0f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  if (p.joined) cluster_sync_all();                       // every block has started, before its memory is written to
  Mag<TY> mag;
  int parity = 0;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * groups + g; r < p.rows; r += step) {
    const TX* row = static_cast<const TX*>(p.x) + r * p.ldx;
    Raw<TX> x[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) load_raw(x[j], row, chunk_col(t, nt, j), p.k);
    float2 s2 = both(0.0f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Chunk c = x[j].get();
#pragma unroll
      for (int i = 0; i < 4; ++i) s2 = add2(s2, c.v[i]);             // 0 past the row's end
    }
    const float own_mean = (s2.x + s2.y) * inv_thread;
    s2 = both(0.0f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      // branches: selects instead of them took registers that spilled (107 -> 139 us at 16384 x 8192)
      if (chunk_col(t, nt, j) < p.k) {
        const Chunk c = x[j].get();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 d = add2(c.v[i], both(-own_mean));
          s2 = fma2(d, d, s2);
        }
      }
    }
    Stats st = join_lanes(n_thread, own_mean, s2.x + s2.y, inv_warp);
    if (gw > 1) {
      if (lane == 0) red[parity][warp] = make_float2(st.mean, st.m2);
      group_sync(g, nt);
      const float2 w = lane < gw ? red[parity][w0 + lane] : make_float2(0.0f, 0.0f);
      parity ^= 1;
      st = join_lanes(n_lane, w.x, w.y, inv_k);
    }
    const float mean = st.mean;
    const float rstd = __frsqrt_rn(fmaf(st.m2 < 0.0f ? 0.0f : st.m2, inv_k, p.eps));   // a NaN stays one
    TY* y = static_cast<TY*>(p.y) + r * p.ldy;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = chunk_col(t, nt, j);
      if (col < p.k) {
        const Chunk gm = load_param_chunk<TP>(p.gamma, col, 1.0f), bt = load_param_chunk<TP>(p.beta, col, 0.0f);
        Chunk c = x[j].get();
#pragma unroll
        for (int i = 0; i < 4; ++i) c.v[i] = fma2(mul2(add2(c.v[i], both(-mean)), both(rstd)), gm.v[i], bt.v[i]);
        store_chunk<TY>(y + col, c, mag);
      }
    }
    if (t == 0) {
      if (p.mean) p.mean[r] = mean;
      if (p.rstd) p.rstd[r] = rstd;
    }
  }
  publish_amax(p, mag.bits(), mags);
}

// Forward of short rows (k <= 32 E) of any alignment: a warp takes RP rows at a
// time, lane l their elements l, l + 32, ..., straight from and to memory, with
// gamma and beta in registers.  The rows' sums are formed two at the price of
// one, and RP rows hide each other's latency.
constexpr int LS_MAX_K = 256;
template <typename TX, typename TY, int E>
__global__ void __launch_bounds__(256, 4) ln_forward_short_kernel(const LnParams p, int) {
  constexpr int RP = E <= 2 ? 4 : 2;
  __shared__ uint32_t mags[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float inv_k = 1.0f / static_cast<float>(p.k);
  float gm[E], bt[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = lane + 32 * e;
    gm[e] = p.gamma && c < p.k ? load_param(p.gamma, p.param_f32, c) : 1.0f;
    bt[e] = p.beta && c < p.k ? load_param(p.beta, p.param_f32, c) : 0.0f;
  }
  if (p.joined) cluster_sync_all();                       // every block has started, before its memory is written to
  uint32_t mag = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 8 * RP;
  for (int64_t r = (static_cast<int64_t>(blockIdx.x) * 8 + warp) * RP; r < p.rows; r += step) {
    float x[RP][E];
    float s[RP], mean[RP], rstd[RP];
#pragma unroll
    for (int q = 0; q < RP; ++q) {
      const TX* row = static_cast<const TX*>(p.x) + (r + q) * p.ldx;
#pragma unroll
      for (int e = 0; e < E; ++e) x[q][e] = r + q < p.rows && lane + 32 * e < p.k ? to_f32(row[lane + 32 * e]) : 0.0f;
    }
#pragma unroll
    for (int q = 0; q < RP; ++q) {
      s[q] = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) s[q] += x[q][e];
    }
#pragma unroll
    for (int q = 0; q < RP; q += 2) {
      const float2 t = warp_sum2(s[q], s[q + 1]);
      mean[q] = t.x * inv_k, mean[q + 1] = t.y * inv_k;
    }
#pragma unroll
    for (int q = 0; q < RP; ++q) {
      s[q] = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = lane + 32 * e < p.k ? x[q][e] - mean[q] : 0.0f;
        s[q] = fmaf(d, d, s[q]);
      }
    }
#pragma unroll
    for (int q = 0; q < RP; q += 2) {
      const float2 t = warp_sum2(s[q], s[q + 1]);
      rstd[q] = __frsqrt_rn(fmaf(t.x, inv_k, p.eps)), rstd[q + 1] = __frsqrt_rn(fmaf(t.y, inv_k, p.eps));
    }
#pragma unroll
    for (int q = 0; q < RP; ++q) {
      if (r + q >= p.rows) break;
      TY* row = static_cast<TY*>(p.y) + (r + q) * p.ldy;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (lane + 32 * e >= p.k) continue;
        const TY o = from_f32<TY>(fmaf((x[q][e] - mean[q]) * rstd[q], gm[e], bt[e]));
        row[lane + 32 * e] = o;
        mag = max(mag, mag_bits(o));
      }
      if (lane == 0) {
        if (p.mean) p.mean[r + q] = mean[q];
        if (p.rstd) p.rstd[r + q] = rstd[q];
      }
    }
  }
  publish_amax(p, mag, mags);
}

// Forward of bf16 rows that start anywhere, of up to LF_MAX_K elements: the
// chunks of the kernel for aligned rows out of the row's image in shared memory, where gamma and
// beta lie too.  A thread holds its chunks in registers, so the next row's image
// is on its way once every thread has read this one's; more images ahead leave
// room for fewer groups and measured slower (16384 x 4095 bf16: one 123 us, two
// 149, three 198).
constexpr int LI_THREADS = 512;
constexpr int LI_SMEM = 216 * 1024;

template <typename TY, int NV>
__global__ void __launch_bounds__(LI_THREADS, NV <= 4 ? 2 : 1) ln_forward_image_kernel(const LnParams p, int nt) {
  using TX = __nv_bfloat16;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 red[2][LI_THREADS / 32];
  __shared__ uint32_t mags[LI_THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = blockDim.x / nt, g = threadIdx.x / nt, t = threadIdx.x - g * nt;
  const int gw = nt >> 5, w0 = g * gw;
  const int k8 = (p.k + 7) / 8 * 8;
  const int row_bytes = odd_bytes(p.k, sizeof(TX)), out_bytes = k8 * static_cast<int>(sizeof(TY));
  float* gamma = reinterpret_cast<float*>(smem);
  float* beta = gamma + k8;
  uint8_t* own = smem + 8 * k8 + static_cast<size_t>(g) * (row_bytes + out_bytes);
  uint8_t* out = own + row_bytes;
  const float inv_k = 1.0f / static_cast<float>(p.k);
  auto count = [&](int first, int lanes) {
    int n = 0;
    for (int j = 0; j < NV; ++j) n += min(max(p.k - 8 * (first + nt * j), 0), 8 * lanes);
    return static_cast<float>(n);
  };
  auto inverse = [](float n) { return n > 0.0f ? 1.0f / n : 0.0f; };
  const float n_thread = count(t, 1), inv_thread = inverse(n_thread);
  const float inv_warp = inverse(count(t - lane, 32));
  const float n_lane = lane < gw ? count(32 * lane, 32) : 0.0f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * groups + g;
  odd_clear<TX>(own, t, nt, p.k);
  group_or_warp_sync(g, nt);
  auto issue = [&](int64_t r) {
    if (r < p.rows) odd_in(own, static_cast<const TX*>(p.x) + r * p.ldx, t, nt, p.k);
    cp_async_commit();
  };
  issue(r0);
  params_in(gamma, beta, p);
  __syncthreads();
  if (p.joined) cluster_sync_all();                       // every block has started, before its memory is written to
  Mag<TY> mag;
  int parity = 0;
  for (int64_t r = r0; r < p.rows; r += step) {
    cp_async_wait<0>();
    group_or_warp_sync(g, nt);                           // the row is there
    const int shift = row_shift(static_cast<const TX*>(p.x) + r * p.ldx);
    Chunk x[NV];
    float2 s2 = both(0.0f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = chunk_col(t, nt, j);
      if (c < p.k) {
        x[j] = odd_chunk<TX>(own, c, shift);
#pragma unroll
        for (int i = 0; i < 4; ++i) s2 = add2(s2, x[j].v[i]);        // 0 past the row's end
      }
    }
    const float own_mean = (s2.x + s2.y) * inv_thread;
    s2 = both(0.0f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = chunk_col(t, nt, j);
      if (c < p.k) {
        Chunk d;
#pragma unroll
        for (int i = 0; i < 4; ++i) d.v[i] = add2(x[j].v[i], both(-own_mean));
        if (c + 8 > p.k) cut_chunk(d, p.k - c, 0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) s2 = fma2(d.v[i], d.v[i], s2);
      }
    }
    Stats st = join_lanes(n_thread, own_mean, s2.x + s2.y, inv_warp);
    if (gw > 1) {
      if (lane == 0) red[parity][warp] = make_float2(st.mean, st.m2);
      group_sync(g, nt);
      const float2 w = lane < gw ? red[parity][w0 + lane] : make_float2(0.0f, 0.0f);
      parity ^= 1;
      st = join_lanes(n_lane, w.x, w.y, inv_k);
    } else {
      __syncwarp();
    }
    issue(r + step);                                     // every thread has read the image
    const float mean = st.mean;
    const float rstd = __frsqrt_rn(fmaf(st.m2 < 0.0f ? 0.0f : st.m2, inv_k, p.eps));   // a NaN stays one
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = chunk_col(t, nt, j);
      if (c < p.k) {
        const Chunk gm = param_chunk(gamma, c), bt = param_chunk(beta, c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[j].v[i] = fma2(mul2(add2(x[j].v[i], both(-mean)), both(rstd)), gm.v[i], bt.v[i]);
        if (c + 8 > p.k) cut_chunk(x[j], p.k - c, 0.0f);
        store_chunk<TY>(reinterpret_cast<TY*>(out) + c, x[j], mag);
      }
    }
    group_or_warp_sync(g, nt);
    odd_out(out, static_cast<TY*>(p.y) + r * p.ldy, t, nt, p.k);
    if (t == 0) {
      if (p.mean) p.mean[r] = mean;
      if (p.rstd) p.rstd[r] = rstd;
    }
  }
  publish_amax(p, mag.bits(), mags);
}

// Forward of fp32 rows that start anywhere, of up to LO_MAX_K elements: the NT
// threads of a group hold elements t, t + NT, ... in registers, so every access
// is of 32 neighbouring elements whatever the alignment, at offsets that are
// constants of the kernel.  Four elements at a time, the ones past the row's end
// skipped by four.  (3001 x 1155: 10.3 us against 16.9 through row images; bf16 rows,
// whose accesses are half as wide: 16384 x 4095 201 against 123 us.)
constexpr int LO_ELEMS = 32;
constexpr int LO_MAX_K = 1024 * LO_ELEMS;

template <typename TY, typename TP, int NT>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT, 1024 / (NT < 256 ? 256 : NT)) ln_forward_odd_kernel(const LnParams p, int) {
  using TX = float;
  constexpr int THREADS = NT < 256 ? 256 : NT, GROUPS = THREADS / NT, GW = NT / 32;
  __shared__ float2 red[2][THREADS / 32];
  __shared__ uint32_t mags[THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = threadIdx.x / NT, t = threadIdx.x % NT, w0 = g * GW;
  const float inv_k = 1.0f / static_cast<float>(p.k);
  const int left = p.k - t;                               // element e of this thread is in the row: e * NT < left
  const int full = p.k / NT, rest = p.k % NT;             // of a group
  auto inverse = [](float n) { return n > 0.0f ? 1.0f / n : 0.0f; };
  const float n_thread = static_cast<float>(full + (t < rest)), inv_thread = inverse(n_thread);
  auto warp_count = [&](int w) { return static_cast<float>(32 * full + min(max(rest - 32 * w, 0), 32)); };
  const float inv_warp = inverse(warp_count(warp - w0));
  const float n_lane = lane < GW ? warp_count(lane) : 0.0f;
  if (p.joined) cluster_sync_all();                       // every block has started, before its memory is written to
  uint32_t mag = 0;
  int parity = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * GROUPS;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * GROUPS + g; r < p.rows; r += step) {
    const TX* row = static_cast<const TX*>(p.x) + r * p.ldx + t;
    float x[LO_ELEMS];
#pragma unroll
    for (int e = 0; e < LO_ELEMS; e += 4)
      if (e * NT < p.k) {
#pragma unroll
        for (int i = e; i < e + 4; ++i) x[i] = i * NT < left ? to_f32(row[i * NT]) : 0.0f;
      }
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < LO_ELEMS; e += 4)
      if (e * NT < p.k) s += (x[e] + x[e + 1]) + (x[e + 2] + x[e + 3]);
    const float own_mean = s * inv_thread;
    s = 0.0f;
#pragma unroll
    for (int e = 0; e < LO_ELEMS; e += 4)
      if (e * NT < p.k) {
#pragma unroll
        for (int i = e; i < e + 4; ++i) {
          const float d = i * NT < left ? x[i] - own_mean : 0.0f;
          s = fmaf(d, d, s);
        }
      }
    Stats st = join_lanes(n_thread, own_mean, s, inv_warp);
    if constexpr (GW > 1) {
      if (lane == 0) red[parity][warp] = make_float2(st.mean, st.m2);
      if constexpr (GROUPS > 1)
        group_sync(g, NT);
      else
        __syncthreads();
      const float2 w = lane < GW ? red[parity][w0 + lane] : make_float2(0.0f, 0.0f);
      parity ^= 1;
      st = join_lanes(n_lane, w.x, w.y, inv_k);
    }
    const float mean = st.mean;
    const float rstd = __frsqrt_rn(fmaf(st.m2 < 0.0f ? 0.0f : st.m2, inv_k, p.eps));   // a NaN stays one
    TY* y = static_cast<TY*>(p.y) + r * p.ldy + t;
    const TP* gamma = static_cast<const TP*>(p.gamma) + t;
    const TP* beta = static_cast<const TP*>(p.beta) + t;
#pragma unroll
    for (int e = 0; e < LO_ELEMS; e += 4)
      if (e * NT < p.k) {
        float gm[4], bt[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          gm[i] = p.gamma && (e + i) * NT < left ? to_f32(gamma[(e + i) * NT]) : 1.0f;
          bt[i] = p.beta && (e + i) * NT < left ? to_f32(beta[(e + i) * NT]) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((e + i) * NT < left) {
            const TY o = from_f32<TY>(fmaf((x[e + i] - mean) * rstd, gm[i], bt[i]));
            y[(e + i) * NT] = o;
            mag = max(mag, mag_bits(o));
          }
      }
    if (t == 0) {
      if (p.mean) p.mean[r] = mean;
      if (p.rstd) p.rstd[r] = rstd;
    }
  }
  publish_amax(p, mag, mags);
}

// ---------------------------------------------------------------------------
// Backward in one pass
// ---------------------------------------------------------------------------
constexpr int LB_THREADS = 512;        // most threads of a block; 128 registers each
constexpr int LB_NV = 2;               // chunks of 8 elements per thread
constexpr int LB_MAX_COLS = LB_THREADS * 8 * LB_NV;        // columns of a block
constexpr int LB_MAX_CLUSTER = 8;
constexpr int LB_MAX_K = LB_MAX_COLS * LB_MAX_CLUSTER;
constexpr int LB_SMEM = 216 * 1024;

// The block's largest |dx| (in warp 0): to its slot, for the sum over blocks
// to join, or straight to the maximum where no such kernel follows.
__device__ __forceinline__ void publish_block(const LnBwdParams& p, uint32_t mag, uint32_t* mag_out) {
  if (threadIdx.x != 0) return;
  if (mag_out)
    mag_out[blockIdx.x] = mag;
  else if (p.amax)
    atomicMax(reinterpret_cast<unsigned int*>(p.amax), mag);
}

// Bytes of one ring stage of a group (vector: slots of nt threads; odd: images).
template <typename TX, typename TDY, bool kOdd>
__host__ __device__ constexpr int lb_stage_bytes(int k, int nt, bool res) {
  return kOdd ? odd_bytes(k, sizeof(TDY)) + odd_bytes(k, sizeof(TX)) * (res ? 2 : 1)
              : nt * 8 * LB_NV * static_cast<int>(sizeof(TDY) + sizeof(TX) * (res ? 2 : 1));
}
// Bytes of a group: its ring, and for odd rows the image of its dx.
template <typename TX, typename TDY, bool kOdd, int S>
__host__ __device__ constexpr int lb_group_bytes(int k, int nt, bool res) {
  return S * lb_stage_bytes<TX, TDY, kOdd>(k, nt, res) + (kOdd ? odd_bytes(k, sizeof(TX)) : 0);
}

// Backward of rows of up to LB_MAX_K elements.  A block has G groups of nt
// threads; a group takes one row at a time, a thread the same columns of every
// row, so dgamma and dbeta are sums in its registers until the end.  The rows
// ahead are on their way into a ring of S in shared memory (the accumulators
// leave no room for a second row in registers).  Rows longer than a block's
// columns are cut between the blocks of a cluster (kc columns each, one group
// per block), which exchange the row's two sums through each other's shared
// memory.  At the end the groups' column sums meet in shared memory and the
// block writes one partial; the sum over blocks (sum_partials_kernel) runs in
// block order, so results do not depend on timing.
template <typename TX, typename TDY, bool kOdd, bool kCluster, int S>
__global__ void __launch_bounds__(LB_THREADS, 1) ln_backward_rows_kernel(const LnBwdParams p, int nt, int kc,
                                                                          uint32_t* mag_out) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 red[2][LB_THREADS / 32];
  __shared__ float2 peers[2][LB_MAX_CLUSTER];            // the row's sums of each block of the cluster
  __shared__ uint32_t mags[LB_THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = blockDim.x / nt, g = threadIdx.x / nt, t = threadIdx.x - g * nt;
  const int gw = nt >> 5, w0 = g * gw;                   // warps of a group, its first
  const int cluster = kCluster ? (p.k + kc - 1) / kc : 1;            // blocks that share a row
  const int rank = kCluster ? static_cast<int>(cluster_ctarank()) : 0;
  const int c0 = rank * kc, k = kCluster ? min(kc, p.k - c0) : p.k;  // this block's columns
  const int dy_bytes = kOdd ? odd_bytes(k, sizeof(TDY)) : nt * 8 * LB_NV * static_cast<int>(sizeof(TDY));
  const int x_bytes = kOdd ? odd_bytes(k, sizeof(TX)) : nt * 8 * LB_NV * static_cast<int>(sizeof(TX));
  const int stage_bytes = lb_stage_bytes<TX, TDY, kOdd>(k, nt, p.res != nullptr);
  uint8_t* own = ring + static_cast<size_t>(g) * lb_group_bytes<TX, TDY, kOdd, S>(k, nt, p.res != nullptr);
  uint8_t* out = own + S * stage_bytes;                  // odd: the image of dx
  const float inv_k = 1.0f / static_cast<float>(p.k);
  const int64_t step = static_cast<int64_t>(gridDim.x / cluster) * groups;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x / cluster) * groups + g;
  const TDY* dy_base = static_cast<const TDY*>(p.dy) + c0;
  const TX* x_base = static_cast<const TX*>(p.x) + c0;
  const TX* res_base = static_cast<const TX*>(p.res) + c0;

  auto issue = [&](int64_t r, int stage) {
    if (r < p.rows) {
      uint8_t* b = own + stage * stage_bytes;
      if constexpr (kOdd) {
        odd_in(b, dy_base + r * p.lddy, t, nt, k);
        odd_in(b + dy_bytes, x_base + r * p.ldx, t, nt, k);
        if (p.res) odd_in(b + dy_bytes + x_bytes, res_base + r * p.ldr, t, nt, k);
      } else {
        stage_in<TDY, LB_NV>(b, dy_base + r * p.lddy, t, nt, k);
        stage_in<TX, LB_NV>(b + dy_bytes, x_base + r * p.ldx, t, nt, k);
        if (p.res) stage_in<TX, LB_NV>(b + dy_bytes + x_bytes, res_base + r * p.ldr, t, nt, k);
      }
    }
    cp_async_commit();
  };
  if constexpr (kCluster) cluster_sync_all();             // every block of the cluster has started
  if constexpr (kOdd) {
    for (int i = 0; i < S; ++i) {
      uint8_t* b = own + i * stage_bytes;
      odd_clear<TDY>(b, t, nt, k);
      odd_clear<TX>(b + dy_bytes, t, nt, k);
      if (p.res) odd_clear<TX>(b + dy_bytes + x_bytes, t, nt, k);
    }
    group_or_warp_sync(g, nt);
  }
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(r0 + i * step, i);

  Chunk gam[LB_NV], dg[LB_NV], db[LB_NV];
#pragma unroll
  for (int j = 0; j < LB_NV; ++j) {
    const int c = chunk_col(t, nt, j);
#pragma unroll
    for (int i = 0; i < 4; ++i) dg[j].v[i] = db[j].v[i] = both(0.0f);
    if constexpr (kOdd) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        gam[j].v[i].x = p.gamma && c + 2 * i < k ? load_param(p.gamma, p.param_f32, c0 + c + 2 * i) : 1.0f;
        gam[j].v[i].y = p.gamma && c + 2 * i + 1 < k ? load_param(p.gamma, p.param_f32, c0 + c + 2 * i + 1) : 1.0f;
      }
    } else {
      const int in = c0 + min(c, k - 8);
      gam[j] = p.param_f32 ? load_param_chunk<float>(p.gamma, in, 1.0f) : load_param_chunk<__nv_bfloat16>(p.gamma, in, 1.0f);
    }
  }
  Mag<TX> mag;
  int parity = 0, stage = 0;
  float mean_next = r0 < p.rows ? p.mean[r0] : 0.0f, rstd_next = r0 < p.rows ? p.rstd[r0] : 0.0f;
  for (int64_t r = r0; r < p.rows; r += step) {
    // the slot read in the last turn takes the row S - 1 turns ahead (odd: every
    // thread has read it, by the barrier in front of dx's way out)
    issue(r + (S - 1) * step, stage == 0 ? S - 1 : stage - 1);
    const float mean = mean_next, rstd = rstd_next;
    if (r + step < p.rows) {
      mean_next = p.mean[r + step];
      rstd_next = p.rstd[r + step];
    }
    cp_async_wait<S - 1>();
    if constexpr (kOdd) group_or_warp_sync(g, nt);
    const uint8_t* b = own + stage * stage_bytes;
    int dy_shift = 0, x_shift = 0;
    if constexpr (kOdd) {
      dy_shift = row_shift(dy_base + r * p.lddy);
      x_shift = row_shift(x_base + r * p.ldx);
    }
    Chunk dy[LB_NV], xh[LB_NV];
    float2 sa = both(0.0f), sx = both(0.0f);
#pragma unroll
    for (int j = 0; j < LB_NV; ++j) {
      const int c = chunk_col(t, nt, j);
      if constexpr (kOdd) {
        if (c >= k) continue;
        dy[j] = odd_chunk<TDY>(b, c, dy_shift);
        xh[j] = odd_chunk<TX>(b + dy_bytes, c, x_shift);
      } else {
        dy[j] = stage_out<TDY>(b, t, nt, j);
        xh[j] = stage_out<TX>(b + dy_bytes, t, nt, j);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) xh[j].v[i] = mul2(add2(xh[j].v[i], both(-mean)), both(rstd));
      if (c >= k) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = mul2(dy[j].v[i], gam[j].v[i]);       // 0 past the row's end, as dy is
        sa = add2(sa, a);
        sx = fma2(a, xh[j].v[i], sx);
        dg[j].v[i] = fma2(dy[j].v[i], xh[j].v[i], dg[j].v[i]);
        db[j].v[i] = add2(db[j].v[i], dy[j].v[i]);
      }
    }
    float2 sum = warp_sum2(sa.x + sa.y, sx.x + sx.y);
    if (gw > 1) {
      if (lane == 0) red[parity][warp] = sum;
      group_sync(g, nt);
      const float2 w = lane < gw ? red[parity][w0 + lane] : make_float2(0.0f, 0.0f);
      sum = warp_sum2(w.x, w.y);
    }
    if constexpr (kCluster) {
      // a peer reads the slots of this parity before it arrives at the next row's barrier
      if (threadIdx.x < cluster)
        st_shared_cluster_f32x2(mapa_shared(smem_u32(&peers[parity][rank]), threadIdx.x), sum);
      cluster_sync_all();
      sum = make_float2(0.0f, 0.0f);
      for (int i = 0; i < cluster; ++i) {
        sum.x += peers[parity][i].x;
        sum.y += peers[parity][i].y;
      }
    }
    parity ^= 1;
    const float2 c1 = both(-rstd * (sum.x * inv_k)), c2 = both(-rstd * (sum.y * inv_k));
    TX* dx = static_cast<TX*>(p.dx) + r * p.lddx + c0;
    int res_shift = 0;
    if constexpr (kOdd) res_shift = p.res ? row_shift(res_base + r * p.ldr) : 0;
#pragma unroll
    for (int j = 0; j < LB_NV; ++j) {
      const int c = chunk_col(t, nt, j);
      if (c >= k) continue;
      Chunk v;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v.v[i] = fma2(mul2(dy[j].v[i], gam[j].v[i]), both(rstd), fma2(xh[j].v[i], c2, c1));
      if (p.res) {
        Chunk res;
        if constexpr (kOdd)
          res = odd_chunk<TX>(b + dy_bytes + x_bytes, c, res_shift);
        else
          res = stage_out<TX>(b + dy_bytes + x_bytes, t, nt, j);
#pragma unroll
        for (int i = 0; i < 4; ++i) v.v[i] = add2(v.v[i], res.v[i]);
      }
      if constexpr (kOdd) {
        if (c + 8 > k) cut_chunk(v, k - c, 0.0f);
        store_chunk<TX>(reinterpret_cast<TX*>(out) + c, v, mag);
      } else {
        store_chunk<TX>(dx + c, v, mag);
      }
    }
    if constexpr (kOdd) {
      group_or_warp_sync(g, nt);
      odd_out(out, dx, t, nt, k);
    }
    if (++stage == S) stage = 0;
  }
  cp_async_wait<0>();
  const uint32_t m = block_max(mag.bits(), mags);         // its barrier: every group is done with the ring
  if (p.partial) {
    float* acc = reinterpret_cast<float*>(ring);          // [groups][2][k]
#pragma unroll
    for (int j = 0; j < LB_NV; ++j) {
      const int c = chunk_col(t, nt, j);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < k) {
          acc[(2 * g) * k + c + e] = dg[j].get(e);
          acc[(2 * g + 1) * k + c + e] = db[j].get(e);
        }
    }
    __syncthreads();
    float* part = p.partial + static_cast<int64_t>(blockIdx.x / cluster) * 2 * p.k + c0;
    for (int i = threadIdx.x; i < 2 * k; i += blockDim.x) {
      float s = 0.0f;
      for (int h = 0; h < groups; ++h) s += acc[2 * h * k + i];
      part[i < k ? i : i - k + p.k] = s;
    }
  }
  publish_block(p, m, mag_out);
  if constexpr (kCluster) cluster_sync_all();             // no block leaves while a peer may still write to it
}

// Backward of rows that start anywhere, of up to LB_ODD_K elements: the NT
// threads of a group hold elements t, t + NT, ... as in the forward kernel, and
// their column sums.  A row's loads, sums and stores alternate; the block's other
// groups and the number of elements in flight (three operands) keep the memory
// busy.  dispatch_backward says which rows the ring kernel above takes instead.
constexpr int LB_ODD_ELEMS = 16;
constexpr int LB_ODD_K = LB_THREADS * LB_ODD_ELEMS;
template <typename TX, typename TDY, typename TP, int NT>
__global__ void __launch_bounds__(LB_THREADS, 1) ln_backward_odd_kernel(const LnBwdParams p, uint32_t* mag_out) {
  constexpr int E = LB_ODD_ELEMS, GROUPS = LB_THREADS / NT, GW = NT / 32;
  extern __shared__ __align__(16) uint8_t ring[];         // the groups' column sums [GROUPS][2][k]
  __shared__ float2 red[2][LB_THREADS / 32];
  __shared__ uint32_t mags[LB_THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = threadIdx.x / NT, t = threadIdx.x % NT, w0 = g * GW;
  const float inv_k = 1.0f / static_cast<float>(p.k);
  const int left = p.k - t;                               // element e of this thread is in the row: e * NT < left
  float dg[E], db[E];
#pragma unroll
  for (int e = 0; e < E; ++e) dg[e] = db[e] = 0.0f;
  uint32_t mag = 0;
  int parity = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * GROUPS;
  const TP* gamma = static_cast<const TP*>(p.gamma) + t;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * GROUPS + g; r < p.rows; r += step) {
    const float mean = p.mean[r], rstd = p.rstd[r];
    const TDY* dy = static_cast<const TDY*>(p.dy) + r * p.lddy + t;
    const TX* x = static_cast<const TX*>(p.x) + r * p.ldx + t;
    const TX* z = static_cast<const TX*>(p.res) + r * p.ldr + t;
    float a[E], xh[E], res[E];
#pragma unroll
    for (int e = 0; e < E; e += 4)
      if (e * NT < p.k) {
#pragma unroll
        for (int i = e; i < e + 4; ++i) {
          a[i] = i * NT < left ? to_f32(dy[i * NT]) : 0.0f;
          xh[i] = i * NT < left ? to_f32(x[i * NT]) : 0.0f;
          res[i] = p.res && i * NT < left ? to_f32(z[i * NT]) : 0.0f;
        }
      }
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int e = 0; e < E; e += 4)
      if (e * NT < p.k) {
        float gm[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) gm[i] = p.gamma && (e + i) * NT < left ? to_f32(gamma[(e + i) * NT]) : 1.0f;
#pragma unroll
        for (int i = e; i < e + 4; ++i)
          if (i * NT < left) {
            xh[i] = (xh[i] - mean) * rstd;
            dg[i] = fmaf(a[i], xh[i], dg[i]);
            db[i] += a[i];
            a[i] *= gm[i - e];
            s1 += a[i];
            s2 = fmaf(a[i], xh[i], s2);
          }
      }
    float2 sum = warp_sum2(s1, s2);
    if constexpr (GW > 1) {
      if (lane == 0) red[parity][warp] = sum;
      if constexpr (GROUPS > 1)
        group_sync(g, NT);
      else
        __syncthreads();
      const float2 w = lane < GW ? red[parity][w0 + lane] : make_float2(0.0f, 0.0f);
      parity ^= 1;
      sum = warp_sum2(w.x, w.y);
    }
    const float c1 = -rstd * (sum.x * inv_k), c2 = -rstd * (sum.y * inv_k);
    TX* dx = static_cast<TX*>(p.dx) + r * p.lddx + t;
#pragma unroll
    for (int e = 0; e < E; e += 4)
      if (e * NT < p.k) {
#pragma unroll
        for (int i = e; i < e + 4; ++i)
          if (i * NT < left) {
            const TX o = from_f32<TX>(fmaf(a[i], rstd, fmaf(xh[i], c2, c1)) + res[i]);
            dx[i * NT] = o;
            mag = max(mag, mag_bits(o));
          }
      }
  }
  const uint32_t m = block_max(mag, mags);
  if (p.partial) {
    float* acc = reinterpret_cast<float*>(ring) + 2 * g * p.k + t;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (e * NT < left) acc[e * NT] = dg[e], acc[p.k + e * NT] = db[e];
    __syncthreads();
    const float* sums = reinterpret_cast<const float*>(ring);
    for (int i = threadIdx.x; i < 2 * p.k; i += LB_THREADS) {
      float s = 0.0f;
#pragma unroll
      for (int h = 0; h < GROUPS; ++h) s += sums[2 * h * p.k + i];
      p.partial[static_cast<int64_t>(blockIdx.x) * 2 * p.k + i] = s;
    }
  }
  publish_block(p, m, mag_out);
}

// Backward of short rows of any alignment, as the forward kernel above: a warp
// takes RP rows at a time and keeps its columns' sums in registers.  (For rows of
// up to 256 it measured three times as slow as the kernel for whole chunks.)
constexpr int LB_SHORT_K = 64;
constexpr int LB_SHORT_RP = 4;
constexpr int LB_SHORT_ROWS = LB_THREADS / 32 * LB_SHORT_RP;           // of a block at a time
template <typename TX, typename TDY>
__global__ void __launch_bounds__(LB_THREADS) ln_backward_short_kernel(const LnBwdParams p, uint32_t* mag_out) {
  constexpr int E = LB_SHORT_K / 32, RP = LB_SHORT_RP;
  constexpr int WARPS = LB_THREADS / 32;
  __shared__ float acc[WARPS][2][32 * E];
  __shared__ uint32_t mags[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float inv_k = 1.0f / static_cast<float>(p.k);
  float gm[E], dg[E], db[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    gm[e] = p.gamma && lane + 32 * e < p.k ? load_param(p.gamma, p.param_f32, lane + 32 * e) : 1.0f;
    dg[e] = db[e] = 0.0f;
  }
  uint32_t mag = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * WARPS * RP;
  for (int64_t r = (static_cast<int64_t>(blockIdx.x) * WARPS + warp) * RP; r < p.rows; r += step) {
    float dy[RP][E], xh[RP][E], res[RP][E], mean[RP], rstd[RP];
    float2 sum[RP];
#pragma unroll
    for (int q = 0; q < RP; ++q) {
      const bool on = r + q < p.rows;
      const TDY* d = static_cast<const TDY*>(p.dy) + (r + q) * p.lddy;
      const TX* x = static_cast<const TX*>(p.x) + (r + q) * p.ldx;
      const TX* z = static_cast<const TX*>(p.res) + (r + q) * p.ldr;
      mean[q] = on ? p.mean[r + q] : 0.0f, rstd[q] = on ? p.rstd[r + q] : 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = lane + 32 * e;
        const bool in = on && c < p.k;
        dy[q][e] = in ? to_f32(d[c]) : 0.0f;
        xh[q][e] = in ? to_f32(x[c]) : mean[q];
        res[q][e] = p.res && in ? to_f32(z[c]) : 0.0f;
      }
    }
#pragma unroll
    for (int q = 0; q < RP; ++q) {
      float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (lane + 32 * e >= p.k) continue;
        xh[q][e] = (xh[q][e] - mean[q]) * rstd[q];
        const float a = dy[q][e] * gm[e];
        s1 += a;
        s2 = fmaf(a, xh[q][e], s2);
        dg[e] = fmaf(dy[q][e], xh[q][e], dg[e]);
        db[e] += dy[q][e];
      }
      sum[q] = warp_sum2(s1, s2);
    }
#pragma unroll
    for (int q = 0; q < RP; ++q) {
      if (r + q >= p.rows) break;
      const float c1 = -rstd[q] * (sum[q].x * inv_k), c2 = -rstd[q] * (sum[q].y * inv_k);
      TX* out = static_cast<TX*>(p.dx) + (r + q) * p.lddx;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (lane + 32 * e >= p.k) continue;
        const TX o = from_f32<TX>(fmaf(dy[q][e] * gm[e], rstd[q], fmaf(xh[q][e], c2, c1)) + res[q][e]);
        out[lane + 32 * e] = o;
        mag = max(mag, mag_bits(o));
      }
    }
  }
  const uint32_t m = block_max(mag, mags);
  if (p.partial) {
#pragma unroll
    for (int e = 0; e < E; ++e) acc[warp][0][lane + 32 * e] = dg[e], acc[warp][1][lane + 32 * e] = db[e];
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.k; i += LB_THREADS) {
      const int which = i >= p.k, c = which ? i - p.k : i;
      float s = 0.0f;
      for (int w = 0; w < WARPS; ++w) s += acc[w][which][c];
      p.partial[static_cast<int64_t>(blockIdx.x) * 2 * p.k + i] = s;
    }
  }
  publish_block(p, m, mag_out);
}

// First n0 columns of the blocks' partials [blocks][stride] to out0, the next
// n1 to out1 (either may be null), and the largest of their magnitudes to
// amax.  A block of 8 warps takes 32 columns; warp w sums the partials w, w +
// 8, ..., and the warps' sums are added in order.
__global__ void __launch_bounds__(256) sum_partials_kernel(const float* partial, int blocks, int64_t stride, int n0, int n1,
                                                           float* out0, float* out1, const uint32_t* mags, int n_mags,
                                                           float* amax) {
  __shared__ float part[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");      // launched as a programmatic dependent of the rows' kernel
  const int i = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (i < n0 + n1) {
#pragma unroll 8
    for (int b = warp; b < blocks; b += 8) s += __ldcg(partial + b * stride + i);
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && i < n0 + n1) {
#pragma unroll
    for (int w = 1; w < 8; ++w) s += part[w][lane];
    if (i < n0) {
      if (out0) out0[i] = s;
    } else if (out1) {
      out1[i - n0] = s;
    }
  }
  if (blockIdx.x == 0 && warp == 1 && amax) {
    uint32_t m = 0;
    for (int b = lane; b < n_mags; b += 32) m = max(m, __ldcg(mags + b));
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (lane == 0) *amax = __uint_as_float(m);
  }
}

constexpr int LN_CHUNKS = 64;
constexpr int LB_MAX_BLOCKS = 160;     // of the one-pass backward kernel; a workspace is sized for it

// A kernel's limit of dynamic shared memory is one for the function, whoever
// calls it: set to the most that any call of it asks for, never to a call's own
// size, which another thread's launch between the two steps would find too small.
template <typename Kernel>
cudaError_t allow_shared(Kernel kern, int most) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

// Launches a forward kernel for `need` blocks' worth of rows, `most` of them at
// a time.  Up to a cluster's blocks go as one cluster.
template <typename Kernel>
cudaError_t launch_forward(Kernel kern, LnParams p, int64_t need, int64_t most, int threads, int smem, int nt, cudaStream_t s) {
  if (need <= LF_MAX_CLUSTER) {
    most = LF_MAX_CLUSTER;
    p.joined = 1;
  }
  cudaError_t e = cudaSuccess;
  if (p.amax && !p.joined) e = cudaMemsetAsync(p.amax, 0, sizeof(float), s);
  if (e == cudaSuccess && smem > 0) e = allow_shared(kern, LI_SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(need < most ? need : most));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cfg.gridDim.x;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.joined ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p, nt);
}

template <typename TX, typename TY, typename TP, int NV, int THREADS>
cudaError_t run_forward_rows(const LnParams& p, cudaStream_t s) {
  const int per_warp = 32 * 8 * NV;
  const int nt = (p.k + per_warp - 1) / per_warp * 32;
  int groups = THREADS / nt;
  if (groups > p.rows) groups = static_cast<int>(p.rows);
  return launch_forward(ln_forward_rows_kernel<TX, TY, TP, NV, THREADS>, p, (p.rows + groups - 1) / groups,
                        static_cast<int64_t>(device_sm_count()) * lf_blocks<TX, NV>(THREADS), groups * nt, 0, nt, s);
}

template <typename TX, int NV, int THREADS>
cudaError_t run_forward(const LnParams& p, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  if (p.y_f32)
    return p.param_f32 ? run_forward_rows<TX, float, float, NV, THREADS>(p, s)
                       : run_forward_rows<TX, float, bf16, NV, THREADS>(p, s);
  return p.param_f32 ? run_forward_rows<TX, bf16, float, NV, THREADS>(p, s)
                     : run_forward_rows<TX, bf16, bf16, NV, THREADS>(p, s);
}

template <typename TY, int NV>
cudaError_t run_forward_image(const LnParams& p, int nt, int64_t group_bytes, int64_t params, cudaStream_t s) {
  const int64_t per_sm = NV <= 4 ? 2 : 1;                 // blocks per SM
  int64_t groups = LI_THREADS / nt;
  int64_t fit = (LI_SMEM / per_sm - params) / group_bytes;
  const bool shared_sm = fit >= 1;
  if (!shared_sm) fit = (LI_SMEM - params) / group_bytes;            // one block has the SM
  if (groups > fit) groups = fit;                         // also with fewer rows: all threads fetch gamma and beta
  return launch_forward(ln_forward_image_kernel<TY, NV>, p, (p.rows + groups - 1) / groups,
                        device_sm_count() * (shared_sm ? per_sm : 1), static_cast<int>(groups) * nt,
                        static_cast<int>(groups * group_bytes + params), nt, s);
}

template <typename TY, int NV>
bool try_forward_image(const LnParams& p, cudaStream_t s, cudaError_t* e) {
  const int per_warp = 32 * 8 * NV;
  const int nt = (p.k + per_warp - 1) / per_warp * 32;
  const int64_t row = odd_bytes(p.k, sizeof(__nv_bfloat16)), out = (p.k + 7) / 8 * 8 * static_cast<int64_t>(sizeof(TY));
  const int64_t params = (p.k + 7) / 8 * 64;
  if (nt > LI_THREADS || params + row + out > LI_SMEM) return false;
  *e = run_forward_image<TY, NV>(p, nt, row + out, params, s);
  return true;
}

template <typename TY, typename TP, int NT>
cudaError_t run_forward_odd(const LnParams& p, cudaStream_t s) {
  constexpr int THREADS = NT < 256 ? 256 : NT;
  const int64_t need = (p.rows + THREADS / NT - 1) / (THREADS / NT);
  return launch_forward(ln_forward_odd_kernel<TY, TP, NT>, p, need, static_cast<int64_t>(device_sm_count()) * (1024 / THREADS),
                        THREADS, 0, NT, s);
}

template <typename TY, typename TP>
cudaError_t dispatch_forward_odd(const LnParams& p, cudaStream_t s) {
  if (p.k <= 32 * LO_ELEMS) return run_forward_odd<TY, TP, 32>(p, s);
  if (p.k <= 64 * LO_ELEMS) return run_forward_odd<TY, TP, 64>(p, s);
  if (p.k <= 128 * LO_ELEMS) return run_forward_odd<TY, TP, 128>(p, s);
  if (p.k <= 256 * LO_ELEMS) return run_forward_odd<TY, TP, 256>(p, s);
  if (p.k <= 512 * LO_ELEMS) return run_forward_odd<TY, TP, 512>(p, s);
  return run_forward_odd<TY, TP, 1024>(p, s);
}

template <typename TX, typename TY>
cudaError_t run_forward_short(const LnParams& p, cudaStream_t s) {
  const int rp = p.k <= 64 ? 4 : 2;
  const int64_t need = (p.rows + 8 * rp - 1) / (8 * rp), most = static_cast<int64_t>(device_sm_count()) * 4;
  return p.k <= 64 ? launch_forward(ln_forward_short_kernel<TX, TY, 2>, p, need, most, 256, 0, 32, s)
                   : launch_forward(ln_forward_short_kernel<TX, TY, 8>, p, need, most, 256, 0, 32, s);
}

template <typename TX>
cudaError_t dispatch_forward(const LnParams& p, bool vec, cudaStream_t s) {
  // 32768 rows of 64: 12 us against 18 of the kernel for whole chunks, of 99: 19 against 28 of the one for odd rows;
  // of 200 in whole chunks: 33 against 19
  if (p.k <= 64 || (!vec && p.k <= LS_MAX_K)) return p.y_f32 ? run_forward_short<TX, float>(p, s) : run_forward_short<TX, __nv_bfloat16>(p, s);
  if (vec && p.k <= LF_THREADS * 32) return run_forward<TX, 4, LF_THREADS>(p, s);
  if (vec && p.k <= lf_max_k<4>()) return run_forward<TX, 4, 512>(p, s);
  if (vec && p.k <= LF_MAX_K) return run_forward<TX, 8, 512>(p, s);
  cudaError_t e;
  using bf16 = __nv_bfloat16;
  if constexpr (sizeof(TX) == 4) {
    if (!vec && p.k <= LO_MAX_K) {
      if (p.y_f32) return p.param_f32 ? dispatch_forward_odd<float, float>(p, s) : dispatch_forward_odd<float, bf16>(p, s);
      return p.param_f32 ? dispatch_forward_odd<bf16, float>(p, s) : dispatch_forward_odd<bf16, bf16>(p, s);
    }
  } else if (!vec && p.k <= LF_MAX_K) {
    if (p.k <= lf_max_k<4>()) {
      if (p.y_f32 ? try_forward_image<float, 4>(p, s, &e) : try_forward_image<bf16, 4>(p, s, &e)) return e;
    } else if (p.y_f32 ? try_forward_image<float, 8>(p, s, &e) : try_forward_image<bf16, 8>(p, s, &e)) {
      return e;
    }
  }
  if (p.amax) {
    e = cudaMemsetAsync(p.amax, 0, sizeof(float), s);
    if (e != cudaSuccess) return e;
  }
  const int grid = static_cast<int>(p.rows < 8 * device_sm_count() ? p.rows : 8 * device_sm_count());
  ln_forward_long_kernel<TX><<<grid, LN_THREADS, 0, s>>>(p);
  return cudaGetLastError();
}

// Every row of the operand starts on a 16-byte boundary.
bool rows_aligned16(const void* p, int64_t ld, bool f32) { return aligned16(p) && (ld * (f32 ? 4 : 2)) % 16 == 0; }

template <typename TX, typename TDY>
cudaError_t run_backward_long(const LnBwdParams& p, float* dgamma, float* dbeta, cudaStream_t s) {
  if (p.amax) {
    const cudaError_t e = cudaMemsetAsync(p.amax, 0, sizeof(float), s);
    if (e != cudaSuccess) return e;
  }
  const int grid = static_cast<int>(p.rows < 8 * device_sm_count() ? p.rows : 8 * device_sm_count());
  ln_backward_dx_long_kernel<TX><<<grid, LN_THREADS, 0, s>>>(p);
  if (p.partial) {
    const int per = static_cast<int>((p.rows + LN_CHUNKS - 1) / LN_CHUNKS);
    const int chunks = static_cast<int>((p.rows + per - 1) / per);
    const int cols = (p.k + LN_THREADS - 1) / LN_THREADS;
    ln_backward_params_long_kernel<TX><<<dim3(cols, chunks), LN_THREADS, 0, s>>>(p, per);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_sum_partials(p.partial, chunks, 2 * static_cast<int64_t>(p.k), p.k, p.k, dgamma, dbeta, nullptr, 0, nullptr, s);
  }
  return cudaGetLastError();
}

// Rows that start anywhere, fp32 dy and x: up to LB_ODD_K elements the kernel
// without a ring takes them at every size (dispatch_backward), so only rows cut
// between blocks are left for the ring.
template <typename TX, typename TDY, bool kOdd>
constexpr bool kRingAlone = !(kOdd && sizeof(TX) + sizeof(TDY) == 8);

// A launch of the one-pass backward kernel: rows cut between `cluster` blocks.
template <typename TX, typename TDY, bool kOdd, int S>
cudaError_t run_backward_rows(const LnBwdParams& p, int cluster, int kc, float* dgamma, float* dbeta, uint32_t* mags,
                              cudaStream_t s) {
  const int per_warp = 32 * 8 * LB_NV;
  const int nt = (kc + per_warp - 1) / per_warp * 32;
  const int64_t each = lb_group_bytes<TX, TDY, kOdd, S>(kc, nt, p.res != nullptr);
  int64_t groups = cluster > 1 ? 1 : LB_THREADS / nt;
  if (groups > LB_SMEM / each) groups = LB_SMEM / each;
  if (groups > p.rows) groups = p.rows;
  int64_t smem = groups * each;
  if (groups * 2 * kc * 4 > smem) smem = groups * 2 * kc * 4;        // the column sums
  const int64_t sms = (device_sm_count() < LB_MAX_BLOCKS ? device_sm_count() : LB_MAX_BLOCKS) / cluster;
  const int64_t need = (p.rows + groups - 1) / groups;
  const int blocks = static_cast<int>(need < sms ? need : sms) * cluster;
  auto kern = ln_backward_rows_kernel<TX, TDY, kOdd, true, S>;
  if constexpr (kRingAlone<TX, TDY, kOdd>)
    if (cluster == 1) kern = ln_backward_rows_kernel<TX, TDY, kOdd, false, S>;
  static_assert(LB_THREADS * 8 * LB_NV * 2 * 4 <= LB_SMEM, "the column sums of all groups fit where the rings do");
  cudaError_t e = allow_shared(kern, LB_SMEM);
  // the sum over blocks also joins their maxima: only without it has *amax to be cleared
  if (e == cudaSuccess && p.amax && !p.partial) e = cudaMemsetAsync(p.amax, 0, sizeof(float), s);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(groups * nt));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, p, nt, kc, mags);
  if (e != cudaSuccess || !p.partial) return e;
  return launch_sum_partials(p.partial, blocks / cluster, 2 * static_cast<int64_t>(p.k), p.k, p.k, dgamma, dbeta, mags, blocks,
                             p.amax, s);
}

// The smallest cluster whose blocks hold their share of a row and a ring of
// it: four stages, or three or two of long rows.
template <typename TX, typename TDY, bool kOdd>
bool try_backward_rows(const LnBwdParams& p, float* dgamma, float* dbeta, uint32_t* mags, cudaStream_t s, cudaError_t* e) {
  for (int cluster = kRingAlone<TX, TDY, kOdd> ? 1 : 2; cluster <= LB_MAX_CLUSTER; cluster *= 2) {
    const int64_t kc = ((static_cast<int64_t>(p.k) + cluster - 1) / cluster + 7) / 8 * 8;
    if (kc > LB_MAX_COLS || kc * (cluster - 1) >= p.k) continue;
    const int cols = static_cast<int>(kc);
    const int per_warp = 32 * 8 * LB_NV;
    const int nt = (cols + per_warp - 1) / per_warp * 32;
    const bool res = p.res != nullptr;
    if (lb_group_bytes<TX, TDY, kOdd, 4>(cols, nt, res) <= LB_SMEM)
      *e = run_backward_rows<TX, TDY, kOdd, 4>(p, cluster, cols, dgamma, dbeta, mags, s);
    else if (lb_group_bytes<TX, TDY, kOdd, 3>(cols, nt, res) <= LB_SMEM)
      *e = run_backward_rows<TX, TDY, kOdd, 3>(p, cluster, cols, dgamma, dbeta, mags, s);
    else if (lb_group_bytes<TX, TDY, kOdd, 2>(cols, nt, res) <= LB_SMEM)
      *e = run_backward_rows<TX, TDY, kOdd, 2>(p, cluster, cols, dgamma, dbeta, mags, s);
    else
      continue;
    return true;
  }
  return false;
}

template <typename TX, typename TDY>
cudaError_t run_backward_short(const LnBwdParams& p, float* dgamma, float* dbeta, uint32_t* mags, cudaStream_t s) {
  const int64_t need = (p.rows + LB_SHORT_ROWS - 1) / LB_SHORT_ROWS;
  const int64_t most = device_sm_count() < LB_MAX_BLOCKS ? device_sm_count() : LB_MAX_BLOCKS;
  const int blocks = static_cast<int>(need < most ? need : most);
  cudaError_t e = cudaSuccess;
  if (p.amax && !p.partial) e = cudaMemsetAsync(p.amax, 0, sizeof(float), s);
  if (e != cudaSuccess) return e;
  ln_backward_short_kernel<TX, TDY><<<blocks, LB_THREADS, 0, s>>>(p, mags);
  e = cudaGetLastError();
  if (e != cudaSuccess || !p.partial) return e;
  return launch_sum_partials(p.partial, blocks, 2 * static_cast<int64_t>(p.k), p.k, p.k, dgamma, dbeta, mags, blocks, p.amax, s);
}

template <typename TX, typename TDY, typename TP, int NT>
cudaError_t run_backward_odd(const LnBwdParams& p, float* dgamma, float* dbeta, uint32_t* mags, cudaStream_t s) {
  constexpr int GROUPS = LB_THREADS / NT;
  const int64_t need = (p.rows + GROUPS - 1) / GROUPS;
  const int64_t most = device_sm_count() < LB_MAX_BLOCKS ? device_sm_count() : LB_MAX_BLOCKS;
  const int blocks = static_cast<int>(need < most ? need : most);
  const int smem = p.partial ? GROUPS * 2 * p.k * static_cast<int>(sizeof(float)) : 0;
  auto kern = ln_backward_odd_kernel<TX, TDY, TP, NT>;
  cudaError_t e = allow_shared(kern, LB_THREADS * LB_ODD_ELEMS * 2 * static_cast<int>(sizeof(float)));   // GROUPS * k at most
  if (e == cudaSuccess && p.amax && !p.partial) e = cudaMemsetAsync(p.amax, 0, sizeof(float), s);
  if (e != cudaSuccess) return e;
  kern<<<blocks, LB_THREADS, smem, s>>>(p, mags);
  e = cudaGetLastError();
  if (e != cudaSuccess || !p.partial) return e;
  return launch_sum_partials(p.partial, blocks, 2 * static_cast<int64_t>(p.k), p.k, p.k, dgamma, dbeta, mags, blocks, p.amax, s);
}

template <typename TX, typename TDY, typename TP>
cudaError_t dispatch_backward_odd(const LnBwdParams& p, float* dgamma, float* dbeta, uint32_t* mags, cudaStream_t s) {
  if (p.k <= 32 * LB_ODD_ELEMS) return run_backward_odd<TX, TDY, TP, 32>(p, dgamma, dbeta, mags, s);
  if (p.k <= 64 * LB_ODD_ELEMS) return run_backward_odd<TX, TDY, TP, 64>(p, dgamma, dbeta, mags, s);
  if (p.k <= 128 * LB_ODD_ELEMS) return run_backward_odd<TX, TDY, TP, 128>(p, dgamma, dbeta, mags, s);
  if (p.k <= 256 * LB_ODD_ELEMS) return run_backward_odd<TX, TDY, TP, 256>(p, dgamma, dbeta, mags, s);
  return run_backward_odd<TX, TDY, TP, 512>(p, dgamma, dbeta, mags, s);
}

template <typename TX, typename TDY>
cudaError_t dispatch_backward(const LnBwdParams& p, bool vec, float* dgamma, float* dbeta, uint32_t* mags, cudaStream_t s) {
  if (p.k <= LB_SHORT_K) return run_backward_short<TX, TDY>(p, dgamma, dbeta, mags, s);
  // The kernel without a ring: fp32 rows at every size, whose accesses fill whole sectors (1500 x 1155 13.9 us against
  // 23.9 of the ring, 20000 x 1155 88 against 176, 3000 x 8001 105 against 196).  With a 16-bit type up to 2^23 bytes of dy
  // and x.  Where these lie in L2, behind the kernels that wrote them, its blocks' earlier start wins (device time, without
  // and ring): bf16 100 x 1155 8.4 and 11.2 us, 1537 x 1155 (7 MB) 14.9 and 17.5, 8000 x 301 (10 MB) 16.5 and 19.9, 20000 x
  // 1155 (92 MB) 153 and 93.  Out of memory the ring's loads ahead win earlier: 100 x 1155 10.1 and 11.5, 4000 x 301 (5 MB)
  // 14.0 and 15.6, 1537 x 1155 20.6 and 17.7, 8000 x 301 22.1 and 21.9, 3000 x 1155 (14 MB) 33.4 and 23.6.  The bound lies
  // between the two; fp32 with bf16 likewise (1537 x 1155, 11 MB: 16.1 and 18.8 out of L2, 24.5 and 19.5 out of memory).
  if (!vec && p.k <= LB_ODD_K &&
      (!kRingAlone<TX, TDY, true> ||
       p.rows * p.k * static_cast<int64_t>(sizeof(TX) + sizeof(TDY)) <= (int64_t{1} << 23)))
    return p.param_f32 ? dispatch_backward_odd<TX, TDY, float>(p, dgamma, dbeta, mags, s)
                       : dispatch_backward_odd<TX, TDY, __nv_bfloat16>(p, dgamma, dbeta, mags, s);
  cudaError_t e = cudaSuccess;
  if (vec ? try_backward_rows<TX, TDY, false>(p, dgamma, dbeta, mags, s, &e)
          : try_backward_rows<TX, TDY, true>(p, dgamma, dbeta, mags, s, &e))
    return e;
  return run_backward_long<TX, TDY>(p, dgamma, dbeta, s);
}

}  // namespace

cudaError_t launch_sum_partials(const float* partial, int blocks, int64_t stride, int n0, int n1, float* out0, float* out1,
                                const uint32_t* mags, int n_mags, float* amax, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(n0) + n1 + 31) / 32));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sum_partials_kernel, partial, blocks, stride, n0, n1, out0, out1, mags, n_mags, amax);
}

// [blocks][2][k] partials, then one magnitude per block.
size_t layernorm_backward_workspace_bytes(int64_t rows, int64_t k) {
  const int64_t blocks = k > LB_MAX_K ? LN_CHUNKS : LB_MAX_BLOCKS;
  return static_cast<size_t>(round_up(blocks * 2 * k * 4, 256) + round_up(4 * LB_MAX_BLOCKS, 256));
}

nvfp4_status launch_layernorm(const LayerNorm& a, cudaStream_t s) {
  if (a.rows == 0) return a.amax ? launch_status(cudaMemsetAsync(a.amax, 0, sizeof(float), s)) : NVFP4_OK;
  const bool xf = a.x_dtype == NVFP4_DTYPE_F32, yf = a.y_dtype == NVFP4_DTYPE_F32;
  const LnParams p{a.x, a.ldx, a.gamma, a.beta, a.param_dtype == NVFP4_DTYPE_F32, a.eps, a.y, a.ldy,
                   yf, a.mean, a.rstd, a.amax, a.rows, static_cast<int>(a.k), 0};
  const bool vec = a.k % 8 == 0 && rows_aligned16(a.x, a.ldx, xf) && rows_aligned16(a.y, a.ldy, yf) && aligned16(a.gamma) && aligned16(a.beta);
  return launch_status(xf ? dispatch_forward<float>(p, vec, s) : dispatch_forward<__nv_bfloat16>(p, vec, s));
}

nvfp4_status launch_layernorm_backward(const LayerNormBackward& a, cudaStream_t s) {
  const bool sums = a.dgamma || a.dbeta;
  cudaError_t e = cudaSuccess;
  if (a.rows == 0) {
    if (a.amax) e = cudaMemsetAsync(a.amax, 0, sizeof(float), s);
    if (e == cudaSuccess && a.dgamma) e = cudaMemsetAsync(a.dgamma, 0, a.k * sizeof(float), s);
    if (e == cudaSuccess && a.dbeta) e = cudaMemsetAsync(a.dbeta, 0, a.k * sizeof(float), s);
    return launch_status(e);
  }
  const bool xf = a.x_dtype == NVFP4_DTYPE_F32, df = a.dy_dtype == NVFP4_DTYPE_F32;
  const LnBwdParams p{a.dy, a.lddy, df, a.x, a.ldx, a.mean, a.rstd, a.gamma,
                      a.param_dtype == NVFP4_DTYPE_F32, a.residual, a.ldr, a.dx, a.lddx,
                      sums ? static_cast<float*>(a.workspace) : nullptr, a.amax, a.rows, static_cast<int>(a.k)};
  const bool vec = a.k % 8 == 0 && rows_aligned16(a.dy, a.lddy, df) && rows_aligned16(a.x, a.ldx, xf) && rows_aligned16(a.dx, a.lddx, xf) &&
                   aligned16(a.gamma) && (!a.residual || rows_aligned16(a.residual, a.ldr, xf));
  uint32_t* mags = sums ? reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.workspace) +
                                                      layernorm_backward_workspace_bytes(a.rows, a.k) -
                                                      round_up(4 * LB_MAX_BLOCKS, 256))
                        : nullptr;
  using bf16 = __nv_bfloat16;
  if (xf)
    e = df ? dispatch_backward<float, float>(p, vec, a.dgamma, a.dbeta, mags, s)
           : dispatch_backward<float, bf16>(p, vec, a.dgamma, a.dbeta, mags, s);
  else
    e = df ? dispatch_backward<bf16, float>(p, vec, a.dgamma, a.dbeta, mags, s)
           : dispatch_backward<bf16, bf16>(p, vec, a.dgamma, a.dbeta, mags, s);
  return launch_status(e);
}

}  // namespace nvfp4
