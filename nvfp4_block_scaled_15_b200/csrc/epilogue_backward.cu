// Gradient of the product epilogue D = act(pre) [+ residual], pre = alpha acc + bias:
//   dpre = dD act'(pre),  dbias = sum over rows of dpre  (dresidual = dD)
//
// A block takes a strip of columns over a chunk of rows; a thread the same
// columns of every row, so dbias is a sum in its registers.  The chunks' sums
// leave as partials that sum_partials_kernel adds in order: results do not
// depend on timing.  Bound by memory where rows are aligned (three tensors,
// 4096 x 28672 bf16); the activation's ex2 and rcp take half of that time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "epilogue.cuh"
#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int EB_THREADS = 256;
constexpr int EB_WARPS = EB_THREADS / 32;
constexpr int EB_BLOCKS_PER_SM = 4;
constexpr int EB_MAX_CHUNKS = 64;
constexpr int EB_MAX_BLOCKS = 4096;    // of a grid whose columns alone need fewer; a workspace is sized for it
constexpr int EO_COLS = 4;             // columns of a thread whose rows start anywhere, 32 apart
constexpr int EO_BLOCKS_PER_SM = 3;

struct EpiBwdParams {
  const void* dd;
  int64_t ldd;
  const void* pre;
  int64_t ldp;
  int act;
  void* dpre;            // null: only dbias
  int64_t lddp;
  float* partial;        // [chunks][N], null: no dbias
  uint32_t* mags;        // [blocks] largest |dpre| as fp32 bits, with partial
  float* amax;
  int64_t M;
  int N;
  int rows_per_chunk;
};

__device__ __forceinline__ void publish_block_mag(const EpiBwdParams& p, uint32_t mag, uint32_t* warp_mags) {
  if (!p.amax) return;
  mag = __reduce_max_sync(0xFFFFFFFFu, mag);
  if ((threadIdx.x & 31) == 0) warp_mags[threadIdx.x >> 5] = mag;
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int w = 1; w < EB_WARPS; ++w) mag = max(mag, warp_mags[w]);
  if (p.mags)
    p.mags[blockIdx.y * gridDim.x + blockIdx.x] = mag;      // joined by the sum over chunks
  else
    atomicMax(reinterpret_cast<unsigned int*>(p.amax), mag);
}

// 8 elements; not through the read-only path, since dpre may be dd.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
template <typename T>
__device__ __forceinline__ void load_raw(Raw8<T>& x, const T* p) {
#pragma unroll
  for (int h = 0; h < static_cast<int>(sizeof(T)) / 2; ++h) x.w[h] = ld_stream(p + h * (16 / sizeof(T)));
}
template <typename T>
__device__ __forceinline__ Chunk chunk_of(const Raw8<T>& x) {
  if constexpr (sizeof(T) == 2) {
    return unpack_chunk(x.w[0]);
  } else {
    Chunk c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      c.v[2 * h] = make_float2(__uint_as_float(x.w[h].x), __uint_as_float(x.w[h].y));
      c.v[2 * h + 1] = make_float2(__uint_as_float(x.w[h].z), __uint_as_float(x.w[h].w));
    }
    return c;
  }
}

// Rows of whole 16-byte aligned 8-element chunks: a warp takes 256 columns (8
// per lane) of rows w, w + 8, ... of the chunk, U rows' loads in flight.
template <typename T, int kAct>
__global__ void __launch_bounds__(EB_THREADS, EB_BLOCKS_PER_SM) epilogue_backward_kernel(const EpiBwdParams p) {
  constexpr int U = 2;
  const int down = static_cast<int>(blockDim.x >> 5);    // rows between a warp's; as a constant it measured slower (131 against 124 us)
  __shared__ float4 sums[EB_WARPS][2][32];
  __shared__ uint32_t warp_mags[EB_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 256 + lane * 8;
  const bool in = c < p.N;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * p.rows_per_chunk;
  const int64_t r1 = min(p.M, r0 + p.rows_per_chunk);
  const T* dd = static_cast<const T*>(p.dd) + c;
  const T* pre = static_cast<const T*>(p.pre) + c;
  T* dpre = static_cast<T*>(p.dpre) + c;
  Chunk s;
#pragma unroll
  for (int i = 0; i < 4; ++i) s.v[i] = both(0.0f);
  Mag<T> mag;
  if (in) {
    for (int64_t r = r0 + warp; r < r1; r += U * down) {
      Raw8<T> a[U], b[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t q = r + u * down;
        if (q < r1) {
          load_raw(a[u], dd + q * p.ldd);
          if constexpr (kAct != NVFP4_ACT_NONE) load_raw(b[u], pre + q * p.ldp);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t q = r + u * down;
        if (q >= r1) break;
        Chunk d = chunk_of(a[u]);
        if constexpr (kAct != NVFP4_ACT_NONE) {
          const Chunk v = chunk_of(b[u]);
#pragma unroll
          for (int i = 0; i < 4; ++i) d.v[i] = mul2(d.v[i], slope_pair<kAct>(v.v[i]));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s.v[i] = add2(s.v[i], d.v[i]);
        store_chunk<T>(p.dpre ? dpre + q * p.lddp : nullptr, d, mag);
      }
    }
  }
  if (p.partial) {
    sums[warp][0][lane] = make_float4(s.v[0].x, s.v[0].y, s.v[1].x, s.v[1].y);
    sums[warp][1][lane] = make_float4(s.v[2].x, s.v[2].y, s.v[3].x, s.v[3].y);
    __syncthreads();
    // thread i adds the warps' sums of column i of the strip: lane i / 8, element i % 8
    const int i = threadIdx.x;
    const float* first = reinterpret_cast<const float*>(&sums[0][(i >> 2) & 1][i >> 3]) + (i & 3);
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < EB_WARPS; ++w) sum += first[w * 2 * 32 * 4];
    const int col = blockIdx.x * 256 + i;
    if (col < p.N) p.partial[static_cast<int64_t>(blockIdx.y) * p.N + col] = sum;
  }
  publish_block_mag(p, mag.bits(), warp_mags);
}

// Rows that start anywhere: a thread takes EO_COLS columns 32 apart, a warp's
// accesses are 32 neighbouring elements; EO_COLS x U elements' loads in flight.
template <typename T, int kAct>
__global__ void __launch_bounds__(EB_THREADS, EO_BLOCKS_PER_SM) epilogue_backward_odd_kernel(const EpiBwdParams p) {
  constexpr int U = 4;
  __shared__ float sums[EB_WARPS][EO_COLS][32];
  __shared__ uint32_t warp_mags[EB_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = blockIdx.x * (32 * EO_COLS) + lane;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * p.rows_per_chunk;
  const int64_t r1 = min(p.M, r0 + p.rows_per_chunk);
  const T* dd = static_cast<const T*>(p.dd) + c0;
  const T* pre = static_cast<const T*>(p.pre) + c0;
  T* dpre = static_cast<T*>(p.dpre) + c0;
  float s[EO_COLS];
  bool in[EO_COLS];
#pragma unroll
  for (int j = 0; j < EO_COLS; ++j) s[j] = 0.0f, in[j] = c0 + 32 * j < p.N;
  uint32_t mag = 0;
  for (int64_t r = r0 + warp; r < r1; r += U * EB_WARPS) {
    T a[U][EO_COLS], b[U][EO_COLS];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t q = r + u * EB_WARPS;
#pragma unroll
      for (int j = 0; j < EO_COLS; ++j) {
        const bool on = in[j] && q < r1;
        a[u][j] = on ? dd[q * p.ldd + 32 * j] : from_f32<T>(0.0f);
        b[u][j] = kAct != NVFP4_ACT_NONE && on ? pre[q * p.ldp + 32 * j] : from_f32<T>(0.0f);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t q = r + u * EB_WARPS;
      if (q >= r1) break;
#pragma unroll
      for (int j = 0; j < EO_COLS; j += 2) {
        float2 d = make_float2(to_f32(a[u][j]), to_f32(a[u][j + 1]));
        if constexpr (kAct != NVFP4_ACT_NONE) d = mul2(d, slope_pair<kAct>(make_float2(to_f32(b[u][j]), to_f32(b[u][j + 1]))));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!in[j + h]) continue;
          const float v = h ? d.y : d.x;
          s[j + h] += v;
          const T o = from_f32<T>(v);
          if (p.dpre) dpre[q * p.lddp + 32 * (j + h)] = o;
          mag = max(mag, mag_bits(o));
        }
      }
    }
  }
  if (p.partial) {
#pragma unroll
    for (int j = 0; j < EO_COLS; ++j) sums[warp][j][lane] = s[j];
    __syncthreads();
    if (warp < EO_COLS && c0 + 32 * warp < p.N) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < EB_WARPS; ++w) sum += sums[w][warp][lane];
      p.partial[static_cast<int64_t>(blockIdx.y) * p.N + c0 + 32 * warp] = sum;
    }
  }
  publish_block_mag(p, mag, warp_mags);
}

template <typename T, int kAct>
void launch_rows(const EpiBwdParams& p, bool vec, dim3 grid, cudaStream_t s) {
  if (vec)
    epilogue_backward_kernel<T, kAct><<<grid, EB_THREADS, 0, s>>>(p);
  else
    epilogue_backward_odd_kernel<T, kAct><<<grid, EB_THREADS, 0, s>>>(p);
}

template <typename T>
void launch_act(const EpiBwdParams& p, bool vec, dim3 grid, cudaStream_t s) {
  switch (p.act) {
    case NVFP4_ACT_RELU: return launch_rows<T, NVFP4_ACT_RELU>(p, vec, grid, s);
    case NVFP4_ACT_GELU: return launch_rows<T, NVFP4_ACT_GELU>(p, vec, grid, s);
    case NVFP4_ACT_GELU_TANH: return launch_rows<T, NVFP4_ACT_GELU_TANH>(p, vec, grid, s);
    case NVFP4_ACT_SILU: return launch_rows<T, NVFP4_ACT_SILU>(p, vec, grid, s);
    default: return launch_rows<T, NVFP4_ACT_NONE>(p, vec, grid, s);
  }
}

// Chunks of rows: the fewest whose blocks fill the last wave of SMs to within a
// few percent (4096 x 28672, 112 strips: one wave of three chunks leaves a
// quarter of the SMs idle), each of at least two rows per warp.
int64_t chunk_count(int64_t strips, int64_t M, bool vec) {
  const int64_t slots = static_cast<int64_t>(device_sm_count()) * (vec ? EB_BLOCKS_PER_SM : EO_BLOCKS_PER_SM);
  int64_t most = EB_MAX_BLOCKS / strips;
  const int64_t by_rows = (M + 2 * EB_WARPS - 1) / (2 * EB_WARPS);
  if (most > by_rows) most = by_rows;
  if (most > EB_MAX_CHUNKS) most = EB_MAX_CHUNKS;
  int64_t best = 1;
  double best_fill = 0.0;
  for (int64_t c = 1; c <= most; ++c) {
    const int64_t blocks = strips * c, waves = (blocks + slots - 1) / slots;
    const double fill = static_cast<double>(blocks) / static_cast<double>(waves * slots);
    if (fill > best_fill + 0.02) best = c, best_fill = fill;
  }
  return best;
}

// Most blocks that a grid for N columns has.
int64_t most_blocks(int64_t N) {
  const int64_t strips = (N + 32 * EO_COLS - 1) / (32 * EO_COLS);     // the narrower strips
  return strips > EB_MAX_BLOCKS ? strips : EB_MAX_BLOCKS;
}

}  // namespace

// [chunks][N] partials, then one magnitude per block.
size_t epilogue_backward_workspace_bytes(int64_t M, int64_t N) {
  const int64_t chunks = M < EB_MAX_CHUNKS ? (M > 0 ? M : 1) : EB_MAX_CHUNKS;
  return static_cast<size_t>(round_up(chunks * N * 4, 256) + round_up(4 * most_blocks(N), 256));
}

nvfp4_status launch_epilogue_backward(const EpilogueBackward& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  // with dbias the last kernel also joins the blocks' maxima: no clearing needed
  if (a.amax && (a.M == 0 || !a.dbias)) e = cudaMemsetAsync(a.amax, 0, sizeof(float), s);
  if (a.M == 0) {
    if (e == cudaSuccess && a.dbias) e = cudaMemsetAsync(a.dbias, 0, a.N * sizeof(float), s);
    return launch_status(e);
  }
  if (e != cudaSuccess) return launch_status(e);
  const bool f32 = a.dtype == NVFP4_DTYPE_F32;
  const auto aligned = [&](const void* q, int64_t ld) { return aligned16(q) && (ld * (f32 ? 4 : 2)) % 16 == 0; };
  const bool vec = a.N % 8 == 0 && aligned(a.dd, a.ldd) && (a.act == NVFP4_ACT_NONE || aligned(a.pre, a.ldp)) &&
                   (!a.dpre || aligned(a.dpre, a.lddp));
  const int width = vec ? 256 : 32 * EO_COLS;
  const int64_t strips = (a.N + width - 1) / width;
  int64_t chunks = chunk_count(strips, a.M, vec);
  const int64_t per = (a.M + chunks - 1) / chunks;
  chunks = (a.M + per - 1) / per;
  EpiBwdParams p{a.dd, a.ldd, a.pre, a.ldp, a.act, a.dpre, a.lddp,
                 a.dbias ? static_cast<float*>(a.workspace) : nullptr, nullptr, a.amax, a.M, static_cast<int>(a.N),
                 static_cast<int>(per)};
  if (a.dbias)
    p.mags = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.workspace) + epilogue_backward_workspace_bytes(a.M, a.N) -
                                         round_up(4 * most_blocks(a.N), 256));
  const dim3 grid(static_cast<unsigned>(strips), static_cast<unsigned>(chunks));
  if (f32)
    launch_act<float>(p, vec, grid, s);
  else
    launch_act<__nv_bfloat16>(p, vec, grid, s);
  e = cudaGetLastError();
  if (e == cudaSuccess && a.dbias)
    e = launch_sum_partials(p.partial, static_cast<int>(chunks), a.N, static_cast<int>(a.N), 0, a.dbias, nullptr, p.mags,
                            static_cast<int>(strips * chunks), a.amax, s);
  return launch_status(e);
}

}  // namespace nvfp4
