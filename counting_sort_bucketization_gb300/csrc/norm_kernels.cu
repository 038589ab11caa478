// norm_kernels.cu -- root-mean-square norm of the residual stream, and its gradient.
//
//   forward   z = x + residual, rounded to the stream's type (bf16 or fp32) and kept;
//             r = 1 / sqrt(mean_j z_j^2 + eps); y = z r w, in bf16, in e4m3 with one fp32
//             scale for each 1x128 block (as quantize_rows makes them, from the 32-bit
//             y), or both
//   gradient  g = dy w, h = z r: dz = r (g - h mean_j(g_j h_j)) + dresidual,
//             dw_j = sum over rows of dy_j h_j
//
// The norm is of the rounded z, which is what the next layer and the gradient read.
//
// A row's threads hold it in registers as it was loaded, 16 bytes of bf16 a thread and step (16
// threads have a scale block), so it is read once; a warp has a row of up to 1024 columns, a
// CTA a longer one.  Statistics are fp32 sums in a fixed order; each rounding to 16 or 8 bits is
// the one that the output's type asks for.
//
// HBM bound: 9 bytes a value (bf16 stream, both outputs), the gradient 8.  One call after another:
//   32768 x 4096   178 us, 6.8 TB/s (a copy's rate); stream in fp32 250, 7.0
//   32768 x 7168   305, 7.0;  508, 6.0          16384 x 16384  367, 6.6;  766, 4.6
//   8192 x 32768   394, 6.2;  770, 4.5
// the gradient with the weight's
//   32768 x 4096   176, 6.1;  284, 6.6          32768 x 7168   331, 5.7;  603, 5.5
//   16384 x 16384  375, 5.7;  730, 5.2          8192 x 32768   592, 3.6; 1410, 2.7
// The weight's sums take the registers of the warps that would fill the gradient's phases.  Past
// 8192 columns (the gradient: 16384) a thread has eight vectors, which in fp32 leave one CTA
// an SM; past 16384 they no longer fit its registers in fp32 (176 bytes of spills a thread), nor
// in the gradient (488, fp32 740).  64 x 7168: 8 us a call, of which the host takes 7.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxRowThreads = 512;
constexpr int kShortThreads = 256;       // of a CTA whose warps have a row each

// Eight values of the stream as they were loaded.
template <bool FP32>
struct Raw8 {
  uint4 v[FP32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    if constexpr (FP32) {
      v[0] = load_v4(static_cast<const float*>(base) + at);
      v[1] = load_v4(static_cast<const float*>(base) + at + 4);
    } else {
      v[0] = load_v4(static_cast<const uint16_t*>(base) + at);
    }
  }
  // Rounds to the stream's type.
  __device__ __forceinline__ void set(const float* f) {
    if constexpr (FP32) {
      v[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
      v[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
    } else {
      v[0] = pack8(f);
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t at) const {
    if constexpr (FP32) {
      ptx::st_v4(static_cast<float*>(base) + at, v[0]);
      ptx::st_v4(static_cast<float*>(base) + at + 4, v[1]);
    } else {
      ptx::st_v4(static_cast<uint16_t*>(base) + at, v[0]);
    }
  }
  __device__ __forceinline__ void get(float* f) const {
    if constexpr (FP32) {
      f[0] = __uint_as_float(v[0].x), f[1] = __uint_as_float(v[0].y), f[2] = __uint_as_float(v[0].z), f[3] = __uint_as_float(v[0].w);
      f[4] = __uint_as_float(v[1].x), f[5] = __uint_as_float(v[1].y), f[6] = __uint_as_float(v[1].z), f[7] = __uint_as_float(v[1].w);
    } else {
      unpack8(v[0], f);
    }
  }
};
// Eight of the weight: read by every row, so they may stay in the L1.
__device__ __forceinline__ void load_weight(const NormArgs& a, int64_t at, float* f) {
  if (a.weight_fp32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.weight) + at);
    const float4 x = __ldg(p), y = __ldg(p + 1);
    f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w, f[4] = y.x, f[5] = y.y, f[6] = y.z, f[7] = y.w;
  } else {
    unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.weight) + at)), f);
  }
}
__device__ __forceinline__ void store_fp32(float* p, const float* f) {
  ptx::st_v4(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
  ptx::st_v4(p + 4, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])));
}

// The sum over a row's threads, the same in all of them and in a fixed order.  `part` has
// a word a warp; with ROW_WARPS a row's threads are the CTA's.
template <bool CTA_ROW>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  if constexpr (CTA_ROW) {
    __syncthreads();                     // the last sum is read
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.0f;
    for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) v += part[w];
  }
  return v;
}

// MAXT: threads of a row at most; 32: each warp of a CTA has a row.  A CTA a row (or eight):
// a wave of CTAs that walk the rows, with the next row's copies under way, took 200 us in
// place of 182 on 32768 x 4096, 330 in place of 254 with the stream in fp32 (L2 flushed): SMs are
// not equally fast, and the block scheduler evens that out.
template <int NV, int MAXT, bool FP32>
__global__ void __launch_bounds__(MAXT == 32 ? kShortThreads : MAXT, NV <= 4 ? 4 : 1) norm_kernel(NormArgs a) {
  constexpr bool CTA_ROW = MAXT > 32;
  __shared__ float part[kMaxRowThreads / 32];
  ptx::grid_dependency_wait();
  const int threads = CTA_ROW ? static_cast<int>(blockDim.x) : 32;
  const int tid = CTA_ROW ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x) % 32;
  int64_t rows = a.rows;
  if (a.total_rows != nullptr) rows = min64(rows, *a.total_rows);
  const int64_t row = CTA_ROW ? static_cast<int64_t>(blockIdx.x)
                              : static_cast<int64_t>(blockIdx.x) * (kShortThreads / 32) + threadIdx.x / 32;
  if (row >= rows) return;               // a whole CTA, or a whole warp
  const int64_t base = row * a.cols;
  const int cols = static_cast<int>(a.cols);
  Raw8<false> x[NV];
  Raw8<FP32> z[NV];                      // the residual, then z
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = 8 * (j * threads + tid);
    if (c < cols) {
      x[j].load(a.x, base + c);
      if (a.residual != nullptr) z[j].load(a.residual, base + c);
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = 8 * (j * threads + tid);
    if (c >= cols) break;
    float f[8];
    x[j].get(f);
    if (a.residual != nullptr) {
      float g[8];
      z[j].get(g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] += g[i];
    }
    z[j].set(f);
    if (a.residual != nullptr) z[j].store(a.residual_out, base + c);
    z[j].get(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(f[i], f[i], sum);
  }
  sum = row_sum<CTA_ROW>(sum, part);
  float r = 1.0f / sqrtf(sum / static_cast<float>(cols) + a.eps);
  if (!(sum < INFINITY)) {               // squares beyond fp32: eps, at most 2^88, is nothing beside a mean from 2^113 on
    sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (8 * (j * threads + tid) >= cols) break;
      float f[8];
      z[j].get(f);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(f[i] * 0x1p-80f, f[i] * 0x1p-80f, sum);
    }
    sum = row_sum<CTA_ROW>(sum, part);
    r = 0x1p-80f / sqrtf(sum / static_cast<float>(cols));
  }
  if (a.rstd != nullptr && tid == 0) a.rstd[row] = r;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = 8 * (j * threads + tid);
    const bool in = c < cols;
    float f[8] = {};
    if (in) {
      float w[8];
      load_weight(a, c, w);
      z[j].get(f);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = f[i] * r * w[i];
      if (a.y != nullptr) ptx::st_v4(a.y + base + c, pack8(f));
    }
    if (a.q != nullptr) {
      float m = kAmaxFloor;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(f[i]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(kFull, m, o));
      const float sf = __fdiv_rn(m, kE4m3Max);
      const float inv = __fdiv_rn(1.0f, sf);
      if (in) {
        *reinterpret_cast<uint2*>(a.q + base + c) = quantize8(f, inv);
        if (tid % 16 == 0) a.sf[row * a.sf_row_stride + c / kBlock * a.sf_block_stride] = sf;
      }
    }
  }
}

// A CTA walks a share of the rows; a thread keeps its columns' part of the weight's gradient
// over them, and the CTAs' parts are added by the kernel below.  Shares are fixed, so the
// sums are.  (32768 x 4096, L2 flushed: 184 us; two shares for each CTA that fits, so that SMs
// that are ahead take more, 191, four 203: their parts cost more than they even out.)
//
// CTAs an SM: what is in flight counts, so many with few registers: the same with four 184 us,
// three 190, two 221; the stream in fp32 spills with four (383, 342 with three).
template <int NV, int MAXT, bool FP32>
__global__ void __launch_bounds__(MAXT == 32 ? kShortThreads : MAXT,
                                  NV == 1 ? 4 : NV == 2 ? (MAXT == 256 && !FP32 ? 4 : 3) : MAXT <= 256 ? 2 : 1)
norm_backward_kernel(NormArgs a) {
  constexpr bool CTA_ROW = MAXT > 32;
  __shared__ float part[kMaxRowThreads / 32];
  extern __shared__ float sum_s[];       // [cols], where warps have a row each
  ptx::grid_dependency_wait();
  const int threads = CTA_ROW ? static_cast<int>(blockDim.x) : 32;
  const int tid = CTA_ROW ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x) % 32;
  constexpr int kRows = CTA_ROW ? 1 : kShortThreads / 32;
  const int mine = CTA_ROW ? 0 : static_cast<int>(threadIdx.x) / 32;
  int64_t rows = a.rows;
  if (a.total_rows != nullptr) rows = min64(rows, *a.total_rows);
  const int cols = static_cast<int>(a.cols);
  const float inv_cols = 1.0f / static_cast<float>(cols);
  float dw[NV][8] = {};
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + mine; row < rows; row += static_cast<int64_t>(gridDim.x) * kRows) {
    const int64_t base = row * a.cols;
    Raw8<false> dy[NV];
    Raw8<FP32> z[NV], dres[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (j * threads + tid);
      if (c < cols) {
        dy[j].load(a.x, base + c);
        z[j].load(a.residual, base + c);
        if (a.dresidual != nullptr) dres[j].load(a.dresidual, base + c);
      }
    }
    const float r = a.rstd[row];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (j * threads + tid);
      if (c >= cols) break;
      float g[8], h[8], w[8];
      load_weight(a, c, w);
      dy[j].get(g);
      z[j].get(h);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[i] *= r;
        dw[j][i] = fmaf(g[i], h[i], dw[j][i]);
        sum = fmaf(g[i] * w[i], h[i], sum);
      }
    }
    const float mean = row_sum<CTA_ROW>(sum, part) * inv_cols;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (j * threads + tid);
      if (c >= cols) break;
      float g[8], h[8], w[8], d[8] = {};
      load_weight(a, c, w);
      dy[j].get(g);
      z[j].get(h);
      if (a.dresidual != nullptr) dres[j].get(d);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = fmaf(r, fmaf(-h[i] * r, mean, g[i] * w[i]), d[i]);
      Raw8<FP32> out;
      out.set(d);
      out.store(a.residual_out, base + c);
      if (a.y != nullptr) ptx::st_v4(a.y + base + c, pack8(d));
    }
  }
  if (a.dweight == nullptr) return;
  float* out = a.partial + static_cast<int64_t>(blockIdx.x) * a.cols;
  if constexpr (CTA_ROW) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (j * threads + tid);
      if (c < cols) store_fp32(out + c, dw[j]);
    }
  } else {
    for (int w = 0; w < kRows; ++w) {    // one after the other: a fixed order
      if (w == mine) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = 8 * (j * threads + tid);
          if (c >= cols) break;
#pragma unroll
          for (int i = 0; i < 8; ++i) sum_s[c + i] = w == 0 ? dw[j][i] : sum_s[c + i] + dw[j][i];
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < cols; c += kShortThreads) out[c] = sum_s[c];
  }
}

// The weight's gradient from the CTAs' parts: a warp's lanes have 32 columns, its CTA's
// 32 warps every 32nd part, added in their order.
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads) norm_weight_kernel(const float* partial, int parts, int64_t cols, float* dweight,
                                                                  bool accumulate) {
  __shared__ float sum_s[kSumThreads / 32][32];
  ptx::grid_dependency_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (c < cols)
#pragma unroll 8
    for (int p = warp; p < parts; p += kSumThreads / 32) s += partial[p * cols + c];
  sum_s[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
    for (int w = 1; w < kSumThreads / 32; ++w) s += sum_s[w][lane];
    dweight[c] = accumulate ? dweight[c] + s : s;
  }
}

// Vectors of a thread and threads of a row.  A warp has up to 1024 columns, a CTA two
// vectors a thread up to 4096, four up to 8192, then eight; the gradient, which holds more,
// four and twice the threads up to 16384 (375 us; eight vectors took 559 on 16384 x 16384).
struct Shape {
  int nv;
  int max_threads;
  int threads;
};
Shape shape_of(int64_t cols, bool backward) {
  const int64_t vecs = ceil_div64(cols, 8);
  if (vecs <= 128) return {vecs <= 32 ? 1 : vecs <= 64 ? 2 : 4, 32, kShortThreads};
  const int nv = vecs <= 512 ? 2 : vecs <= (backward ? 2048 : 1024) ? 4 : 8;
  const int threads = static_cast<int>(ceil_div64(ceil_div64(vecs, nv), 32) * 32);
  return {nv, threads <= 256 ? 256 : 512, threads};
}

template <bool BACKWARD, typename F>
cudaError_t with_shape(const Shape& s, bool fp32, F run) {
#define MOE_NORM_CASE(NV, MAXT) \
  if (s.nv == NV && s.max_threads == MAXT) return fp32 ? run.template operator()<NV, MAXT, true>() : run.template operator()<NV, MAXT, false>();
  MOE_NORM_CASE(1, 32)
  MOE_NORM_CASE(2, 32)
  MOE_NORM_CASE(4, 32)
  MOE_NORM_CASE(2, 256)
  MOE_NORM_CASE(4, 256)
  if constexpr (BACKWARD) {
    MOE_NORM_CASE(4, 512)
  } else {
    MOE_NORM_CASE(8, 256)
  }
  MOE_NORM_CASE(8, 512)
#undef MOE_NORM_CASE
  return cudaErrorInvalidValue;
}

struct Forward {
  const NormArgs& a;
  const Shape& s;
  cudaStream_t stream;
  template <int NV, int MAXT, bool FP32>
  cudaError_t operator()() const {
    const int64_t grid = MAXT > 32 ? a.rows : ceil_div64(a.rows, kShortThreads / 32);
    return launch_pdl(norm_kernel<NV, MAXT, FP32>, dim3(static_cast<unsigned>(grid)), s.threads, 0, stream, a);
  }
};

struct Backward {
  const NormArgs& a;
  const Shape& s;
  cudaStream_t stream;
  template <int NV, int MAXT, bool FP32>
  cudaError_t operator()() const {
    const auto kernel = norm_backward_kernel<NV, MAXT, FP32>;
    const size_t smem = MAXT > 32 ? 0 : 4 * static_cast<size_t>(a.cols);
    const int ctas = cached_occupancy(kernel, s.threads, smem);
    const int64_t most = min64(static_cast<int64_t>(ctas > 0 ? ctas : 1) * device_sm_count(), norm_parts(a.cols));
    const int64_t units = MAXT > 32 ? a.rows : ceil_div64(a.rows, kShortThreads / 32);
    const int64_t grid = max64(1, min64(units, most));
    count_launch();
    cudaError_t e = launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), s.threads, smem, stream, a);
    if (e != cudaSuccess || a.dweight == nullptr) return e;
    count_launch();
    return launch_pdl(norm_weight_kernel, dim3(static_cast<unsigned>(ceil_div64(a.cols, 32))), kSumThreads, 0, stream,
                      static_cast<const float*>(a.partial), static_cast<int>(grid), a.cols, a.dweight, a.accumulate);
  }
};

}  // namespace

// The norm writes rows and scales that the dispatch may read before its
// griddepcontrol.wait, so it never releases its dependents early.
cudaError_t launch_norm(const NormArgs& a, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  const Shape s = shape_of(a.cols, false);
  count_launch();
  return with_shape<false>(s, a.stream_fp32, Forward{a, s, stream});
}

int64_t norm_parts(int64_t cols) { return 160 * max64(1, 1024 / shape_of(cols, true).threads); }

// Without rows the gradient of the weight is still written.
cudaError_t launch_norm_backward(const NormArgs& a, cudaStream_t stream) {
  if (a.rows == 0 && a.dweight == nullptr) return cudaSuccess;
  const Shape s = shape_of(a.cols, true);
  return with_shape<true>(s, a.stream_fp32, Backward{a, s, stream});
}

}  // namespace moe
