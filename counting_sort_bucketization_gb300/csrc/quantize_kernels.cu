// quantize_kernels.cu -- 8-bit rows for dispatch and for the expert products,
// and the gated activation between two products.
//
//   quantize_rows_kernel   bf16 [rows, cols] -> e4m3 with one fp32 scale for
//                          each 1x128 block; with SWIGLU the input is
//                          [rows, 2*cols] = (gate | up) and the quantised value
//                          is silu(gate) * up, never rounded in between.
//   quantize_cols_kernel   receive rows -> transposed e4m3 [cols, rows] with
//                          one scale for each 128x1 block (weight gradients
//                          sum over rows, so their blocks run down a column).
//   swiglu_backward_kernel gradient of silu(gate) * up.
//
// Block scale: sf = max(|x|, 1e-30) / 448, q = e4m3(x * (1 / sf)), both
// divisions IEEE.  The floor keeps 1/sf finite for a block of zeros, whose
// codes are zeros; 448 is e4m3's largest value.  The one rounding to 8 bits is
// the purpose of the kernel; everything before it is fp32.
//
// All of them move a few bytes an element once and are bound by HBM.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kBlock = 128;            // values that share a scale
constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 1e-30f;

__device__ __forceinline__ void unpack8(uint4 v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Two floats to two e4m3 codes (lo in the low byte), round to nearest even.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t cvt_e4m3x4(float a, float b, float c, float d) {
  return cvt_e4m3x2(a, b) | (cvt_e4m3x2(c, d) << 16);
}

__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// The larger of two magnitudes; a NaN on either side stays (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// ---------------------------------------------------------------- rows
// A half-warp owns one block of 128 columns (16 bytes of bf16 a lane); a CTA
// of 8 warps covers 16 rows x 4 blocks.  Each half-warp takes the four blocks
// of its row in turn with all loads issued first, so a lane has 4 (SWIGLU: 8)
// 16-byte loads in flight, and the 16 rows of a CTA make 64-byte runs of a
// column-major scale column.
constexpr int kRowsThreads = 256;
constexpr int kRowsPerCta = kRowsThreads / 16;
constexpr int kBlocksPerLane = 4;

template <bool SWIGLU>
__global__ void __launch_bounds__(kRowsThreads) quantize_rows_kernel(QuantRowsArgs a) {
  ptx::grid_dependency_wait();
  const int64_t nb = (a.cols + kBlock - 1) / kBlock;
  const int64_t chunks = (nb + kBlocksPerLane - 1) / kBlocksPerLane;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) / chunks * kRowsPerCta;
  const int64_t b0 = static_cast<int64_t>(blockIdx.x) % chunks * kBlocksPerLane;
  const int64_t row = row0 + threadIdx.x / 16;
  const int sub = threadIdx.x % 16;
  int64_t rows = a.rows;
  if (a.total_rows != nullptr) rows = min64(rows, *a.total_rows);
  if (row0 >= rows) return;
  // A half-warp past the last row still takes part in the warp's shuffles.
  const bool live = row < rows;

  const int64_t in_cols = SWIGLU ? 2 * a.cols : a.cols;
  const uint16_t* src = a.x + row * in_cols;
  uint4 v[kBlocksPerLane], u[kBlocksPerLane];
#pragma unroll
  for (int j = 0; j < kBlocksPerLane; ++j) {
    const int64_t c = (b0 + j) * kBlock + sub * 8;
    v[j] = u[j] = make_uint4(0, 0, 0, 0);
    if (live && c < a.cols) {
      v[j] = ptx::ld_nc_v4(src + c);
      if (SWIGLU) u[j] = ptx::ld_nc_v4(src + a.cols + c);
    }
  }
#pragma unroll
  for (int j = 0; j < kBlocksPerLane; ++j) {
    if (b0 + j >= nb) break;   // the same for the whole CTA
    const int64_t c = (b0 + j) * kBlock + sub * 8;
    float f[8];
    unpack8(v[j], f);
    if (SWIGLU) {
      float g[8];
      unpack8(u[j], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = f[i] * sigmoid(f[i]) * g[i];
    }
    float m = kAmaxFloor;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(f[i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float sf = __fdiv_rn(m, kE4m3Max);
    const float inv = __fdiv_rn(1.0f, sf);
    if (live && c < a.cols) {
      uint2 q;
      q.x = cvt_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
      q.y = cvt_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
      *reinterpret_cast<uint2*>(a.q + row * a.cols + c) = q;
    }
    if (live && sub == 0) a.sf[row * a.sf_row_stride + (b0 + j) * a.sf_block_stride] = sf;
  }
}

// ---------------------------------------------------------------- columns
// A CTA transposes a tile of 128 rows (one scale block; segments start at
// multiples of 128, so it lies in one expert) x 64 columns.  A thread holds 4
// consecutive rows x 8 columns, so its codes of a column make one 32-bit word
// of the transposed tile; words go through shared memory at a pitch of 33 and
// leave as 128-byte runs of a transposed row.
constexpr int kColsThreads = 256;
constexpr int kTileCols = 64;
constexpr int kPitch = 33;

__global__ void __launch_bounds__(kColsThreads) quantize_cols_kernel(QuantColsArgs a) {
  __shared__ uint32_t tile[kTileCols * kPitch];
  __shared__ float wmax[kColsThreads / 32][kTileCols];
  __shared__ int valid_s;
  ptx::grid_dependency_wait();
  const int64_t chunks = (a.cols + kTileCols - 1) / kTileCols;
  const int64_t rb = static_cast<int64_t>(blockIdx.x) / chunks;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) % chunks * kTileCols;
  const int64_t r0 = rb * kBlock;
  const int total = a.expert_offset[a.num_experts];
  if (r0 >= total || total > a.capacity) {
    if (total > a.capacity && blockIdx.x == 0 && threadIdx.x == 0) set_error(a.err, MOE_ERR_CAPACITY);
    return;
  }
  if (threadIdx.x == 0) {
    // The expert whose segment holds row r0: the last one that starts at or before it.
    int lo = 0, hi = a.num_experts;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.expert_offset[mid] <= r0) lo = mid; else hi = mid;
    }
    const int64_t end = static_cast<int64_t>(a.expert_offset[lo]) + a.expert_count[lo];
    valid_s = static_cast<int>(max64(0, min64(kBlock, end - r0)));
  }
  __syncthreads();
  const int valid = valid_s;
  const int g = threadIdx.x / 8, c8 = threadIdx.x % 8;   // rows 4g..4g+3, columns 8*c8..+7
  const int64_t c = c0 + c8 * 8;
  uint4 v[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int r = 4 * g + p;
    v[p] = make_uint4(0, 0, 0, 0);
    if (r < valid && c < a.cols) v[p] = ptx::ld_nc_v4(a.x + (r0 + r) * a.cols + c);
  }
  float f[4][8], m[8];
#pragma unroll
  for (int p = 0; p < 4; ++p) unpack8(v[p], f[p]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = kAmaxFloor;
#pragma unroll
    for (int p = 0; p < 4; ++p) m[i] = max_nan(m[i], fabsf(f[p][i]));
    m[i] = max_nan(m[i], __shfl_xor_sync(0xffffffffu, m[i], 8));
    m[i] = max_nan(m[i], __shfl_xor_sync(0xffffffffu, m[i], 16));
  }
  const int warp = threadIdx.x / 32;
  if (threadIdx.x % 32 < 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) wmax[warp][c8 * 8 + i] = m[i];
  }
  __syncthreads();
  if (threadIdx.x < kTileCols) {
    float t = wmax[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < kColsThreads / 32; ++w) t = max_nan(t, wmax[w][threadIdx.x]);
    const float sf = __fdiv_rn(t, kE4m3Max);
    if (c0 + threadIdx.x < a.cols) a.sf[rb * a.cols + c0 + threadIdx.x] = sf;
    wmax[0][threadIdx.x] = __fdiv_rn(1.0f, sf);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float inv = wmax[0][c8 * 8 + i];
    tile[(c8 * 8 + i) * kPitch + g] = cvt_e4m3x4(f[0][i] * inv, f[1][i] * inv, f[2][i] * inv, f[3][i] * inv);
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kTileCols * 8 / kColsThreads; ++j) {
    const int unit = threadIdx.x + j * kColsThreads;
    const int col = unit / 8, part = unit % 8;
    if (c0 + col < a.cols) {
      const uint32_t* t = tile + col * kPitch + part * 4;
      ptx::st_v4(a.q + (c0 + col) * a.ld + r0 + part * 16, make_uint4(t[0], t[1], t[2], t[3]));
    }
  }
}

// ---------------------------------------------------------------- SwiGLU gradient
// With s = sigmoid(g): d gate = dh * u * s * (1 + g * (1 - s)), d up = dh * g * s.
// A thread owns 8 columns of a row (16-byte accesses throughout).
constexpr int kBwdThreads = 256;

__global__ void __launch_bounds__(kBwdThreads) swiglu_backward_kernel(SwigluBackwardArgs a) {
  ptx::grid_dependency_wait();
  const int64_t per_row = a.width / 8;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kBwdThreads + threadIdx.x;
  int64_t rows = a.rows;
  if (a.total_rows != nullptr) rows = min64(rows, *a.total_rows);
  const int64_t row = id / per_row, c = id % per_row * 8;
  if (row >= rows) return;
  const uint16_t* gu = a.gate_up + row * 2 * a.width + c;
  const uint4 gv = ptx::ld_nc_v4(gu), uv = ptx::ld_nc_v4(gu + a.width);
  const uint4 dv = ptx::ld_nc_v4(a.dh + row * a.width + c);
  float g[8], u[8], d[8], dg[8], du[8];
  unpack8(gv, g);
  unpack8(uv, u);
  unpack8(dv, d);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = sigmoid(g[i]);
    dg[i] = d[i] * u[i] * s * (1.0f + g[i] * (1.0f - s));
    du[i] = d[i] * g[i] * s;
  }
  uint16_t* out = a.dgate_up + row * 2 * a.width + c;
  ptx::st_v4(out, make_uint4(pack_bf16(dg[0], dg[1]), pack_bf16(dg[2], dg[3]), pack_bf16(dg[4], dg[5]),
                             pack_bf16(dg[6], dg[7])));
  ptx::st_v4(out + a.width, make_uint4(pack_bf16(du[0], du[1]), pack_bf16(du[2], du[3]), pack_bf16(du[4], du[5]),
                                       pack_bf16(du[6], du[7])));
}

constexpr int64_t kMaxGrid = 2147483647;

}  // namespace

// These kernels never release their dependents early: the dispatch permutes
// may read x and sf before their own griddepcontrol.wait.
cudaError_t launch_quantize_rows(const QuantRowsArgs& a, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  const int64_t nb = ceil_div64(a.cols, kBlock);
  const int64_t grid = ceil_div64(a.rows, kRowsPerCta) * ceil_div64(nb, kBlocksPerLane);
  if (grid > kMaxGrid) return cudaErrorInvalidConfiguration;
  count_launch();
  const dim3 g(static_cast<unsigned>(grid));
  return a.swiglu ? launch_pdl(quantize_rows_kernel<true>, g, kRowsThreads, 0, stream, a)
                  : launch_pdl(quantize_rows_kernel<false>, g, kRowsThreads, 0, stream, a);
}

cudaError_t launch_quantize_cols(const QuantColsArgs& a, cudaStream_t stream) {
  if (a.capacity == 0) return cudaSuccess;
  const int64_t grid = ceil_div64(a.capacity, kBlock) * ceil_div64(a.cols, kTileCols);
  if (grid > kMaxGrid) return cudaErrorInvalidConfiguration;
  count_launch();
  return launch_pdl(quantize_cols_kernel, dim3(static_cast<unsigned>(grid)), kColsThreads, 0, stream, a);
}

cudaError_t launch_swiglu_backward(const SwigluBackwardArgs& a, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  const int64_t grid = ceil_div64(a.rows * (a.width / 8), kBwdThreads);
  if (grid > kMaxGrid) return cudaErrorInvalidConfiguration;
  count_launch();
  return launch_pdl(swiglu_backward_kernel, dim3(static_cast<unsigned>(grid)), kBwdThreads, 0, stream, a);
}

}  // namespace moe
