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
// All of them move a few bytes an element once and are bound by HBM (a copy
// reaches 6.76 TB/s): rows of 32768 x 7168 in 113 us (6.3 TB/s), SwiGLU of
// 34816 x (2 x 2048) in 57 us (6.3), its gradient on 10007 x (2 x 1936) in
// 29.8 us (6.5), the columns of 32768 receive rows x 4096 in 72 us (5.8; the
// barriers between the steps of a tile are what is left).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace moe {
namespace {

// 1 / (1 + 2^(-g log2 e)).  The product's rounding adds 2^-24 |g| to the relative error where e^-g
// counts, 2^-18 at -64, and results below 2^-126 are zero: every use is rounded to 16 or 8
// bits (2^-9, 2^-4) right after.
__device__ __forceinline__ float sigmoid(float g) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  return __fdividef(1.0f, 1.0f + e);
}

// ---------------------------------------------------------------- rows
// A half-warp owns one block of 128 columns (16 bytes of bf16 a lane); a CTA
// of 8 warps covers 16 rows x 4 blocks.  Each half-warp takes the four blocks
// of its row in turn with all loads issued first, so a lane has 4 (SWIGLU: 8)
// 16-byte loads in flight (with 2 and 4 the same rows take 133 us, SwiGLU 60), and
// the 16 rows of a CTA make 64-byte runs of a column-major scale column.
constexpr int kRowsThreads = 256;
constexpr int kRowsPerCta = kRowsThreads / 16;
constexpr int kBlocksPerLane = 4;

template <bool SWIGLU>
__global__ void __launch_bounds__(kRowsThreads, SWIGLU ? 4 : 6) quantize_rows_kernel(QuantRowsArgs a) {
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
// A CTA transposes tiles of 128 rows (one scale block; segments start at
// multiples of 128, so it lies in one expert) x 64 columns, kColTiles of them
// side by side with the next tile's rows on their way.  A thread holds 4
// consecutive rows x 8 columns, so its codes of a column make one 32-bit word
// of the transposed tile; words go through shared memory at a pitch of 33 and
// leave as 128-byte runs of a transposed row.  (Five CTAs an SM: 72 us where four
// take 76 and three 82.  A warp a tile of 16 columns, without barriers, took 115: its
// 32-byte pieces of rows cost more than the barriers.)
constexpr int kColsThreads = 256;
constexpr int kTileCols = 64;
constexpr int kColTiles = 4;
constexpr int kPitch = 33;

// Larger magnitudes of two pairs of bf16 (exact: no rounding); NaN stays.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7fff7fffu), "r"(b & 0x7fff7fffu));
  return r;
}

__global__ void __launch_bounds__(kColsThreads, 5) quantize_cols_kernel(QuantColsArgs a) {
  __shared__ uint32_t tile[kTileCols * kPitch];
  __shared__ uint32_t wmax[kColsThreads / 32][kTileCols / 2];
  __shared__ float inv_s[kTileCols];
  __shared__ int valid_s;
  __shared__ bool off_grid_s;
  ptx::grid_dependency_wait();
  const int64_t chunks = (a.cols + kColTiles * kTileCols - 1) / (kColTiles * kTileCols);
  const int64_t rb = static_cast<int64_t>(blockIdx.x) / chunks;
  const int64_t c_first = static_cast<int64_t>(blockIdx.x) % chunks * (kColTiles * kTileCols);
  const int64_t r0 = rb * kBlock;
  const int g = threadIdx.x / 8, c8 = threadIdx.x % 8;   // rows 4g..4g+3, columns 8*c8..+7
  const int warp = threadIdx.x / 32;
  const uint16_t* src = a.x + (r0 + 4 * g) * a.cols + c8 * 8;
  uint4 v[4], next[4];
  // Rows in the buffer; gap rows among them are dropped below.
  const auto load = [&](int64_t c0, uint4* to) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      to[p] = make_uint4(0, 0, 0, 0);
      if (r0 + 4 * g + p < a.capacity && c0 + c8 * 8 < a.cols) to[p] = ptx::ld_nc_v4(src + p * a.cols + c0);
    }
  };
  load(c_first, next);
  // The expert whose segment holds row r0 says how many of the block's rows are real.
  const int total = a.expert_offset[a.num_experts];
  if (threadIdx.x == 0) valid_s = 0, off_grid_s = false;
  __syncthreads();
  for (int e = threadIdx.x; e < a.num_experts; e += kColsThreads) {
    const int start = a.expert_offset[e];
    if (start % kBlock != 0) off_grid_s = true;
    if (start <= r0 && r0 < a.expert_offset[e + 1])
      valid_s = static_cast<int>(max64(0, min64(kBlock, static_cast<int64_t>(start) + a.expert_count[e] - r0)));
  }
  if (r0 >= total || total > a.capacity) {
    if (total > a.capacity && blockIdx.x == 0 && threadIdx.x == 0) set_error(a.err, MOE_ERR_CAPACITY);
    return;
  }
  __syncthreads();
  if (off_grid_s) {   // a block could lie in two experts
    if (blockIdx.x == 0 && threadIdx.x == 0) set_error(a.err, MOE_ERR_INVALID_ARG);
    return;
  }
  const int valid = valid_s;
  for (int ct = 0; ct < kColTiles; ++ct) {
    const int64_t c0 = c_first + ct * kTileCols;
    if (c0 >= a.cols) break;
#pragma unroll
    for (int p = 0; p < 4; ++p) v[p] = 4 * g + p < valid ? next[p] : make_uint4(0, 0, 0, 0);
    if (ct + 1 < kColTiles) load(c0 + kTileCols, next);
    uint32_t m[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      m[0] = max_abs_bf16x2(m[0], v[p].x);
      m[1] = max_abs_bf16x2(m[1], v[p].y);
      m[2] = max_abs_bf16x2(m[2], v[p].z);
      m[3] = max_abs_bf16x2(m[3], v[p].w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = max_abs_bf16x2(m[i], __shfl_xor_sync(0xffffffffu, m[i], 8));
      m[i] = max_abs_bf16x2(m[i], __shfl_xor_sync(0xffffffffu, m[i], 16));
    }
    if (threadIdx.x % 32 < 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) wmax[warp][c8 * 4 + i] = m[i];
    }
    __syncthreads();
    if (threadIdx.x < kTileCols) {
      uint32_t t = wmax[0][threadIdx.x / 2];
#pragma unroll
      for (int w = 1; w < kColsThreads / 32; ++w) t = max_abs_bf16x2(t, wmax[w][threadIdx.x / 2]);
      const float amax = __uint_as_float(threadIdx.x % 2 ? t & 0xffff0000u : t << 16);
      const float sf = __fdiv_rn(max_nan(amax, kAmaxFloor), kE4m3Max);
      if (c0 + threadIdx.x < a.cols) a.sf[rb * a.cols + c0 + threadIdx.x] = sf;
      inv_s[threadIdx.x] = __fdiv_rn(1.0f, sf);
    }
    __syncthreads();
    float f[4][8];
#pragma unroll
    for (int p = 0; p < 4; ++p) unpack8(v[p], f[p]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float inv = inv_s[c8 * 8 + i];
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
  const int64_t grid = ceil_div64(a.capacity, kBlock) * ceil_div64(a.cols, kColTiles * kTileCols);
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
