// combine_backward_kernel.cu -- gradient of the combine's weighted sum.
//
//   out_t = sum_k w_tk y[slot(t, k)]:   dy[slot(t, k)] = w_tk dout_t   (bf16, one rounding)
//                                       dw_tk = <dout_t, y[slot(t, k)]> (fp32)
//
// A token's columns go to one or more warps, 16 bytes a lane and step: a lane reads dout
// once for up to 8 slots, reads the slots' expert rows, adds to their dot products and
// writes their rows of dy.  HBM bound: 2 + 4 K bytes a column and token.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSlots = 8;                // slots of a token done together

// WARPS: of a token.
template <int WARPS, bool DOT>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(CombineBackwardArgs a) {
  __shared__ float part_s[kWarps][kSlots];
  ptx::grid_dependency_wait();
  constexpr int kTokens = kWarps / WARPS, kLanes = 32 * WARPS;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int tid = threadIdx.x % kLanes;
  const int64_t H = a.hidden;
  const int K = a.topk;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens; t0 < a.num_tokens; t0 += static_cast<int64_t>(gridDim.x) * kTokens) {
    const int64_t t = t0 + warp / WARPS;
    const bool live = t < a.num_tokens;
    for (int k0 = 0; k0 < K; k0 += kSlots) {
      int64_t at[kSlots];                // a slot's row, -1 without one
      float w[kSlots], dot[kSlots];
#pragma unroll
      for (int q = 0; q < kSlots; ++q) {
        at[q] = -1;
        w[q] = dot[q] = 0.0f;
        if (live && k0 + q < K) {
          const int s = __ldg(a.dst_slot + t * K + k0 + q);
          w[q] = __ldg(a.weights + t * K + k0 + q);
          if (s >= a.capacity) {
            if (tid == 0) set_error(a.err, MOE_ERR_CAPACITY);
          } else if (s >= 0) {
            at[q] = s * H;
          }
        }
      }
      if (live) {
        for (int64_t c = 8 * tid; c < H; c += 8 * kLanes) {
          uint4 y[kSlots];
          const uint4 dv = ptx::ld_nc_v4(a.dout + t * H + c);
          if (DOT) {
#pragma unroll
            for (int q = 0; q < kSlots; ++q) {
              y[q] = make_uint4(0, 0, 0, 0);
              if (at[q] >= 0) y[q] = load_v4(a.expert_out + at[q] + c);
            }
          }
          float d[8];
          unpack8(dv, d);
#pragma unroll
          for (int q = 0; q < kSlots; ++q) {
            if (at[q] < 0) continue;
            float v[8];
            if (DOT) {
              unpack8(y[q], v);
#pragma unroll
              for (int i = 0; i < 8; ++i) dot[q] = fmaf(d[i], v[i], dot[q]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = w[q] * d[i];
            ptx::st_v4(a.dy + at[q] + c, pack8(v));
          }
        }
      }
      if (DOT) {
#pragma unroll
        for (int q = 0; q < kSlots; ++q)
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) dot[q] += __shfl_xor_sync(kFull, dot[q], o);
        if (WARPS > 1) {
          __syncthreads();               // the last slots' parts are read
          if (lane == 0)
#pragma unroll
            for (int q = 0; q < kSlots; ++q) part_s[warp][q] = dot[q];
          __syncthreads();
        }
        if (live && tid == 0)
#pragma unroll
          for (int q = 0; q < kSlots; ++q) {
            if (k0 + q >= K) break;
            float s = dot[q];
            for (int v = 1; v < WARPS; ++v) s += part_s[warp + v][q];
            a.dweights[t * K + k0 + q] = s;
          }
      }
    }
  }
  if (!a.zero_pad) return;
  // Alignment-gap rows, an eighth of an expert's a CTA.
  constexpr int kShares = 8;
  for (int64_t u = blockIdx.x; u < static_cast<int64_t>(a.num_experts) * kShares; u += gridDim.x) {
    const int e = static_cast<int>(u / kShares);
    const int64_t end = min64(a.expert_offset[e + 1], a.capacity);
    for (int64_t r = static_cast<int64_t>(a.expert_offset[e]) + a.expert_count[e] + u % kShares; r < end; r += kShares)
      if (r >= 0)
        for (int64_t c = 8 * static_cast<int64_t>(threadIdx.x); c < H; c += 8 * kThreads)
          ptx::st_v4(a.dy + r * H + c, make_uint4(0, 0, 0, 0));
  }
}

}  // namespace

cudaError_t launch_combine_backward(const CombineBackwardArgs& a, cudaStream_t stream) {
  if (a.num_tokens == 0 && !a.zero_pad) return cudaSuccess;
  count_launch();
  const auto run = [&](auto kernel, int tokens) {
    const int ctas = cached_occupancy(kernel, kThreads, 0);
    const int64_t most = static_cast<int64_t>(ctas > 0 ? ctas : 1) * device_sm_count();
    int64_t units = ceil_div64(a.num_tokens, tokens);
    if (a.zero_pad) units = max64(units, static_cast<int64_t>(a.num_experts) * 8);
    const int64_t grid = max64(1, min64(units, most));
    return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), kThreads, 0, stream, a);
  };
  // A warp a token where there are enough of them to fill the GPU.
  const bool many = a.num_tokens >= static_cast<int64_t>(kWarps) * device_sm_count() || a.hidden <= 256;
  if (a.dweights != nullptr)
    return many ? run(combine_backward_kernel<1, true>, kWarps) : run(combine_backward_kernel<kWarps, true>, 1);
  return many ? run(combine_backward_kernel<1, false>, kWarps) : run(combine_backward_kernel<kWarps, false>, 1);
}

}  // namespace moe
