// combine_backward_kernel.cu -- gradient of the combine's weighted sum.
//
//   out_t = sum_k w_tk y[slot(t, k)]:   dy[slot(t, k)] = w_tk dout_t   (bf16, one rounding)
//                                       dw_tk = <dout_t, y[slot(t, k)]> (fp32)
//
// A token's columns go to one or more warps, 16 bytes a lane and step: a lane reads dout
// once for up to 8 slots, reads the slots' expert rows, adds to their dot products and
// writes their rows of dy.  HBM bound: 2 + 4 K bytes a column and token.  32768 tokens x top-8 x
// 4096 in 652 us (6.8 TB/s, a copy's rate), 4096 x top-8 x 7168 186 (6.6), 131072 x top-2 x 512
// 108 (6.2); 48 x top-8 x 7168 10 us a call (host 8).
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
constexpr int kGapCtas = 4;              // that share an expert's gap rows

// Alignment-gap rows to zero, by the first CTAs of the grid.  A layout of more rows than there
// are has no slots, and its gaps are not touched either, as by the permutes.
__device__ __forceinline__ void zero_gaps(const CombineBackwardArgs& a) {
  if (a.expert_offset[a.num_experts] > a.capacity) return;
  const int e = static_cast<int>(blockIdx.x) / kGapCtas;
  const int64_t end = min64(a.expert_offset[e + 1], a.capacity);
  int64_t r = max64(0, static_cast<int64_t>(a.expert_offset[e]) + a.expert_count[e]) + blockIdx.x % kGapCtas;
  for (; r < end; r += kGapCtas)
    for (int64_t c = 8 * static_cast<int64_t>(threadIdx.x); c < a.hidden; c += 8 * kThreads)
      ptx::st_v4(a.dy + r * a.hidden + c, make_uint4(0, 0, 0, 0));
}

// A slot's row, -1 without one.
__device__ __forceinline__ int slot_row(const CombineBackwardArgs& a, int64_t pair, bool report) {
  const int s = __ldg(a.dst_slot + pair);
  if (s < a.capacity) return max(s, -1);
  if (report) set_error(a.err, MOE_ERR_CAPACITY);
  return -1;
}

// A token's columns go to WARPS warps, SLOTS of its slots at a time.  Reads in flight are what
// counts: as many CTAs an SM as the slots' registers allow, and each CTA ends with its tokens,
// so that the block scheduler keeps the faster SMs busy (32768 x top-8 x 4096: 655 us; one
// wave of two CTAs an SM that walk the tokens, 706).
template <int WARPS, int SLOTS, bool DOT>
__global__ void __launch_bounds__(kThreads, SLOTS == 8 ? 3 : SLOTS == 4 ? 4 : 6) combine_backward_kernel(CombineBackwardArgs a) {
  __shared__ float part_s[kWarps][SLOTS];
  ptx::grid_dependency_wait();
  constexpr int kTokens = kWarps / WARPS, kLanes = 32 * WARPS;
  const int gaps = a.zero_pad ? a.num_experts * kGapCtas : 0;
  if (static_cast<int>(blockIdx.x) < gaps) return zero_gaps(a);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int tid = threadIdx.x % kLanes;
  const int64_t H = a.hidden;
  const int K = a.topk;
  const int64_t t = static_cast<int64_t>(blockIdx.x - gaps) * kTokens + warp / WARPS;
  const bool live = t < a.num_tokens;    // the same for a whole warp
  for (int k0 = 0; k0 < K; k0 += SLOTS) {
    int at[SLOTS];
    float w[SLOTS], dot[SLOTS];
#pragma unroll
    for (int q = 0; q < SLOTS; ++q) {
      at[q] = -1;
      w[q] = dot[q] = 0.0f;
      if (live && k0 + q < K) {
        at[q] = slot_row(a, t * K + k0 + q, tid == 0);
        w[q] = __ldg(a.weights + t * K + k0 + q);
      }
    }
    for (int64_t c = 8 * tid; live && c < H; c += 8 * kLanes) {
      uint4 y[SLOTS];
      const uint4 dv = ptx::ld_nc_v4(a.dout + t * H + c);
      if (DOT) {
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
          y[q] = make_uint4(0, 0, 0, 0);
          if (at[q] >= 0) y[q] = load_v4(a.expert_out + at[q] * H + c);
        }
      }
      float d[8];
      unpack8(dv, d);
#pragma unroll
      for (int q = 0; q < SLOTS; ++q) {
        if (at[q] < 0) continue;
        float v[8];
        if (DOT) {
          unpack8(y[q], v);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[q] = fmaf(d[i], v[i], dot[q]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = w[q] * d[i];
        ptx::st_v4(a.dy + at[q] * H + c, pack8(v));
      }
    }
    if (DOT) {
#pragma unroll
      for (int q = 0; q < SLOTS; ++q)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[q] += __shfl_xor_sync(kFull, dot[q], o);
      if (WARPS > 1) {
        __syncthreads();                 // the last slots' parts are read
        if (lane == 0)
#pragma unroll
          for (int q = 0; q < SLOTS; ++q) part_s[warp][q] = dot[q];
        __syncthreads();
      }
      if (live && tid == 0)
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
          if (k0 + q >= K) break;
          float s = dot[q];
          for (int v = 1; v < WARPS; ++v) s += part_s[warp + v][q];
          a.dweights[t * K + k0 + q] = s;
        }
    }
  }
}

// A CTA a slot: dout is read for each of them, from the L2 but for the first.
constexpr int kSteps = 4;
template <bool DOT>
__global__ void __launch_bounds__(kThreads) combine_backward_slot_kernel(CombineBackwardArgs a) {
  __shared__ float part_s[kWarps];
  ptx::grid_dependency_wait();
  const int gaps = a.zero_pad ? a.num_experts * kGapCtas : 0;
  if (static_cast<int>(blockIdx.x) < gaps) return zero_gaps(a);
  const int64_t pair = static_cast<int64_t>(blockIdx.x) - gaps, t = pair / a.topk, H = a.hidden;
  const int at = slot_row(a, pair, threadIdx.x == 0);
  const float w = __ldg(a.weights + pair);
  float dot = 0.0f;
  if (at >= 0)
    for (int64_t c0 = 8 * static_cast<int64_t>(threadIdx.x); c0 < H; c0 += 8 * kSteps * kThreads) {
      uint4 dv[kSteps], y[kSteps];
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const int64_t c = c0 + 8 * j * kThreads;
        dv[j] = y[j] = make_uint4(0, 0, 0, 0);
        if (c < H) {
          dv[j] = ptx::ld_nc_v4(a.dout + t * H + c);
          if (DOT) y[j] = load_v4(a.expert_out + at * H + c);
        }
      }
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const int64_t c = c0 + 8 * j * kThreads;
        float d[8], v[8];
        unpack8(dv[j], d);
        unpack8(y[j], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dot = fmaf(d[i], v[i], dot);
          d[i] *= w;
        }
        if (c < H) ptx::st_v4(a.dy + at * H + c, pack8(d));
      }
    }
  if (DOT) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
    if (threadIdx.x % 32 == 0) part_s[threadIdx.x / 32] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int v = 1; v < kWarps; ++v) dot += part_s[v];
      a.dweights[pair] = dot;
    }
  }
}

}  // namespace

cudaError_t launch_combine_backward(const CombineBackwardArgs& args, cudaStream_t stream) {
  const CombineBackwardArgs a = args;
  const int64_t gaps = a.zero_pad ? static_cast<int64_t>(a.num_experts) * kGapCtas : 0;
  if (a.num_tokens == 0 && gaps == 0) return cudaSuccess;
  const auto run = [&](auto kernel, int64_t ctas) {
    if (gaps + ctas > 2147483647) return cudaErrorInvalidConfiguration;
    count_launch();
    return launch_pdl(kernel, dim3(static_cast<unsigned>(gaps + ctas)), kThreads, 0, stream, a);
  };
  const bool dot = a.dweights != nullptr;
  // Few long rows: a CTA a slot.  top-8, 7168 columns, against a CTA a token (cold L2, with
  // the launch): 1 token 8 to 12 us, 48 tokens 14 to 18, 128 18 to 20, 256 the same.
  const int64_t pairs = a.num_tokens * a.topk;
  if (pairs <= 1024 && a.hidden >= 2048)
    return dot ? run(combine_backward_slot_kernel<true>, pairs) : run(combine_backward_slot_kernel<false>, pairs);
  // Two vectors a lane at least; more warps where tokens alone do not fill the SMs.  32768
  // tokens x top-8 x 4096: 8 warps 655 us, one 678; 20000 x top-4 x 2048: 145 and 125.
  int warps = a.hidden >= 4096 ? 8 : a.hidden >= 2048 ? 4 : a.hidden >= 1024 ? 2 : 1;
  while (warps < kWarps && a.num_tokens * warps < static_cast<int64_t>(kWarps) * device_sm_count()) warps *= 2;
  const int64_t ctas = ceil_div64(a.num_tokens, kWarps / warps);
#define MOE_COMBINE_CASE(W, S)    \
  if (warps == W && slots == S)   \
    return dot ? run(combine_backward_kernel<W, S, true>, ctas) : run(combine_backward_kernel<W, S, false>, ctas);
#define MOE_COMBINE_SLOTS(W) MOE_COMBINE_CASE(W, 2) MOE_COMBINE_CASE(W, 4) MOE_COMBINE_CASE(W, 8)
  const int slots = a.topk <= 2 ? 2 : a.topk <= 4 ? 4 : 8;
  MOE_COMBINE_SLOTS(1)
  MOE_COMBINE_SLOTS(2)
  MOE_COMBINE_SLOTS(4)
  MOE_COMBINE_SLOTS(8)
#undef MOE_COMBINE_SLOTS
#undef MOE_COMBINE_CASE
  return cudaErrorInvalidValue;
}

}  // namespace moe
