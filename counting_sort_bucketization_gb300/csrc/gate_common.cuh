// gate_common.cuh -- what the top-k gate (gate_kernels.cu) and the routing by scores and
// groups (route_kernels.cu) share: rows of logits a warp at a time, scores, shares of
// picks, and the sums over tokens.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kGateThreads = 256;
constexpr int kGateWarps = kGateThreads / 32;
constexpr int kGateMaxVpl = 32;              // columns of a lane: MOE_MAX_EXPERTS / 32
constexpr float kTinySum = 0x1p-30f;         // sums of sigmoids below it are taken of e^(l - max) instead
constexpr unsigned kKeyNegInf = 0x007fffffu; // sortable keys of -inf and +inf
constexpr unsigned kKeyInf = 0xff800000u;

// Ordinary loads: the gradient may be written over the logits.
__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }

__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  *p = *reinterpret_cast<const uint16_t*>(&b);
}

// Unsigned integers in the order of the floats; never 0.  The NaN of an addition
// (0x7fffffff) comes after +inf.
__device__ __forceinline__ unsigned sortable(float f) {
  const int b = __float_as_int(f);
  return static_cast<unsigned>(b ^ (b >> 31 | static_cast<int>(0x80000000u)));
}
__device__ __forceinline__ float unsortable(unsigned u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// e^x for x <= 0 (-inf too): 2^t with t = x log2 e rounded, times e^(x - t ln 2), whose
// exponent is at most 2^-24 |x| and enters to first order.  (Without it the product's
// rounding errs by 2^-24 |x| of the result; expf takes 5 us more on 131072 x 384, both
// directions.)  ln 2 as one float is good to 2^-28, so what is left is 2^-28 |x| and the
// approximation's 2^-22.  Results below 2^-126 are zero.
__device__ __forceinline__ float exp_neg(float x) {
  x = fmaxf(x, -128.0f);
  const float t = x * 1.4426950408889634f;
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return fmaf(r, fmaf(-t, 0.6931471805599453f, x), r);
}
// sigmoid(|x|) and sigmoid(-|x|).  The smaller is not taken as a difference from one, which
// would have no bits left from 17 on.
__device__ __forceinline__ void sigmoids(float x, float& large, float& small) {
  const float e = exp_neg(-fabsf(x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(large) : "f"(1.0f + e));   // of 1 to 2: 1 ulp
  small = e * large;
}
__device__ __forceinline__ float sigmoid(float x) {
  float large, small;
  sigmoids(x, large, small);
  return x >= 0.0f ? large : small;
}

// A share of a sum of scores.  The sum is zero only where a caller's own ids are of closed
// experts alone.
__device__ __forceinline__ float share(float v, float sum) { return sum > 0.0f ? __fdividef(v, sum) : 0.0f; }

// The column of a lane's i-th value.
template <bool VEC>
__device__ __forceinline__ int column(int lane, int i) {
  return VEC ? (i / 4) * 128 + lane * 4 + i % 4 : lane + 32 * i;
}

__device__ __forceinline__ void load4(const float* p, float* l) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  l[0] = v.x, l[1] = v.y, l[2] = v.z, l[3] = v.w;
}
__device__ __forceinline__ void load4(const uint16_t* p, float* l) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  l[0] = __uint_as_float(v.x << 16), l[1] = __uint_as_float(v.x & 0xffff0000u);
  l[2] = __uint_as_float(v.y << 16), l[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float* v) { *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void store4(uint16_t* p, const float* v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// One row's logits in registers; -inf past E (a multiple of 4 with VEC).
template <int VPL, typename T, bool VEC>
__device__ __forceinline__ void load_row(const T* row, bool live, int lane, int E, float* l) {
#pragma unroll
  for (int i = 0; i < VPL; i += VEC ? 4 : 1) {
    const int col = column<VEC>(lane, i);
    if constexpr (VEC) {
      l[i] = l[i + 1] = l[i + 2] = l[i + 3] = -INFINITY;
      if (live && col < E) load4(row + col, l + i);
    } else {
      l[i] = live && col < E ? load_logit(row + col) : -INFINITY;
    }
  }
}
template <int VPL, typename T, bool VEC>
__device__ __forceinline__ void store_row(T* row, int lane, int E, const float* v) {
#pragma unroll
  for (int i = 0; i < VPL; i += VEC ? 4 : 1) {
    const int col = column<VEC>(lane, i);
    if (col < E) {
      if constexpr (VEC) store4(row + col, v + i);
      else store_logit(row + col, v[i]);
    }
  }
}

template <int VPL>
__device__ __forceinline__ float row_max(const float* l) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
  return unsortable(__reduce_max_sync(kFull, sortable(m)));
}

// Scores of a routed row in place of its logits, up to a common factor; returns their
// sum.  `m` is the row's largest logit (softmax).  Sigmoids whose sum is below 2^-30 are
// e^l to 2^-30 each: e^(l - max) stand in their place, which neither vanish nor lose
// bits, and `tiny` says so, with the largest logit in `m`.  With `g`, the scores' sum
// weighted by it goes to `dot`, and a sigmoid's slope s (1 - s) in the score's place.
template <int VPL, typename T, bool SIGMOID, bool VEC>
__device__ __forceinline__ float scores(float* l, float& m, bool& tiny, const T* row, int lane, int E,
                                        const float* g = nullptr, float* dot = nullptr) {
  float s = 0.0f, d = 0.0f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    // exp(-inf) = 0, and sigmoid(-inf) = 0 / (1 + 0): closed experts score nothing
    if (SIGMOID && g != nullptr) {
      float large, small;
      sigmoids(l[i], large, small);
      const float score = l[i] >= 0.0f ? large : small;
      s += score;
      d += score * g[i];
      l[i] = large * small;
    } else {
      l[i] = SIGMOID ? sigmoid(l[i]) : exp_neg(l[i] - m);
      s += l[i];
    }
  }
  s = warp_sum(s);
  if (!SIGMOID && g != nullptr) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) d += l[i] * g[i];
  }
  tiny = SIGMOID && s < kTinySum;
  if (tiny) {
    load_row<VPL, T, VEC>(row, true, lane, E, l);
    m = row_max<VPL>(l);
    s = d = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      s += l[i] = exp_neg(l[i] - m);       // its own slope: 1 - s is 1
      if (g != nullptr) d += l[i] * g[i];
    }
    s = warp_sum(s);
  }
  if (g != nullptr) *dot = warp_sum(d);
  return s;
}

// A pick's share of the picks' scores, of which `top` is the largest's logit (softmax).
// Each is taken relative to that one's, however small beside the row's; sigmoids only
// where their sum is tiny.
template <bool SIGMOID>
__device__ __forceinline__ float share_of_picks(bool pick, float l, float score, float top) {
  float v = SIGMOID ? score : pick ? exp_neg(l - top) : 0.0f;
  float sum = warp_sum(v);
  if (SIGMOID && sum < kTinySum) {
    top = unsortable(__reduce_max_sync(kFull, pick ? sortable(l) : 0u));
    v = pick ? exp_neg(l - top) : 0.0f;
    sum = warp_sum(v);
  }
  return share(v, sum);
}

// Adds the warps' sums over their tokens (acc: the scores' shares of a lane's columns) to the
// CTA's, one warp after the other, so the order is fixed.
template <int VPL, typename F>
__device__ __forceinline__ void add_columns(const float* acc, int E, float* sum_s, F column_of) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int w = 0; w < kGateWarps; ++w) {
    if (w == warp) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int col = column_of(lane, i);
        if (col < E) sum_s[col] += acc[i];
      }
    }
    __syncthreads();
  }
}

// The CTAs' sums (sum_s: [E]; cnt_s: [E + 1], picks of each expert and routed tokens) to the
// results over the batch.  All threads of every CTA of the grid call it after a barrier.
__device__ __forceinline__ void finish_sums(const GateArgs& a, float* sum_s, int* cnt_s, float* red_s, bool& last_s) {
  const int E = a.num_experts, K = a.topk;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  // Partials of CTAs, then of groups of CTAs: whoever finishes last in a group (and the
  // last group) adds them in their order.
  const int groups = (static_cast<int>(gridDim.x) + kGateGroup - 1) / kGateGroup;
  const int group = static_cast<int>(blockIdx.x) / kGateGroup;
  for (int level = 0; level < 2; ++level) {
    const int first = level == 0 ? group * kGateGroup : kGateMaxCtas;   // rows of partials; the groups' follow the CTAs'
    const int rows = level == 0 ? min(kGateGroup, static_cast<int>(gridDim.x) - first) : groups;
    const int64_t own = level == 0 ? static_cast<int64_t>(blockIdx.x) : kGateMaxCtas + group;
    if (rows == 1) continue;               // the partial in shared memory is the sum
    for (int e = threadIdx.x; e < E; e += kGateThreads) a.part_sum[own * E + e] = sum_s[e];
    for (int e = threadIdx.x; e <= E; e += kGateThreads) a.part_cnt[own * (E + 1) + e] = cnt_s[e];
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      unsigned* ticket = a.ticket + (level == 0 ? 1 + group : 0);
      last_s = atomicAdd(ticket, 1u) == static_cast<unsigned>(rows) - 1;
      if (last_s) *ticket = 0;
    }
    __syncthreads();
    if (!last_s) return;
    __threadfence();
    for (int e = threadIdx.x; e <= E; e += kGateThreads) {
      float sum = 0.0f;
      int c = 0;
#pragma unroll 8
      for (int b = first; b < first + rows; ++b) {
        if (e < E) sum += __ldcg(a.part_sum + static_cast<int64_t>(b) * E + e);
        c += __ldcg(a.part_cnt + static_cast<int64_t>(b) * (E + 1) + e);
      }
      if (e < E) sum_s[e] = sum;
      cnt_s[e] = c;
    }
    __syncthreads();
  }
  const float inv_tokens = 1.0f / static_cast<float>(max(cnt_s[E], 1));
  float part = 0.0f;
  for (int e = threadIdx.x; e < E; e += kGateThreads) {
    const float mean = sum_s[e] * inv_tokens;
    part += mean * static_cast<float>(cnt_s[e]);
    a.expert_count[e] = cnt_s[e];
    a.prob_mean[e] = mean;
  }
  part = warp_sum(part);
  if (lane == 0) red_s[warp] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.0f;
    for (int w = 0; w < kGateWarps; ++w) s += red_s[w];
    *a.routed_tokens = cnt_s[E];
    *a.balance_loss = a.balance_coef * static_cast<float>(E) * s * inv_tokens / static_cast<float>(K);
  }
}

}  // namespace
}  // namespace moe
