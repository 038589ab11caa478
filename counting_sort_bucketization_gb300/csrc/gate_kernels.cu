// gate_kernels.cu -- the top-k gate of a mixture-of-experts layer with its
// balance loss, and the gradient of both with respect to the logits.
//
// One warp owns a token; lane j holds the columns j, j+32, ... in registers (or
// 4j..4j+3, 4j+128.., where rows can be read four values at a time), so a row is
// read once and every reduction over experts is a warp reduction.
//
//   key_e = l_e + bias_e (one fp32 addition), as integers that sort like the
//   floats.  The K-th largest of the lanes' own maxima bounds the K-th largest key
//   from below; the few keys that reach it are listed in shared memory and each
//   counts those before it (larger, or equal with a lower id): its slot.  If more
//   than 32 reach it, the keys are taken one after the other by redux.max /
//   redux.min.  A key of -inf is not taken.
//   s = softmax(l) or sigmoid(l), q = s / sum(s); w_k = scale * s_k / D, with D the sum of
//   the picks' s (or 1), each quotient taken relative to its own largest score.
//   Balance loss: coef * E * sum_e f_e P_e with P_e the mean of q over the
//   routed tokens and f_e = count_e / (K * routed tokens).
//
// A row without a key above -inf routes nowhere: ids -1, weights 0, not counted
// as routed.  A row with a NaN or +inf key is treated the same and recorded in
// the error word.
//
// The sums over tokens are kept in fp32 a lane and column while a warp walks
// its tokens, then summed over warps, CTAs and last over the CTAs' partials in
// a fixed order, so results do not change from run to run.
//
// 131072 x 384 fp32, top-8: forward 112 us (214 MB), backward 72 us (415 MB, 5.8
// TB/s).  The backward pass is bound by HBM, the forward pass by the issue of its
// ~720 instructions a token, most of them for the choice (bf16 logits, half the
// bytes, take 124 us).  Listing the candidates took it from 210 us, where each pick was
// a pass over all keys, to 131 us; rows four values at a time and the next row's loads a
// token ahead did the rest.  64 x 256, top-8: 7 us, the launch and one reduction.
// From 513 experts on a lane's 32 columns and the next token's do not fit its registers
// (up to 420 bytes of spills a thread): 65536 x 1000, 171 us forward, 85 backward.
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

template <int VPL, typename T, bool SIGMOID, bool VEC>
__global__ void __launch_bounds__(kGateThreads, VPL <= 8 ? 4 : VPL <= 12 ? 3 : 2) gate_forward_kernel(GateArgs a) {
  extern __shared__ uint8_t smem[];
  const int E = a.num_experts, K = a.topk;
  float* sum_s = reinterpret_cast<float*>(smem);       // [E]
  int* cnt_s = reinterpret_cast<int*>(smem) + E;       // [E + 1]: picks of each expert, routed tokens
  __shared__ bool last_s;
  __shared__ uint64_t list_s[kGateWarps][32];
  __shared__ float list_l_s[kGateWarps][32];
  __shared__ float red_s[kGateWarps];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  uint64_t* list = list_s[warp];
  float* list_l = list_l_s[warp];
  float* bias_s = reinterpret_cast<float*>(smem) + 2 * E + 1;   // [32 * VPL], with a bias
  for (int e = threadIdx.x; e < E; e += kGateThreads) sum_s[e] = 0.0f;
  for (int e = threadIdx.x; e <= E; e += kGateThreads) cnt_s[e] = 0;
  __syncthreads();
  ptx::grid_dependency_wait();
  const bool biased = a.bias != nullptr;
  if (biased)
    for (int e = threadIdx.x; e < 32 * VPL; e += kGateThreads) bias_s[e] = e < E ? a.bias[e] : 0.0f;
  __syncthreads();

  float acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
  const T* logits = static_cast<const T*>(a.logits);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kGateWarps;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + warp;
  int routed = 0;
  float next[VPL];
  load_row<VPL, T, VEC>(logits + t * a.logits_stride, t < a.num_tokens, lane, E, next);
  for (; t < a.num_tokens; t += stride) {
    const T* row = logits + t * a.logits_stride;
    float l[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = next[i];
    load_row<VPL, T, VEC>(row + stride * a.logits_stride, t + stride < a.num_tokens, lane, E, next);

    unsigned u[VPL], best = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      // the addition turns -0 into +0 (they tie) and any NaN into the one that sorts above +inf
      const float key = l[i] + (biased ? bias_s[column<VEC>(lane, i)] : 0.0f);
      u[i] = sortable(key);
      best = max(best, u[i]);
    }
    unsigned top = __reduce_max_sync(kFull, best);
    if (top >= kKeyInf && lane == 0) set_error(a.err, MOE_ERR_INVALID_ARG);
    const bool route = top < kKeyInf && top > kKeyNegInf;
    int mine = -1, slot = lane;            // this lane's pick and its place among the K
    float w = 0.0f;
    if (route) {
      // without a bias the largest key is the largest logit
      float m = SIGMOID ? 0.0f : !biased ? unsortable(top) : row_max<VPL>(l);

      // The K-th largest lane maximum (equal ones go together: a lower bound still).
      unsigned floor = top;
      {
        unsigned rest = best;
        for (int k = 1; k < K && floor > kKeyNegInf; ++k) {
          if (rest == floor) rest = 0;
          floor = __reduce_max_sync(kFull, rest);
        }
        floor = max(floor, kKeyNegInf + 1);
      }
      int found = 0;
      float picked = 0.0f;                 // the pick's logit
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const unsigned who = __ballot_sync(kFull, u[i] >= floor);
        if (who == 0) continue;
        if (u[i] >= floor) {
          const int at = found + __popc(who & ptx::lanemask_lt());
          if (at < 32) {
            list[at] = static_cast<uint64_t>(u[i]) << 32 | ~static_cast<unsigned>(column<VEC>(lane, i));
            if (biased) list_l[at] = l[i];
          }
        }
        found += __popc(who);
      }
      __syncwarp();
      if (found <= 32) {
        const uint64_t own = lane < found ? list[lane] : 0;
        picked = biased ? list_l[lane] : unsortable(static_cast<unsigned>(own >> 32));
        int before = 0;
#pragma unroll 4
        for (int j = 0; j < found; ++j) before += list[j] > own;
        if (lane < found) {
          if (before < K) mine = static_cast<int>(~static_cast<unsigned>(own));
          slot = before;
        }
      } else {
        for (int k = 0; k < K && top > kKeyNegInf; ++k) {
          unsigned lowest = kFull;
#pragma unroll
          for (int i = VPL - 1; i >= 0; --i)
            if (u[i] == top) lowest = static_cast<unsigned>(column<VEC>(lane, i));
          const unsigned id = __reduce_min_sync(kFull, lowest);
          if (lane == k) {
            mine = static_cast<int>(id);
            picked = load_logit(row + mine);
          }
          best = 0;
#pragma unroll
          for (int i = 0; i < VPL; ++i) {
            if (column<VEC>(lane, i) == static_cast<int>(id)) u[i] = 0;
            best = max(best, u[i]);
          }
          top = __reduce_max_sync(kFull, best);
        }
      }
      __syncwarp();   // the list is read
      bool tiny;
      const float inv = __fdividef(1.0f, scores<VPL, T, SIGMOID, VEC>(l, m, tiny, row, lane, E));
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] += l[i] * inv;
      ++routed;
      const bool pick = mine >= 0;
      if (pick) atomicAdd(&cnt_s[mine], 1);
      float s = 0.0f;
      if (pick && (SIGMOID || !a.normalize)) s = SIGMOID ? sigmoid(picked) : exp_neg(picked - m) * inv;
      if (a.normalize) {
        // without a bias the largest pick is the largest logit
        const float top_pick = SIGMOID || !biased ? m : unsortable(__reduce_max_sync(kFull, pick ? sortable(picked) : 0u));
        s = share_of_picks<SIGMOID>(pick, picked, s, top_pick);
      }
      w = a.scale * s;
    }
    if (slot < K) {
      a.topk_idx[t * K + slot] = mine;
      a.weights[t * K + slot] = w;
    }
  }

  // The CTA's sums: warps one after the other, so the order is fixed.
  if (lane == 0 && routed > 0) atomicAdd(&cnt_s[E], routed);
  for (int w = 0; w < kGateWarps; ++w) {
    if (w == warp) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int col = column<VEC>(lane, i);
        if (col < E) sum_s[col] += acc[i];
      }
    }
    __syncthreads();
  }
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

// Gradient.  With g_e = dloss * coef * E * f_e / routed and A = sum_e q_e g_e, the
// balance loss gives log s_e the gradient q_e (g_e - A).  The weights give that of a pick
//   d_k = scale * r_k * (dw_k - sum_j r_j dw_j), r_k = s_k / D   (normalised)
//   d_k = scale * s_k * dw_k                                     (not),
// and d log s_e / d l_j is (e == j) - p_j for softmax, where only the second d has a sum
// c over the picks, and (1 - s_e) on the diagonal for sigmoid.  The picked columns are
// written by lane k after the row, over the value the row store left there.
//
// Sigmoids take more registers: a CTA an SM fewer than softmax measured faster where more
// spill (131072 x 256, 53 against 76 us; x 384, 71 against 87; 65536 x 1000, 104 against 113).
template <int VPL, typename T, bool SIGMOID, bool VEC>
__global__ void __launch_bounds__(kGateThreads, VPL <= 8 ? (SIGMOID ? 4 : 5) : VPL <= 12 ? (SIGMOID ? 3 : 4) : VPL <= 16 || !SIGMOID ? 2 : 1) gate_backward_kernel(GateArgs a) {
  const int E = a.num_experts, K = a.topk;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  ptx::grid_dependency_wait();
  float g[VPL];
  const float routed = static_cast<float>(max(*a.routed_tokens, 1));
  const float coef = a.dloss != nullptr ? *a.dloss * a.balance_coef * static_cast<float>(E) /
                                              (static_cast<float>(K) * routed * routed) : 0.0f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int col = column<VEC>(lane, i);
    g[i] = col < E ? coef * static_cast<float>(a.expert_count[col]) : 0.0f;
  }
  const T* logits = static_cast<const T*>(a.logits);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kGateWarps;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + warp;
  float next[VPL];
  load_row<VPL, T, VEC>(logits + t * a.logits_stride, t < a.num_tokens, lane, E, next);
  // the token's picks and their gradients, also a token ahead
  const auto load_pick = [&](int64_t tok, int64_t* id, float* d) {
    const bool in = lane < K && tok < a.num_tokens;
    *id = in ? a.topk_idx[tok * K + lane] : -1;
    *d = in && a.dweights != nullptr ? a.dweights[tok * K + lane] : 0.0f;
  };
  int64_t next_id;
  float next_dw;
  load_pick(t, &next_id, &next_dw);
  for (; t < a.num_tokens; t += stride) {
    const T* row = logits + t * a.logits_stride;
    T* out = static_cast<T*>(a.dlogits) + t * a.dlogits_stride;
    float l[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = next[i];
    load_row<VPL, T, VEC>(row + stride * a.logits_stride, t + stride < a.num_tokens, lane, E, next);
    int64_t mine = next_id;
    float dw = next_dw;
    load_pick(t + stride, &next_id, &next_dw);
    if (mine >= E) {
      mine = -1;
      set_error(a.err, MOE_ERR_BAD_EXPERT_ID);
    }
    if (!__any_sync(kFull, mine >= 0)) {   // routed nowhere: no gradient
      const float zero[VPL] = {};
      store_row<VPL, T, VEC>(out, lane, E, zero);
      continue;
    }
    float m = SIGMOID ? 0.0f : row_max<VPL>(l);
    bool tiny;
    float dot;
    const float inv = share(1.0f, scores<VPL, T, SIGMOID, VEC>(l, m, tiny, row, lane, E, g, &dot));
    const float A = dot * inv;

    const bool pick = mine >= 0;
    const float lk = pick ? load_logit(row + mine) : 0.0f;
    if (!pick) dw = 0.0f;
    float q = 0.0f, s = 0.0f, rest = 1.0f; // the pick's share of the row, its score, and what that lacks to 1
    if (pick) {
      if (!SIGMOID || tiny) q = exp_neg(lk - m) * inv;
      if (SIGMOID) {
        float large, small;
        sigmoids(lk, large, small);
        s = lk >= 0.0f ? large : small;
        rest = lk >= 0.0f ? small : large;
      } else {
        s = q;
      }
      if (SIGMOID && !tiny) q = s * inv;
    }
    float d;                               // of the weights, with respect to the logarithm of the pick's score
    float c = 0.0f;
    if (a.normalize) {
      const float top = SIGMOID ? 0.0f : unsortable(__reduce_max_sync(kFull, pick ? sortable(lk) : 0u));
      const float r = share_of_picks<SIGMOID>(pick, lk, s, top);
      d = a.scale * r * (dw - warp_sum(r * dw));
    } else {
      d = a.scale * s * dw;
      if (!SIGMOID) c = warp_sum(d);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      l[i] = l[i] * inv * ((g[i] - A) - c);
    __syncwarp();   // every lane has its pick's logit, which may lie where another stores
    store_row<VPL, T, VEC>(out, lane, E, l);
    __syncwarp();
    if (pick) {
      const float gk = coef * static_cast<float>(a.expert_count[mine]);
      store_logit(out + mine, SIGMOID ? rest * (q * (gk - A) + d) : q * ((gk - A) - c) + d);
    }
  }
}

template <typename T, bool SIGMOID>
cudaError_t launch_gate(const GateArgs& a, bool backward, cudaStream_t stream) {
  const int vpl = (a.num_experts + 31) / 32;
  const size_t smem = backward ? 0 : 4 * (static_cast<size_t>(2 * a.num_experts + 1) + 32 * kGateMaxVpl);
  count_launch();
  // One wave of CTAs walks the tokens.
  const auto run = [&](auto kernel) {
    const int ctas = cached_occupancy(kernel, kGateThreads, smem);
    const int64_t most = min64(static_cast<int64_t>(ctas > 0 ? ctas : 1) * device_sm_count(), kGateMaxCtas);
    const int64_t grid = max64(1, min64(ceil_div64(a.num_tokens, kGateWarps), most));
    return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), kGateThreads, smem, stream, a);
  };
  // Four values at a time where every row starts on a vector's boundary.
  const uintptr_t vec = 4 * sizeof(T);
  const bool wide = a.num_experts % 4 == 0 && a.logits_stride % 4 == 0 && aligned(a.logits, vec) &&
                    (!backward || (a.dlogits_stride % 4 == 0 && aligned(a.dlogits, vec)));
#define MOE_GATE_CASE(V)                                                                            \
  if (vpl <= V)                                                                                     \
    return backward ? (wide ? run(gate_backward_kernel<V, T, SIGMOID, true>)                        \
                            : run(gate_backward_kernel<V, T, SIGMOID, false>))                      \
                    : (wide ? run(gate_forward_kernel<V, T, SIGMOID, true>)                         \
                            : run(gate_forward_kernel<V, T, SIGMOID, false>));
  // Up to 64 columns a lane has one or two of its own.
#define MOE_GATE_NARROW(V)                                               \
  if (vpl <= V)                                                          \
    return backward ? run(gate_backward_kernel<V, T, SIGMOID, false>)    \
                    : run(gate_forward_kernel<V, T, SIGMOID, false>);
  MOE_GATE_NARROW(1)
  MOE_GATE_NARROW(2)
#undef MOE_GATE_NARROW
  MOE_GATE_CASE(4)
  MOE_GATE_CASE(8)
  MOE_GATE_CASE(12)
  MOE_GATE_CASE(16)
  MOE_GATE_CASE(32)
#undef MOE_GATE_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

// The gate writes topk_idx, which the layout kernels may read before their
// griddepcontrol.wait, so it never releases its dependents early.
cudaError_t launch_gate(const GateArgs& a, bool backward, cudaStream_t stream) {
  if (backward && a.num_tokens == 0) return cudaSuccess;
  if (a.logits_bf16)
    return a.sigmoid ? launch_gate<uint16_t, true>(a, backward, stream) : launch_gate<uint16_t, false>(a, backward, stream);
  return a.sigmoid ? launch_gate<float, true>(a, backward, stream) : launch_gate<float, false>(a, backward, stream);
}

}  // namespace moe
