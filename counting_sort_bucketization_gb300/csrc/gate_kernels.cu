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
#include "gate_common.cuh"

namespace moe {
namespace {

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

  if (lane == 0 && routed > 0) atomicAdd(&cnt_s[E], routed);
  add_columns<VPL>(acc, E, sum_s, [](int l, int i) { return column<VEC>(l, i); });
  finish_sums(a, sum_s, cnt_s, red_s, last_s);
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
