// route_kernels.cu -- routing by scores: the forward pass of a top-k gate whose choice of
// experts goes by score + bias, limited to the best groups of experts.  (Its gradient is
// the gate's: the choice carries none.)
//
//   s = softmax(l) or sigmoid(l); key_e = s_e + bias_e, -inf where l_e is (a closed expert).
//   Groups are E / G experts side by side.  A group's score is the sum of its 1 or 2 largest
//   keys above -inf; the best topk_groups stay, then the K largest keys of those.  Ties go to
//   the lower id.  Weights, counts and balance loss are the gate's.
//
// Keys are numbers, not their approximations in 32 bits: two of them may lie closer than
// those err (their order then hangs on how a sigmoid was computed).  So a warp compares in
// 32 bits with the errors' bound in hand, and where a decision lies within it, the token
// is done again in 64 bits (choose_exact).  Equal logits with equal biases tie exactly, and
// where no bias differs from another the order of the logits is that of the keys; neither
// needs 64 bits.
//
// One warp a token, as in the gate (gate_kernels.cu, whose list of candidates this is).
// The groups' two largest keys: 32 / G lanes a group walk its keys in shared memory.
#include "gate_common.cuh"

namespace moe {
namespace {

// Bounds of what a 32-bit score errs by, of the row's largest score.  Sigmoid: e^-x 2^-21.4,
// the sum and the reciprocal 2^-22 (of itself), so 2^-20 of a small one and 2^-21 at 1/2 and
// above.  Softmax: two exponentials, a sum of up to 37 additions one after the other, a
// quotient.
constexpr float kErrSigmoid = 0x1p-20f;
constexpr float kErrSoftmax = 0x1p-18f;

struct Pick64 {
  double key;
  int id;
};
__device__ __forceinline__ Pick64 warp_best(Pick64 p) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double k = __shfl_xor_sync(kFull, p.key, o);
    const int id = __shfl_xor_sync(kFull, p.id, o);
    if (k > p.key || (k == p.key && id < p.id)) p.key = k, p.id = id;
  }
  return p;
}

// The token's picks in 64 bits: lane k < K gets pick k's id, or -1.  `key` is the warp's.
template <typename T, bool SIGMOID>
__device__ __noinline__ int choose_exact(const T* row, float m, const float* bias, double* key, int E, int K, int G,
                                         int topk_groups, int group_sum, bool biased) {
  const int lane = threadIdx.x % 32;
  const double none = -INFINITY;
  double sum = 0.0;
  for (int e = lane; e < E; e += 32) {
    const double l = static_cast<double>(load_logit(row + e));
    const double s = SIGMOID ? 1.0 / (1.0 + exp(-l)) : exp(l - static_cast<double>(m));
    sum += s;
    key[e] = s;
  }
  if (!SIGMOID) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  }
  for (int e = lane; e < E; e += 32) {
    const double s = SIGMOID ? key[e] : key[e] / sum;
    key[e] = load_logit(row + e) > -INFINITY ? s + static_cast<double>(bias[e]) : none;
  }
  __syncwarp();
  unsigned kept = kFull;
  const int per = E / G;
  if (topk_groups < G) {
    Pick64 own{none, lane};
    if (lane < G) {
      double hi = none, lo = none;
      for (int e = lane * per; e < (lane + 1) * per; ++e) {
        const double k = key[e];
        if (k > hi) lo = hi, hi = k;
        else if (k > lo) lo = k;
      }
      own.key = group_sum == 2 && lo > none ? hi + lo : hi;
    }
    kept = 0;
    for (int j = 0; j < topk_groups; ++j) {
      const Pick64 best = warp_best(own);
      if (!(best.key > none)) break;
      kept |= 1u << best.id;
      if (lane == best.id) own.key = none;
    }
  }
  if (!biased) {
    __syncwarp();
    for (int e = lane; e < E; e += 32) key[e] = static_cast<double>(load_logit(row + e));
    __syncwarp();
  }
  int mine = -1;
  for (int k = 0; k < K; ++k) {
    Pick64 own{none, E};
    for (int e = lane; e < E; e += 32)
      if (key[e] > own.key && (kept >> (e / per) & 1)) own.key = key[e], own.id = e;
    const Pick64 best = warp_best(own);
    if (!(best.key > none)) break;
    if (lane == k) mine = best.id;
    __syncwarp();
    if (lane == 0) key[best.id] = none;
    __syncwarp();
  }
  __syncwarp();
  return mine;
}

template <int VPL, typename T, bool SIGMOID, bool VEC>
__global__ void __launch_bounds__(kGateThreads, VPL <= 8 ? 4 : VPL <= 12 ? 3 : 2) route_forward_kernel(GateArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int E = a.num_experts, K = a.topk, G = a.num_groups, per = E / G;
  __shared__ bool last_s;
  __shared__ uint64_t list_s[kGateWarps][32];
  __shared__ float list_l_s[kGateWarps][32];
  __shared__ float red_s[kGateWarps];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  uint64_t* list = list_s[warp];
  float* list_l = list_l_s[warp];
  // a warp's keys: 32 bits each for the groups, 64 where they are done again
  double* key64 = reinterpret_cast<double*>(smem) + static_cast<size_t>(warp) * (32 * VPL);
  float* key_s = reinterpret_cast<float*>(key64);
  float* sum_s = reinterpret_cast<float*>(reinterpret_cast<double*>(smem) + kGateWarps * 32 * VPL);   // [E]
  int* cnt_s = reinterpret_cast<int*>(sum_s) + E;   // [E + 1]: picks of each expert, routed tokens
  float* bias_s = sum_s + 2 * E + 1;                // [32 * VPL]
  for (int e = threadIdx.x; e < E; e += kGateThreads) sum_s[e] = 0.0f;
  for (int e = threadIdx.x; e <= E; e += kGateThreads) cnt_s[e] = 0;
  ptx::grid_dependency_wait();
  // biases that are all the same number change no order
  bool differ = false;
  for (int e = threadIdx.x; e < 32 * VPL; e += kGateThreads) {
    const float b = a.bias != nullptr && e < E ? a.bias[e] : 0.0f;
    bias_s[e] = b;
    differ |= a.bias != nullptr && e < E && (!(b == a.bias[0]) || !(fabsf(b) < INFINITY));
  }
  const bool biased = __syncthreads_or(differ);

  // lanes of a group, and where each starts in it: apart, so that groups meet no bank together
  const bool limited = a.topk_groups < G;
  int lanes = 32;
  while (lanes * G > 32) lanes /= 2;
  const int group = lane / lanes, sub = lane % lanes;
  const int turn = limited ? (group * lanes) % per : 0;
  const unsigned inverse = (0x400000u + per - 1) / per;   // e / per = e * inverse >> 22 for e < 1024

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
    unsigned u[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = next[i];
    load_row<VPL, T, VEC>(row + stride * a.logits_stride, t + stride < a.num_tokens, lane, E, next);

    // The addition turns -0 into +0 and any NaN into the one that sorts above +inf.
    unsigned best = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      u[i] = sortable(l[i] + 0.0f);
      best = max(best, u[i]);
    }
    unsigned top = __reduce_max_sync(kFull, best);
    bool bad = top >= kKeyInf;
    bool route = !bad && top > kKeyNegInf;
    int mine = -1, slot = lane;            // this lane's pick and its place among the K
    float w = 0.0f;
    if (route) {
      float m = unsortable(top);
      const float m0 = m;
      bool tiny;
      const float inv = __fdividef(1.0f, scores<VPL, T, SIGMOID, VEC>(l, m, tiny, row, lane, E));
      const float factor = SIGMOID ? (tiny ? exp_neg(m0) : 1.0f) : inv;   // to the score itself
      const float most = SIGMOID ? sigmoid(m0) : inv;
      const float err = (SIGMOID ? kErrSigmoid * fminf(most, 0.5f) : kErrSoftmax * most) + 0x1p-120f;
      bool exact = false;                  // some decision lies within the errors

      if (biased) {
        best = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const float key = fmaf(l[i], factor, bias_s[column<VEC>(lane, i)]);
          u[i] = u[i] > kKeyNegInf ? sortable(key + 0.0f) : kKeyNegInf;
          best = max(best, u[i]);
        }
        top = __reduce_max_sync(kFull, best);
        bad = top >= kKeyInf;
        route = !bad && top > kKeyNegInf;
      }
      if (route && limited) {
        const bool by_logit = !biased && a.group_sum == 1;   // the best key is the best logit's
#pragma unroll
        for (int i = 0; i < VPL; i += VEC ? 4 : 1) {
          float k[4];
#pragma unroll
          for (int j = 0; j < (VEC ? 4 : 1); ++j)
            k[j] = u[i + j] <= kKeyNegInf ? -INFINITY
                   : biased || by_logit   ? unsortable(u[i + j])
                                          : fmaf(l[i + j], factor, bias_s[column<VEC>(lane, i + j)]);
          if constexpr (VEC) store4(key_s + column<VEC>(lane, i), k);
          else key_s[column<VEC>(lane, i)] = k[0];
        }
        __syncwarp();
        float hi = -INFINITY, lo = -INFINITY;
        if (group < G)
          for (int j = sub; j < per; j += lanes) {
            int at = j + turn;
            if (at >= per) at -= per;
            const float k = key_s[group * per + at];
            lo = fmaxf(lo, fminf(hi, k));
            hi = fmaxf(hi, k);
          }
        for (int o = lanes / 2; o > 0; o /= 2) {
          const float h2 = __shfl_xor_sync(kFull, hi, o), l2 = __shfl_xor_sync(kFull, lo, o);
          lo = fmaxf(fmaxf(lo, l2), fminf(hi, h2));
          hi = fmaxf(hi, h2);
        }
        const float score = a.group_sum == 2 && lo > -INFINITY ? hi + lo : hi;
        const float off = 2.0f * err + 0x1p-23f * (fabsf(hi) + (lo > -INFINITY ? fabsf(lo) : 0.0f));
        unsigned rest = group < G ? sortable(score + 0.0f) : kKeyNegInf, kept = 0;
        unsigned last = 0;
        float worst = 0.0f;                // of the bounds
        for (int j = 0; j < a.topk_groups; ++j) {
          const unsigned b = __reduce_max_sync(kFull, rest);
          if (b <= kKeyNegInf) break;
          const int g = (__ffs(__ballot_sync(kFull, rest == b)) - 1) / lanes;
          kept |= 1u << g;
          last = b;
          if (group == g) rest = kKeyNegInf, worst = off;
        }
        const unsigned out = __reduce_max_sync(kFull, rest);
        if (out > kKeyNegInf && !by_logit) {
          if (rest == out) worst = fmaxf(worst, off);
          worst = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(worst)));
          exact = unsortable(last) - unsortable(out) <= 2.0f * worst;
        }
        best = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const unsigned g = static_cast<unsigned>(column<VEC>(lane, i)) * inverse >> 22;
          if (!(kept >> (g & 31) & 1)) u[i] = min(u[i], kKeyNegInf);
          best = max(best, u[i]);
        }
        top = __reduce_max_sync(kFull, best);
        __syncwarp();                      // the keys are read
      }
      // Two keys closer than this may be in either order.
      const auto near = [&](float x, float y) {
        return biased && fabsf(x - y) <= 2.0f * err + 0x1p-23f * fmaxf(fabsf(x), fabsf(y));
      };
      float picked = 0.0f;                 // the pick's logit
      if (route && !exact) {
        // The K-th largest lane maximum (equal ones go together: a lower bound still).
        unsigned floor = top;
        {
          unsigned rest = best;
          for (int k = 1; k < K && floor > kKeyNegInf; ++k) {
            if (rest == floor) rest = 0;
            floor = __reduce_max_sync(kFull, rest);
          }
          if (biased && floor > kKeyNegInf) {
            const float f = unsortable(floor);
            floor = sortable(f - (2.0f * err + 0x1p-22f * fabsf(f)));
          }
          floor = max(floor, kKeyNegInf + 1);
        }
        int found = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const unsigned who = __ballot_sync(kFull, u[i] >= floor);
          if (who == 0) continue;
          if (u[i] >= floor) {
            const int at = found + __popc(who & ptx::lanemask_lt());
            if (at < 32) list[at] = static_cast<uint64_t>(u[i]) << 32 | ~static_cast<unsigned>(column<VEC>(lane, i));
          }
          found += __popc(who);
        }
        __syncwarp();
        if (found <= 32) {
          const uint64_t own = lane < found ? list[lane] : 0;
          const int id = static_cast<int>(~static_cast<unsigned>(own));
          picked = lane < found ? (biased ? load_logit(row + id) : unsortable(static_cast<unsigned>(own >> 32))) : 0.0f;
          int before = 0;
#pragma unroll 4
          for (int j = 0; j < found; ++j) before += list[j] > own;
          if (lane < found) {
            if (before < K) mine = id;
            slot = before;
          }
          if (biased) {
            __syncwarp();                  // the list is read
            if (lane < found) list[before] = own, list_l[before] = picked;
            __syncwarp();
            if (mine >= 0 && before + 1 < found) {
              const uint64_t follow = list[before + 1];
              const int other = static_cast<int>(~static_cast<unsigned>(follow));
              if (near(unsortable(static_cast<unsigned>(own >> 32)), unsortable(static_cast<unsigned>(follow >> 32))))
                exact = picked != list_l[before + 1] || bias_s[id] != bias_s[other];
            }
          }
        } else {
          float last_key = INFINITY, last_l = 0.0f, last_b = 0.0f;
          for (int k = 0; k <= K && top > kKeyNegInf; ++k) {
            unsigned lowest = kFull;
#pragma unroll
            for (int i = VPL - 1; i >= 0; --i)
              if (u[i] == top) lowest = static_cast<unsigned>(column<VEC>(lane, i));
            const unsigned id = __reduce_min_sync(kFull, lowest);
            const float lk = load_logit(row + id), bk = bias_s[id], key = unsortable(top);
            if (near(last_key, key) && (lk != last_l || bk != last_b)) exact = true;
            last_key = key, last_l = lk, last_b = bk;
            if (lane == k && k < K) mine = static_cast<int>(id), picked = lk;
            best = 0;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
              if (column<VEC>(lane, i) == static_cast<int>(id)) u[i] = 0;
              best = max(best, u[i]);
            }
            top = __reduce_max_sync(kFull, best);
          }
        }
        __syncwarp();                      // the list is read
      }
      if (route && __any_sync(kFull, exact)) {
        mine = choose_exact<T, SIGMOID>(row, m0, bias_s, key64, E, K, G, a.topk_groups, a.group_sum, biased);
        picked = mine >= 0 ? load_logit(row + mine) : 0.0f;
        slot = lane;
      }
      if (route) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] += l[i] * inv;
        ++routed;
        const bool pick = mine >= 0;
        if (pick) atomicAdd(&cnt_s[mine], 1);
        float s = 0.0f;
        if (pick && (SIGMOID || !a.normalize)) s = SIGMOID ? sigmoid(picked) : exp_neg(picked - m) * inv;
        if (a.normalize) {
          const float top_pick = SIGMOID ? m : unsortable(__reduce_max_sync(kFull, pick ? sortable(picked) : 0u));
          s = share_of_picks<SIGMOID>(pick, picked, s, top_pick);
        }
        w = a.scale * s;
      }
    }
    if (bad && lane == 0) set_error(a.err, MOE_ERR_INVALID_ARG);
    if (slot < K) {
      a.topk_idx[t * K + slot] = mine;
      a.weights[t * K + slot] = w;
    }
  }
  finish_sums<VPL, VEC>(a, acc, routed, sum_s, cnt_s, red_s, last_s);
}

template <typename T, bool SIGMOID>
cudaError_t launch_typed(const GateArgs& a, cudaStream_t stream) {
  const int vpl = (a.num_experts + 31) / 32;
  const bool wide = a.num_experts % 4 == 0 && a.logits_stride % 4 == 0 && aligned(a.logits, 4 * sizeof(T));
  count_launch();
  // One wave of CTAs walks the tokens.
  const auto run = [&](auto kernel, int v) {
    const size_t smem = 8 * static_cast<size_t>(kGateWarps) * 32 * v + 4 * (static_cast<size_t>(2 * a.num_experts + 1) + 32 * v);
    if (cudaError_t e = ensure_smem_limit(kernel, smem)) return e;
    const int ctas = cached_occupancy(kernel, kGateThreads, smem);
    const int64_t most = min64(static_cast<int64_t>(ctas > 0 ? ctas : 1) * device_sm_count(), kGateMaxCtas);
    const int64_t grid = max64(1, min64(ceil_div64(a.num_tokens, kGateWarps), most));
    return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), kGateThreads, smem, stream, a);
  };
  // Up to 64 columns a lane has one or two of its own; four at a time where every row starts
  // on a vector's boundary.
#define MOE_ROUTE_CASE(V) \
  if (vpl <= V) return wide && V >= 4 ? run(route_forward_kernel<V, T, SIGMOID, (V >= 4)>, V) : run(route_forward_kernel<V, T, SIGMOID, false>, V);
  MOE_ROUTE_CASE(1)
  MOE_ROUTE_CASE(2)
  MOE_ROUTE_CASE(4)
  MOE_ROUTE_CASE(8)
  MOE_ROUTE_CASE(12)
  MOE_ROUTE_CASE(16)
  MOE_ROUTE_CASE(32)
#undef MOE_ROUTE_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

// Writes topk_idx, which the layout kernels may read before their griddepcontrol.wait, so
// it never releases its dependents early.
cudaError_t launch_route(const GateArgs& a, cudaStream_t stream) {
  if (a.logits_bf16) return a.sigmoid ? launch_typed<uint16_t, true>(a, stream) : launch_typed<uint16_t, false>(a, stream);
  return a.sigmoid ? launch_typed<float, true>(a, stream) : launch_typed<float, false>(a, stream);
}

}  // namespace moe
