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
// 32 bits with the errors' bound in hand, and a token with a decision within it (a few in ten
// thousand) is done again with keys of two floats after the loop over the tokens: one that
// has its candidates listed from those (exact_rank, about 1 us), others from all experts
// (exact_picks, about 8).  Calls within the loop cost all tokens registers (131072 x 384 in 16
// groups 194 us, 168 without them, when both were tried).  Equal logits with equal biases tie exactly, experts and
// groups whose largest keys are such, and where no bias differs from another the order of the
// logits is that of the keys; none of these is left open.
//
// One warp a token, as in the gate (gate_kernels.cu).  A lane has V columns side by side where
// they are of one group and rows lie on vectors' boundaries: the groups' two largest keys then
// come from registers and shuffles (else 32 / G lanes a group walk its keys in shared
// memory).  Candidates are the keys from a bound on: what the token before had as its K-th
// key, a little lower; or, if fewer than K or more than 32 reach that, the K-th largest of the
// lanes' two largest.  The bound changes the work, not the result.  It stays above -inf, the
// key of closed experts and of columns past E, which are never listed.  Where more than 32 keys
// reach it still (equal ones, K near 32, groups that few lanes hold) they are picked one after
// the other: 131072 x 128, top-32, 645 us, and 131072 x 1024, one group of 16, top-8, 564.
//
// 131072 x 384, sigmoid with bias, top-8, the L2 flushed: 137 us, in 16 groups of which 4 stay
// 175 (256 experts in 8 groups 158); the logits once are 201 MB, 30 us.  A token takes 780
// instructions (128 experts 645, so most do not depend on their number; 440 are the choice and
// the weights), in 16 groups 960, which is 100 us of issue slots; the rest is their chain, with
// 24 warps an SM (ncu: issue slots 56 % busy, ALU 58 %, DRAM 16 %).  Half a
// warp a token has two chains a warp and took 158 in place of 188 when it was tried, with 4 us
// more for 64 tokens and twice the code.  64 x 256 in 8 groups: 8.9 us a call, the launch and one
// token's chain.  Rows of zeros (padding): 351 us for 131072 x 384 in 16 groups.
#include <cfloat>

#include "gate_common.cuh"

namespace moe {
namespace {

// Bounds of what a 32-bit score errs by, of the row's largest score (a sigmoid counts as 1/8
// at most), u = 2^-24.
// Sigmoid: e^-x as 2^(-x log2 e) errs by (1.5 |x| + 4) u of itself, 1 + e^-x and the reciprocal by
// 3 u more; |x| <= 28 unless the scores' sum is tiny (then they are e^(x - max)).  48 u of a small
// score; of one near 1 e^-x's error counts s (1 - s): 4.4 u.
constexpr float kErrSigmoid = 0x1p-18f;
// Softmax: e^x errs by (2.5 |x| + 4) u of itself, 5 u of the largest; the sum by as much in the
// mean, where |x| is at most log E, and by V + 5 additions; the quotient by 5 u.
template <int V>
constexpr float kErrSoftmax = (V + 48) * 0x1p-24f;

// Numbers as sums of two floats, good to about 2^-46: hi is the sum rounded, lo the rest.
// (The 64-bit unit does 2 multiply-adds a cycle and SM; a token redone with it took 40 us.)
// Knuth's sum of two numbers with its error, Dekker's where the first is the larger, and his
// product with the error by one fused multiply-add.  Intrinsics, so that no addition is fused
// with a product.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two quick_sum(float a, float b) {   // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Two exact_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two add(Two a, Two b) {
  const Two s = exact_sum(a.hi, b.hi);
  return quick_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ Two mul(Two a, Two b) {
  const float p = __fmul_rn(a.hi, b.hi);
  const float e = __fmaf_rn(a.hi, b.hi, -p);
  return quick_sum(p, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, e)));
}
__device__ __forceinline__ Two reciprocal(Two d) {
  const float q = __frcp_rn(d.hi);
  const float rest = __fmaf_rn(-q, d.lo, __fmaf_rn(-q, d.hi, 1.0f));
  return quick_sum(q, __fmul_rn(rest, q));
}
// e^x, x <= 0: x = n ln 2 + r, the Taylor series of e^r (its terms from r^7 on need one float),
// times 2^n.  ln 2 comes in three parts, of which n times the first two is exact (Cody and
// Waite's reduction).  Below
// 2^-125 zero.
__device__ __forceinline__ Two two_exp(Two x) {
  if (!(x.hi > -86.0f)) return {0.0f, 0.0f};
  const float n = rintf(x.hi * 1.4426950408889634f);
  const Two a = exact_sum(__fmaf_rn(-n, 0x1.62e4p-1f, x.hi), __fmul_rn(-n, 0x1.7f7cp-20f));
  const Two r = quick_sum(a.hi, __fadd_rn(a.lo, __fmaf_rn(-n, 0x1.1cf79ap-36f, x.lo)));
  float q = 1.0f / 479001600.0f;
  q = fmaf(q, r.hi, 1.0f / 39916800.0f);
  q = fmaf(q, r.hi, 1.0f / 3628800.0f);
  q = fmaf(q, r.hi, 1.0f / 362880.0f);
  q = fmaf(q, r.hi, 1.0f / 40320.0f);
  q = fmaf(q, r.hi, 1.0f / 5040.0f);
  Two p = add(mul(r, {q, 0.0f}), {0x1.6c16c2p-10f, -0x1.27d27ep-35f});   // 1/720
  p = add(mul(r, p), {0x1.111112p-7f, -0x1.dddddep-32f});                // 1/120
  p = add(mul(r, p), {0x1.555556p-5f, -0x1.555556p-30f});                // 1/24
  p = add(mul(r, p), {0x1.555556p-3f, -0x1.555556p-28f});                // 1/6
  p = add(mul(r, p), {0.5f, 0.0f});
  p = add(mul(r, p), {1.0f, 0.0f});
  p = add(mul(r, p), {1.0f, 0.0f});
  const float scale = __uint_as_float(static_cast<unsigned>(static_cast<int>(n) + 127) << 23);
  return {p.hi * scale, p.lo * scale};
}
__device__ __forceinline__ Two two_sigmoid(float l) {
  const Two e = two_exp({-fabsf(l), 0.0f});
  const Two s = reciprocal(add({1.0f, 0.0f}, e));
  return l >= 0.0f ? s : mul(e, s);
}

// Keys of two floats as integers in their order; 0 is none.
__device__ __forceinline__ uint64_t ordered(Two k) {
  return static_cast<uint64_t>(sortable(k.hi + 0.0f)) << 32 | sortable(k.lo + 0.0f);
}
__device__ __forceinline__ Two number(uint64_t u) {
  return {unsortable(static_cast<unsigned>(u >> 32)), unsortable(static_cast<unsigned>(u))};
}
__device__ __forceinline__ Two half(Two k) { return {0.5f * k.hi, 0.5f * k.lo}; }
__device__ __forceinline__ Two plus_bias(Two s, float b) {
  const Two k = exact_sum(s.hi, b);
  return quick_sum(k.hi, __fadd_rn(k.lo, s.lo));
}
// The largest of the lanes' keys.
__device__ __forceinline__ uint64_t warp_best(uint64_t key) {
  const unsigned hi = __reduce_max_sync(kFull, static_cast<unsigned>(key >> 32));
  const unsigned lo = __reduce_max_sync(kFull, static_cast<unsigned>(key >> 32) == hi ? static_cast<unsigned>(key) : 0u);
  return static_cast<uint64_t>(hi) << 32 | lo;
}

// One over the softmax's sum (sigmoid: 1).
template <typename T, bool SIGMOID>
__device__ __forceinline__ Two exact_scale(const T* row, float m, int E) {
  if (SIGMOID) return {1.0f, 0.0f};
  Two sum{0.0f, 0.0f};
#pragma unroll 2
  for (int e = threadIdx.x % 32; e < E; e += 32) sum = add(sum, two_exp(exact_sum(load_logit(row + e), -m)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum = add(sum, {__shfl_xor_sync(kFull, sum.hi, o), __shfl_xor_sync(kFull, sum.lo, o)});
  return reciprocal(sum);
}
template <typename T, bool SIGMOID>
__device__ __forceinline__ uint64_t exact_key(const T* row, float m, Two scale, const float* bias, int e) {
  const float l = load_logit(row + e), b = bias[e];
  const Two s = SIGMOID ? two_sigmoid(l) : mul(two_exp(exact_sum(l, -m)), scale);
  return l > -INFINITY && b > -INFINITY ? ordered(plus_bias(s, b)) : 0;
}

// How many of `found` <= 32 candidates, a lane each, come before the lane's.
template <typename T, bool SIGMOID>
__device__ __noinline__ int exact_rank(const T* row, float m, const float* bias, int E, int id, int found) {
  const Two scale = exact_scale<T, SIGMOID>(row, m, E);
  const uint64_t own = threadIdx.x % 32 < found ? exact_key<T, SIGMOID>(row, m, scale, bias, id) : 0;
  int before = 0;
  for (int j = 0; j < found; ++j) {
    const uint64_t k = __shfl_sync(kFull, own, j);
    const int other = __shfl_sync(kFull, id, j);
    before += k > own || (k == own && other < id);
  }
  return before;
}

// A token's picks from such keys: lane k < K gets pick k's id, or -1.  `key` is the warp's,
// [E]; `m` the row's largest logit.
template <typename T, bool SIGMOID>
__device__ __noinline__ int exact_picks(const GateArgs& a, const T* row, float m, const float* bias, bool biased, uint64_t* key) {
  const int lane = threadIdx.x % 32;
  const int E = a.num_experts, per = E / a.num_groups;
  const Two scale = exact_scale<T, SIGMOID>(row, m, E);
#pragma unroll 2
  for (int e = lane; e < E; e += 32) key[e] = exact_key<T, SIGMOID>(row, m, scale, bias, e);
  __syncwarp();
  if (a.topk_groups < a.num_groups) {
    uint64_t score = 0;                  // of group `lane`
    if (lane < a.num_groups) {
      uint64_t hi = 0, lo = 0;
#pragma unroll 4
      for (int j = 0; j < per; ++j) {
        const uint64_t k = key[lane * per + j];
        lo = max(lo, min(hi, k));
        hi = max(hi, k);
      }
      // Halves, which add without an overflow; a group's only key is halved too.
      if (a.group_sum == 1 || hi == 0) score = hi;
      else score = ordered(lo > 0 ? add(half(number(hi)), half(number(lo))) : half(number(hi)));
    }
    unsigned kept = 0;
    for (int j = 0; j < a.topk_groups; ++j) {
      const uint64_t best = warp_best(score);
      if (best == 0) break;
      const int g = __ffs(__ballot_sync(kFull, score == best)) - 1;
      kept |= 1u << g;
      if (lane == g) score = 0;
    }
    __syncwarp();
    for (int e = lane; e < E; e += 32) {
      if (!(kept >> (e / per) & 1)) key[e] = 0;
      else if (!biased && key[e] > 0) key[e] = static_cast<uint64_t>(sortable(load_logit(row + e) + 0.0f)) << 32;
    }
  }
  int mine = -1;
  for (int k = 0; k < a.topk; ++k) {
    __syncwarp();
    uint64_t own = 0;
    unsigned id = kFull;
#pragma unroll 4
    for (int e = lane; e < E; e += 32)
      if (key[e] > own) own = key[e], id = e;
    const uint64_t best = warp_best(own);
    if (best == 0) break;
    id = __reduce_min_sync(kFull, own == best ? id : kFull);
    if (lane == k) mine = static_cast<int>(id);
    if (id % 32 == lane) key[id] = 0;
  }
  __syncwarp();
  return mine;
}

// Where a token's choice is left open, its first id says so until the loop over the tokens is
// over; one token whose candidates are listed is kept by its warp instead.
constexpr int64_t kOpen = -2;
struct Late {
  int64_t token = 0;
  int found = 0;                         // candidates
  float m = 0.0f;                        // the row's largest logit
  int* ids;                              // shared memory, [32]
};

// Ids and weights of a token from its picks: a lane's pick (or -1) and its place.
template <typename T, bool SIGMOID>
__device__ __forceinline__ void settle(const GateArgs& a, int* cnt_s, int64_t token, float m, int mine, int slot) {
  const T* row = static_cast<const T*>(a.logits) + token * a.logits_stride;
  const bool pick = mine >= 0;
  const float picked = pick ? load_logit(row + mine) : 0.0f;
  float p = 0.0f;
  if (pick) atomicAdd(&cnt_s[mine], 1);
  if (SIGMOID) {
    if (pick) p = sigmoid(picked);
  } else if (!a.normalize) {
    float sum = 0.0f;
    for (int e = threadIdx.x % 32; e < a.num_experts; e += 32) sum += exp_neg(load_logit(row + e) - m);
    p = share(pick ? exp_neg(picked - m) : 0.0f, warp_sum(sum));
  }
  if (a.normalize)
    p = share_of_picks<SIGMOID>(pick, picked, p, unsortable(__reduce_max_sync(kFull, pick ? sortable(picked) : 0u)));
  if (slot < a.topk) {
    a.topk_idx[token * a.topk + slot] = mine;
    a.weights[token * a.topk + slot] = a.scale * p;
  }
}

// The warp's choices left open, from exact keys.  Its i-th token is first + i * stride.
template <typename T, bool SIGMOID>
__device__ __noinline__ void settle_open(const GateArgs& a, const float* bias_s, bool biased, uint64_t* key64, int* cnt_s,
                                         const Late& late, bool any_open, int64_t first, int64_t stride) {
  const int lane = threadIdx.x % 32, E = a.num_experts, K = a.topk;
  const T* logits = static_cast<const T*>(a.logits);
  if (late.found > 0) {
    const int id = lane < late.found ? late.ids[lane] : 0;
    const int before = exact_rank<T, SIGMOID>(logits + late.token * a.logits_stride, late.m, bias_s, E, id, late.found);
    settle<T, SIGMOID>(a, cnt_s, late.token, late.m, lane < late.found && before < K ? id : -1, lane < late.found ? before : lane);
    __syncwarp();
  }
  if (!any_open) return;
  for (int64_t base = first; base < a.num_tokens; base += 32 * stride) {
    const int64_t own = base + lane * stride;
    unsigned open = __ballot_sync(kFull, own < a.num_tokens && a.topk_idx[own * K] == kOpen);
    for (; open != 0; open &= open - 1) {
      const int64_t tok = base + (__ffs(open) - 1) * stride;
      const T* row = logits + tok * a.logits_stride;
      float m = -INFINITY;
      for (int e = lane; e < E; e += 32) m = fmaxf(m, load_logit(row + e));
      m = unsortable(__reduce_max_sync(kFull, sortable(m + 0.0f)));
      settle<T, SIGMOID>(a, cnt_s, tok, m, exact_picks<T, SIGMOID>(a, row, m, bias_s, biased, key64), lane);
    }
  }
}

__device__ __forceinline__ void add_best(float& hi, float& lo, float k) {
  lo = fmaxf(lo, fminf(hi, k));
  hi = fmaxf(hi, k);
}
// The two largest of a lane's and another's two largest.
__device__ __forceinline__ void merge_best(float& hi, float& lo, float h2, float l2) {
  lo = fmaxf(fmaxf(lo, l2), fminf(hi, h2));
  hi = fmaxf(hi, h2);
}

// Biases to shared memory ([padded], zeros past E), and what is to be known of them.
// Biases that are all the same number change no order.  Others than numbers close experts
// (-inf) or spoil the tokens that have them open (NaN, +inf).  All threads of the CTA.
struct Biases {
  bool differ;
  bool odd;
};
__device__ __forceinline__ Biases load_biases(const GateArgs& a, float* bias_s, int padded) {
  bool differ = false, odd = false;
  for (int e = threadIdx.x; e < padded; e += kGateThreads) {
    const float b = a.bias != nullptr && e < a.num_experts ? a.bias[e] : 0.0f;
    bias_s[e] = b;
    if (a.bias != nullptr && e < a.num_experts) {
      differ |= b != a.bias[0];
      odd |= !(fabsf(b) < INFINITY);
    }
  }
  Biases r;
  r.odd = __syncthreads_or(odd);
  r.differ = __syncthreads_or(differ) || r.odd;
  return r;
}

// The column of a lane's i-th value: V side by side (BLOCKED), or 32 apart.
template <int V, bool BLOCKED>
__device__ __forceinline__ int route_column(int lane, int i) {
  return BLOCKED ? lane * V + i : lane + 32 * i;
}
template <int V, typename T, bool BLOCKED>
__device__ __forceinline__ void load_route_row(const T* row, bool live, int lane, int E, float* l) {
  constexpr int kStep = BLOCKED && V % 4 == 0 ? 4 : 1;
#pragma unroll
  for (int i = 0; i < V; i += kStep) {
    const int col = route_column<V, BLOCKED>(lane, i);
#pragma unroll
    for (int j = 0; j < kStep; ++j) l[i + j] = -INFINITY;
    if (live && col < E) {
      if constexpr (kStep == 4) load4(row + col, l + i);
      else l[i] = load_logit(row + col);
    }
  }
}

template <int V, typename T, bool SIGMOID, bool BLOCKED>
__global__ void __launch_bounds__(kGateThreads, V <= 4 ? 4 : V <= 12 ? 3 : 2) route_forward_kernel(GateArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int E = a.num_experts, K = a.topk, G = a.num_groups, per = E / G;
  __shared__ bool last_s;
  __shared__ __align__(16) float list_k_s[kGateWarps][32];
  __shared__ int list_id_s[kGateWarps][32];
  __shared__ float red_s[kGateWarps];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  float* list_k = list_k_s[warp];
  int* list_id = list_id_s[warp];
  uint64_t* key64 = reinterpret_cast<uint64_t*>(smem) + static_cast<size_t>(warp) * (32 * V);   // for exact_picks
  float* key_s = reinterpret_cast<float*>(key64);                                                // for groups not BLOCKED
  float* sum_s = reinterpret_cast<float*>(reinterpret_cast<uint64_t*>(smem) + kGateWarps * 32 * V);   // [E]
  float* bias_s = sum_s + 32 * V;                   // [32 * V]
  int* cnt_s = reinterpret_cast<int*>(bias_s + 32 * V);   // [E + 1]: picks of each expert, routed tokens
  for (int e = threadIdx.x; e < E; e += kGateThreads) sum_s[e] = 0.0f;
  for (int e = threadIdx.x; e <= E; e += kGateThreads) cnt_s[e] = 0;
  ptx::grid_dependency_wait();
  const Biases biases = load_biases(a, bias_s, 32 * V);
  const bool biased = biases.differ, check_keys = biases.odd;

  constexpr int kLine = 128 / static_cast<int>(sizeof(T));   // values
  const bool limited = a.topk_groups < G;
  const bool by_logit = !biased && a.group_sum == 1;   // a group's score is in the order of its best logit
  // Lanes of a group (BLOCKED: those that hold it), the lane's group, its place there.
  int lanes = BLOCKED ? max(1, per / V) : 32;
  if (!BLOCKED)
    while (lanes * G > 32) lanes /= 2;
  const int group = lane / lanes, sub = lane % lanes;
  const int turn = limited && !BLOCKED ? (group * lanes) % per : 0;   // groups start apart, so that they meet no bank together
  const unsigned inverse = (0x400000u + per - 1) / per;   // e / per = e * inverse >> 22 for e < 1024

  bool any_open = false;
  Late late;
  late.ids = reinterpret_cast<int*>(key64) + 32 * V;        // past the groups' keys
  // Keys from `guess` on are candidates, if between K and 32 reach it: a little below the
  // K-th best key of the token before.
  float guess = INFINITY, slack = 0.0f;

  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  const T* logits = static_cast<const T*>(a.logits);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kGateWarps;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + warp;
  int routed = 0;
  for (; t < a.num_tokens; t += stride) {
    const T* row = logits + t * a.logits_stride;
    float key[V], s[V];                  // key: first the logit
    load_route_row<V, T, BLOCKED>(row, true, lane, E, key);
    // The next token's row on its way to the L2 (in registers it costs spills: 131072 x 384 147
    // us in place of 139).
    if (t + stride < a.num_tokens)
      for (int c = lane * kLine; c < E; c += 32 * kLine)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(row + stride * a.logits_stride + c));
    float m = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, key[i]);
    m = unsortable(__reduce_max_sync(kFull, sortable(m + 0.0f)));

    // Scores; a NaN among the logits shows in their sum.  (What they err by is no matter for
    // the means, and the picks' weights come from better ones.)
    float sum = 0.0f;
    const float finite = fmaxf(m, -FLT_MAX);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float x = (SIGMOID ? -key[i] : key[i] - finite) * 1.4426950408889634f;
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(s[i]) : "f"(x));
      if (SIGMOID) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s[i]) : "f"(1.0f + s[i]));
      sum += s[i];
    }
    sum = warp_sum(sum);
    bool bad = !(m < INFINITY) || !(sum < INFINITY);
    bool route = !bad && m > -INFINITY;
    int64_t mine = -1;                   // this lane's pick
    int slot = lane;                     // and its place among the K
    float w = 0.0f;
    if (route) {
      float factor = SIGMOID ? 1.0f : __fdividef(1.0f, sum);       // of s to the score
      if (SIGMOID && sum < kTinySum) {   // sigmoids that are e^l to 2^-30: e^(l - m) in their place
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) sum += s[i] = exp_neg(key[i] - m);
        sum = warp_sum(sum);
        factor = exp_neg(m);
      }
      const float inv = __fdividef(1.0f, sum);
      float b[V];
      if (biased) {
        if constexpr (BLOCKED && V % 4 == 0) {
#pragma unroll
          for (int i = 0; i < V; i += 4) load4(bias_s + lane * V + i, b + i);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) b[i] = bias_s[route_column<V, BLOCKED>(lane, i)];
        }
      }
      if (check_keys) {
        bool open = false;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (key[i] > -INFINITY) open |= b[i] != -INFINITY, bad |= !(b[i] < INFINITY);
        bad = __any_sync(kFull, bad);
        route = __any_sync(kFull, open) && !bad;
      }
      if (route)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += s[i] * inv;

      // What a key may err by, but for its own rounding.
      // (a sigmoid is below e^m)
      float most = factor;
      if (SIGMOID) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(most) : "f"(m * 1.4426950408889634f));
      const float err = (SIGMOID ? 1.01f * kErrSigmoid * fminf(most, 0.125f) : kErrSoftmax<V> * most) + 0x1p-120f;
      const auto near = [&](float x, float y) {
        return biased && fabsf(x - y) <= 2.0f * err + 0x1p-23f * fmaxf(fabsf(x), fabsf(y));
      };
      bool exact = false;                // the choice is left open
      float hi = -INFINITY, lo = -INFINITY;   // the lane's largest keys
      if (limited && !by_logit) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (biased) key[i] = key[i] > -INFINITY ? fmaf(s[i], factor, b[i]) : -INFINITY;
          if (BLOCKED) add_best(hi, lo, key[i]);
          else key_s[route_column<V, BLOCKED>(lane, i)] = key[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (biased) key[i] = key[i] > -INFINITY ? fmaf(s[i], factor, b[i]) : -INFINITY;
          if (limited && !BLOCKED) key_s[route_column<V, BLOCKED>(lane, i)] = key[i];
          hi = fmaxf(hi, key[i]);
        }
      }
      float own_hi = hi, own_lo = lo;    // of the lane's keys, for the choice
      bool held = true;                  // the lane's experts (BLOCKED) are of a kept group
      unsigned kept = kFull;
      if (limited) {
        if (BLOCKED) {
          if ((lanes & (lanes - 1)) == 0) {
            for (int o = lanes / 2; o > 0; o /= 2)
              merge_best(hi, lo, __shfl_xor_sync(kFull, hi, o), __shfl_xor_sync(kFull, lo, o));
          } else {
            const float h1 = hi, l1 = lo;
            for (int j = 1; j < lanes; ++j) {
              const int from = group * lanes + (sub + j >= lanes ? sub + j - lanes : sub + j);
              merge_best(hi, lo, __shfl_sync(kFull, h1, from & 31), __shfl_sync(kFull, l1, from & 31));
            }
          }
        } else {
          __syncwarp();
          hi = lo = -INFINITY;
          if (group < G)
            for (int j = sub; j < per; j += lanes) {
              int at = j + turn;
              if (at >= per) at -= per;
              add_best(hi, lo, key_s[group * per + at]);
            }
          for (int o = lanes / 2; o > 0; o /= 2)
            merge_best(hi, lo, __shfl_xor_sync(kFull, hi, o), __shfl_xor_sync(kFull, lo, o));
          __syncwarp();                  // the keys are read
        }
        // Without a bias hi and lo are logits: the keys are their scores and the bias that all have.
        const auto key_of = [&](float l) {
          return l > -INFINITY ? (SIGMOID ? sigmoid(l) : exp_neg(fminf(l - m, 0.0f)) * inv) + bias_s[0] : -INFINITY;
        };
        const float k1 = biased || by_logit ? hi : key_of(hi), k2 = biased || by_logit ? lo : key_of(lo);
        // Half the sum of two (two keys of the lowest value would add to -inf, a closed group's score), and
        // what it may err by: half of two keys' errors, their roundings and the sum's.
        const float second = k2 > -INFINITY ? 0.5f * k2 : 0.0f;
        const float score = group >= G ? -INFINITY : a.group_sum == 2 ? 0.5f * k1 + second : k1;
        const float off = by_logit ? 0.0f : err + 0x1p-23f * (0.5f * fabsf(k1) + fabsf(second));
        unsigned rest = sortable(score + 0.0f);
        kept = 0;
        held = false;
        for (int j = 0; j < a.topk_groups; ++j) {
          const unsigned best = __reduce_max_sync(kFull, rest);
          if (best <= kKeyNegInf) break;
          const int g = __shfl_sync(kFull, group, __ffs(__ballot_sync(kFull, rest == best)) - 1);
          kept |= 1u << g;
          if (group == g) rest = kKeyNegInf, held = true;
        }
        if (!by_logit) {
          // What a group left may reach, and the least that a kept one may be.
          const bool there = score > -INFINITY;
          const unsigned high = sortable(score + off), low = sortable(score - off);
          const unsigned reach = __reduce_max_sync(kFull, there && !held ? high : 0u);
          const unsigned least = __reduce_min_sync(kFull, held ? low : kFull);
          if (route && reach >= least) {
            // Groups that may be on either side are left open unless they tie exactly: equal logits as their two
            // largest (keys: and nothing near one of them that is not the same logit and bias).
            const bool between = held ? low <= reach : there && high >= least;
            const unsigned own1 = sortable(hi + 0.0f), own2 = a.group_sum == 2 ? sortable(lo + 0.0f) : 0u;
            const unsigned h1 = __reduce_max_sync(kFull, between ? own1 : 0u), h2 = __reduce_max_sync(kFull, between ? own2 : 0u);
            exact = __any_sync(kFull, between && (own1 != h1 || own2 != h2));
            if (biased && !exact) {
              const unsigned groups = __reduce_or_sync(kFull, between ? 1u << group : 0u);
              const float top1 = unsortable(h1), top2 = h2 > kKeyNegInf ? unsortable(h2) : top1;
              const auto in_groups = [&](int i) {
                return (groups >> (BLOCKED ? group : static_cast<unsigned>(route_column<V, BLOCKED>(lane, i)) * inverse >> 22 & 31) & 1) != 0;
              };
              unsigned at1 = E - 1, at2 = E - 1;
#pragma unroll
              for (int i = 0; i < V; ++i) {
                const unsigned col = route_column<V, BLOCKED>(lane, i);
                if (key[i] == top1 && in_groups(i)) at1 = min(at1, col);
                if (key[i] == top2 && in_groups(i)) at2 = min(at2, col);
              }
              at1 = __reduce_min_sync(kFull, at1);
              at2 = __reduce_min_sync(kFull, at2);
              const float l1 = load_logit(row + at1), b1 = bias_s[at1], l2 = load_logit(row + at2), b2 = bias_s[at2];
              exact = top1 != top2 && near(top1, top2);
#pragma unroll
              for (int i = 0; i < V; ++i) {
                if (!(key[i] > -INFINITY) || !in_groups(i)) continue;
                const bool first = near(key[i], top1);
                if (!first && !near(key[i], top2)) continue;
                const int col = route_column<V, BLOCKED>(lane, i);
                exact |= load_logit(row + col) != (first ? l1 : l2) || bias_s[col] != (first ? b1 : b2);
              }
              exact = __any_sync(kFull, exact);
            }
          }
        }
        if (!BLOCKED) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const unsigned g = static_cast<unsigned>(route_column<V, BLOCKED>(lane, i)) * inverse >> 22;
            if (!(kept >> (g & 31) & 1)) key[i] = -INFINITY;
          }
        } else if (!held) {
          own_hi = own_lo = -INFINITY;
        }
      }
      // Few lanes have keys left, or many picks are wanted: a lane's second counts too.
      if ((limited && !(BLOCKED && biased && !by_logit)) || (!limited && K > 8)) {
        own_hi = own_lo = -INFINITY;
        if (!BLOCKED || held)
#pragma unroll
          for (int i = 0; i < V; ++i) add_best(own_hi, own_lo, key[i]);
      }
      if (route && !exact) {
        // Keys from `least` on, which is above -inf: that is the key of closed experts and past E.
        const auto mark = [&](float least) {
          unsigned bits = 0;
          if (!BLOCKED || held)
#pragma unroll
            for (int i = 0; i < V; ++i)
              if (key[i] >= least) bits |= 1u << i;
          return bits;
        };
        // How many are marked in all and by the lanes before this one.
        int found, at;
        const auto count = [&](unsigned bits) {
          const int c = __popc(bits);
          found = at = 0;
#pragma unroll
          for (int j = 0; (1 << j) <= V; ++j) {
            const unsigned who = __ballot_sync(kFull, c >> j & 1);
            found += __popc(who) << j;
            at += __popc(who & ptx::lanemask_lt()) << j;
          }
        };
        unsigned bits = mark(guess);
        count(bits);
        unsigned top = 0;
        float edge = guess;              // what is not marked lies below it
        const bool few = found < K, many = found > 32;
        if (few || many) {
          // The K-th largest of the lanes' largest (equal ones of two lanes go together: a
          // lower bound still), less what it may err by.
          unsigned rest = sortable(own_hi + 0.0f), second = sortable(own_lo + 0.0f);
          top = __reduce_max_sync(kFull, rest);
          unsigned floor = top;
          for (int k = 1; k < K && floor > kKeyNegInf; ++k) {
            if (rest == floor) rest = second, second = 0;
            floor = __reduce_max_sync(kFull, rest);
          }
          float least = -FLT_MAX;
          if (floor > kKeyNegInf) {
            least = unsortable(floor);
            if (biased) least = fmaxf(least - (2.0f * err + 0x1p-22f * fabsf(least)), -FLT_MAX);
          }
          bits = mark(least);
          count(bits);
          edge = -FLT_MAX;               // further below
        }
        float picked = 0.0f, score = 0.0f;   // the pick's logit and score
        int candidate = 0;
        bool beyond = false;             // what is not listed may belong to the picks
        if (found <= 32) {
          // Ids, keys; then both in the keys' order.
          for (; bits != 0; bits &= bits - 1) list_id[at++] = route_column<V, BLOCKED>(lane, __ffs(bits) - 1);
          __syncwarp();
          const int id = lane < found ? list_id[lane] : 0;
          const float l = lane < found ? load_logit(row + id) : 0.0f;
          const float bias = bias_s[id];
          score = SIGMOID ? sigmoid(l) : exp_neg(fminf(l - m, 0.0f)) * inv;
          const float k = lane >= found ? -INFINITY : biased ? score + bias : l;
          list_k[lane] = k;
          __syncwarp();
          int before = 0;
          for (int j = 0; j < found; j += 4) {
            const float4 o = *reinterpret_cast<const float4*>(list_k + j);
            before += (o.x > k) + (o.y > k) + (o.z > k) + (o.w > k);
          }
          // Equal keys: the lower id first, which is the lower lane where a lane's columns are
          // side by side.
          unsigned same = __match_any_sync(kFull, lane < found ? before : 32 + lane);
          if (BLOCKED) {
            before += __popc(same & ptx::lanemask_lt());
          } else {
            const int mates = __reduce_max_sync(kFull, __popc(same));
            int earlier = 0;
            if (mates > 1)
              for (int j = 0; j < found; ++j) {
                const int other = __shfl_sync(kFull, id, j);
                earlier += (same >> j & 1) != 0 && other < id;
              }
            before += earlier;
          }
          __syncwarp();
          if (lane < found) list_k[before] = k, list_id[before] = id;
          __syncwarp();
          // A pick is compared with the next one, and every key behind the picks with the last of them: where
          // neither is near, or is the same logit and bias, the order is that of the numbers.
          if (biased && lane < found) {
            const int mate = before < K - 1 ? before + 1 : K - 1;
            if (before == K - 1) {
              exact = beyond = near(k, edge);
            } else if (mate < found && near(k, list_k[mate])) {
              const int other = list_id[mate];
              exact = load_logit(row + other) != l || bias_s[other] != bias;
            }
          }
          // The next token's guess.  A key may be the type's lowest value.  What a row whose K-th key is a mask leaves
          // as slack is gone after one ordinary row: only halved, -1e9 took 25 and the lowest value over 100.
          if (found >= K) {
            const float last = list_k[K - 1];
            if (few) slack = fminf(fmaxf(2.0f * slack, 0x1p-4f * (list_k[0] - last) + 0x1p-8f * fabsf(last)), FLT_MAX);
            else if (many || found > 20) slack = fminf((many ? 0.5f : 0.75f) * slack, list_k[0] - last + 0x1p-4f * fabsf(last));
            guess = fmaxf(last - slack, -FLT_MAX);
          }
          candidate = id;
          if (lane < found) {
            if (before < K) mine = id, picked = l;
            slot = before;
          }
        } else {
          // More than a list holds: one pick after the other, each near no other number, nor what is left the last.
          const float first = unsortable(top);
          float last_key = first, last_l = 0.0f, last_b = 0.0f;
          float h;
          for (int k = 0; k < K && top > kKeyNegInf; ++k) {
            const float want = unsortable(top);
            unsigned lowest = kFull;
            if (!BLOCKED || held)
#pragma unroll
              for (int i = V - 1; i >= 0; --i)
                if (key[i] == want) lowest = static_cast<unsigned>(route_column<V, BLOCKED>(lane, i));
            const unsigned id = __reduce_min_sync(kFull, lowest);
            const float lk = load_logit(row + id), bk = bias_s[id];
            if (k > 0 && near(last_key, want) && (lk != last_l || bk != last_b)) exact = true;
            last_key = want, last_l = lk, last_b = bk;
            if (k == K - 1 && want < first) {      // (a padding row's equal keys say nothing)
              slack = fminf(fmaxf(few ? 2.0f * slack : 0.0f, 0x1p-4f * (first - want) + 0x1p-8f * fabsf(want)), FLT_MAX);
              guess = fmaxf(want - slack, -FLT_MAX);
            }
            if (lane == k) mine = id, picked = lk, score = SIGMOID ? sigmoid(lk) : exp_neg(lk - m) * inv;
            h = -INFINITY;
            if (!BLOCKED || held)
#pragma unroll
              for (int i = 0; i < V; ++i) {
                if (route_column<V, BLOCKED>(lane, i) == static_cast<int>(id)) key[i] = -INFINITY;
                h = fmaxf(h, key[i]);
              }
            top = __reduce_max_sync(kFull, sortable(h + 0.0f));
          }
          if (biased && top > kKeyNegInf && (!BLOCKED || held))
#pragma unroll
            for (int i = 0; i < V; ++i)
              if (key[i] > -INFINITY && near(key[i], last_key)) {
                const int col = route_column<V, BLOCKED>(lane, i);
                exact |= load_logit(row + col) != last_l || bias_s[col] != last_b;
              }
        }
        __syncwarp();                    // the list is read
        exact = __any_sync(kFull, exact);
        if (exact) {
          mine = -1;
          if (found <= 32 && late.found == 0 && !__any_sync(kFull, beyond)) {
            late.token = t, late.found = found, late.m = m;
            if (lane < found) late.ids[slot] = candidate;
            exact = false;
            slot = 32;                   // nothing is written yet
          }
        }
        const bool pick = mine >= 0;
        if (pick) atomicAdd(&cnt_s[mine], 1);
        float p = pick ? score : 0.0f;
        if (a.normalize) {
          const float top_pick = SIGMOID ? m : unsortable(__reduce_max_sync(kFull, pick ? sortable(picked) : 0u));
          p = share_of_picks<SIGMOID>(pick, picked, p, top_pick);
        }
        w = a.scale * p;
      }
      if (route) ++routed;
      if (exact) {
        any_open = true;
        slot = lane;
        if (lane == 0) mine = kOpen;
      }
    }
    if (bad && lane == 0) set_error(a.err, MOE_ERR_INVALID_ARG);
    if (slot < K) {
      a.topk_idx[t * K + slot] = mine;
      a.weights[t * K + slot] = w;
    }
  }
  __syncwarp();
  if (late.found > 0 || any_open)
    settle_open<T, SIGMOID>(a, bias_s, biased, key64, cnt_s, late, any_open,
                            static_cast<int64_t>(blockIdx.x) * kGateWarps + warp, stride);
  if (lane == 0 && routed > 0) atomicAdd(&cnt_s[E], routed);
  add_columns<V>(acc, E, sum_s, [](int l, int i) { return route_column<V, BLOCKED>(l, i); });
  finish_sums(a, sum_s, cnt_s, red_s, last_s);
}

template <typename T, bool SIGMOID>
cudaError_t launch_typed(const GateArgs& a, cudaStream_t stream) {
  const int v = (a.num_experts + 31) / 32, per = a.num_experts / a.num_groups;
  // Columns side by side where a lane's are of one group, and (from 4 a lane on) every row
  // starts on a vector's boundary.
  const bool wide = a.num_experts % 4 == 0 && a.logits_stride % 4 == 0 && aligned(a.logits, 4 * sizeof(T));
  const auto blocked = [&](int V) { return (V < 4 || wide) && (a.topk_groups == a.num_groups || per % V == 0); };
  count_launch();
  // One wave of CTAs walks the tokens.
  const auto run = [&](auto kernel, int V) {
    const size_t smem = 8 * static_cast<size_t>(kGateWarps) * 32 * V + 4 * (2 * 32 * static_cast<size_t>(V) + a.num_experts + 1);
    if (cudaError_t e = ensure_smem_limit(kernel, smem)) return e;
    const int ctas = cached_occupancy(kernel, kGateThreads, smem);
    const int64_t most = min64(static_cast<int64_t>(ctas > 0 ? ctas : 1) * device_sm_count(), kGateMaxCtas);
    const int64_t grid = max64(1, min64(ceil_div64(a.num_tokens, kGateWarps), most));
    return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), kGateThreads, smem, stream, a);
  };
#define MOE_ROUTE_CASE(V) \
  if (v <= V) return blocked(V) ? run(route_forward_kernel<V, T, SIGMOID, true>, V) : run(route_forward_kernel<V, T, SIGMOID, false>, V);
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
