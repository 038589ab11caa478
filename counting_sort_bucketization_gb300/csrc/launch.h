// launch.h -- host-side launchers of the library's kernels (internal).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"

namespace moe {

size_t count_smem_bytes(const moe_layout_desc& d, const TilePlan& p);
size_t rank_smem_bytes(const moe_layout_desc& d, const TilePlan& p);

// topk_idx as int64 (the default) or int32.
struct IdsRef {
  const void* ptr;
  bool i32;
};

// count_tiles_kernel + scan_columns_kernel.
cudaError_t launch_count(const moe_layout_desc& d, const TilePlan& p, IdsRef ids, int32_t* expert_count,
                         int32_t* rank_count, int* err, int32_t* hist, int32_t* rhist, cudaStream_t stream);

// rank_maps_kernel.
cudaError_t launch_rank(const moe_layout_desc& d, const TilePlan& p, IdsRef ids, const int32_t* hist_prefix,
                        const int32_t* expert_count, const int32_t* rank_count, int32_t* expert_offset,
                        int32_t* rank_psum, int32_t* dst_slot, int32_t* src_idx, int64_t capacity,
                        int32_t* total_rows, int* err, cudaStream_t stream);

// Count + scan + rank: one cooperative kernel when every tile fits on the
// GPU at once, else the three kernels above.
cudaError_t launch_build(const moe_layout_desc& d, const TilePlan& p, IdsRef ids, int32_t* expert_count,
                         int32_t* rank_count, int32_t* hist, int32_t* rhist, unsigned* barrier_words,
                         int32_t* expert_offset, int32_t* rank_psum, int32_t* dst_slot, int32_t* src_idx,
                         int64_t capacity, int32_t* total_rows, int* err, cudaStream_t stream);

// cumulative[e] += expert_count[e] (int64 running totals across calls).
cudaError_t launch_accumulate_stats(const int32_t* expert_count, int E, int64_t* cumulative, cudaStream_t stream);

// rank_rows_kernel: the non-expand (rank-contiguous) slot map.
cudaError_t launch_rank_rows(const moe_layout_desc& d, const TilePlan& p, IdsRef ids, const int32_t* rhist_prefix,
                             const int32_t* rank_count, int32_t* rank_slot, int32_t* rank_src, int64_t capacity,
                             int* err, cudaStream_t stream);

struct PermuteArgs {
  const uint8_t* x;
  const uint8_t* sf;
  int64_t row_bytes;
  int64_t sf_row_bytes;
  const int32_t* dst_slot;
  const int32_t* total_rows;     // rows the layout uses (checked against capacity)
  const int32_t* expert_offset;  // gap rows (zero_pad only)
  const int32_t* expert_count;
  uint8_t* recv_x;
  uint8_t* recv_sf;
  int64_t capacity;
  int64_t num_tokens;
  int topk;
  int num_experts;
  int zero_pad;
  int* err;
  unsigned* work;                // [2] token counter + finished-CTA counter (zero between launches)
  bool non_expand;               // rows of the non-expand layout (sizes the dynamic kernel's pieces)
  uint64_t wait_ns;              // bound on each mbarrier wait (set by launch_permute)
  unsigned extra_tx;             // test hook: bytes no copy delivers, on each CTA's first stage
};

cudaError_t launch_permute(const PermuteArgs& a, cudaStream_t stream);

struct CombineArgs {
  const uint16_t* expert_out;  // bf16 bits
  int64_t expert_out_rows;
  int64_t hidden;
  const int32_t* dst_slot;
  const float* weights;
  uint16_t* out;               // bf16 bits
  int64_t num_tokens;
  int topk;
  int* err;
  unsigned* work;              // [2] token counter + finished-CTA counter (zero between launches)
  uint64_t wait_ns;            // bound on each mbarrier wait (set by launch_combine)
};

cudaError_t launch_combine(const CombineArgs& a, cudaStream_t stream);

struct SfColMajorArgs {
  const uint32_t* sf;          // [num_tokens, cols] 4-byte scale words
  int64_t cols;
  const int32_t* src;          // token of each receive row; -1 = gap row
  const int32_t* total_rows;   // rows in use (checked against capacity)
  uint32_t* out;               // column j at out + j * ld
  int64_t ld;
  int64_t capacity;
  int64_t num_tokens;
  int zero_pad;
  int* err;
};

cudaError_t launch_sf_col_major(const SfColMajorArgs& a, cudaStream_t stream);

// Argument checks shared by the C entry points (moe_layout_api.cu).
int check_desc(const moe_layout_desc* d);
int check_workspace(const moe_layout_desc* d, const void* ws, size_t ws_bytes, WorkspaceLayout* out);
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

// ------------------------------------------------ gate (gate_kernels.cu)
// CTAs of the forward kernel at most: each leaves one partial of the sums over
// tokens in the gate's workspace, and each group of kGateGroup CTAs one of its own:
// [error word | tickets | pad to 256 B][fp32 kGatePartials x E]
// [int32 kGatePartials x (E + 1)].
constexpr int kGateMaxCtas = 608;
constexpr int kGateGroup = 24;
constexpr int kGatePartials = kGateMaxCtas + (kGateMaxCtas + kGateGroup - 1) / kGateGroup;
static_assert(16 + 4 * (1 + (kGateMaxCtas + kGateGroup - 1) / kGateGroup) <= 256, "tickets");

struct GateArgs {
  const void* logits;
  const float* bias;             // may be null
  int64_t logits_stride;         // elements
  int64_t num_tokens;
  int num_experts;
  int topk;
  bool logits_bf16;
  bool sigmoid;
  bool normalize;
  float scale;
  float balance_coef;
  int64_t* topk_idx;             // written forward, read backward
  float* weights;
  int32_t* expert_count;         // written forward, read backward
  float* prob_mean;
  int32_t* routed_tokens;        // written forward, read backward
  float* balance_loss;
  float* part_sum;
  int32_t* part_cnt;
  unsigned* ticket;              // of all, then of each group; zero between launches
  int* err;
  const float* dweights;         // backward; may be null
  const float* dloss;            // backward; may be null
  void* dlogits;
  int64_t dlogits_stride;
};

cudaError_t launch_gate(const GateArgs& a, bool backward, cudaStream_t stream);

// ------------------------------------------------ 8-bit rows (quantize_kernels.cu)
struct QuantRowsArgs {
  const uint16_t* x;             // bf16 bits [rows, cols], or [rows, 2 * cols] with swiglu
  int64_t rows;
  int64_t cols;
  const int32_t* total_rows;     // rows in use, or null: all
  uint8_t* q;                    // e4m3 [rows, cols]
  float* sf;                     // scale of (row, block) at row * sf_row_stride + block * sf_block_stride
  int64_t sf_row_stride;
  int64_t sf_block_stride;
  bool swiglu;
};

cudaError_t launch_quantize_rows(const QuantRowsArgs& a, cudaStream_t stream);

struct QuantColsArgs {
  const uint16_t* x;             // bf16 bits [capacity, cols]
  int64_t capacity;
  int64_t cols;
  const int32_t* expert_offset;
  const int32_t* expert_count;
  int num_experts;
  uint8_t* q;                    // e4m3 [cols, ld]
  int64_t ld;
  float* sf;                     // [capacity / 128, cols]
  int* err;
};

cudaError_t launch_quantize_cols(const QuantColsArgs& a, cudaStream_t stream);

struct SwigluBackwardArgs {
  const uint16_t* gate_up;       // bf16 bits [rows, 2 * width]
  const uint16_t* dh;            // bf16 bits [rows, width]
  int64_t rows;
  int64_t width;
  const int32_t* total_rows;     // rows in use, or null: all
  uint16_t* dgate_up;
};

cudaError_t launch_swiglu_backward(const SwigluBackwardArgs& a, cudaStream_t stream);

// ------------------------------------------------ expert products (expert_gemm_kernel.cu)
struct ExpertGemmArgs {
  const void* x;                 // e4m3: receive rows [capacity, width_in]; gradient: [width_in, sf_ld]
  const float* x_sf;
  int64_t sf_ld;                 // pitch of x_sf; gradient: pitch of both operands
  int64_t capacity;
  int64_t width_in;
  const void* w;                 // e4m3: weights [E, width_out, width_in]; gradient: dy [width_out, sf_ld]
  const float* w_sf;
  int64_t width_out;
  const int32_t* expert_offset;
  const int32_t* expert_count;
  void* out;
  bool out_fp32;
  bool accumulate;
  int num_experts;
  int64_t pairs;                 // (token, slot) pairs the layout was built for
  int* err;
};

// The kernel's view of either product: rows of out come from receive rows
// (gradient: rows of dy), its columns from the weights (gradient: rows of x^T).
struct GemmParams {
  const float* row_sf;           // scale of (k-block, row) at k-block * row_sf_pitch + row
  int64_t row_sf_pitch;
  const float* col_sf;           // weights' scales; gradient: x_sf
  int out_cols;                  // columns (and pitch) of out
  int dy_rows;                   // gradient: rows of out of an expert
  int kblocks;                   // forward: k-blocks of a row
  int splits;                    // CTAs that share a tile's k-blocks (kFew)
  int num_experts;
  const int32_t* expert_offset;
  const int32_t* expert_count;
  int64_t capacity;
  void* out;
  bool out_fp32;
  bool accumulate;
  int* err;
  uint64_t wait_ns;              // bound on each mbarrier wait
  unsigned extra_tx;             // test hook: bytes no copy delivers, on each CTA's (pair's) first stage
};

cudaError_t launch_expert_gemm(const ExpertGemmArgs& a, cudaStream_t stream);
cudaError_t launch_expert_wgrad(const ExpertGemmArgs& a, cudaStream_t stream);

// Limit of every in-kernel wait and the test hooks that make a wait run out
// (moe_debug_set_waits); the launchers copy them into the kernels' arguments.
struct WaitConfig {
  uint64_t limit_ns;        // bound on any in-kernel wait (default kWaitLimitNs)
  unsigned barrier_extra;   // added to the fused layout's grid-barrier targets (0 in normal use)
  unsigned extra_tx;        // bytes added to each CTA's first permute stage (0 in normal use)
};
WaitConfig wait_config();

// Streaming multiprocessors of the current device (cached per device).
int device_sm_count();

// Host-side launch settings, looked up once instead of on every call.
//   ensure_smem_limit: raise `func`'s dynamic shared-memory limit to at least
//     `smem` bytes in the current context; the runtime call is made only when
//     the limit must grow (cached per context, so a context created after a
//     device reset sets it again).
//   cached_occupancy: resident CTAs per SM of `func` at (threads, smem) on
//     the current device, 0 if the query failed (then not cached).
//   cooperative_launch_supported: the current device's attribute, cached.
//   current_context_id: a nonzero identity of the current context, 0 if none.
cudaError_t ensure_smem_limit(const void* func, size_t smem);
int cached_occupancy(const void* func, int threads, size_t smem);
bool cooperative_launch_supported();
uint64_t current_context_id();

template <typename... KArgs>
cudaError_t ensure_smem_limit(void (*func)(KArgs...), size_t smem) {
  return ensure_smem_limit(reinterpret_cast<const void*>(func), smem);
}
template <typename... KArgs>
int cached_occupancy(void (*func)(KArgs...), int threads, size_t smem) {
  return cached_occupancy(reinterpret_cast<const void*>(func), threads, smem);
}

}  // namespace moe
