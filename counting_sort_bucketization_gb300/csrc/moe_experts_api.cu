// moe_experts_api.cu -- the extern "C" entry points around the layout: gate,
// 8-bit rows, gated activation and expert products.  Argument checks and
// launches; semantics are documented in include/moe_layout.h.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "launch.h"

namespace moe {
namespace {

size_t gate_workspace(int E) {
  const size_t words = static_cast<size_t>(kGatePartials) * static_cast<size_t>(2 * E + 1);
  return (256 + 4 * words + 255) / 256 * 256;
}

int gate_args(const moe_layout_desc* desc, const moe_gate_desc* gate, const void* logits, int64_t logits_stride,
              const float* bias, void* workspace, size_t workspace_bytes, GateArgs* out) {
  if (int st = check_desc(desc)) return st;
  if (gate == nullptr || workspace == nullptr || !aligned(workspace, 256) ||
      workspace_bytes < gate_workspace(desc->num_experts))
    return MOE_ERR_INVALID_ARG;
  if (desc->num_tokens > 0 && (logits == nullptr || logits_stride < desc->num_experts)) return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, gate->logits_bf16 ? 2 : 4) || !aligned(bias, 4)) return MOE_ERR_INVALID_ARG;
  if (logits_stride > MOE_MAX_ROW_BYTES / 4) return MOE_ERR_UNSUPPORTED;
  GateArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.logits_stride = logits_stride;
  a.num_tokens = desc->num_tokens;
  a.num_experts = desc->num_experts;
  a.topk = desc->topk;
  a.logits_bf16 = gate->logits_bf16 != 0;
  a.sigmoid = gate->sigmoid != 0;
  a.normalize = gate->normalize != 0;
  a.scale = gate->scale;
  a.balance_coef = gate->balance_coef;
  a.err = at<int>(workspace, 0);
  a.ticket = at<unsigned>(workspace, 16);
  a.part_sum = at<float>(workspace, 256);
  a.part_cnt = at<int32_t>(workspace, 256 + 4 * static_cast<size_t>(kGatePartials) * desc->num_experts);
  *out = a;
  return MOE_OK;
}

// Whether the gradient's rows may lie on the logits' in a way that the kernel cannot
// take: anything but the same rows or none.  (Ranges that interleave with unlike strides
// count as overlapping.)
bool rows_clash(const void* x, int64_t x_stride, const void* y, int64_t y_stride, int64_t rows, int64_t width) {
  if (x == y && (x_stride == y_stride || rows <= 1)) return false;
  const int64_t a = reinterpret_cast<int64_t>(x), b = reinterpret_cast<int64_t>(y);
  if (a + (rows - 1) * x_stride + width <= b || b + (rows - 1) * y_stride + width <= a) return false;
  if (x_stride != y_stride) return true;
  const int64_t off = ((b - a) % x_stride + x_stride) % x_stride;   // of a row of y in a row of x
  return off < width || off + width > x_stride;
}

// Row and column counts of the 8-bit row kernels.
int check_rows(int64_t rows, int64_t cols, int64_t multiple) {
  if (rows < 0 || cols <= 0 || cols % multiple != 0) return MOE_ERR_INVALID_ARG;
  if (rows >= (int64_t{1} << 31) || cols > MOE_MAX_ROW_BYTES / 4) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Whether two ranges of bytes touch; `same`: the same base is allowed (in place).
bool touch(const void* x, int64_t x_bytes, const void* y, int64_t y_bytes, bool same) {
  if (x == nullptr || y == nullptr || (same && x == y)) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  return a < b + static_cast<uintptr_t>(y_bytes) && b < a + static_cast<uintptr_t>(x_bytes);
}

// eps: squares that vanish in fp32 (below 2^-149) are nothing beside 2^-126, and 2^88 is nothing
// beside a mean of squares whose sum overflows.
int check_norm(const moe_norm_desc* d) {
  if (d == nullptr || !(d->eps >= 0x1p-126f) || !(d->eps <= 0x1p88f)) return MOE_ERR_INVALID_ARG;
  if (int st = check_rows(d->rows, d->cols, 16)) return st;
  return d->cols > MOE_MAX_NORM_COLS ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_gate_workspace_bytes(const moe_layout_desc* desc, size_t* bytes) {
  if (int st = check_desc(desc)) return st;
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = gate_workspace(desc->num_experts);
  return MOE_OK;
}

int moe_gate_forward(const moe_layout_desc* desc, const moe_gate_desc* gate, const void* logits,
                     int64_t logits_stride, const float* bias, int64_t* topk_idx, float* weights,
                     int32_t* expert_count, float* prob_mean, int32_t* routed_tokens, float* balance_loss,
                     void* workspace, size_t workspace_bytes, void* stream) {
  GateArgs a;
  if (int st = gate_args(desc, gate, logits, logits_stride, bias, workspace, workspace_bytes, &a)) return st;
  if ((desc->num_tokens > 0 && (topk_idx == nullptr || weights == nullptr)) || expert_count == nullptr ||
      prob_mean == nullptr || routed_tokens == nullptr || balance_loss == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (!aligned(topk_idx, 8) || !aligned(weights, 4)) return MOE_ERR_INVALID_ARG;
  a.topk_idx = topk_idx;
  a.weights = weights;
  a.expert_count = expert_count;
  a.prob_mean = prob_mean;
  a.routed_tokens = routed_tokens;
  a.balance_loss = balance_loss;
  return cuda_status(launch_gate(a, false, static_cast<cudaStream_t>(stream)));
}

int moe_gate_forward_grouped(const moe_layout_desc* desc, const moe_gate_desc* gate, const moe_gate_groups* groups,
                             const void* logits, int64_t logits_stride, const float* bias, int64_t* topk_idx,
                             float* weights, int32_t* expert_count, float* prob_mean, int32_t* routed_tokens,
                             float* balance_loss, void* workspace, size_t workspace_bytes, void* stream) {
  GateArgs a;
  if (int st = gate_args(desc, gate, logits, logits_stride, bias, workspace, workspace_bytes, &a)) return st;
  if (groups == nullptr || groups->num_groups < 1 || desc->num_experts % groups->num_groups != 0 ||
      groups->topk_groups < 1 || groups->topk_groups > groups->num_groups || groups->group_sum < 1 ||
      groups->group_sum > 2)
    return MOE_ERR_INVALID_ARG;
  if (groups->num_groups > MOE_MAX_GROUPS) return MOE_ERR_UNSUPPORTED;
  if ((desc->num_tokens > 0 && (topk_idx == nullptr || weights == nullptr)) || expert_count == nullptr ||
      prob_mean == nullptr || routed_tokens == nullptr || balance_loss == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (!aligned(topk_idx, 8) || !aligned(weights, 4)) return MOE_ERR_INVALID_ARG;
  a.num_groups = groups->num_groups;
  a.topk_groups = groups->topk_groups;
  a.group_sum = groups->group_sum;
  a.topk_idx = topk_idx;
  a.weights = weights;
  a.expert_count = expert_count;
  a.prob_mean = prob_mean;
  a.routed_tokens = routed_tokens;
  a.balance_loss = balance_loss;
  return cuda_status(launch_route(a, static_cast<cudaStream_t>(stream)));
}

int moe_gate_backward(const moe_layout_desc* desc, const moe_gate_desc* gate, const void* logits,
                      int64_t logits_stride, const int64_t* topk_idx, const int32_t* expert_count,
                      const int32_t* routed_tokens, const float* dweights, const float* dloss, void* dlogits, int64_t dlogits_stride, void* workspace,
                      size_t workspace_bytes, void* stream) {
  GateArgs a;
  if (int st = gate_args(desc, gate, logits, logits_stride, nullptr, workspace, workspace_bytes, &a)) return st;
  if (expert_count == nullptr || routed_tokens == nullptr) return MOE_ERR_INVALID_ARG;
  if (desc->num_tokens > 0 &&
      (topk_idx == nullptr || dlogits == nullptr || dlogits_stride < desc->num_experts))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(topk_idx, 8) || !aligned(dweights, 4) || !aligned(dlogits, gate->logits_bf16 ? 2 : 4))
    return MOE_ERR_INVALID_ARG;
  if (dlogits_stride > MOE_MAX_ROW_BYTES / 4) return MOE_ERR_UNSUPPORTED;
  const int64_t size = gate->logits_bf16 ? 2 : 4;
  if (desc->num_tokens > 0 && rows_clash(logits, size * logits_stride, dlogits, size * dlogits_stride, desc->num_tokens,
                                         size * desc->num_experts))
    return MOE_ERR_INVALID_ARG;
  a.topk_idx = const_cast<int64_t*>(topk_idx);
  a.expert_count = const_cast<int32_t*>(expert_count);
  a.routed_tokens = const_cast<int32_t*>(routed_tokens);
  a.dweights = dweights;
  a.dloss = dloss;
  a.dlogits = dlogits;
  a.dlogits_stride = dlogits_stride;
  return cuda_status(launch_gate(a, true, static_cast<cudaStream_t>(stream)));
}

int moe_combine_backward(const moe_layout_desc* desc, const void* dout, int64_t hidden, const int32_t* dst_slot,
                         const float* weights, const void* expert_out, void* dy, int64_t capacity_rows,
                         float* dweights, const int32_t* expert_offset, const int32_t* expert_count, int zero_pad,
                         void* workspace, size_t workspace_bytes, void* stream) {
  if (int st = check_desc(desc)) return st;
  WorkspaceLayout w;
  if (int st = check_workspace(desc, workspace, workspace_bytes, &w)) return st;
  if (int st = check_rows(capacity_rows, hidden, 8)) return st;
  if (hidden > MOE_MAX_ROW_BYTES / 2) return MOE_ERR_UNSUPPORTED;
  if (zero_pad != 0 && (expert_offset == nullptr || expert_count == nullptr)) return MOE_ERR_INVALID_ARG;
  if (capacity_rows > 0 && dy == nullptr) return MOE_ERR_INVALID_ARG;
  if (desc->num_tokens > 0 && (dout == nullptr || dst_slot == nullptr || weights == nullptr ||
                               (dweights != nullptr && expert_out == nullptr && capacity_rows > 0)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(dout, 16) || !aligned(expert_out, 16) || !aligned(dy, 16) || !aligned(weights, 4) || !aligned(dweights, 4) ||
      !aligned(dst_slot, 4) || !aligned(expert_offset, 4) || !aligned(expert_count, 4))
    return MOE_ERR_INVALID_ARG;
  const int64_t dense = 2 * hidden * desc->num_tokens, rows = 2 * hidden * capacity_rows;
  const int64_t pairs = 4 * desc->num_tokens * desc->topk;
  if (touch(dy, rows, dout, dense, false) || touch(dy, rows, expert_out, rows, true) || touch(dy, rows, weights, pairs, false) ||
      touch(dy, rows, dst_slot, pairs, false) || touch(dweights, pairs, dout, dense, false) ||
      touch(dweights, pairs, expert_out, rows, false) || touch(dweights, pairs, dy, rows, false) ||
      touch(dweights, pairs, weights, pairs, false) || touch(dweights, pairs, dst_slot, pairs, false))
    return MOE_ERR_INVALID_ARG;
  const int64_t E = desc->num_experts;
  if (zero_pad != 0 && (touch(dy, rows, expert_offset, 4 * (E + 1), false) || touch(dy, rows, expert_count, 4 * E, false) ||
                        touch(dweights, pairs, expert_offset, 4 * (E + 1), false) ||
                        touch(dweights, pairs, expert_count, 4 * E, false)))
    return MOE_ERR_INVALID_ARG;
  CombineBackwardArgs a{};
  a.dout = static_cast<const uint16_t*>(dout);
  a.hidden = hidden;
  a.dst_slot = dst_slot;
  a.weights = weights;
  a.expert_out = static_cast<const uint16_t*>(expert_out);
  a.dy = static_cast<uint16_t*>(dy);
  a.capacity = capacity_rows;
  a.dweights = dweights;
  a.expert_offset = expert_offset;
  a.expert_count = expert_count;
  a.zero_pad = zero_pad != 0 && desc->alignment > 1;   // else there are no gaps
  a.num_tokens = desc->num_tokens;
  a.topk = desc->topk;
  a.num_experts = desc->num_experts;
  a.err = at<int>(workspace, w.err_off);
  return cuda_status(launch_combine_backward(a, static_cast<cudaStream_t>(stream)));
}

int moe_rms_norm(const moe_norm_desc* norm, const void* x, const void* residual, const void* weight,
                 const int32_t* total_rows, void* residual_out, void* y, void* q, float* sf, int64_t sf_ld,
                 float* rstd, void* stream) {
  if (int st = check_norm(norm)) return st;
  const int64_t rows = norm->rows, cols = norm->cols, n = rows * cols, nb = ceil_div64(cols, 128);
  const bool wide = norm->stream_fp32 != 0;
  if (rows == 0) return MOE_OK;
  if ((residual == nullptr) != (residual_out == nullptr) || (residual == nullptr && wide)) return MOE_ERR_INVALID_ARG;
  if ((y == nullptr && q == nullptr) || (q == nullptr) != (sf == nullptr) || weight == nullptr) return MOE_ERR_INVALID_ARG;
  if (q != nullptr && sf_ld != 0 && (sf_ld < rows || sf_ld % 4 != 0)) return MOE_ERR_INVALID_ARG;
  if (x == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(residual_out, 16) || !aligned(y, 16) ||
      !aligned(q, 16) || !aligned(sf, 4) || !aligned(rstd, 4) || !aligned(total_rows, 4))
    return MOE_ERR_INVALID_ARG;
  // Outputs against inputs and against each other.
  const int64_t size = wide ? 4 : 2, scales = 4 * (sf_ld == 0 ? rows * nb : sf_ld * nb), wbytes = (norm->weight_fp32 ? 4 : 2) * cols;
  const struct { const void* p; int64_t bytes; bool bf16; } out[] = {
      {residual_out, size * n, !wide}, {y, 2 * n, true}, {q, n, false}, {sf, scales, false}, {rstd, 4 * rows, false}};
  for (int i = 0; i < 5; ++i) {
    if (touch(out[i].p, out[i].bytes, x, 2 * n, out[i].bf16) ||
        touch(out[i].p, out[i].bytes, residual, size * n, i == 0 || (out[i].bf16 && !wide)) ||
        touch(out[i].p, out[i].bytes, weight, wbytes, false) || touch(out[i].p, out[i].bytes, total_rows, 4, false))
      return MOE_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (touch(out[i].p, out[i].bytes, out[j].p, out[j].bytes, false)) return MOE_ERR_INVALID_ARG;
  }
  NormArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.residual = residual;
  a.weight = weight;
  a.total_rows = total_rows;
  a.rows = rows;
  a.cols = cols;
  a.eps = norm->eps;
  a.stream_fp32 = wide;
  a.weight_fp32 = norm->weight_fp32 != 0;
  a.residual_out = residual_out;
  a.y = static_cast<uint16_t*>(y);
  a.q = static_cast<uint8_t*>(q);
  a.sf = sf;
  a.sf_row_stride = sf_ld == 0 ? nb : 1;
  a.sf_block_stride = sf_ld == 0 ? 1 : sf_ld;
  a.rstd = rstd;
  return cuda_status(launch_norm(a, static_cast<cudaStream_t>(stream)));
}

int moe_rms_norm_workspace_bytes(const moe_norm_desc* norm, size_t* bytes) {
  if (int st = check_norm(norm)) return st;
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = 4 * static_cast<size_t>(norm_parts(norm->cols)) * static_cast<size_t>(norm->cols);
  return MOE_OK;
}

int moe_rms_norm_backward(const moe_norm_desc* norm, const void* dy, const void* z, const float* rstd,
                          const void* weight, const void* dresidual, const int32_t* total_rows, void* dz, void* dx,
                          float* dweight, int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  if (int st = check_norm(norm)) return st;
  const int64_t rows = norm->rows, cols = norm->cols, n = rows * cols;
  const bool wide = norm->stream_fp32 != 0;
  if (weight == nullptr || (rows > 0 && (dy == nullptr || z == nullptr || rstd == nullptr || dz == nullptr)))
    return MOE_ERR_INVALID_ARG;
  const int64_t need = 4 * norm_parts(cols) * cols;
  if (dweight != nullptr && (workspace == nullptr || static_cast<int64_t>(workspace_bytes) < need)) return MOE_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(z, 16) || !aligned(rstd, 4) || !aligned(weight, 16) || !aligned(dresidual, 16) ||
      !aligned(dz, 16) || !aligned(dx, 16) || !aligned(dweight, 4) || !aligned(workspace, 16) || !aligned(total_rows, 4))
    return MOE_ERR_INVALID_ARG;
  const int64_t size = wide ? 4 : 2, wbytes = (norm->weight_fp32 ? 4 : 2) * cols;
  const struct { const void* p; int64_t bytes; bool bf16, stream; } out[] = {
      {dz, size * n, !wide, true}, {dx, 2 * n, true, !wide}, {dweight, 4 * cols, false, false},
      {dweight != nullptr ? workspace : nullptr, need, false, false}};
  for (int i = 0; i < 4; ++i) {
    if (touch(out[i].p, out[i].bytes, dy, 2 * n, out[i].bf16) || touch(out[i].p, out[i].bytes, z, size * n, out[i].stream) ||
        touch(out[i].p, out[i].bytes, dresidual, size * n, out[i].stream) || touch(out[i].p, out[i].bytes, rstd, 4 * rows, false) ||
        touch(out[i].p, out[i].bytes, weight, wbytes, false) || touch(out[i].p, out[i].bytes, total_rows, 4, false))
      return MOE_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (touch(out[i].p, out[i].bytes, out[j].p, out[j].bytes, false)) return MOE_ERR_INVALID_ARG;
  }
  NormArgs a{};
  a.x = static_cast<const uint16_t*>(dy);
  a.residual = z;
  a.weight = weight;
  a.total_rows = total_rows;
  a.rows = rows;
  a.cols = cols;
  a.eps = norm->eps;
  a.stream_fp32 = wide;
  a.weight_fp32 = norm->weight_fp32 != 0;
  a.residual_out = dz;
  a.y = static_cast<uint16_t*>(dx);
  a.rstd = const_cast<float*>(rstd);
  a.dresidual = dresidual;
  a.dweight = dweight;
  a.partial = static_cast<float*>(workspace);
  a.accumulate = accumulate != 0;
  return cuda_status(launch_norm_backward(a, static_cast<cudaStream_t>(stream)));
}

int moe_quantize_rows(const void* x, int64_t rows, int64_t cols, const int32_t* total_rows, void* q, float* sf,
                      int64_t sf_ld, void* stream) {
  if (int st = check_rows(rows, cols, 16)) return st;
  if (sf_ld != 0 && (sf_ld < rows || sf_ld % 4 != 0)) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (x == nullptr || q == nullptr || sf == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(sf, 4)) return MOE_ERR_INVALID_ARG;
  QuantRowsArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.rows = rows;
  a.cols = cols;
  a.total_rows = total_rows;
  a.q = static_cast<uint8_t*>(q);
  a.sf = sf;
  a.sf_row_stride = sf_ld == 0 ? ceil_div64(cols, 128) : 1;
  a.sf_block_stride = sf_ld == 0 ? 1 : sf_ld;
  return cuda_status(launch_quantize_rows(a, static_cast<cudaStream_t>(stream)));
}

int moe_swiglu_quantize(const void* gate_up, int64_t rows, int64_t width, const int32_t* total_rows, void* q,
                        float* sf, int64_t sf_ld, void* stream) {
  if (int st = check_rows(rows, width, 16)) return st;
  if (sf_ld < rows || sf_ld % 4 != 0) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (gate_up == nullptr || q == nullptr || sf == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned(gate_up, 16) || !aligned(q, 16) || !aligned(sf, 4)) return MOE_ERR_INVALID_ARG;
  QuantRowsArgs a{};
  a.x = static_cast<const uint16_t*>(gate_up);
  a.rows = rows;
  a.cols = width;
  a.total_rows = total_rows;
  a.q = static_cast<uint8_t*>(q);
  a.sf = sf;
  a.sf_row_stride = 1;
  a.sf_block_stride = sf_ld;
  a.swiglu = true;
  return cuda_status(launch_quantize_rows(a, static_cast<cudaStream_t>(stream)));
}

int moe_swiglu_backward(const void* gate_up, const void* dh, int64_t rows, int64_t width,
                        const int32_t* total_rows, void* dgate_up, void* stream) {
  if (int st = check_rows(rows, width, 8)) return st;
  if (rows > 0 && (gate_up == nullptr || dh == nullptr || dgate_up == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned(gate_up, 16) || !aligned(dh, 16) || !aligned(dgate_up, 16)) return MOE_ERR_INVALID_ARG;
  SwigluBackwardArgs a{};
  a.gate_up = static_cast<const uint16_t*>(gate_up);
  a.dh = static_cast<const uint16_t*>(dh);
  a.rows = rows;
  a.width = width;
  a.total_rows = total_rows;
  a.dgate_up = static_cast<uint16_t*>(dgate_up);
  return cuda_status(launch_swiglu_backward(a, static_cast<cudaStream_t>(stream)));
}

int moe_quantize_cols(const moe_layout_desc* desc, const void* x, int64_t capacity_rows, int64_t cols,
                      const int32_t* expert_offset, const int32_t* expert_count, void* q, int64_t ld, float* sf,
                      void* workspace, size_t workspace_bytes, void* stream) {
  if (int st = check_desc(desc)) return st;
  WorkspaceLayout w;
  if (int st = check_workspace(desc, workspace, workspace_bytes, &w)) return st;
  if (int st = check_rows(capacity_rows, cols, 8)) return st;
  if (desc->alignment % 128 != 0) return MOE_ERR_UNSUPPORTED;
  if (ld % 128 != 0 || ld < capacity_rows || expert_offset == nullptr || expert_count == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (capacity_rows > 0 && (x == nullptr || q == nullptr || sf == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(sf, 4)) return MOE_ERR_INVALID_ARG;
  QuantColsArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.capacity = capacity_rows;
  a.cols = cols;
  a.expert_offset = expert_offset;
  a.expert_count = expert_count;
  a.num_experts = desc->num_experts;
  a.q = static_cast<uint8_t*>(q);
  a.ld = ld;
  a.sf = sf;
  a.err = at<int>(workspace, w.err_off);
  return cuda_status(launch_quantize_cols(a, static_cast<cudaStream_t>(stream)));
}

int moe_expert_gemm_fp8(const moe_layout_desc* desc, const void* x, const float* x_sf, int64_t sf_ld,
                        int64_t capacity_rows, int64_t width_in, const void* w, const float* w_sf,
                        int64_t width_out, const int32_t* expert_offset, const int32_t* expert_count, void* out,
                        void* workspace, size_t workspace_bytes, void* stream) {
  if (int st = check_desc(desc)) return st;
  WorkspaceLayout wl;
  if (int st = check_workspace(desc, workspace, workspace_bytes, &wl)) return st;
  if (int st = check_rows(capacity_rows, width_in, 16)) return st;
  if (int st = check_rows(0, width_out, 8)) return st;
  if (sf_ld < capacity_rows || sf_ld % 4 != 0 || expert_offset == nullptr || expert_count == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (w == nullptr || w_sf == nullptr ||
      (capacity_rows > 0 && (x == nullptr || x_sf == nullptr || out == nullptr)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(x_sf, 4) || !aligned(w_sf, 4))
    return MOE_ERR_INVALID_ARG;
  if (capacity_rows == 0) return MOE_OK;
  ExpertGemmArgs a{};
  a.x = x;
  a.x_sf = x_sf;
  a.sf_ld = sf_ld;
  a.capacity = capacity_rows;
  a.width_in = width_in;
  a.w = w;
  a.w_sf = w_sf;
  a.width_out = width_out;
  a.expert_offset = expert_offset;
  a.expert_count = expert_count;
  a.out = out;
  a.num_experts = desc->num_experts;
  a.pairs = desc->num_tokens * desc->topk;
  a.err = at<int>(workspace, wl.err_off);
  return cuda_status(launch_expert_gemm(a, static_cast<cudaStream_t>(stream)));
}

int moe_expert_wgrad_fp8(const moe_layout_desc* desc, const void* dy, const float* dy_sf, const void* x,
                         const float* x_sf, int64_t ld, int64_t capacity_rows, int64_t width_out, int64_t width_in,
                         const int32_t* expert_offset, const int32_t* expert_count, void* dw, int dw_fp32,
                         int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  if (int st = check_desc(desc)) return st;
  WorkspaceLayout wl;
  if (int st = check_workspace(desc, workspace, workspace_bytes, &wl)) return st;
  if (int st = check_rows(capacity_rows, width_in, 8)) return st;
  if (int st = check_rows(0, width_out, 1)) return st;
  if (desc->alignment % 128 != 0) return MOE_ERR_UNSUPPORTED;
  if (ld % 128 != 0 || ld < capacity_rows || ld <= 0 || expert_offset == nullptr || expert_count == nullptr ||
      dw == nullptr || (accumulate != 0 && dw_fp32 == 0))
    return MOE_ERR_INVALID_ARG;
  if (ld >= (int64_t{1} << 31)) return MOE_ERR_UNSUPPORTED;
  if (dy == nullptr || dy_sf == nullptr || x == nullptr || x_sf == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dw, 16) || !aligned(dy_sf, 4) || !aligned(x_sf, 4))
    return MOE_ERR_INVALID_ARG;
  ExpertGemmArgs a{};
  a.x = x;
  a.x_sf = x_sf;
  a.sf_ld = ld;
  a.capacity = capacity_rows;
  a.width_in = width_in;
  a.w = dy;
  a.w_sf = dy_sf;
  a.width_out = width_out;
  a.expert_offset = expert_offset;
  a.expert_count = expert_count;
  a.out = dw;
  a.out_fp32 = dw_fp32 != 0;
  a.accumulate = accumulate != 0;
  a.num_experts = desc->num_experts;
  a.pairs = desc->num_tokens * desc->topk;
  a.err = at<int>(workspace, wl.err_off);
  return cuda_status(launch_expert_wgrad(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
