// expert_gemm_kernel.cu -- products of e4m3 operands with an fp32 scale for
// each block of 128, over the segments of the receive buffer:
//
//   forward (and input gradient)  out[r, o] = sum_b sx[b, r] sw[e, o/128, b] <x_r, w_o>_b
//   weight gradient               dw[e, o, i] = sum_b sdy[b, o] sx[b, i] <dy_o, x_i>_b
//
// A scale that changes every 128 values of K means the tensor core can sum one
// k-block only.  Each k-block's product lands in tensor memory, and epilogue
// warps add it, times its scales, to fp32 sums in registers:
//
//   warp 0      TMA loads of P and Q tiles (128-byte rows, one k-block wide)
//   warps 1-2   tcgen05.mma, 4 per k-block, each into an accumulator of its own
//   warp 3      the k-block's scales to shared memory
//   warps 4-    tensor memory -> fp32 sums; at the tile's end rows of out
//
// D[p, q] = <P_p, Q_q>: P gives the 128 accumulator rows (tensor-memory lanes) of
// a CTA, Q its columns.  Three kinds:
//
//   kMany   P = receive rows, Q = weights; a pair of CTAs shares 256 x 256 tiles,
//           each loading half of Q.  A thread owns a receive row, and both scales
//           of a k-block and 128-column block multiply to one number for it.
//   kFew    P = weights, Q = receive rows; one CTA.  The tensor core takes any
//           multiple of 16 columns, so an expert with one token does not pay for
//           128.  Bound by the reading of the weights.  With fewer tiles than half
//           the SMs, a cluster of CTAs takes a tile, each a share of K, and the
//           first adds the others' sums, in their order, from distributed shared
//           memory.
//   kWgrad  P = x^T, Q = dy^T (so that columns of dw run along lanes); a pair.
//
// What shaped it, measured on 16 experts of about 1024 rows, 7168 -> 4096 (before and after
// each step, as the kernel was then):
//  - From an MMA's issue to a waiting warp it takes ~280 cycles more than the MMA
//    (512 a k-block), and ~210 for the peer's word that a buffer was read.  Tensor
//    memory has room for two buffers of 256 columns, so a tile is two accumulators of
//    128 with buffers and barriers of their own: 435 -> 412 us.
//  - Issuing an MMA takes ~53 cycles whatever its size, so each accumulator has an
//    MMA warp: 377 -> 367 us.  Loop bounds and tile numbers of the issuing warps are kept in
//    uniform registers; from ordinary ones every operand is moved over one by one.
//  - Rows of out leave by tensor-map stores from a block of 32 x 32 a warp, so the tile
//    after does not wait for 152 SMs that write at once: 380 -> 367 us (16 k-blocks: 222
//    -> 205), with one stage of operands less (6 -> 5; 4, and room for two blocks: 375).
//    kWgrad, whose tiles have few k-blocks, 390 -> 316 us (8 experts of 1024 rows,
//    4096 x 7168, bf16), and 280 when its loop's bounds stay in uniform registers too.
//    Rows of dw along lanes would read tensor memory at 1.2 cycles, but came to 295.
//  - Scales come two k-blocks ahead: 363 us, 425 with one; kWgrad 280, 294 with one, and
//    302 with three, which spill.
//  - The epilogue is bound by its chain of latencies (wait, load, add), so kMany has 16
//    warps of 64 columns, 412 -> 386 us; 32 columns of tensor memory in flight,
//    386 -> 375 us.
//  - tcgen05.ld of the 32x32-bit shape moves a register of an SM quarter in 1.2 cycles,
//    the 16x256-bit one in 2.0; kFew and kWgrad take the latter for its pairs of columns.
//
// What it comes to, of twice the bf16 rate that a library product reaches (3781
// TFLOP/s): 16 experts of about 1024 rows, 7168 -> 4096, kMany 366 us (2630 TFLOP/s, 70 %;
// the epilogue's adds to fp32 sums are what is left, the tensor core waits for them; 325 us
// if each has 1024 exactly, so four row tiles, not five); 256 experts 5.7 ms with pauses
// between calls (2700), 6.5-6.7 ms one call after the other, when the power cap holds the
// SMs at 1.47-1.51 GHz of 2.07.  16 tokens to top-8 of 256 experts, kFew 0.47 ms (6.4 TB/s
// of 6.76); one row, 7168 -> 4096, its 29 MB of weights from HBM, 13.5 us.  32 experts of
// about 1024 rows, 4096 x 7168, kWgrad 1.18 ms in bf16 (1630 TFLOP/s: two scales a value and
// k-block, 1.9 GB of results), 1.31 in fp32, 1.64 added to fp32.
//
// One persistent CTA (or pair) per SM walks the tiles of all experts.  All sums
// are fp32; the result is rounded once.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "common.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

enum Kind { kMany, kFew, kWgrad };

constexpr int kKBlock = 128;                       // values (and bytes) of K in a scale block
constexpr int kPRows = 128;                        // accumulator rows of a CTA
constexpr int kPBytes = kPRows * kKBlock;
constexpr int kQBytes = 128 * kKBlock;             // a CTA loads at most 128 rows of Q
constexpr int kStageBytes = kPBytes + kQBytes;
constexpr int kBatchCols = 32;                     // columns of one tensor-memory load
constexpr int kSlotWords = 128 + kPRows;           // scales of columns or rows, then (kWgrad) of rows
constexpr int kTmemCols = 512;
constexpr int kAccCols = 128;                      // columns of an accumulator
constexpr int kOutBytes = 64 * 64;                 // a warp's 64 rows x 32 columns of bf16 (kFew, kWgrad)
constexpr int kRowsBytes = 32 * 64;                // 32 x 32 (kMany)

template <Kind KIND>
struct Config {
  static constexpr int kCtas = KIND == kFew ? 1 : 2;
  static constexpr int kAccs = KIND == kFew ? 1 : 2;           // accumulators of a tile
  static constexpr int kTileCols = kAccs * kAccCols;
  static constexpr int kBuffers = kTmemCols / kTileCols;       // of an accumulator
  static constexpr int kUnit = 16 * kCtas;                     // column granularity: each CTA of a pair holds n / 2 rows of Q
  static constexpr int kQRows = kAccCols / kCtas;              // rows of Q of an accumulator a CTA loads at most
  static constexpr int kSplit = 2;                             // epilogue warps side by side in an accumulator
  static constexpr int kWarpCols = kAccCols / kSplit;
  static constexpr int kEpilogueWarps = 4 * kAccs * kSplit;
  static constexpr int kThreads = 128 + 32 * kEpilogueWarps;
  static constexpr int kStages = KIND == kMany ? 5 : KIND == kFew ? 5 : 4;   // what the staging of out leaves room for
  // Registers a thread: sums, and values of tensor memory.
  static constexpr int kLaunchRegs = KIND == kFew ? 168 : 96;
  static constexpr int kEpilogueRegs = KIND == kFew ? 224 : 104, kOtherRegs = KIND == kFew ? 56 : 64;
  static_assert(32 * kEpilogueWarps * kEpilogueRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs,
                "register split above the launch's total");
  static_assert(kAccs * kQRows * kKBlock <= kQBytes, "shared memory of Q");
};

// What the roles share besides the tiles.
struct Shared {
  alignas(16) float scale[2][4][kSlotWords];       // [accumulator][buffer]
  int tile_end[MOE_MAX_EXPERTS];                   // tiles of experts 0..e
  int seg_start[MOE_MAX_EXPERTS];
  int seg_count[MOE_MAX_EXPERTS];
  uint64_t full[6], empty[6];
  uint64_t acc_full[2][4], acc_empty[2][4];        // full: product and scales are there
  uint64_t scale_empty[2][4];
  uint32_t tmem;
  int warp_sum[20];
};
template <Kind KIND>
struct Smem {
  alignas(1024) uint8_t stage[Config<KIND>::kStages][kStageBytes];
  alignas(1024) uint8_t out[Config<KIND>::kEpilogueWarps * (KIND == kMany ? kRowsBytes : kOutBytes)];
  Shared s;
};
// The dynamic base is only known to be 16-byte aligned: room to align it.
template <Kind KIND>
constexpr size_t kSmemBytes = sizeof(Smem<KIND>) + 1024;
static_assert(kSmemBytes<kMany> <= 232448 && kSmemBytes<kFew> <= 232448 && kSmemBytes<kWgrad> <= 232448,
              "shared memory of one SM");

struct Tile {
  int expert;
  int p0;          // first row of P for this CTA
  int p_valid;     // rows of P that exist
  int q0;          // first row of Q
  int q_valid;     // rows of Q that exist
  int n[2];        // columns of the two accumulators; the second may have none
  int k0;          // first k (kWgrad: the segment's first row)
  int kblocks;
  bool last;       // the expert's last tile along the receive rows
};

__host__ __device__ constexpr int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Tiles along the receive rows (kWgrad: rows of dy) of an expert, and across.
template <Kind KIND>
__device__ __forceinline__ int row_tiles(const GemmParams& p, int count) {
  return ceil_div(KIND == kWgrad ? p.dy_rows : count, KIND == kMany ? 256 : Config<KIND>::kTileCols);
}
template <Kind KIND>
__device__ __forceinline__ int col_tiles(const GemmParams& p) {
  return ceil_div(p.out_cols, KIND == kMany ? Config<KIND>::kTileCols : kPRows * Config<KIND>::kCtas);
}

template <Kind KIND>
__device__ __forceinline__ Tile get_tile(const GemmParams& p, const Shared& s, int t, int rank, int split) {
  using C = Config<KIND>;
  int lo = 0, hi = p.num_experts - 1;     // first expert whose tiles end after t
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (s.tile_end[mid] > t) hi = mid; else lo = mid + 1;
  }
  const int count = s.seg_count[lo], start = s.seg_start[lo], nr = row_tiles<KIND>(p, count);
  const int local = t - (lo == 0 ? 0 : s.tile_end[lo - 1]);
  const int row = local % nr, col = local / nr;
  Tile r;
  r.expert = lo;
  r.last = row == nr - 1;
  r.k0 = KIND == kWgrad ? start : 0;
  r.kblocks = KIND == kWgrad ? ceil_div(count, kKBlock) : p.kblocks;
  if (KIND == kFew) {   // this CTA's share of K
    const int first = p.kblocks * split / p.splits;
    r.k0 = first * kKBlock;
    r.kblocks = p.kblocks * (split + 1) / p.splits - first;
  }
  if (KIND == kMany) {
    const int at = row * 256 + rank * kPRows;
    r.p0 = start + at;
    r.p_valid = max(0, min(kPRows, count - at));
    r.q0 = col * C::kTileCols;
    r.q_valid = min(C::kTileCols, p.out_cols - r.q0);
  } else {
    // columns shared evenly over the tiles along the rows
    const int rows = KIND == kWgrad ? p.dy_rows : count;
    const int per = ceil_div(ceil_div(rows, nr), C::kUnit) * C::kUnit;
    r.p0 = (col * C::kCtas + rank) * kPRows;
    r.p_valid = max(0, min(kPRows, p.out_cols - r.p0));
    r.q0 = (KIND == kWgrad ? 0 : start) + row * per;
    r.q_valid = max(0, min(per, rows - row * per));
  }
  // kMany: an accumulator is one scale block of the weights; kWgrad: the two are of
  // like size, the first in whole batches
  const int n = max(C::kUnit, ceil_div(r.q_valid, C::kUnit) * C::kUnit);
  r.n[0] = n <= kAccCols ? n : KIND == kMany ? kAccCols : ceil_div(n / 2, kBatchCols) * kBatchCols;
  r.n[1] = n - r.n[0];
  return r;
}

// Place of a column's scale: a lane reads those of its four pairs among 32
// columns as two vectors.
__device__ __forceinline__ int scale_place(int j) {
  return (j & ~15) + ((j & 7) >> 1) * 4 + ((j & 8) >> 3) * 2 + (j & 1);
}
__device__ __forceinline__ void load_scales(const float* at, uint64_t* q) {
  const float4 lo = *reinterpret_cast<const float4*>(at), hi = *reinterpret_cast<const float4*>(at + 16);
  q[0] = tc::pack2(lo.x, lo.y), q[1] = tc::pack2(lo.z, lo.w), q[2] = tc::pack2(hi.x, hi.y), q[3] = tc::pack2(hi.z, hi.w);
}

// Position in a ring of N buffers, and the parity of the phase it is in.
template <int N>
struct Ring {
  uint32_t i = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++i == N) i = 0, phase ^= 1;
  }
};

// A value all lanes have, in a uniform register: addresses, descriptors and loop
// bounds built on it then stay there.  (From ordinary registers each MMA or TMA
// operand is moved over one by one, and issuing takes longer than the MMAs.)
__device__ __forceinline__ int uniform(int v) {
  return __reduce_max_sync(0xffffffffu, v);
}

// The whole warp waits, and leaves together (tcgen05.ld needs all lanes).
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, limit_ns));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Rows of out from sums whose thread owns a row (kMany): row `quarter` * 32 + lane of
// the tile, acc[c][i] column 32 c + 2 i, +1 after its column `col`.
__device__ __forceinline__ void store_rows(const GemmParams& p, const Tile& t, int quarter, int lane, int col, uint8_t* stage,
                                           const CUtensorMap* map_out, const uint64_t (*acc)[16]) {
  using C = Config<kMany>;
  const int oc = t.q0 + col, row = t.p0 + quarter * 32;
  const int rows = t.p_valid - quarter * 32, cols = p.out_cols - oc;
  const bool whole = rows >= 32;   // else a box would reach into the next segment
#pragma unroll
  for (int c = 0; c < C::kWarpCols / kBatchCols; ++c) {
    const int at = c * kBatchCols;
    uint4 v[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = tc::unpack2(acc[c][4 * h + i]);
        w[i] = pack_bf16(f.x, f.y);
      }
      v[h] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (whole) {
      // A block of 32 x 32, which the next tile's k-blocks do not wait for: 64 bytes a
      // row, its pieces swapped as the tensor map has them.
      if (lane == 0) ptx::bulk_wait_read<0>();
      __syncwarp();
#pragma unroll
      for (int h = 0; h < 4; ++h) *reinterpret_cast<uint4*>(stage + lane * 64 + (h ^ lane / 2 % 4) * 16) = v[h];
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (at < cols) tc::store_box(map_out, oc + at, row, 0, ptx::smem_addr(stage));
        ptx::bulk_commit();
      }
    } else if (lane < rows) {
      uint16_t* out = static_cast<uint16_t*>(p.out) + (static_cast<int64_t>(row) + lane) * p.out_cols + oc;
#pragma unroll
      for (int h = 0; h < 4; ++h)
        if (at + 8 * h < cols) ptx::st_v4(out + at + 8 * h, v[h]);
    }
  }
}

// Rows of out from sums whose columns are rows of out (kFew, kWgrad).
// acc[c][8 * up + 2 * h + r]: row 16 * up + 8 * r + lane / 4 of the warp's 32,
// columns 32 * c + 8 * h + 2 * (lane % 4), +1 of its accumulator columns.
template <Kind KIND>
__device__ __forceinline__ void store_columns(const GemmParams& p, const Tile& t, int quarter, int acc_id, int part, int lane,
                                              uint8_t* stage, const CUtensorMap* map_out, const uint64_t (*acc)[16]) {
  using C = Config<KIND>;
  const int n = (acc_id == 0 ? t.n[0] : t.n[1]) - part * C::kWarpCols;
  const int row = (acc_id == 0 ? 0 : t.n[0]) + part * C::kWarpCols;   // of the tile
  const int col0 = t.p0 + quarter * 32;                     // the warp's first column of out
  const int rows = min(n, t.q_valid - row);
  if (KIND == kWgrad && p.out_fp32) {
    // A block of 32 x 32 at a time, 128 bytes a row, pieces swapped as the tensor map has
    // them: a store meets no bank twice.
#pragma unroll
    for (int c = 0; c < C::kWarpCols / kBatchCols; ++c) {
      if (lane == 0) ptx::bulk_wait_read<0>();
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int at = 8 * (i / 2 % 4) + 2 * (lane % 4), piece = 4 * (i / 8) + 2 * (i % 2) + lane / 16;
        const float2 f = tc::unpack2(acc[c][i]);
        float* to = reinterpret_cast<float*>(stage + at * 128) + lane / 4 % 4;
        to[(piece ^ at % 8) * 4] = f.x;
        to[32 + (piece ^ (at + 1) % 8) * 4] = f.y;
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (c * kBatchCols < rows && col0 < p.out_cols) {
          const uint32_t from = ptx::smem_addr(stage);
          if (p.accumulate) tc::add_box(map_out, col0, t.q0 + row + c * kBatchCols, t.expert, from);
          else tc::store_box(map_out, col0, t.q0 + row + c * kBatchCols, t.expert, from);
        }
        ptx::bulk_commit();
      }
    }
    return;
  }
  // All of the warp's rows through shared memory at once: 64 bytes a row, its 16-byte
  // pieces swapped by the row so that stmatrix meets no bank twice (as the tensor map of
  // out has them).
  if (KIND == kWgrad && lane == 0) ptx::bulk_wait_read<0>();
  __syncwarp();   // the last tile's rows are read
#pragma unroll
  for (int c = 0; c < C::kWarpCols / kBatchCols; ++c)
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = tc::unpack2(acc[c][8 * (i / 2) + 2 * h + i % 2]);
        v[i] = pack_bf16(f.x, f.y);
      }
      // four matrices of 8 columns of out, transposed to 8 rows of 64 bytes
      const int r = c * kBatchCols + 8 * h + lane % 8, piece = (lane / 8) ^ (r / 2 % 4);
      tc::stmatrix_x4_trans(ptx::smem_addr(stage) + r * 64 + piece * 16, v[0], v[1], v[2], v[3]);
    }
  if (KIND == kWgrad) {
    // Boxes of 32 rows, which the next tile's k-blocks do not wait for.  A tile's rows end
    // at a multiple of 32 or with the matrix, whose edges the tensor map clips.
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
#pragma unroll
      for (int c = 0; c < C::kWarpCols / kBatchCols; ++c)
        if (c * kBatchCols < rows && col0 < p.out_cols)
          tc::store_box(map_out, col0, t.q0 + row + c * kBatchCols, t.expert, ptx::smem_addr(stage) + c * kBatchCols * 64);
      ptx::bulk_commit();
    }
    return;
  }
  __syncwarp();
  const int oc = col0 + (lane % 4) * 8;
  uint16_t* out = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(t.q0 + row) * p.out_cols + oc;
#pragma unroll
  for (int h = 0; h < C::kWarpCols / 8; ++h) {
    const int r = 8 * h + lane / 4;
    const uint4 w = ptx::ld_shared_v4(stage + r * 64 + ((lane % 4) ^ (r / 2 % 4)) * 16);
    if (r < rows && oc < p.out_cols) ptx::st_v4(out + static_cast<int64_t>(r) * p.out_cols, w);
  }
}

// Alignment-gap rows of the expert's segment: zeros, 16 bytes a lane.
template <Kind KIND>
__device__ __forceinline__ void zero_gap(const GemmParams& p, const Shared& s, const Tile& t, int rank, int ew, int lane) {
  using C = Config<KIND>;
  const int64_t end = min64(p.expert_offset[t.expert + 1], p.capacity);
  int64_t r = static_cast<int64_t>(s.seg_start[t.expert]) + s.seg_count[t.expert];
  // the tile's columns of out, a share of the rows for each warp (of both CTAs)
  const int c0 = KIND == kMany ? t.q0 : t.p0, cols = KIND == kMany ? t.q_valid : t.p_valid;
  const int warps = KIND == kMany ? C::kCtas * C::kEpilogueWarps : C::kEpilogueWarps;
  for (r += KIND == kMany ? rank * C::kEpilogueWarps + ew : ew; r < end; r += warps)
    for (int c = lane * 8; c < cols; c += 256)
      ptx::st_v4(static_cast<uint16_t*>(p.out) + r * p.out_cols + c0 + c, make_uint4(0, 0, 0, 0));
}

template <Kind KIND>
__global__ void __launch_bounds__(Config<KIND>::kThreads, 1)
expert_gemm_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                   const __grid_constant__ CUtensorMap map_c /* kFew: Q in boxes of 16 rows; else out */, const GemmParams p) {
  using C = Config<KIND>;
  constexpr int CTAS = C::kCtas, NBUF = C::kBuffers, ACCS = C::kAccs, kStages = C::kStages, kThreads = C::kThreads;
  extern __shared__ uint8_t smem_raw[];
  // The same offset in both CTAs of a pair: the bases are equal.
  Smem<KIND>& mem = *reinterpret_cast<Smem<KIND>*>(smem_raw + ((1024 - (ptx::smem_addr(smem_raw) & 1023)) & 1023));
  Shared& s = mem.s;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = CTAS == 2 ? static_cast<int>(tc::cluster_rank()) : 0;
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    tc::prefetch_map(&map_p);
    tc::prefetch_map(&map_q);
    if (KIND == kFew) tc::prefetch_map(&map_c);
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&s.full[i], 1);
      ptx::mbar_init(&s.empty[i], ACCS);           // a commit of each MMA warp
    }
    for (int i = 0; i < NBUF; ++i)
      for (int h = 0; h < ACCS; ++h) {
        ptx::mbar_init(&s.acc_full[h][i], 2);      // the commit, and the scales' warp
        ptx::mbar_init(&s.acc_empty[h][i], 4 * C::kSplit * CTAS);
        ptx::mbar_init(&s.scale_empty[h][i], 4 * C::kSplit);
      }
    ptx::fence_mbar_init();
  }
  if (warp == 1) tc::tmem_alloc<CTAS>(&s.tmem, kTmemCols);
  ptx::grid_dependency_wait();

  // Segments and the running count of tiles.  A segment that does not lie in
  // the buffer (a layout that overflowed its capacity, or a start that is not a
  // block boundary for the gradient) is left out and recorded.
  const int across = col_tiles<KIND>(p);
  int running = 0;
  for (int base = 0; base < p.num_experts; base += kThreads) {
    const int e = base + static_cast<int>(threadIdx.x);
    int tiles = 0;
    if (e < p.num_experts) {
      const int start = p.expert_offset[e];
      int count = p.expert_count[e];
      const bool fits = start >= 0 && count >= 0 && static_cast<int64_t>(start) + count <= p.capacity;
      const bool whole = KIND != kWgrad || start % kKBlock == 0;
      if (!fits || !whole) {
        set_error(p.err, fits ? MOE_ERR_INVALID_ARG : MOE_ERR_CAPACITY);
        count = 0;
      }
      s.seg_start[e] = count > 0 ? start : 0;
      s.seg_count[e] = count;
      tiles = row_tiles<KIND>(p, count) * across;
      if (KIND == kWgrad && p.accumulate && count == 0) tiles = 0;   // nothing to add (8 experts of 4096 x 7168, half empty: 402 -> 218 us)
    }
    int sum = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) s.warp_sum[warp] = sum;
    __syncthreads();
    int before = running;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += s.warp_sum[w];
      running += s.warp_sum[w];
    }
    if (e < p.num_experts) s.tile_end[e] = before + sum;
    __syncthreads();
  }
  const int tiles = uniform(running);
  tc::fence_before();
  __syncthreads();
  if (CTAS == 2) tc::cluster_sync();   // the pair's barriers and tensor memory exist
  tc::fence_after();
  const uint32_t tmem = static_cast<uint32_t>(uniform(static_cast<int>(s.tmem)));
  const int splits = KIND == kFew ? p.splits : 1;   // CTAs that share a tile's K
  const int split = splits > 1 ? static_cast<int>(tc::cluster_rank()) : 0;
  const int first_tile = static_cast<int>(blockIdx.x) / (CTAS * splits), step = static_cast<int>(gridDim.x) / (CTAS * splits);
  bool ok = true;
  // Every warp of a cluster that shares tiles meets twice at a tile's end: when the
  // sums are in shared memory, and when they are read.  A warp whose wait ran out
  // still comes.
  const auto meet = [&] {
    if (KIND == kFew && splits > 1) tc::cluster_sync();
  };

  if (warp < 4) {
    tc::reg_dec<C::kOtherRegs>();
    if (warp == 0) {
      // ---- loads ---------------------------------------------------------
      // The warp stays together so that addresses live in uniform registers; one
      // lane issues.
      Ring<kStages> ring;
      uint32_t loads = 0;
      for (int t = first_tile; t < tiles; t += step, meet(), meet()) {
        if (!ok) continue;
        const Tile tile = get_tile<KIND>(p, s, t, rank, split);
        // Q rows of each accumulator, an equal share by each CTA of a pair, in boxes of 64;
        // 16 for the shortest segments
        const int n0 = uniform(tile.n[0]), n1 = uniform(tile.n[1]);
        const bool small = KIND == kFew && n0 <= 16, two = KIND == kFew ? n0 > 64 : n1 > 0;
        const int q0 = uniform(tile.q0 + rank * (n0 / CTAS));
        const int q1 = KIND == kFew ? q0 + 64 : uniform(tile.q0 + n0 + rank * (n1 / CTAS));
        const uint32_t bytes = CTAS * (kPBytes + (two ? 128 : small ? 16 : 64) * kKBlock);
        const int expert = uniform(tile.expert), p0 = uniform(tile.p0), kblocks = uniform(tile.kblocks);
        const int p_plane = KIND == kFew ? expert : 0, q_plane = KIND == kMany ? expert : 0;
        int x = uniform(tile.k0);
#pragma unroll 1
        for (int kb = 0; kb < kblocks; ++kb, x += kKBlock) {
          if (!(ok = wait_warp(&s.empty[ring.i], ring.phase ^ 1, p.wait_ns))) break;
          if (tc::elect_one()) {
            uint32_t bar = ptx::smem_addr(&s.full[ring.i]);
            const uint32_t dst = ptx::smem_addr(mem.stage[ring.i]);
            if (leader) ptx::mbar_arrive_expect_tx(&s.full[ring.i], bytes + (loads == 0 ? p.extra_tx : 0));
            if (CTAS == 2) bar = tc::map_to_rank(bar, 0);
            tc::load_box<CTAS>(dst, &map_p, x, p0, p_plane, bar);
            if (small) tc::load_box<CTAS>(dst + kPBytes, &map_c, x, q0, q_plane, bar);
            else tc::load_box<CTAS>(dst + kPBytes, &map_q, x, q0, q_plane, bar);
            if (two) tc::load_box<CTAS>(dst + kPBytes + 64 * kKBlock, &map_q, x, q1, q_plane, bar);
          }
          __syncwarp();
          ring.next();
          ++loads;
        }
      }
      // Every stage handed back: no copy or remote arrival is left in flight.
#pragma unroll 1
      for (uint32_t i = 0; ok && i < kStages; ++i, ring.next())
        if (loads + i >= kStages) ok = wait_warp(&s.empty[ring.i], ring.phase ^ 1, p.wait_ns);
      // After a wait that ran out the stages will not be handed back, but their copies (the
      // peer's too, which count on the leader's barriers) are waited for; the cluster's
      // barrier at the end keeps the peer's shared memory until then.
      if (!ok && leader)
#pragma unroll 1
        for (uint32_t n = loads < kStages ? 0 : loads - kStages; n < loads; ++n)
          wait_warp(&s.full[n % kStages], n / kStages & 1, p.wait_ns);
    } else if (warp < 3) {
      // ---- MMA: warp 1 + h into accumulator h -----------------------------
      // The barriers of a k-block are asked together: a ready one answers after ~60
      // cycles.
      const int h = warp - 1;
      if (leader && h < ACCS) {
        Ring<kStages> ring;
        Ring<NBUF> buf;
        uint32_t used = 0;
        const uint64_t p_desc = tc::operand_desc(ptx::smem_addr(mem.stage[0]));
        const uint32_t q_off = (kPBytes + h * C::kQRows * kKBlock) >> 4;
        for (int t = first_tile; t < tiles; t += step, meet(), meet()) {
          if (!ok) continue;
          const Tile tile = get_tile<KIND>(p, s, t, rank, split);
          const int kblocks = uniform(tile.kblocks), n = uniform(h == 0 ? tile.n[0] : tile.n[1]);
          const uint32_t idesc = tc::instr_desc(kPRows * CTAS, n);
#pragma unroll 1
          for (int kb = 0; kb < kblocks; ++kb) {
            const bool in = ptx::mbar_try_wait_parity(&s.full[ring.i], ring.phase);
            const bool free = ptx::mbar_try_wait_parity(&s.acc_empty[h][buf.i], buf.phase ^ 1);
            if (!__all_sync(0xffffffffu, in && free)) {
              ok = wait_warp(&s.full[ring.i], ring.phase, p.wait_ns) &&
                   wait_warp(&s.acc_empty[h][buf.i], buf.phase ^ 1, p.wait_ns);
              if (!ok) break;
            }
            tc::fence_after();
            if (tc::elect_one()) {
              if (n > 0) {
                const uint64_t a = p_desc + ring.i * (kStageBytes >> 4);
                const uint64_t q = a + q_off;
                const uint32_t d = tmem + buf.i * C::kTileCols + h * kAccCols;
#pragma unroll
                for (int k = 0; k < kKBlock / 32; ++k) tc::mma_e4m3<CTAS>(d, a + 2 * k, q + 2 * k, idesc, k > 0);
              }
              tc::commit<CTAS>(&s.acc_full[h][buf.i]);
              tc::commit<CTAS>(&s.empty[ring.i]);
            }
            __syncwarp();
            ring.next();
            buf.next();
            ++used;
          }
        }
        for (uint32_t i = 0; i < NBUF; ++i, ++used, buf.next())   // the epilogues' last (remote) arrivals
          if (used >= NBUF) ok &= wait_warp(&s.acc_empty[h][buf.i], buf.phase ^ 1, p.wait_ns);
      } else {
        for (int t = first_tile; t < tiles; t += step, meet(), meet()) {}
      }
    } else {
      // ---- scales --------------------------------------------------------
      // Through registers and kAhead k-blocks ahead: one for each receive row (kMany:
      // accumulator row, else column), times the weights' one; kWgrad: one for each
      // column and row.
      constexpr int kAhead = 2, kRows = 128 / 32;
      constexpr int kSets = KIND == kWgrad ? 2 : 1;            // of row scales: kMany's are the same for both accumulators
      constexpr int kWeights = KIND == kWgrad ? kRows : ACCS;
      Ring<NBUF> ring;
      for (int t = first_tile; t < tiles; t += step, meet(), meet()) {
        if (!ok) continue;
        const Tile tile = get_tile<KIND>(p, s, t, rank, split);
        const int kblocks = uniform(tile.kblocks);
        const int64_t kb0 = tile.k0 / kKBlock;
        const int valid = (KIND == kMany ? tile.p_valid : tile.q_valid) - lane;
        const float* rs = p.row_sf + kb0 * p.row_sf_pitch + (KIND == kMany ? tile.p0 : tile.q0) + lane;
        const int block = KIND == kMany ? tile.q0 / 128 : tile.p0 / 128;
        const int blocks = ceil_div(p.out_cols, 128);
        const float* ws = KIND == kWgrad ? p.col_sf + kb0 * p.out_cols + tile.p0 + lane
                                         : p.col_sf + (static_cast<int64_t>(tile.expert) * blocks + block) * p.kblocks;
        float r[kAhead][kSets][kRows], w[kAhead][kWeights];
        const auto fetch = [&](int kb, float (*rv)[kRows], float* wv) {
          const bool in = kb < kblocks;
#pragma unroll
          for (int h = 0; h < kSets; ++h)
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
              const int j = (h == 0 ? 0 : tile.n[0]) + i * 32;
              rv[h][i] = in && j < valid ? __ldg(rs + kb * p.row_sf_pitch + j) : 0.0f;
            }
          if (KIND == kWgrad) {
#pragma unroll
            for (int i = 0; i < kRows; ++i)
              wv[i] = in && lane + i * 32 < tile.p_valid ? __ldg(ws + static_cast<int64_t>(kb) * p.out_cols + i * 32) : 0.0f;
          } else {
            wv[0] = in && block < blocks ? __ldg(ws + kb0 + kb) : 0.0f;
            if (KIND == kMany) wv[ACCS - 1] = in && block + 1 < blocks ? __ldg(ws + p.kblocks + kb) : 0.0f;
          }
        };
#pragma unroll
        for (int d = 0; d < kAhead; ++d) fetch(d, r[d], w[d]);
        for (int kb = 0; kb < kblocks && ok; kb += kAhead) {
#pragma unroll
          for (int d = 0; d < kAhead; ++d) {
            if (kb + d >= kblocks) break;
#pragma unroll
            for (int h = 0; h < ACCS; ++h) {
              if (!(ok = wait_warp(&s.scale_empty[h][ring.i], ring.phase ^ 1, p.wait_ns))) break;
              float* to = s.scale[h][ring.i];
#pragma unroll
              for (int i = 0; i < kRows; ++i) {
                const int j = lane + i * 32;
                const float v = r[d][kSets == 2 ? h : 0][i];
                if (KIND == kMany) to[j] = v * w[d][h];
                if (KIND == kFew) to[scale_place(j)] = v * w[d][h];
                if (KIND == kWgrad) to[scale_place(j)] = v;
                if (KIND == kWgrad) to[128 + j] = w[d][i];
              }
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(&s.acc_full[h][ring.i]);
            }
            if (!ok) break;
            ring.next();
            fetch(kb + d + kAhead, r[d], w[d]);
          }
        }
      }
    }
  } else {
    // ---- epilogue --------------------------------------------------------
    // Warp w reads tensor-memory lanes 32 (w % 4) .. + 31 of one accumulator.
    tc::reg_inc<C::kEpilogueRegs>();
    constexpr int kBatches = C::kWarpCols / kBatchCols;
    const int uw = uniform(warp);
    const int ew = uw - 4, quarter = uw % 4, half = ew / (4 * C::kSplit), part = ew / 4 % C::kSplit;   // half: the accumulator
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * kAccCols + part * C::kWarpCols;
    uint32_t freed = ptx::smem_addr(&s.acc_empty[half][0]);   // the leader's barriers
    if (CTAS == 2) freed = tc::map_to_rank(freed, 0);
    Ring<NBUF> buf;
    for (int t = first_tile; t < tiles; t += step) {
      if (!ok) {
        meet();
        meet();
        continue;
      }
      int n, kblocks;                                         // all that lives over the k-blocks
      {
        const Tile tile = get_tile<KIND>(p, s, t, rank, split);
        n = (half == 0 ? tile.n[0] : tile.n[1]) - part * C::kWarpCols;
        kblocks = tile.kblocks;
        // kWgrad, 8 experts x 1024 rows: 304 -> 280 us (no spills).  kMany is slower so.
        if (KIND == kWgrad) n = uniform(n), kblocks = uniform(kblocks);
      }
      uint64_t acc[kBatches][16];                             // pairs of sums: see store_rows, store_columns
#pragma unroll
      for (int c = 0; c < kBatches; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[c][i] = 0;
#pragma unroll 1
      for (int kb = 0; kb < kblocks; ++kb) {
        if (!(ok = wait_warp(&s.acc_full[half][buf.i], buf.phase, p.wait_ns))) break;
        tc::fence_after();
        const float* sc = s.scale[half][buf.i];
        const uint32_t from = lane_base + buf.i * C::kTileCols;
        uint64_t ps[4];
        if (KIND == kMany) {
          const float v = sc[quarter * 32 + lane];
          ps[0] = tc::pack2(v, v);
          __syncwarp();
          if (tc::elect_one()) ptx::mbar_arrive(&s.scale_empty[half][buf.i]);
        }
        if (KIND == kWgrad) {
          const float* rows = sc + 128 + quarter * 32 + lane / 4;
#pragma unroll
          for (int i = 0; i < 4; ++i) ps[i] = tc::pack2(rows[8 * i], rows[8 * i]);
        }
        if constexpr (KIND == kMany) {
          // columns past n are read and added for nothing: only the last tile across has any
#pragma unroll
          for (int c = 0; c < kBatches; ++c) {
            float v[2][16];
            tc::ld_32x16(from + c * kBatchCols, v[0]);
            tc::ld_32x16(from + c * kBatchCols + 16, v[1]);
            tc::wait_ld();
            if (c == kBatches - 1) {   // all is in registers: the tensor core may have the buffer back
              tc::fence_before();
              __syncwarp();
              if (tc::elect_one()) tc::mbar_arrive_cluster_relaxed(freed + buf.i * 8);
            }
#pragma unroll
            for (int d = 0; d < 2; ++d)
#pragma unroll
              for (int i = 0; i < 8; ++i)
                acc[c][8 * d + i] = tc::fma2(tc::pack2(v[d][2 * i], v[d][2 * i + 1]), ps[0], acc[c][8 * d + i]);
          }
        } else {
          sc += part * C::kWarpCols + (lane % 4) * 4;
          if constexpr (KIND == kFew) {
            if (n > 0) {
              float v[kBatches][32];
#pragma unroll
              for (int c = 0; c < kBatches; ++c) {
                tc::ld_16x32(from + c * kBatchCols, v[c]);
                tc::ld_16x32(from + c * kBatchCols + (16u << 16), v[c] + 16);
              }
              uint64_t q[kBatches][4];
#pragma unroll
              for (int c = 0; c < kBatches; ++c) load_scales(sc + c * kBatchCols, q[c]);
              tc::wait_ld();
              tc::fence_before();
              __syncwarp();
              if (tc::elect_one()) tc::mbar_arrive_cluster_relaxed(freed + buf.i * 8);
#pragma unroll
              for (int c = 0; c < kBatches; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  acc[c][i] = tc::fma2(tc::pack2(v[c][16 * (i / 8) + 4 * (i / 2 % 4) + 2 * (i % 2)],
                                                    v[c][16 * (i / 8) + 4 * (i / 2 % 4) + 2 * (i % 2) + 1]), q[c][i / 2 % 4], acc[c][i]);
            }
          } else if (n > 0) {
#pragma unroll
            for (int c = 0; c < kBatches; ++c) {
              uint64_t q[4];
              load_scales(sc + c * kBatchCols, q);
#pragma unroll
              for (int up = 0; up < 2; ++up) {
                float v[16];
                tc::ld_16x32(from + c * kBatchCols + (static_cast<uint32_t>(16 * up) << 16), v);
                tc::wait_ld();
                if (c == kBatches - 1 && up == 1) {
                  tc::fence_before();
                  __syncwarp();
                  if (tc::elect_one()) tc::mbar_arrive_cluster_relaxed(freed + buf.i * 8);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  acc[c][8 * up + i] = tc::fma2(tc::mul2(tc::pack2(v[2 * i], v[2 * i + 1]), ps[2 * up + i % 2]), q[i / 2],
                                                acc[c][8 * up + i]);
              }
            }
          }
        }
        __syncwarp();
        if (KIND != kMany && tc::elect_one()) {
          if (n <= 0) tc::mbar_arrive_cluster_relaxed(freed + buf.i * 8);
          ptx::mbar_arrive(&s.scale_empty[half][buf.i]);
        }
        buf.next();
      }
      if (KIND == kFew && splits > 1) {
        // pair r of epilogue thread j at r * 256 + j of the stages, which are free
        uint64_t* sums = reinterpret_cast<uint64_t*>(mem.stage) + (threadIdx.x - 128);
        if (split > 0 && n > 0)
#pragma unroll
          for (int c = 0; c < kBatches; ++c)
            if (c * kBatchCols < n)
#pragma unroll
              for (int i = 0; i < 16; ++i) sums[(c * 16 + i) * 256] = acc[c][i];
        meet();
        if (split == 0 && n > 0)
          for (int q = 1; q < splits; ++q) {
            const uint32_t from = tc::map_to_rank(ptx::smem_addr(sums), q);
#pragma unroll
            for (int c = 0; c < kBatches; ++c)
              if (c * kBatchCols < n)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[c][i] = tc::add2(acc[c][i], tc::ld_cluster(from + (c * 16 + i) * 256 * 8));
          }
        ptx::fence_proxy_async_smem();   // the next tile's loads come through the async proxy
        meet();
      }
      if (!ok) continue;
      if (split > 0) continue;

      const Tile tile = get_tile<KIND>(p, s, t, rank, split);
      if constexpr (KIND == kMany) store_rows(p, tile, quarter, lane, half * kAccCols + part * C::kWarpCols,
                                                mem.out + ew * kRowsBytes, &map_c, acc);
      else store_columns<KIND>(p, tile, quarter, half, part, lane, mem.out + ew * kOutBytes, &map_c, acc);
      if (KIND != kWgrad && tile.last) zero_gap<KIND>(p, s, tile, rank, ew, lane);
    }
    if (KIND != kFew && lane == 0) ptx::bulk_wait<0>();
  }

  if (!ok) set_error(p.err, MOE_ERR_TIMEOUT);
  tc::fence_before();
  __syncthreads();
  if (CTAS == 2) tc::cluster_sync();   // no arrival or MMA of the peer is left
  if (warp == 1) {
    tc::fence_after();
    tc::tmem_free<CTAS>(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- host
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(f);
  });
  return fn;
}

// [planes, rows, width] of 1 (operands), 2 or 4 bytes (bf16 or fp32 results), with boxes
// of box_rows x 128 values of an operand or 32 of a result; what lies outside reads as zero
// and is not written.
cudaError_t encode(CUtensorMap* m, const void* base, int64_t width, int64_t rows, int64_t planes, int box_rows,
                   int bytes = 1) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return cudaErrorNotSupported;
  const int64_t pitch = bytes * width;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(planes)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch), static_cast<cuuint64_t>(pitch * rows)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(bytes == 1 ? kKBlock : kBatchCols), static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t unit[3] = {1, 1, 1};
  const CUtensorMapDataType type = bytes == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  const CUresult r = fn(m, type, 3, const_cast<void*>(base), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        bytes == 2 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <Kind KIND>
cudaError_t launch(const CUtensorMap& map_p, const CUtensorMap& map_q, const CUtensorMap& map_c, const GemmParams& p,
                   cudaStream_t stream) {
  const int cluster = Config<KIND>::kCtas * p.splits;
  const auto kernel = expert_gemm_kernel<KIND>;
  cudaError_t e = ensure_smem_limit(kernel, kSmemBytes<KIND>);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(device_sm_count() / cluster * cluster));
  cfg.blockDim = dim3(Config<KIND>::kThreads);
  cfg.dynamicSmemBytes = kSmemBytes<KIND>;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kernel, map_p, map_q, map_c, p);
}

GemmParams common_params(const ExpertGemmArgs& a) {
  GemmParams p{};
  p.num_experts = a.num_experts;
  p.expert_offset = a.expert_offset;
  p.expert_count = a.expert_count;
  p.capacity = a.capacity;
  p.out = a.out;
  p.out_fp32 = a.out_fp32;
  p.accumulate = a.accumulate;
  p.err = a.err;
  p.wait_ns = wait_config().limit_ns;
  p.extra_tx = wait_config().extra_tx;
  p.splits = 1;
  return p;
}

}  // namespace

cudaError_t launch_expert_gemm(const ExpertGemmArgs& a, cudaStream_t stream) {
  GemmParams p = common_params(a);
  p.row_sf = a.x_sf;
  p.row_sf_pitch = a.sf_ld;
  p.col_sf = a.w_sf;
  p.out_cols = static_cast<int>(a.width_out);
  p.kblocks = static_cast<int>(ceil_div64(a.width_in, kKBlock));
  // kFew's tile holds 128 rows of an expert, kMany's 256.  Up to a mean of 112 rows
  // (nearly all experts in one tile) kFew measures faster, from 128 on kMany.  32 experts,
  // tokens routed at random, kFew against kMany: 7168 -> 4096, mean of 64 rows 165 to 194 us,
  // 112 173 to 201, 120 198 to 201, 128 205 to 198, 144 251 to 199; 2048 -> 7168, 112 96
  // to 107, 120 107 to 107, 128 117 to 108.
  const int64_t mean = a.pairs / a.num_experts;
  const bool many = mean >= 120;
  if (!many) {
    // The tiles if the pairs are what they are said to be; at least 4 k-blocks a share.
    const int64_t tiles = (min64(a.num_experts, max64(a.pairs, 1)) + a.pairs / 128) * ceil_div64(a.width_out, kPRows);
    while (p.splits < 8 && 2 * p.splits * tiles <= device_sm_count() && 8 * p.splits <= p.kblocks) p.splits *= 2;
  }
  CUtensorMap rows, third, weights;
  cudaError_t e = encode(&rows, a.x, a.width_in, a.capacity, 1, many ? kPRows : 64);
  if (e == cudaSuccess)
    e = many ? encode(&third, a.out, a.width_out, a.capacity, 1, kBatchCols, 2) : encode(&third, a.x, a.width_in, a.capacity, 1, 16);
  if (e == cudaSuccess) e = encode(&weights, a.w, a.width_in, a.width_out, a.num_experts, many ? 64 : kPRows);
  if (e != cudaSuccess) return e;
  return many ? launch<kMany>(rows, weights, third, p, stream) : launch<kFew>(weights, rows, third, p, stream);
}

cudaError_t launch_expert_wgrad(const ExpertGemmArgs& a, cudaStream_t stream) {
  GemmParams p = common_params(a);
  p.row_sf = a.w_sf;
  p.row_sf_pitch = a.width_out;
  p.col_sf = a.x_sf;
  p.out_cols = static_cast<int>(a.width_in);
  p.dy_rows = static_cast<int>(a.width_out);
  CUtensorMap x, dy, out;
  cudaError_t e = encode(&x, a.x, a.sf_ld, a.width_in, 1, kPRows);
  if (e == cudaSuccess) e = encode(&dy, a.w, a.sf_ld, a.width_out, 1, 64);
  if (e == cudaSuccess) e = encode(&out, a.out, a.width_in, a.width_out, a.num_experts, kBatchCols, a.out_fp32 ? 4 : 2);
  return e == cudaSuccess ? launch<kWgrad>(x, dy, out, p, stream) : e;
}

}  // namespace moe
