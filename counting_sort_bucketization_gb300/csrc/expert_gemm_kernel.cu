// expert_gemm_kernel.cu -- products of e4m3 operands with an fp32 scale for
// each block of 128, over the segments of the receive buffer:
//
//   forward (and input gradient)  out[r, o] = sum_b sx[b, r] sw[e, o/128, b] <x_r, w_o>_b
//   weight gradient               dw[e, o, i] = sum_b sdy[b, o] sx[b, i] <dy_o, x_i>_b
//
// Both are D[p, q] = sum_b sp sq <P_p, Q_q>_b written to out[q * pitch + p]:
// P = weights (forward) or x^T (gradient) gives the 128 accumulator rows of a
// CTA, Q = receive rows or dy^T its columns.
//
// Why this orientation: the tensor core takes any multiple of 16 columns, so a
// tile has as many columns as the segment has rows left and an expert with one
// token does not pay for 128; and a CTA's 128 weight rows are one scale block, so
// their scale is one number a k-block.
//
// A scale that changes every 128 values of K means the tensor core can sum one
// k-block only.  Each k-block's product lands in tensor memory, and epilogue
// warps add it, times its scales, to fp32 sums in registers:
//
//   warp 0      TMA loads of P and Q tiles (128-byte rows, one k-block wide)
//   warp 1      tcgen05.mma, 4 per k-block, into one of NBUF tensor-memory buffers
//   warps 2-3   the k-block's scales to shared memory
//   warps 4-19  tensor memory -> fp32 sums; at the tile's end bf16 (fp32) rows out
//
// More than 128 columns are two accumulators, each with its own barriers and 8
// of the 16 epilogue warps: the tensor core fills one while the other is read.
//
// One persistent CTA (or pair: CTAS == 2, one 256-row MMA over two SMs, each
// loading half of Q) per SM walks the tiles of all experts.  All sums are fp32;
// the result is rounded once.
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

constexpr int kThreads = 640;
constexpr int kEpilogueWarps = 16;
constexpr int kHalfCols = 128;                     // columns of an accumulator
constexpr int kBatchCols = 32;                     // columns a warp loads at a time
constexpr int kBatches = 2;                        // of a warp: 8 warps, 4 of them side by side in rows
constexpr int kKBlock = 128;                       // values (and bytes) of K in a scale block
constexpr int kPRows = 128;                        // accumulator rows of a CTA
constexpr int kPBytes = kPRows * kKBlock;
constexpr int kQBytes = 128 * kKBlock;             // Q rows a CTA holds at most: 128
constexpr int kStageBytes = kPBytes + kQBytes;
constexpr int kStages = 6;
constexpr int kScaleSlots = 6;
constexpr int kSlotWords = 256 + kPRows;           // Q scales, then P scales (forward: one word)
constexpr int kOutPitch = 80;                      // bytes; 64 of data, conflict-free for stmatrix
constexpr int kOutBytes = 8 * kOutPitch;           // a warp's 8 rows x 32 columns of bf16
constexpr int kTmemCols = 512;
constexpr int kScaleThreads = 64;
// Registers a thread: each SM quarter holds 4 epilogue warps and one other.
constexpr int kLaunchRegs = 96, kEpilogueRegs = 104, kOtherRegs = 64;
static_assert(512 * kEpilogueRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "register split above the launch's total");

struct Smem {
  alignas(1024) uint8_t stage[kStages][kStageBytes];
  alignas(16) float scale[kScaleSlots][kSlotWords];
  alignas(16) uint8_t out[kEpilogueWarps][kOutBytes];
  int tile_end[MOE_MAX_EXPERTS];                   // tiles of experts 0..e
  int seg_start[MOE_MAX_EXPERTS];
  int seg_count[MOE_MAX_EXPERTS];
  uint64_t full[kStages], empty[kStages];
  uint64_t scale_full[kScaleSlots], scale_empty[kScaleSlots];
  uint64_t acc_full[2][4], acc_empty[2][4];        // [half][buffer]
  uint32_t tmem;
  int warp_sum[kThreads / 32];
};
// The dynamic base is only known to be 16-byte aligned: room to align it.
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory of one SM");

struct Tile {
  int expert;
  int p0;          // first row of P for this CTA
  int q0;          // first row of Q
  int q_valid;     // rows of Q that exist
  int n[2];        // columns of the two accumulators; the second may have none
  int k0;          // first k (forward 0, gradient: the segment's first row)
  int kblocks;
  bool last_q;     // the expert's last tile along Q
};

__host__ __device__ constexpr int ceil_div(int a, int b) { return (a + b - 1) / b; }

template <int CTAS, int MAXN, bool WGRAD>
struct Tiling {
  static constexpr int kUnit = 16 * CTAS;   // column granularity: each CTA of a pair holds n / 2 rows of Q

  __device__ static int q_tiles(const GemmParams& p, int count) {
    return WGRAD ? ceil_div(p.q_rows, MAXN) : ceil_div(count, MAXN);
  }
  __device__ static Tile get(const GemmParams& p, const Smem& s, int t, uint32_t rank) {
    int lo = 0, hi = p.num_experts - 1;     // first expert whose tiles end after t
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (s.tile_end[mid] > t) hi = mid; else lo = mid + 1;
    }
    const int first = lo == 0 ? 0 : s.tile_end[lo - 1];
    const int count = s.seg_count[lo], nq = q_tiles(p, count);
    const int local = t - first, q = local % nq, pt = local / nq;
    const int q_rows = WGRAD ? p.q_rows : count;
    // columns shared evenly over the tiles along Q
    const int per = ceil_div(ceil_div(q_rows, nq), kUnit) * kUnit;
    Tile r;
    r.expert = lo;
    r.p0 = (pt * CTAS + static_cast<int>(rank)) * kPRows;
    r.q_valid = max(0, min(per, q_rows - q * per));
    r.q0 = (WGRAD ? 0 : s.seg_start[lo]) + q * per;
    const int n = max(kUnit, ceil_div(r.q_valid, kUnit) * kUnit);
    r.n[0] = n <= kHalfCols ? n : ceil_div(n / 2, 32) * 32;
    r.n[1] = n - r.n[0];
    r.k0 = WGRAD ? s.seg_start[lo] : 0;
    r.kblocks = WGRAD ? ceil_div(count, kKBlock) : p.kblocks;
    r.last_q = q == nq - 1;
    return r;
  }
};

// Place of column j's scale: a lane reads the four it needs of 16 columns as one vector.
__device__ __forceinline__ int scale_place(int j) {
  return (j & ~15) + ((j & 7) >> 1) * 4 + ((j & 8) >> 3) * 2 + (j & 1);
}

// The whole warp waits, and leaves together (tcgen05.ld needs all lanes).
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, limit_ns));
}

template <int CTAS, int MAXN, bool WGRAD>
__global__ void __launch_bounds__(kThreads, 1)
expert_gemm_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q64,
                   const __grid_constant__ CUtensorMap map_q16, const GemmParams p) {
  constexpr int NBUF = kTmemCols / MAXN;
  static_assert(NBUF <= 4 && (MAXN <= kHalfCols || CTAS == 2), "tensor memory and shared memory of Q");
  using T = Tiling<CTAS, MAXN, WGRAD>;
  extern __shared__ uint8_t smem_raw[];
  // The same offset in both CTAs of a pair: the bases are equal.
  Smem& s = *reinterpret_cast<Smem*>(smem_raw + ((1024 - (ptx::smem_addr(smem_raw) & 1023)) & 1023));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = CTAS == 2 ? tc::cluster_rank() : 0;
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    tc::prefetch_map(&map_p);
    tc::prefetch_map(&map_q64);
    tc::prefetch_map(&map_q16);
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&s.full[i], 1);
      ptx::mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < kScaleSlots; ++i) {
      ptx::mbar_init(&s.scale_full[i], kScaleThreads);
      ptx::mbar_init(&s.scale_empty[i], kEpilogueWarps);
    }
    for (int i = 0; i < NBUF; ++i)
      for (int h = 0; h < 2; ++h) {
        ptx::mbar_init(&s.acc_full[h][i], 1);
        ptx::mbar_init(&s.acc_empty[h][i], kEpilogueWarps / 2 * CTAS);
      }
    ptx::fence_mbar_init();
  }
  if (warp == 1) tc::tmem_alloc<CTAS>(&s.tmem, kTmemCols);
  ptx::grid_dependency_wait();

  // Segments and the running count of tiles.  A segment that does not lie in
  // the buffer (a layout that overflowed its capacity, or a start that is not a
  // block boundary for the gradient) is left out and recorded.
  const int p_tiles = ceil_div(p.p_rows, kPRows * CTAS);
  int running = 0;
  for (int base = 0; base < p.num_experts; base += kThreads) {
    const int e = base + static_cast<int>(threadIdx.x);
    int tiles = 0;
    if (e < p.num_experts) {
      const int start = p.expert_offset[e];
      int count = p.expert_count[e];
      const bool fits = start >= 0 && count >= 0 && static_cast<int64_t>(start) + count <= p.capacity;
      const bool whole = !WGRAD || start % kKBlock == 0;
      if (!fits || !whole) {
        set_error(p.err, fits ? MOE_ERR_INVALID_ARG : MOE_ERR_CAPACITY);
        count = 0;
      }
      s.seg_start[e] = count > 0 ? start : 0;
      s.seg_count[e] = count;
      tiles = T::q_tiles(p, count) * p_tiles;
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
  const int tiles = running;
  tc::fence_before();
  __syncthreads();
  if (CTAS == 2) tc::cluster_sync();   // the pair's barriers and tensor memory exist
  tc::fence_after();
  const uint32_t tmem = s.tmem;
  const int first_tile = static_cast<int>(blockIdx.x) / CTAS, step = static_cast<int>(gridDim.x) / CTAS;
  bool ok = true;

  if (warp < 4) {
    tc::reg_dec<kOtherRegs>();
    if (warp == 0 && lane == 0) {
      // ---- loads ---------------------------------------------------------
      uint32_t it = 0;
      for (int t = first_tile; t < tiles && ok; t += step) {
        const Tile tile = T::get(p, s, t, rank);
        const uint32_t bytes = CTAS * kPBytes + (tile.n[0] + tile.n[1]) * kKBlock;
        for (int kb = 0; kb < tile.kblocks; ++kb, ++it) {
          const uint32_t st = it % kStages;
          if (!(ok = tc::mbar_wait(&s.empty[st], (it / kStages & 1) ^ 1, p.wait_ns))) break;
          if (leader) ptx::mbar_arrive_expect_tx(&s.full[st], bytes + (it == 0 ? p.extra_tx : 0));
          uint32_t bar = ptx::smem_addr(&s.full[st]);
          if (CTAS == 2) bar = tc::map_to_rank(bar, 0);
          const uint32_t dst = ptx::smem_addr(s.stage[st]);
          const int x = tile.k0 + kb * kKBlock;
          tc::load_box<CTAS>(dst, &map_p, x, tile.p0, WGRAD ? 0 : tile.expert, bar);
          // the columns of each accumulator, half of them by each CTA of a pair
#pragma unroll
          for (int h = 0; h < CTAS; ++h) {
            const int rows = tile.n[h] / CTAS;
            const int q = tile.q0 + (h == 0 ? 0 : tile.n[0]) + static_cast<int>(rank) * rows;
            const uint32_t to = dst + kPBytes + h * (kHalfCols / CTAS) * kKBlock;
            int r = 0;
            for (; r + 64 <= rows; r += 64) tc::load_box<CTAS>(to + r * kKBlock, &map_q64, x, q + r, 0, bar);
            for (; r < rows; r += 16) tc::load_box<CTAS>(to + r * kKBlock, &map_q16, x, q + r, 0, bar);
          }
        }
      }
      // Every stage handed back: no copy or remote arrival is left in flight.
      for (uint32_t i = 0; i < kStages; ++i, ++it)
        if (it >= kStages) ok &= tc::mbar_wait(&s.empty[it % kStages], (it / kStages & 1) ^ 1, p.wait_ns);
    } else if (warp == 1 && lane == 0 && leader) {
      // ---- MMA -----------------------------------------------------------
      uint32_t it = 0, used[2] = {0, 0};
      for (int t = first_tile; t < tiles && ok; t += step) {
        const Tile tile = T::get(p, s, t, rank);
        for (int kb = 0; kb < tile.kblocks && ok; ++kb, ++it) {
          const uint32_t st = it % kStages;
          if (!(ok = tc::mbar_wait(&s.full[st], it / kStages & 1, p.wait_ns))) break;
          const uint64_t a = tc::operand_desc(ptx::smem_addr(s.stage[st]));
#pragma unroll
          for (int h = 0; h < CTAS; ++h) {
            if (tile.n[h] == 0) continue;
            const uint32_t b = used[h] % NBUF;
            if (!(ok = tc::mbar_wait(&s.acc_empty[h][b], (used[h] / NBUF & 1) ^ 1, p.wait_ns))) break;
            ++used[h];
            tc::fence_after();
            const uint64_t q =
                tc::operand_desc(ptx::smem_addr(s.stage[st]) + kPBytes + h * (kHalfCols / CTAS) * kKBlock);
            const uint32_t idesc = tc::instr_desc(kPRows * CTAS, tile.n[h]);
#pragma unroll
            for (int k = 0; k < kKBlock / 32; ++k)
              tc::mma_e4m3<CTAS>(tmem + b * MAXN + h * kHalfCols, a + 2 * k, q + 2 * k, idesc, k > 0);
            tc::commit<CTAS>(&s.acc_full[h][b]);
          }
          if (ok) tc::commit<CTAS>(&s.empty[st]);
        }
      }
      for (int h = 0; h < 2; ++h)   // the epilogues' last (remote) arrivals
        for (uint32_t i = 0; i < NBUF; ++i, ++used[h])
          if (used[h] >= NBUF)
            ok &= tc::mbar_wait(&s.acc_empty[h][used[h] % NBUF], (used[h] / NBUF & 1) ^ 1, p.wait_ns);
    } else if (warp >= 2) {
      // ---- scales --------------------------------------------------------
      // Through registers, kAhead k-blocks ahead; the forward product's P scale is
      // one number a k-block and goes into the Q scales here.
      constexpr int kAhead = 3, kQ = MAXN / kScaleThreads, kP = WGRAD ? kPRows / kScaleThreads : 1;
      const int j0 = static_cast<int>(threadIdx.x) - 64;
      uint32_t it = 0;
      for (int t = first_tile; t < tiles && ok; t += step) {
        const Tile tile = T::get(p, s, t, rank);
        const int64_t kb0 = tile.k0 / kKBlock;
        const float* qs = p.q_sf + kb0 * p.q_sf_pitch + tile.q0 + j0;
        const float* ps = WGRAD ? p.p_sf + kb0 * p.p_rows + tile.p0 + j0
                                : p.p_sf + (static_cast<int64_t>(tile.expert) * ceil_div(p.p_rows, kKBlock) +
                                            tile.p0 / kKBlock) * p.kblocks;
        float q[kAhead][kQ], w[kAhead][kP];
        const auto fetch = [&](int kb, float* qv, float* wv) {
          const bool in = kb < tile.kblocks;
#pragma unroll
          for (int i = 0; i < kQ; ++i)
            qv[i] = in && j0 + i * kScaleThreads < tile.q_valid ? __ldg(qs + kb * p.q_sf_pitch + i * kScaleThreads) : 0.0f;
#pragma unroll
          for (int i = 0; i < kP; ++i)
            wv[i] = !in || tile.p0 + (WGRAD ? j0 + i * kScaleThreads : 0) >= p.p_rows ? 0.0f
                    : WGRAD ? __ldg(ps + static_cast<int64_t>(kb) * p.p_rows + i * kScaleThreads) : __ldg(ps + kb);
        };
#pragma unroll
        for (int d = 0; d < kAhead; ++d) fetch(d, q[d], w[d]);
        for (int kb = 0; kb < tile.kblocks && ok; kb += kAhead) {
#pragma unroll
          for (int d = 0; d < kAhead; ++d) {
            if (kb + d >= tile.kblocks) break;
            const uint32_t sl = it % kScaleSlots;
            if (!(ok = tc::mbar_wait(&s.scale_empty[sl], (it / kScaleSlots & 1) ^ 1, p.wait_ns))) break;
            ++it;
#pragma unroll
            for (int i = 0; i < kQ; ++i)
              s.scale[sl][scale_place(j0 + i * kScaleThreads)] = WGRAD ? q[d][i] : q[d][i] * w[d][0];
            if (WGRAD) {
#pragma unroll
              for (int i = 0; i < kP; ++i) s.scale[sl][256 + j0 + i * kScaleThreads] = w[d][i];
            }
            ptx::mbar_arrive(&s.scale_full[sl]);
            fetch(kb + d + kAhead, q[d], w[d]);
          }
        }
      }
    }
  } else {
    // ---- epilogue --------------------------------------------------------
    // Warp w reads tensor-memory lanes 32 (w % 4) .. + 31 of one accumulator:
    // 32 columns, and the 32 columns 64 further on.
    tc::reg_inc<kEpilogueRegs>();
    const int ew = warp - 4, quarter = warp % 4, half = ew / 8, sub = ew / 4 % 2;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * kHalfCols + sub * kBatchCols;
    uint8_t* stage = s.out[ew];
    uint32_t it = 0, used = 0;
    for (int t = first_tile; t < tiles && ok; t += step) {
      // Only these three values stay in registers over the k-blocks.
      int n, first, kblocks;
      {
        const Tile tile = T::get(p, s, t, rank);
        n = half == 0 ? tile.n[0] : tile.n[1];
        first = half == 0 ? 0 : tile.n[0];                  // column of the tile the accumulator starts at
        kblocks = tile.kblocks;
      }
      uint64_t acc[kBatches][16];
#pragma unroll
      for (int c = 0; c < kBatches; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[c][i] = 0;
      for (int kb = 0; kb < kblocks; ++kb, ++it) {
        const uint32_t b = used % NBUF, sl = it % kScaleSlots;
        if (!(ok = wait_warp(&s.scale_full[sl], it / kScaleSlots & 1, p.wait_ns))) break;
        if (n > 0) {
          if (!(ok = wait_warp(&s.acc_full[half][b], used / NBUF & 1, p.wait_ns))) break;
          ++used;
          tc::fence_after();
          const float* sc = s.scale[sl];
          uint64_t pw[4];
          if (WGRAD) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float v = sc[256 + quarter * 32 + 8 * i + lane / 4];
              pw[i] = tc::pack2(v, v);
            }
          }
          sc += first + sub * kBatchCols + (lane % 4) * 4;
#pragma unroll
          for (int c = 0; c < kBatches; ++c) {
            if (c * 2 * kBatchCols + sub * kBatchCols < n) {
              uint32_t v[32];
              tc::ld_16x32(lane_base + b * MAXN + c * 2 * kBatchCols, v);
              tc::ld_16x32(lane_base + b * MAXN + c * 2 * kBatchCols + (16u << 16), v + 16);
              const float4 q4[2] = {*reinterpret_cast<const float4*>(sc + c * 2 * kBatchCols),
                                    *reinterpret_cast<const float4*>(sc + c * 2 * kBatchCols + 16)};
              tc::wait_ld();
              // acc[c][8 * up + 2 * h + r]: rows 16 * up + 8 * r + lane / 4, columns 8 * h + 2 * (lane % 4), +1
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                const uint64_t qs = h % 2 == 0 ? tc::pack2(q4[h / 2].x, q4[h / 2].y) : tc::pack2(q4[h / 2].z, q4[h / 2].w);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int up = i / 2, r = i % 2;
                  uint64_t v2 = tc::pack2(v[16 * up + 4 * h + 2 * r], v[16 * up + 4 * h + 2 * r + 1]);
                  if (WGRAD) v2 = tc::mul2(v2, pw[i]);
                  acc[c][8 * up + 2 * h + r] = tc::fma2(v2, qs, acc[c][8 * up + 2 * h + r]);
                }
              }
            }
          }
          tc::fence_before();
        }
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(&s.scale_empty[sl]);
          if (n > 0) {
            if (CTAS == 2) tc::mbar_arrive_cluster_relaxed(tc::map_to_rank(ptx::smem_addr(&s.acc_empty[half][b]), 0));
            else ptx::mbar_arrive(&s.acc_empty[half][b]);
          }
        }
      }
      if (!ok) break;

      const Tile tile = T::get(p, s, t, rank);
      const int col0 = tile.p0 + quarter * 32;              // the warp's first column of out
      const int64_t row0 = (WGRAD ? static_cast<int64_t>(tile.expert) * p.q_rows : 0) + tile.q0;
#pragma unroll
      for (int c = 0; c < kBatches; ++c) {
        const int col = c * 2 * kBatchCols + sub * kBatchCols;
        if (col >= n) break;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int row = first + col + 8 * h;              // of the tile; 8 of them
          if (WGRAD && p.out_fp32) {
            float* out = static_cast<float*>(p.out) + row0 * p.p_rows;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 v = tc::unpack2(acc[c][8 * (i / 2) + 2 * h + i % 2]);
              const int oc = col0 + 8 * i + lane / 4, r = row + 2 * (lane % 4);
              float* o = out + static_cast<int64_t>(r) * p.p_rows + oc;
              if (oc < p.p_rows && r < tile.q_valid) *o = p.accumulate ? *o + v.x : v.x;
              if (oc < p.p_rows && r + 1 < tile.q_valid) o[p.p_rows] = p.accumulate ? o[p.p_rows] + v.y : v.y;
            }
            continue;
          }
          uint32_t v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = tc::unpack2(acc[c][8 * (i / 2) + 2 * h + i % 2]);
            const __nv_bfloat162 h2 = __floats2bfloat162_rn(f.x, f.y);
            v[i] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          // four matrices of 8 columns of out, transposed to 8 rows of 64 bytes
          tc::stmatrix_x4_trans(ptx::smem_addr(stage) + (lane % 8) * kOutPitch + (lane / 8) * 16, v[0], v[1], v[2], v[3]);
          __syncwarp();
          const int r = row + lane / 4, oc = col0 + (lane % 4) * 8;
          const uint4 w = ptx::ld_shared_v4(stage + lane / 4 * kOutPitch + (lane % 4) * 16);
          if (r < tile.q_valid && oc < p.p_rows) ptx::st_v4(static_cast<uint16_t*>(p.out) + (row0 + r) * p.p_rows + oc, w);
          __syncwarp();
        }
      }
      if (!WGRAD && tile.last_q) {
        // gap rows of the segment: zeros, the four warps of the same columns in turn
        const int64_t end = min64(p.expert_offset[tile.expert + 1], p.capacity);
        const int oc = col0 + (lane % 4) * 8;
        if (oc < p.p_rows)
          for (int64_t r = static_cast<int64_t>(tile.q0) + tile.q_valid + ew / 4 * 8 + lane / 4; r < end; r += 32)
            ptx::st_v4(static_cast<uint16_t*>(p.out) + r * p.p_rows + oc, make_uint4(0, 0, 0, 0));
      }
    }
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

// Bytes [planes, rows, width] with boxes of box_rows x 128 bytes, 128-byte swizzle;
// what lies outside reads as zero.
cudaError_t encode(CUtensorMap* m, const void* base, int64_t width, int64_t rows, int64_t planes, int box_rows) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(planes)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(width * rows)};
  const cuuint32_t box[3] = {kKBlock, static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t unit[3] = {1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, unit,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int CTAS, int MAXN, bool WGRAD>
cudaError_t launch(const CUtensorMap* maps, const GemmParams& p, cudaStream_t stream) {
  const auto kernel = expert_gemm_kernel<CTAS, MAXN, WGRAD>;
  cudaError_t e = ensure_smem_limit(kernel, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(device_sm_count() / CTAS * CTAS));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CTAS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kernel, maps[0], maps[1], maps[2], p);
}

}  // namespace

cudaError_t launch_expert_gemm(const ExpertGemmArgs& a, cudaStream_t stream) {
  GemmParams p{};
  p.p_sf = a.w_sf;
  p.q_sf = a.x_sf;
  p.q_sf_pitch = a.sf_ld;
  p.p_rows = static_cast<int>(a.width_out);
  p.kblocks = static_cast<int>(ceil_div64(a.width_in, kKBlock));
  p.num_experts = a.num_experts;
  p.expert_offset = a.expert_offset;
  p.expert_count = a.expert_count;
  p.capacity = a.capacity;
  p.out = a.out;
  p.err = a.err;
  p.wait_ns = wait_config().limit_ns;
  p.extra_tx = wait_config().extra_tx;
  CUtensorMap maps[3];
  cudaError_t e = encode(&maps[0], a.w, a.width_in, a.width_out, a.num_experts, kPRows);
  if (e == cudaSuccess) e = encode(&maps[1], a.x, a.width_in, a.capacity, 1, 64);
  if (e == cudaSuccess) e = encode(&maps[2], a.x, a.width_in, a.capacity, 1, 16);
  if (e != cudaSuccess) return e;
  // Rows an expert has in the mean: many fill the 256 columns of a pair's tile.
  if (a.pairs / a.num_experts >= 192) return launch<2, 256, false>(maps, p, stream);
  return launch<1, 128, false>(maps, p, stream);
}

cudaError_t launch_expert_wgrad(const ExpertGemmArgs& a, cudaStream_t stream) {
  GemmParams p{};
  p.p_sf = a.x_sf;
  p.q_sf = a.w_sf;
  p.q_sf_pitch = a.width_out;
  p.p_rows = static_cast<int>(a.width_in);
  p.q_rows = static_cast<int>(a.width_out);
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
  CUtensorMap maps[3];
  cudaError_t e = encode(&maps[0], a.x, a.sf_ld, a.width_in, 1, kPRows);
  if (e == cudaSuccess) e = encode(&maps[1], a.w, a.sf_ld, a.width_out, 1, 64);
  if (e == cudaSuccess) e = encode(&maps[2], a.w, a.sf_ld, a.width_out, 1, 16);
  if (e != cudaSuccess) return e;
  return launch<2, 256, true>(maps, p, stream);
}

}  // namespace moe
