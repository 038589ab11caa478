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
//   warps 4-11  tensor memory -> fp32 sums; at the tile's end bf16 (fp32) rows out
//
// More than 128 columns are two accumulators, each with its own barriers and 4
// of the 8 epilogue warps: the tensor core fills one while the other is read.
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

constexpr int kThreads = 384;
constexpr int kEpilogueWarps = 8;
constexpr int kHalfCols = 128;                     // columns of an accumulator
constexpr int kBatchCols = 32;                     // columns a warp loads at a time
constexpr int kBatches = kHalfCols / kBatchCols;
constexpr int kKBlock = 128;                       // values (and bytes) of K in a scale block
constexpr int kPRows = 128;                        // accumulator rows of a CTA
constexpr int kPBytes = kPRows * kKBlock;
constexpr int kQBytes = 128 * kKBlock;             // Q rows a CTA holds at most: 128
constexpr int kStageBytes = kPBytes + kQBytes;
constexpr int kStages = 6;
constexpr int kSlotWords = kHalfCols + kPRows;     // scales of an accumulator's columns, then (gradient) of its rows
constexpr int kOutPitch = 96;                      // bytes; 64 of data, 4 rows' 32-byte pieces in different banks
constexpr int kOutBytes = 8 * kOutPitch;           // a warp's 8 rows x 32 columns of bf16
constexpr int kTmemCols = 512;
// Registers a thread: 128 sums, two batches of tensor memory in flight.
constexpr int kLaunchRegs = 168, kEpilogueRegs = 224, kOtherRegs = 56;
static_assert(256 * kEpilogueRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "register split above the launch's total");

struct Smem {
  alignas(1024) uint8_t stage[kStages][kStageBytes];
  alignas(16) float scale[2][4][kSlotWords];       // [half][buffer]
  alignas(16) uint8_t out[kEpilogueWarps][kOutBytes];
  int tile_end[MOE_MAX_EXPERTS];                   // tiles of experts 0..e
  int seg_start[MOE_MAX_EXPERTS];
  int seg_count[MOE_MAX_EXPERTS];
  uint64_t full[kStages], empty[kStages];
  uint64_t acc_full[2][4], acc_empty[2][4];        // [half][buffer]; full: product and scales are there
  uint64_t scale_empty[2][4];
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

// Place of column j's scale: a lane reads the eight it needs of 32 columns (j % 4
// is the same) as two vectors.
__device__ __forceinline__ int scale_place(int j) {
  return (j & ~31) + ((j & 16) >> 4) * 16 + (j & 3) * 4 + ((j & 15) >> 2);
}

// Position in a ring of N buffers, and the parity of the phase it is in.
template <int N>
struct Ring {
  uint32_t i = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++i == N) i = 0, phase ^= 1;
  }
};

// The whole warp waits, and leaves together (tcgen05.ld needs all lanes).
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, limit_ns));
}

template <int CTAS, int MAXN, bool WGRAD>
__global__ void __launch_bounds__(kThreads, 1)
expert_gemm_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                   const GemmParams p) {
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
    tc::prefetch_map(&map_q);
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&s.full[i], 1);
      ptx::mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < NBUF; ++i)
      for (int h = 0; h < 2; ++h) {
        ptx::mbar_init(&s.acc_full[h][i], 2);      // the commit, and the scales' warp
        ptx::mbar_init(&s.acc_empty[h][i], kEpilogueWarps / 2 * CTAS);
        ptx::mbar_init(&s.scale_empty[h][i], kEpilogueWarps / 2);
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
    if (warp == 0) {
      // ---- loads ---------------------------------------------------------
      // The warp stays together so that addresses live in uniform registers; one
      // lane issues.
      Ring<kStages> ring;
      uint32_t loads = 0;
      for (int t = first_tile; t < tiles && ok; t += step) {
        const Tile tile = T::get(p, s, t, rank);
        // Q rows of each accumulator, an equal share by each CTA of a pair, in whole boxes
        int q[CTAS], boxes[CTAS], all = 0;
#pragma unroll
        for (int h = 0; h < CTAS; ++h) {
          const int rows = tile.n[h] / CTAS;
          q[h] = tile.q0 + (h == 0 ? 0 : tile.n[0]) + static_cast<int>(rank) * rows;
          boxes[h] = ceil_div(rows, p.q_box);
          all += boxes[h];
        }
        const uint32_t bytes = CTAS * (kPBytes + all * p.q_box * kKBlock);
        for (int kb = 0; kb < tile.kblocks; ++kb) {
          if (!(ok = wait_warp(&s.empty[ring.i], ring.phase ^ 1, p.wait_ns))) break;
          if (tc::elect_one()) {
            if (leader) ptx::mbar_arrive_expect_tx(&s.full[ring.i], bytes + (loads == 0 ? p.extra_tx : 0));
            uint32_t bar = ptx::smem_addr(&s.full[ring.i]);
            if (CTAS == 2) bar = tc::map_to_rank(bar, 0);
            const uint32_t dst = ptx::smem_addr(s.stage[ring.i]);
            const int x = tile.k0 + kb * kKBlock;
            tc::load_box<CTAS>(dst, &map_p, x, tile.p0, WGRAD ? 0 : tile.expert, bar);
#pragma unroll
            for (int h = 0; h < CTAS; ++h)
              for (int i = 0; i < boxes[h]; ++i)
                tc::load_box<CTAS>(dst + kPBytes + (h * (kHalfCols / CTAS) + i * p.q_box) * kKBlock, &map_q, x,
                                   q[h] + i * p.q_box, 0, bar);
          }
          __syncwarp();
          ring.next();
          ++loads;
        }
      }
      // Every stage handed back: no copy or remote arrival is left in flight.
      for (uint32_t i = 0; i < kStages; ++i, ++loads, ring.next())
        if (loads >= kStages) ok &= wait_warp(&s.empty[ring.i], ring.phase ^ 1, p.wait_ns);
    } else if (warp == 1 && leader) {
      // ---- MMA -----------------------------------------------------------
      Ring<kStages> ring;
      Ring<NBUF> buf[2];
      uint32_t used[2] = {0, 0};
      const uint64_t p_desc = tc::operand_desc(ptx::smem_addr(s.stage[0]));
      for (int t = first_tile; t < tiles && ok; t += step) {
        const Tile tile = T::get(p, s, t, rank);
        const uint32_t idesc[2] = {tc::instr_desc(kPRows * CTAS, tile.n[0]), tc::instr_desc(kPRows * CTAS, tile.n[1])};
        for (int kb = 0; kb < tile.kblocks && ok; ++kb) {
          if (!(ok = wait_warp(&s.full[ring.i], ring.phase, p.wait_ns))) break;
          const uint64_t a = p_desc + ring.i * (kStageBytes >> 4);
#pragma unroll
          for (int h = 0; h < CTAS; ++h) {
            if (h == 1 && tile.n[1] == 0) continue;
            if (!(ok = wait_warp(&s.acc_empty[h][buf[h].i], buf[h].phase ^ 1, p.wait_ns))) break;
            tc::fence_after();
            if (tc::elect_one()) {
              const uint64_t q = a + ((kPBytes + h * (kHalfCols / CTAS) * kKBlock) >> 4);
              const uint32_t d = tmem + buf[h].i * MAXN + h * kHalfCols;
#pragma unroll
              for (int k = 0; k < kKBlock / 32; ++k) tc::mma_e4m3<CTAS>(d, a + 2 * k, q + 2 * k, idesc[h], k > 0);
              tc::commit<CTAS>(&s.acc_full[h][buf[h].i]);
            }
            __syncwarp();
            buf[h].next();
            ++used[h];
          }
          if (ok && tc::elect_one()) tc::commit<CTAS>(&s.empty[ring.i]);
          __syncwarp();
          ring.next();
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)   // the epilogues' last (remote) arrivals
        for (uint32_t i = 0; i < NBUF; ++i, ++used[h], buf[h].next())
          if (used[h] >= NBUF) ok &= wait_warp(&s.acc_empty[h][buf[h].i], buf[h].phase ^ 1, p.wait_ns);
    } else if (warp >= 2) {
      // ---- scales --------------------------------------------------------
      // Warp 2 + h brings those of accumulator h, through registers and kAhead
      // k-blocks ahead; the forward product's P scale is one number a k-block and
      // goes into the Q scales here.
      constexpr int kAhead = 3, kQ = kHalfCols / 32, kP = WGRAD ? kPRows / 32 : 1;
      const int half = warp - 2;
      Ring<NBUF> ring;
      for (int t = first_tile; t < tiles && ok; t += step) {
        const Tile tile = T::get(p, s, t, rank);
        if ((half == 0 ? tile.n[0] : tile.n[1]) == 0) continue;
        const int64_t kb0 = tile.k0 / kKBlock;
        const int j0 = (half == 0 ? 0 : tile.n[0]) + lane;
        const float* qs = p.q_sf + kb0 * p.q_sf_pitch + tile.q0 + j0;
        const float* ps = WGRAD ? p.p_sf + kb0 * p.p_rows + tile.p0 + lane
                                : p.p_sf + (static_cast<int64_t>(tile.expert) * ceil_div(p.p_rows, kKBlock) +
                                            tile.p0 / kKBlock) * p.kblocks;
        float q[kAhead][kQ], w[kAhead][kP];
        const auto fetch = [&](int kb, float* qv, float* wv) {
          const bool in = kb < tile.kblocks;
#pragma unroll
          for (int i = 0; i < kQ; ++i)
            qv[i] = in && j0 + i * 32 < tile.q_valid ? __ldg(qs + kb * p.q_sf_pitch + i * 32) : 0.0f;
#pragma unroll
          for (int i = 0; i < kP; ++i)
            wv[i] = !in || tile.p0 + (WGRAD ? lane + i * 32 : 0) >= p.p_rows ? 0.0f
                    : WGRAD ? __ldg(ps + static_cast<int64_t>(kb) * p.p_rows + i * 32) : __ldg(ps + kb);
        };
#pragma unroll
        for (int d = 0; d < kAhead; ++d) fetch(d, q[d], w[d]);
        for (int kb = 0; kb < tile.kblocks && ok; kb += kAhead) {
#pragma unroll
          for (int d = 0; d < kAhead; ++d) {
            if (kb + d >= tile.kblocks) break;
            if (!(ok = wait_warp(&s.scale_empty[half][ring.i], ring.phase ^ 1, p.wait_ns))) break;
            float* to = s.scale[half][ring.i];
#pragma unroll
            for (int i = 0; i < kQ; ++i) to[scale_place(lane + i * 32)] = WGRAD ? q[d][i] : q[d][i] * w[d][0];
            if (WGRAD) {
#pragma unroll
              for (int i = 0; i < kP; ++i) to[kHalfCols + lane + i * 32] = w[d][i];
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&s.acc_full[half][ring.i]);
            ring.next();
            fetch(kb + d + kAhead, q[d], w[d]);
          }
        }
      }
    }
  } else {
    // ---- epilogue --------------------------------------------------------
    // Warp w reads tensor-memory lanes 32 (w % 4) .. + 31 of one accumulator, 32
    // columns at a time; the next batch is on its way while one is added.
    tc::reg_inc<kEpilogueRegs>();
    const int ew = warp - 4, quarter = warp % 4, half = ew / 4;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * kHalfCols;
    uint8_t* stage = s.out[ew];
    uint32_t freed = ptx::smem_addr(&s.acc_empty[half][0]);   // the leader's barriers
    if (CTAS == 2) freed = tc::map_to_rank(freed, 0);
    Ring<NBUF> buf;
    for (int t = first_tile; t < tiles && ok; t += step) {
      // Only these three values stay in registers over the k-blocks.
      int n, first, kblocks;
      {
        const Tile tile = T::get(p, s, t, rank);
        n = half == 0 ? tile.n[0] : tile.n[1];
        first = half == 0 ? 0 : tile.n[0];                  // column of the tile the accumulator starts at
        kblocks = n > 0 ? tile.kblocks : 0;
      }
      // acc[c][16 * up + 2 * i + r]: row 16 * up + 8 * r + lane / 4, column 32 * c + 4 * i + lane % 4
      float acc[kBatches][32];
#pragma unroll
      for (int c = 0; c < kBatches; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[c][i] = 0.0f;
      for (int kb = 0; kb < kblocks; ++kb) {
        if (!(ok = wait_warp(&s.acc_full[half][buf.i], buf.phase, p.wait_ns))) break;
        tc::fence_after();
        const float* sc = s.scale[half][buf.i];
        float pw[4];
        if (WGRAD) {
#pragma unroll
          for (int i = 0; i < 4; ++i) pw[i] = sc[kHalfCols + quarter * 32 + 8 * i + lane / 4];
        }
        sc += (lane % 4) * 4;
        const uint32_t from = lane_base + buf.i * MAXN;
        float v[2][32];
        tc::ld_16x32(from, v[0]);
        tc::ld_16x32(from + (16u << 16), v[0] + 16);
#pragma unroll
        for (int c = 0; c < kBatches; ++c) {
          if (c * kBatchCols < n) {
            const float4 lo = *reinterpret_cast<const float4*>(sc + c * kBatchCols);
            const float4 hi = *reinterpret_cast<const float4*>(sc + c * kBatchCols + 16);
            tc::wait_ld();
            if (c + 1 < kBatches && (c + 1) * kBatchCols < n) {
              tc::ld_16x32(from + (c + 1) * kBatchCols, v[(c + 1) % 2]);
              tc::ld_16x32(from + (c + 1) * kBatchCols + (16u << 16), v[(c + 1) % 2] + 16);
            } else {   // everything is in registers: the tensor core may have the buffer back
              tc::fence_before();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive_cluster_relaxed(freed + buf.i * 8);
            }
            const float q[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int up = 0; up < 2; ++up)
#pragma unroll
              for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  float x = v[c % 2][16 * up + 2 * i + r];
                  if (WGRAD) x *= pw[2 * up + r];
                  acc[c][16 * up + 2 * i + r] = fmaf(x, q[i], acc[c][16 * up + 2 * i + r]);
                }
          }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&s.scale_empty[half][buf.i]);
        buf.next();
      }
      if (!ok) break;

      const Tile tile = T::get(p, s, t, rank);
      const int col0 = tile.p0 + quarter * 32;              // the warp's first column of out
      const int64_t row0 = (WGRAD ? static_cast<int64_t>(tile.expert) * p.q_rows : 0) + tile.q0;
#pragma unroll
      for (int c = 0; c < kBatches; ++c) {
        const int col = c * kBatchCols;
        if (col >= n) break;
#pragma unroll
        for (int h = 0; h < 4; ++h) {                       // 8 columns of the accumulator: rows of out
          const int row = first + col + 8 * h;
          if (WGRAD && p.out_fp32) {
            float* out = static_cast<float*>(p.out) + row0 * p.p_rows;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int up = i / 4, r = i % 2, at = row + 4 * (i / 2 % 2) + lane % 4;
              const int oc = col0 + 16 * up + 8 * r + lane / 4;
              if (at < tile.q_valid && oc < p.p_rows) {
                float* o = out + static_cast<int64_t>(at) * p.p_rows + oc;
                const float v = acc[c][16 * up + 4 * h + i % 4];
                *o = p.accumulate ? *o + v : v;
              }
            }
            continue;
          }
          // Lanes j and j ^ 4 hold rows k and k + 1 (k = j/4 even) and the rows 8 further
          // on; they trade so that each has two neighbours: one 32-bit word of out.
          const bool odd = (lane & 4) != 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {                     // up = i / 2, column 4 * (i % 2) + lane % 4
            const float lo = acc[c][16 * (i / 2) + 4 * h + 2 * (i % 2)], hi = acc[c][16 * (i / 2) + 4 * h + 2 * (i % 2) + 1];
            const float other = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 4);
            const __nv_bfloat162 h2 = odd ? __floats2bfloat162_rn(other, hi) : __floats2bfloat162_rn(lo, other);
            *reinterpret_cast<__nv_bfloat162*>(stage + (4 * (i % 2) + lane % 4) * kOutPitch + 32 * (i / 2) +
                                               (odd ? 16 : 0) + lane / 8 * 4) = h2;
          }
          __syncwarp();
          const int r = row + lane / 4, oc = col0 + (lane % 4) * 8;
          const uint4 w = ptx::ld_shared_v4(stage + lane / 4 * kOutPitch + (lane % 4) * 16);
          if (r < tile.q_valid && oc < p.p_rows) ptx::st_v4(static_cast<uint16_t*>(p.out) + (row0 + r) * p.p_rows + oc, w);
          __syncwarp();
        }
      }
      if (!WGRAD && tile.last_q) {
        // gap rows of the segment: zeros, the two warps of the same columns in turn
        const int64_t end = min64(p.expert_offset[tile.expert + 1], p.capacity);
        const int oc = col0 + (lane % 4) * 8;
        if (oc < p.p_rows)
          for (int64_t r = static_cast<int64_t>(tile.q0) + tile.q_valid + half * 8 + lane / 4; r < end; r += 16)
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
  return cudaLaunchKernelEx(&cfg, kernel, maps[0], maps[1], p);
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
  CUtensorMap maps[2];
  cudaError_t e = encode(&maps[0], a.w, a.width_in, a.width_out, a.num_experts, kPRows);
  // Rows an expert has in the mean: many fill the 256 columns of a pair's tile.
  const int64_t mean = a.pairs / a.num_experts;
  const bool pair = mean >= 192;
  p.q_box = pair || mean >= 32 ? 64 : 16;
  if (e == cudaSuccess) e = encode(&maps[1], a.x, a.width_in, a.capacity, 1, p.q_box);
  if (e != cudaSuccess) return e;
  if (pair) return launch<2, 256, false>(maps, p, stream);
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
  CUtensorMap maps[2];
  cudaError_t e = encode(&maps[0], a.x, a.sf_ld, a.width_in, 1, kPRows);
  p.q_box = 64;
  if (e == cudaSuccess) e = encode(&maps[1], a.w, a.sf_ld, a.width_out, 1, p.q_box);
  if (e != cudaSuccess) return e;
  return launch<2, 256, true>(maps, p, stream);
}

}  // namespace moe
