// Matrix product with bias, activation and residual for sm_100a, many rows:
// tcgen05 on CTA pairs (cta_group::2), bf16 operands (kind::f16) or E4M3 rows
// with block scales applied by the tensor core (kind::mxf8f6f4.block_scale).
//
//   out[m][n] = act(sum_k x[m][k] w[n][k] + bias[n]) + residual[m][n]
//
// Tile: 256 rows x BN features per pair of CTAs, each CTA holding 128 rows of x and
// BN / 2 features of w per k-block of 128 bytes; the leader issues M = 256, N = BN
// MMAs, every CTA receives the accumulator of its own 128 rows in its own TMEM, and
// two accumulators take turns, so that one tile's epilogue runs under the next
// tile's products. BN = 256 is for bf16 only (two accumulators fill TMEM); BN = 192
// leaves 128 columns, which hold every stage's scales for E4M3.
//   What bounds it is not the tensor pipe but the operands' way from L2 (without
// loads 4680 x 20480 x 5120 bf16 takes 501 us at 1965 MHz, with them 640, and the
// number of stages changes nothing). So a tile may have two halves of BN = 192
// features that share the row operand (384 wide): 29 % fewer bytes per product,
// but each half has one accumulator. The halves' products are reordered at a
// tile's ends to give the epilogue time; what of it stays exposed, about 3 us per
// tile, pays only for long K: 23400 x 1536 x 6144 E4M3 206 (192) and 194 us (384)
// under the power cap, x 1536 x 1536 bf16 100 (256), 102 (384) and 105 us (192). 512
// wide (two halves of 256) was never the best by more than 2 %. At K = 256 and below
// the epilogue sets the time of every tile: 23400 x 1536 x 256 bf16 with residual 31
// (192) and 36 us (256).
// Tiles are walked in groups of 8 row tiles, feature tiles slowest inside a
// group, so that the tiles in flight cover a near-square patch of the output and
// both operands are re-read from L2.
//   producer warp      TMA producer of its CTA (128-byte swizzled operand boxes,
//                      for E4M3 also the 512-byte scale tiles: one of x, and two
//                      that cover the BN features of w in both CTAs); all bytes
//                      count on the leader's full barrier.
//   MMA warp           leader only: copies the stage's scales into TMEM, then
//                      issues the MMAs; k-steps past K are not issued, so scale
//                      bytes past the last block are never used.
//   Both run as whole warps that elect a lane for each stage: with a branch on the
//   lane number around the loop, the operands of every tcgen05 instruction go
//   through registers, about 140 cycles apiece, and the issue bounds the kernel
//   (4680 x 20480 x 5120 bf16 716 us against 668, 23400 x 1536 x 6144 E4M3 228
//   against 187).
//   the other warps    epilogue: a warpgroup takes 64 (BN = 192) or 128 columns
//                      of the CTA's 128 rows, a thread owns one row and 32
//                      columns at a time. The residual's 32 x 32 box comes in by
//                      TMA one step ahead into the staging buffer that the result
//                      leaves from, so both cross global memory in whole rows; the
//                      bias goes through 32 floats of shared memory per warp.
//                      E4M3 output: the 32 columns are one scale block, so a
//                      thread finds its scale without leaving its registers.
//   Output or residual rows that TMA cannot reach (an odd N, a stride that is not a
//   multiple of 16 bytes) take DIRECT: the staging rows are written and read with
//   a lane per column, 64 bytes of a row at a time, and the residual is loaded in the step
//   that adds it; 23400 x 1535 x 1536 bf16 93-103 us, with residual 114-139, by tile (1536
//   features through TMA: 83-87).
// Every wait is bounded; a timeout is recorded in the row-operator status word.
#include <cuda.h>
#include <cuda_bf16.h>

#include "pipeline.cuh"
#include "rows.cuh"
#include "sm100.cuh"

namespace wf {
namespace {

using namespace sm100;

constexpr uint32_t kBufBytes = 32 * 64;         // 32 rows x 32 bf16 columns
constexpr int kGroup = 8;                       // row tiles per raster group
constexpr int kScaleCols = 384;                 // first TMEM column of the scales
constexpr uint32_t kABytes = 128 * 128;

template <bool MX, int BN, int HALVES>
struct Shape {
  static constexpr uint32_t kHalfBytes = BN / 2 * 128;        // one half's features of w
  static constexpr uint32_t kBBytes = HALVES * kHalfBytes;
  // Scale tiles of 128 rows: one of x, and those that cover HALVES * BN rows of w.
  static constexpr int kScaleTiles = MX ? (HALVES * BN + 127) / 128 : 0;
  static constexpr uint32_t kScaleBytes = MX ? 512 + 512 * kScaleTiles : 0;
  static constexpr uint32_t kStageBytes = kABytes + kBBytes + kScaleBytes;   // per CTA
  static constexpr int kStages = HALVES == 2 ? 4 : 5;
  static constexpr int kBufs = HALVES == 2 ? 2 : 3;           // staging buffers per epilogue warp
  // Epilogue: warpgroups of kCols columns. Three at BN = 192 (registers allow no
  // more at 256, where the accumulator's columns are shared by two).
  static constexpr int kCols = BN == 192 ? 64 : 128;
  static constexpr int kEpiWarps = BN / kCols * 4;
  static constexpr int kProducerWarp = kEpiWarps;
  static constexpr int kMmaWarp = kEpiWarps + 1;
  static constexpr int kThreads = 32 * (kEpiWarps + 2);
  static constexpr int kKElems = MX ? 128 : 64;        // elements of a k-block
  static constexpr int kKStep = MX ? 32 : 16;          // elements per MMA
  // Operands of all stages first (1024-byte aligned for the swizzle), then the
  // scale tiles, the staging buffers, the bias rows and the barriers.
  static constexpr uint32_t kOperandBytes = kABytes + kBBytes;
  static constexpr uint32_t kOffScale = kStages * kOperandBytes;
  static constexpr uint32_t kOffBuf = kOffScale + kStages * kScaleBytes;
  static constexpr uint32_t kOffBias = kOffBuf + kEpiWarps * kBufs * kBufBytes;
  static constexpr uint32_t kOffBar = kOffBias + kEpiWarps * 32 * 4;
  // barriers
  static constexpr int kFull0 = 0;                     // leader: both CTAs' bytes landed
  static constexpr int kEmpty0 = kStages;              // both: stage consumed
  static constexpr int kAccFull0 = 2 * kStages;        // both: accumulator b complete
  static constexpr int kAccEmpty0 = 2 * kStages + 2;   // leader: accumulator b drained by both
  static constexpr int kDrain = 2 * kStages + 4;
  static constexpr int kRes0 = 2 * kStages + 5;        // [warp][buf]: residual box landed
  static constexpr int kNumBars = kRes0 + kEpiWarps * kBufs;
  static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;
  static constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;   // + alignment slack
  static_assert(kOperandBytes % 1024 == 0 && kOffBuf % 512 == 0, "alignment");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
  static_assert(!MX || 2 * BN <= kScaleCols, "TMEM");
  static_assert(HALVES == 1 || 2 * kStages <= kWideMinBlocks, "k-blocks of a wide tile");
  static_assert(!MX || kStages * 4 * (1 + kScaleTiles) <= 512 - kScaleCols, "TMEM");
};

struct PairGrid {
  int m_tiles, n_tiles, total, n_kb, k_steps, out_block_tiles, has_residual;
};

// Tile t: groups of kGroup row tiles; in a group, row tile fastest.
__device__ __forceinline__ void decode(const PairGrid &g, int t, int &mt, int &nt) {
  const int per = kGroup * g.n_tiles;
  const int grp = t / per, r = t - grp * per;
  const int left = g.m_tiles - grp * kGroup;
  const int gm = left < kGroup ? left : kGroup;
  nt = r / gm;
  mt = grp * kGroup + (r - nt * gm);
}

template <bool MX, int BN, int HALVES, bool OUT8, bool DIRECT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Shape<MX, BN, HALVES>::kThreads, 1)
    linear_pair_kernel(const __grid_constant__ LinearParams p, const __grid_constant__ PairGrid g,
                       const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw,
                       const __grid_constant__ CUtensorMap tsx, const __grid_constant__ CUtensorMap tsw,
                       const __grid_constant__ CUtensorMap tr, const __grid_constant__ CUtensorMap to) {
  using S = Shape<MX, BN, HALVES>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::kOffBar);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kOffMisc + 4);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(blockIdx.x >> 1), npairs = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tx);
    tma_prefetch_desc(&tw);
    *abort_flag = 0;
    for (int b = 0; b < S::kNumBars; ++b)
      mbar_init(bars + b, (b == S::kAccEmpty0 || b == S::kAccEmpty0 + 1) ? 2 * S::kEpiWarps : 1);
    fence_barrier_init();
  }
  if (warp == S::kMmaWarp) {                   // same warp in both CTAs, same slot offset
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();                           // barriers of both CTAs initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Ctx ctx{bars, abort_flag, p.status, p.wait_limit};
  grid_wait();
  grid_trigger();

  if (warp == S::kProducerWarp) {
    // ------------------------------------------------------------ producer --
    int q = 0;                              // k-blocks issued by this CTA
    bool ok = true;
    for (int t = pair; ok && t < g.total; t += npairs) {
      int mt, nt;
      decode(g, t, mt, nt);
      const int row0 = mt * 256 + static_cast<int>(rank) * 128;
      const int col0 = nt * (HALVES * BN);
      for (int kb = 0; kb < g.n_kb; ++kb, ++q) {
        const int s = q % S::kStages;
        ok = __all_sync(0xffffffffu, wait_bar(ctx, S::kEmpty0 + s, ((q / S::kStages) & 1) ^ 1));
        if (!ok) break;
        // Test hook: the products stall, since the leader's bytes do not come.
        const bool stall = kb == p.stall_k_block && rank == 0;
        if (!stall && elect_one()) {
          // The leader expects the bytes of both CTAs on its full barrier.
          if (rank == 0) mbar_arrive_expect_tx(bars + S::kFull0 + s, 2 * S::kStageBytes);
          uint8_t *sa = smem + s * S::kOperandBytes;
          const uint32_t lb = leader_bar(bars + S::kFull0 + s);
          tma_load_2d_pair(sa, &tx, lb, kb * S::kKElems, row0);
#pragma unroll
          for (int h = 0; h < HALVES; ++h)
            tma_load_2d_pair(sa + kABytes + h * S::kHalfBytes, &tw, lb, kb * S::kKElems,
                             col0 + h * BN + static_cast<int>(rank) * (BN / 2));
          if constexpr (MX) {
            uint8_t *ss = smem + S::kOffScale + s * S::kScaleBytes;
            tma_load_3d_pair(ss, &tsx, lb, 0, kb, row0 >> 7);
            tma_load_3d_pair(ss + 512, &tsw, lb, 0, kb, col0 >> 7);
          }
        }
        __syncwarp();
      }
    }
    // Tail: every stage this CTA filled has been consumed by the MMAs, so no
    // load of this CTA is in flight when it exits; or they have had time to land.
    for (int s = 0; s < S::kStages && q > 0; ++s) {
      const int fills = q / S::kStages + (s < q % S::kStages ? 1 : 0);
      if (fills > 0) tail_wait(ctx, S::kEmpty0 + s, (fills - 1) & 1);
    }
  } else if (warp == S::kMmaWarp) {
    // ---------------------------------------------------------- MMA issuer --
    if (rank == 0) {
      const uint32_t hi = desc_hi_sw128(1024);
      const uint32_t lo0 = desc_lo_sw128(smem_u32(smem), 16);
      const uint32_t sc0 = smem_u32(smem + S::kOffScale);
      int q = 0, i = 0;                     // k-blocks and accumulators done
      bool ok = true;
      uint32_t shift = 0;
      auto acc_empty = [&](int i) {
        ok = __all_sync(0xffffffffu, wait_bar_cluster(ctx, S::kAccEmpty0 + (i & 1), ((i >> 1) & 1) ^ 1));
        tc_fence_after();
        return ok;
      };
      auto acc_full = [&](int i) {
        if (elect_one()) mma_commit_pair(bars + S::kAccFull0 + (i & 1));
        __syncwarp();
      };
      // Halves [h0, h1) of the products of the k-block at position qq of this CTA's
      // sequence, kb of its tile. `first`: the scales are not in TMEM yet. `last`:
      // the stage is free after it. A half h accumulates in columns BN ((i0 + h) & 1).
      auto block = [&](int qq, int kb, int h0, int h1, int i0, bool first, bool last) {
        const int s = qq % S::kStages;
        if (first) {
          ok = __all_sync(0xffffffffu, wait_bar_cluster(ctx, S::kFull0 + s, (qq / S::kStages) & 1));
          if (!ok) return;
          tc_fence_after();
        }
        const uint32_t a_lo = lo0 + ((s * S::kOperandBytes) >> 4);
        const uint32_t b_lo = a_lo + (kABytes >> 4);
        const int left = g.k_steps - kb * (S::kKElems / S::kKStep);
        if (elect_one()) {
          // A stage's scales have their own columns: the stage is refilled only after its
          // products have completed, and no rule orders a copy behind earlier products.
          const uint32_t sfa = tmem + kScaleCols + 4 * (1 + S::kScaleTiles) * s;
          const uint32_t sfb = sfa + 4;
          if (MX && first) {
            const uint32_t sc = sc0 + s * S::kScaleBytes;
#pragma unroll
            for (int j = 0; j <= S::kScaleTiles; ++j)
              tmem_copy_scales_pair(sfa + 4 * j, make_desc_scale_tile(sc + 512 * j));
          }
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            if (h < h0 || h >= h1) continue;
            const uint32_t d = tmem + BN * ((i0 + h) & 1);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k >= left) continue;
              const uint32_t add = (kb > 0 || k > 0) ? 1u : 0u;
              if constexpr (MX)
                mma_mx_ss2_pair(d, a_lo + k * 2, b_lo + ((h * S::kHalfBytes) >> 4) + k * 2, hi,
                                make_idesc_mx_e4m3(256, BN, k), sfa, sfb + shift + h * (BN / 32), add);
              else
                mma_bf16_ss2_pair(d, a_lo + k * 2, b_lo + ((h * S::kHalfBytes) >> 4) + k * 2, hi,
                                  make_idesc_bf16(256, BN, false), add);
            }
          }
          if (last) mma_commit_pair(bars + S::kEmpty0 + s);
        }
        __syncwarp();
      };
      for (int t = pair; ok && t < g.total; t += npairs) {
        int mt, nt;
        decode(g, t, mt, nt);
        // BN = 192: odd feature tiles start at row 64 of a 128-row scale tile.
        shift = (nt * (HALVES * BN) & 127) >> 5;
        if constexpr (HALVES == 1) {
          if (!acc_empty(i)) break;
          for (int kb = 0; ok && kb < g.n_kb; ++kb, ++q) block(q, kb, 0, 1, i, true, true);
          if (ok) acc_full(i);
          ++i;
        } else {
          // The first k-blocks go through half 0 while the epilogue still drains the
          // last tile's half 1, and the last ones finish half 0 early, so that
          // its epilogue runs under their products of half 1.
          // (The launch sees to n_kb >= 2 kStages.)
          const int head = S::kStages, tail = g.n_kb - S::kStages;
          if (!acc_empty(i)) break;
          for (int kb = 0; ok && kb < head; ++kb) block(q + kb, kb, 0, 1, i, true, false);
          if (!ok || !acc_empty(i + 1)) break;
          for (int kb = 0; kb < head; ++kb) block(q + kb, kb, 1, 2, i, false, true);
          for (int kb = head; ok && kb < tail; ++kb) block(q + kb, kb, 0, 2, i, true, true);
          for (int kb = tail; ok && kb < g.n_kb; ++kb) block(q + kb, kb, 0, 1, i, true, false);
          if (!ok) break;
          acc_full(i);
          for (int kb = tail; kb < g.n_kb; ++kb) block(q + kb, kb, 1, 2, i, false, true);
          acc_full(i + 1);
          q += g.n_kb;
          i += 2;
        }
      }
      // Drain: all MMAs issued by this thread complete before TMEM is freed.
      if (elect_one()) mma_commit_pair(bars + S::kDrain);
      __syncwarp();
      drain_wait(ctx, S::kDrain, 0);
    }
  } else {
    // ------------------------------------------------------------ epilogue --
    constexpr int kSteps = S::kCols / 32;                // 32-column steps of a warpgroup
    const int e = warp >> 2;                             // warpgroup: kCols columns of the tile
    const int wr = (warp & 3) * 32;                      // first row of this warp
    const uint32_t lane_addr = static_cast<uint32_t>(wr) << 16;
    uint8_t *bufs = smem + S::kOffBuf + warp * S::kBufs * kBufBytes;
    float *bias_row = reinterpret_cast<float *>(smem + S::kOffBias) + warp * 32;
    const int res_bar = S::kRes0 + warp * S::kBufs;
    uint32_t res_phase = 0;                              // bit per buffer
    uint32_t res_pending = 0;                            // lane 0: boxes in flight
    // This warp's first row and column; past the last tile: outside out.
    auto place = [&](int i, int &row, int &col) {        // of the i-th accumulator
      const int64_t t = pair + static_cast<int64_t>(i / HALVES) * npairs;
      int mt = 0, nt = 0;
      if (t < g.total) decode(g, static_cast<int>(t), mt, nt);
      row = t < g.total ? mt * 256 + static_cast<int>(rank) * 128 + wr : p.M;
      col = (nt * HALVES + i % HALVES) * BN + e * S::kCols;
    };
    auto fetch = [&](int row, int col, int buf) {        // lane 0: residual box of a step
      if (row < p.M && col < p.N) {
        res_pending |= 1u << buf;
        mbar_arrive_expect_tx(bars + res_bar + buf, kBufBytes);
        tma_load_2d(bufs + buf * kBufBytes, &tr, bars + res_bar + buf, col, row);
      }
    };
    auto bias_at = [&](int col) {                        // this lane's column of a step
      return p.bias && col + lane < p.N ? __ldg(p.bias + col + lane) : 0.f;
    };
    int buf = 0;
    int row0, tile_col, row1, tile_col1;                 // this tile's and the next one's place
    place(0, row1, tile_col1);
    if (!DIRECT && g.has_residual && lane == 0) fetch(row1, tile_col1, 0);
    float bias = bias_at(tile_col1);
    bool ok = true;
    const int tiles = (g.total - pair + npairs - 1) / npairs;
    for (int i = 0; ok && i < HALVES * tiles; ++i) {
      const int b = i & 1;
      row0 = row1;
      tile_col = tile_col1;
      place(i + 1, row1, tile_col1);
      ok = __all_sync(0xffffffffu, wait_bar_cluster(ctx, S::kAccFull0 + b, (i >> 1) & 1));
      if (!ok) break;
      tc_fence_after();
      const uint32_t tcol = tmem + lane_addr + BN * b + e * S::kCols;
      uint32_t cur[32], nxt[32];
      tmem_ld32(tcol, cur);
      tmem_ld_wait();
      reg_fence32(cur);
#pragma unroll
      for (int c = 0; c < kSteps; ++c) {
        if (c + 1 < kSteps) tmem_ld32(tcol + (c + 1) * 32, nxt);
        const int col0 = tile_col + c * 32;
        const bool on = row0 < p.M && col0 < p.N;
        const bool same = c + 1 < kSteps;                // the next step is of this tile
        const int next_row = same ? row0 : row1, next_col = same ? col0 + 32 : tile_col1;
        const int buf1 = buf + 1 == S::kBufs ? 0 : buf + 1;
        // Stores of buf (kBufs steps ago) and buf1 (one step fewer) have been read.
        if (!DIRECT && lane == 0) {
          asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(S::kBufs - 2) : "memory");
          if (g.has_residual) fetch(next_row, next_col, buf1);
        }
        bias_row[lane] = bias;
        bias = bias_at(next_col);
        // DIRECT: the residual's box, lane = column, all rows in flight at once; places
        // outside are clamped into it.
        uint16_t res_rows[DIRECT ? 32 : 1];
        if constexpr (DIRECT) {
          if (g.has_residual && on) {
            const int col = col0 + lane < p.N ? col0 + lane : p.N - 1;
            const uint16_t *r = static_cast<const uint16_t *>(p.residual.data) + col;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              res_rows[j] = r[static_cast<int64_t>(row0 + j < p.M ? row0 + j : p.M - 1) * p.residual.ld];
          }
        }
        __syncwarp();
        if (on) {
          float v[32];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 f = reinterpret_cast<const float4 *>(bias_row)[j];
            v[4 * j] = __uint_as_float(cur[4 * j]) + f.x;
            v[4 * j + 1] = __uint_as_float(cur[4 * j + 1]) + f.y;
            v[4 * j + 2] = __uint_as_float(cur[4 * j + 2]) + f.z;
            v[4 * j + 3] = __uint_as_float(cur[4 * j + 3]) + f.w;
          }
          if (p.act == kGelu) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = activate(v[j], kGelu);
          } else if (p.act == kSilu) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = activate(v[j], kSilu);
          }
          // Staging rows of 64 bytes, 64-byte swizzle: 16-byte chunk j of row r at
          // j ^ (r / 2 % 4).
          const uint32_t addr = smem_u32(bufs + buf * kBufBytes + lane * 64);
          const uint32_t x = (lane >> 1) & 3;
          auto staged = [&](int r, int c) {               // bf16 column c of row r
            return bufs + buf * kBufBytes + r * 64 + (((c >> 3) ^ ((r >> 1) & 3)) << 4) + (c & 7) * 2;
          };
          if constexpr (OUT8) {
            // The warpgroup's 64 columns share a staging row: two scale blocks.
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j) m = fmaxf(m, fabsf(v[j]));
            const int ex = block_exponent(m);
            const float f = block_factor(ex);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                const float *u = v + 16 * j + 4 * h;
                w[h] = pack_e4m3x4(u[0] * f, u[1] * f, u[2] * f, u[3] * f);
              }
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr + (((2 * c + j) ^ x) << 4)),
                           "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                           : "memory");
            }
            if (row0 + lane < p.M)
              p.out.scales[scale_offset(row0 + lane, col0 >> 5, g.out_block_tiles)] =
                  static_cast<uint8_t>(ex + 127);
          } else {
            if (g.has_residual) {
              if constexpr (DIRECT) {
                // The staging rows turn the residual's columns around.
#pragma unroll
                for (int j = 0; j < 32; ++j) *reinterpret_cast<uint16_t *>(staged(j, lane)) = res_rows[j];
                __syncwarp();
              } else {
                ok = __all_sync(0xffffffffu, wait_bar(ctx, res_bar + buf, (res_phase >> buf) & 1));
                if (!ok) break;
                res_phase ^= 1u << buf;
                res_pending &= ~(1u << buf);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t w[4];
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                             : "r"(addr + ((j ^ x) << 4)));
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                  v[8 * j + 2 * h] += __uint_as_float(w[h] << 16);
                  v[8 * j + 2 * h + 1] += __uint_as_float(w[h] & 0xffff0000u);
                }
              }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                const __nv_bfloat162 two = __floats2bfloat162_rn(v[8 * j + 2 * h], v[8 * j + 2 * h + 1]);
                w[h] = *reinterpret_cast<const uint32_t *>(&two);
              }
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr + ((j ^ x) << 4)),
                           "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                           : "memory");
            }
          }
          if constexpr (DIRECT) {
            __syncwarp();
            uint16_t *o = static_cast<uint16_t *>(p.out.data) + static_cast<int64_t>(row0) * p.out.ld + col0 + lane;
#pragma unroll 8
            for (int j = 0; j < 32; ++j)
              if (row0 + j < p.M && col0 + lane < p.N)
                o[j * p.out.ld] = *reinterpret_cast<const uint16_t *>(staged(j, lane));
          } else {
            fence_proxy_async_smem();
          }
        }
        __syncwarp();
        if constexpr (DIRECT) {
          // The one staging buffer is free again.
        } else if constexpr (OUT8) {
          // One store for both steps; columns past N are clipped.
          if (c + 1 == kSteps) {
            if (lane == 0) {
              if (row0 < p.M && tile_col < p.N) tma_store_2d(&to, bufs + buf * kBufBytes, tile_col, row0);
              tma_store_commit();
            }
            buf = buf1;
          }
        } else {
          if (lane == 0) {
            if (on) tma_store_2d(&to, bufs + buf * kBufBytes, col0, row0);
            tma_store_commit();                          // a group per step, empty or not
          }
          buf = buf1;
        }
        if (c + 1 < kSteps) {
          tmem_ld_wait();
          reg_fence32(nxt);
#pragma unroll
          for (int j = 0; j < 32; ++j) cur[j] = nxt[j];
        }
        if (c + 2 == kSteps) {
          // Last TMEM load of this accumulator done: release it to the leader.
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(bars + S::kAccEmpty0 + b, 0);
        }
      }
    }
    if (lane == 0) {
      // A fetch that no step took (another role gave up) must land before exit.
      for (int k = 0; k < S::kBufs; ++k)
        if (res_pending >> k & 1) drain_wait(ctx, res_bar + k, (res_phase >> k) & 1);
      tma_store_wait_all();
    }
    __syncwarp();
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync();                           // no MMA or load of the pair is in flight
  if (warp == S::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <bool MX, int BN, int HALVES, bool OUT8, bool DIRECT>
cudaError_t run_pair(const LinearParams &p, cudaStream_t st) {
  using S = Shape<MX, BN, HALVES>;
  const int elt = MX ? 1 : 2;
  CUtensorMap tx{}, tw{}, tsx{}, tsw{}, tr{}, to{};
  const uint64_t K = static_cast<uint64_t>(p.K), M = static_cast<uint64_t>(p.M), N = static_cast<uint64_t>(p.N);
  const uint64_t xd[2] = {K, M}, wd[2] = {K, N}, od[2] = {N, M};
  const uint64_t xs[1] = {static_cast<uint64_t>(p.x.ld) * elt}, ws[1] = {static_cast<uint64_t>(p.w.ld) * elt};
  const uint32_t xb[2] = {S::kKElems, 128}, wb[2] = {S::kKElems, BN / 2}, ob[2] = {OUT8 ? 64 : 32, 32};
  bool ok = encode_rows_map(&tx, elt, 128, p.x.data, 2, xd, xs, xb) &&
            encode_rows_map(&tw, elt, 128, p.w.data, 2, wd, ws, wb);
  if (MX) {
    // Scale tiles as rows of 128 words: [row tiles][block tiles][128].
    const uint64_t kt = (K + 127) / 128;
    const uint64_t sd[3] = {128, kt, (M + 127) / 128}, qd[3] = {128, kt, (N + 127) / 128};
    const uint64_t ss[2] = {512, 512 * kt};
    const uint32_t sb[3] = {128, 1, 1}, qb[3] = {128, 1, S::kScaleTiles};
    ok = ok && encode_rows_map(&tsx, 4, 0, p.x.scales, 3, sd, ss, sb) &&
         encode_rows_map(&tsw, 4, 0, p.w.scales, 3, qd, ss, qb);
  }
  if (!DIRECT) {
    const int oelt = OUT8 ? 1 : 2;
    const uint64_t os[1] = {static_cast<uint64_t>(p.out.ld) * oelt};
    ok = ok && encode_rows_map(&to, oelt, 64, p.out.data, 2, od, os, ob);
    if (p.residual.data) {
      const uint64_t rs[1] = {static_cast<uint64_t>(p.residual.ld) * 2};
      ok = ok && encode_rows_map(&tr, 2, 64, p.residual.data, 2, od, rs, ob);
    }
  }
  if (!ok) return cudaErrorInvalidValue;
  PairGrid g{};
  const int64_t mt = (static_cast<int64_t>(p.M) + 255) / 256, nt = (static_cast<int64_t>(p.N) + HALVES * BN - 1) / (HALVES * BN);
  if (mt * nt > 0x7fffffff - 65536) return cudaErrorInvalidValue;
  g.m_tiles = static_cast<int>(mt);
  g.n_tiles = static_cast<int>(nt);
  g.total = static_cast<int>(mt * nt);
  g.n_kb = (p.K + S::kKElems - 1) / S::kKElems;
  g.k_steps = (p.K + S::kKStep - 1) / S::kKStep;
  g.out_block_tiles = (p.N + 127) / 128;
  g.has_residual = p.residual.data != nullptr;
  if (HALVES == 2 && g.n_kb < kWideMinBlocks) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> allowed;
  const cudaError_t e = allow_shared(linear_pair_kernel<MX, BN, HALVES, OUT8, DIRECT>, allowed, p.device, S::kSmemBytes);
  if (e != cudaSuccess) return e;
  const int pairs = g.total < p.sms / 2 ? g.total : p.sms / 2;
  return launch_dependent(linear_pair_kernel<MX, BN, HALVES, OUT8, DIRECT>, 2 * pairs, S::kThreads, S::kSmemBytes, 0, st,
                          p, g, tx, tw, tsx, tsw, tr, to);
}

}  // namespace

cudaError_t launch_linear_pair(const LinearParams &p, bool e4m3, bool out_e4m3, bool direct, int bn,
                               cudaStream_t st) {
  if (out_e4m3) {
    if (e4m3) return bn == 384 ? run_pair<true, 192, 2, true, false>(p, st) : run_pair<true, 192, 1, true, false>(p, st);
    return bn == 384 ? run_pair<false, 192, 2, true, false>(p, st) : run_pair<false, 192, 1, true, false>(p, st);
  }
  if (direct) {
    if (e4m3) return bn == 384 ? run_pair<true, 192, 2, false, true>(p, st) : run_pair<true, 192, 1, false, true>(p, st);
    return bn == 384   ? run_pair<false, 192, 2, false, true>(p, st)
           : bn == 256 ? run_pair<false, 256, 1, false, true>(p, st)
                       : run_pair<false, 192, 1, false, true>(p, st);
  }
  if (e4m3) return bn == 384 ? run_pair<true, 192, 2, false, false>(p, st) : run_pair<true, 192, 1, false, false>(p, st);
  return bn == 384   ? run_pair<false, 192, 2, false, false>(p, st)
         : bn == 256 ? run_pair<false, 256, 1, false, false>(p, st)
                     : run_pair<false, 192, 1, false, false>(p, st);
}

}  // namespace wf
