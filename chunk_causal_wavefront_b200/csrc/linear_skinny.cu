// Matrix product with bias, activation and residual for sm_100a, few rows: features
// on the M side.
//
// The bytes of w bound it: with few rows every weight is used only a few times.
// So w streams through the tensor core as the A operand, 128 features per tile,
// and the rows of x (tokens) are the N side, NT = 16 ... 128 of them per tile:
// D[feature][token] in TMEM, NT columns. To have every SM stream, K is split over
// a cluster of S = 1 ... 8 CTAs: each CTA sums its share of the k-blocks, sends the
// token slice that rank j finishes into rank j's shared memory, and rank j adds
// the S partial sums in rank order (no atomics, no workspace, one launch, and
// the same result on every run).
//   A thread owns one feature (TMEM lane), so a warp stores 32 neighbouring
//   features of a token at once with plain stores: any N, any row stride. The 32
//   features are one E4M3 scale block, whose largest magnitude is one warp
//   reduction.
//   warp 0: TMA producer; warp 1: scale copies and MMAs (whole warps that elect a
//   lane for each stage); then all four warps: partial sums and epilogue, up to
//   eight tokens at a time, their residual fetched before.
//   Two CTAs share an SM up to 64 tokens. Each holds 81 KB of shared memory or
//   more, so no CTA of another clustered kernel (all hold over 200 KB) fits beside
//   it: two clusters never wait for each other's tensor memory.
//   Measured (captured graph or burst, weights in HBM): 1 x 6144 x 1536 bf16 6.5-7.0 us
//   (18.9 MB; the weights alone 2.9 us at 6.55 TB/s, the rest is the latency of launch,
//   first loads, cluster barriers and last stores), 24 x 5120 x 5120 E4M3 9.0-9.4 us, 64 x
//   1536 x 1536 bf16 5.3-5.9 us, 1111 x 1000 x 1544 13.3-14.2 us (against 14.6-16 on CTA pairs).
// Every wait is bounded; a timeout is recorded in the row-operator status word.
#include <cuda.h>
#include <cuda_bf16.h>

#include "pipeline.cuh"
#include "rows.cuh"
#include "sm100.cuh"

namespace wf {
namespace {

using namespace sm100;

constexpr int kThreads = 128;
constexpr uint32_t kABytes = 128 * 128;         // 128 features x 128 bytes of K

template <bool MX, int NT>
struct Shape {
  static constexpr uint32_t kBBytes = NT * 128;
  static constexpr uint32_t kOperandBytes = kABytes + kBBytes;
  static constexpr uint32_t kScaleBytes = MX ? 1024 : 0;   // 512 of w, 512 of x
  static constexpr uint32_t kStageBytes = kOperandBytes + kScaleBytes;
  static constexpr int kStages = NT == 64 ? 3 : 4;         // NT < 128: two CTAs fit an SM
  static constexpr int kKElems = MX ? 128 : 64;
  static constexpr int kKStep = MX ? 32 : 16;
  static constexpr uint32_t kOffScale = kStages * kOperandBytes;
  static constexpr uint32_t kOffPart = kOffScale + kStages * kScaleBytes;   // [rank][token][feature]
  static constexpr uint32_t kOffBar = kOffPart + NT * 128 * 4;
  static constexpr int kFull0 = 0, kEmpty0 = kStages, kAcc = 2 * kStages, kNumBars = 2 * kStages + 1;
  static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;
  static constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;   // + alignment slack
  // D, then every stage's scales (4 columns of w, 4 of x each).
  static constexpr uint32_t kTmemCols = !MX ? (NT < 32 ? 32 : NT) : (NT <= 32 ? 64 : 2 * NT);
  static_assert(kOperandBytes % 1024 == 0, "alignment");
  static_assert(!MX || NT + 8 * kStages <= static_cast<int>(kTmemCols), "TMEM");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

struct SkinnyGrid {
  int t_tiles, n_kb, k_steps, out_block_tiles;
};

template <bool MX, int NT, int SPLIT, bool OUT8>
__global__ void __launch_bounds__(kThreads)
    linear_skinny_kernel(const __grid_constant__ LinearParams p, const __grid_constant__ SkinnyGrid g,
                         const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw,
                         const __grid_constant__ CUtensorMap tsx,
                         const __grid_constant__ CUtensorMap tsw) {
  using S = Shape<MX, NT>;
  constexpr int kPer = NT / SPLIT;               // tokens that a CTA finishes
  constexpr int kG = kPer < 8 ? kPer : 8;        // of them at a time
  constexpr int kHold = kPer < 64 ? kPer : 64;   // residuals held ahead
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::kOffBar);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kOffMisc + 4);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = SPLIT > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  // Token tiles fastest: the CTAs that share a weight tile run side by side.
  const int tile = static_cast<int>(blockIdx.x) / SPLIT;
  const int ft = tile / g.t_tiles, tt = tile - ft * g.t_tiles;
  const int f0 = ft * 128, t0 = tt * NT;
  const int kb0 = static_cast<int>(static_cast<int64_t>(g.n_kb) * rank / SPLIT);
  const int kb1 = static_cast<int>(static_cast<int64_t>(g.n_kb) * (rank + 1) / SPLIT);

  // The producer warp initialises the barriers and fills the empty ring before
  // anyone else is ready, so the first bytes are under way during the set-up.
  auto load = [&](int kb, int s) {
    uint64_t *full = bars + S::kFull0 + s;
    mbar_arrive_expect_tx(full, S::kStageBytes);
    uint8_t *sa = smem + s * S::kOperandBytes;
    tma_load_2d(sa, &tw, full, kb * S::kKElems, f0);
    tma_load_2d(sa + kABytes, &tx, full, kb * S::kKElems, t0);
    if constexpr (MX) {
      uint8_t *ss = smem + S::kOffScale + s * S::kScaleBytes;
      tma_load_3d(ss, &tsw, full, 0, kb, ft);
      tma_load_3d(ss + 512, &tsx, full, 0, kb, t0 >> 7);
    }
  };
  const int filled = kb1 - kb0 < S::kStages ? kb1 - kb0 : S::kStages;
  if (warp == 0) {
    if (elect_one()) {
      *abort_flag = 0;
      for (int b = 0; b < S::kNumBars; ++b) mbar_init(bars + b, 1);
      fence_barrier_init();
    }
    grid_wait();
    if (elect_one())
      for (int s = 0; s < filled; ++s) load(kb0 + s, s);
    __syncwarp();
  } else if (warp == 1) {
    tmem_alloc(tmem_slot, S::kTmemCols);
    tmem_relinquish();
  }
  if constexpr (SPLIT > 1) cluster_arrive_relaxed();   // waited for before the first remote store
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Ctx ctx{bars, abort_flag, p.status, p.wait_limit};
  grid_wait();
  grid_trigger();

  // This thread's feature and this CTA's tokens. The residual is fetched while the
  // products run (64 tokens of it at most); addresses past the end are clamped
  // into the operand, so no load waits on a branch.
  const int f = f0 + static_cast<int>(threadIdx.x);
  const bool f_on = f < p.N;
  const int fc = f_on ? f : p.N - 1;
  const int first = t0 + rank * kPer;
  const int end = p.M - first < kPer ? p.M : first + kPer;
  const uint16_t *res = OUT8 ? nullptr : static_cast<const uint16_t *>(p.residual.data);
  uint16_t held[kHold];
  auto fetch = [&](int tok) {
#pragma unroll
    for (int j = 0; j < kHold; ++j) {
      const int t = tok + j < p.M ? tok + j : p.M - 1;
      held[j] = res[static_cast<int64_t>(t) * p.residual.ld + fc];
    }
  };
#pragma unroll
  for (int j = 0; j < kHold; ++j) held[j] = 0;
  if (res) fetch(first);
  const float bias = p.bias ? __ldg(p.bias + fc) : 0.f;

  if (warp == 0) {
    // ------------------------------------------------------------ producer --
    int q = filled;
    for (int kb = kb0 + q; kb < kb1; ++kb, ++q) {
      const int s = q % S::kStages;
      if (!__all_sync(0xffffffffu, wait_bar(ctx, S::kEmpty0 + s, ((q / S::kStages) & 1) ^ 1))) break;
      if (elect_one()) load(kb, s);
      __syncwarp();
    }
    // Tail: every filled stage has been consumed, so no load is in flight when
    // the CTA exits; or its loads have had time to land.
    for (int s = 0; s < S::kStages; ++s) {
      const int fills = q / S::kStages + (s < q % S::kStages ? 1 : 0);
      if (fills > 0) tail_wait(ctx, S::kEmpty0 + s, (fills - 1) & 1);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer --
    const uint32_t hi = desc_hi_sw128(1024);
    const uint32_t lo0 = desc_lo_sw128(smem_u32(smem), 16);
    const uint32_t sc0 = smem_u32(smem + S::kOffScale);
    // Tokens 32 j .. of a 128-row scale tile are its columns j ..
    const uint32_t shift = (t0 & 127) >> 5;
    int q = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++q) {
      const int s = q % S::kStages;
      const bool stall = kb == p.stall_k_block;       // test hook: kAcc is not complete before the end
      if (!__all_sync(0xffffffffu, wait_bar(ctx, stall ? S::kAcc : S::kFull0 + s, stall ? 0 : (q / S::kStages) & 1))) break;
      tc_fence_after();
      const uint32_t a_lo = lo0 + ((s * S::kOperandBytes) >> 4);
      const uint32_t b_lo = a_lo + (kABytes >> 4);
      const int left = g.k_steps - kb * (S::kKElems / S::kKStep);
      if (elect_one()) {
        if constexpr (MX) {
          const uint32_t sc = sc0 + s * S::kScaleBytes;
          const uint32_t sfa = tmem + NT + 8 * s;         // a stage's own columns
          const uint32_t sfb = sfa + 4;
          tmem_copy_scales(sfa, make_desc_scale_tile(sc));
          tmem_copy_scales(sfb, make_desc_scale_tile(sc + 512));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < left)
              mma_mx_ss2(tmem, a_lo + k * 2, b_lo + k * 2, hi, make_idesc_mx_e4m3(128, NT, k), sfa,
                         sfb + shift, (q > 0 || k > 0) ? 1u : 0u);
        } else {
          constexpr uint32_t idesc = make_idesc_bf16(128, NT, false);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < left)
              mma_bf16_ss2(tmem, a_lo + k * 2, b_lo + k * 2, hi, idesc, (q > 0 || k > 0) ? 1u : 0u);
        }
        mma_commit(bars + S::kEmpty0 + s);
      }
      __syncwarp();
    }
    if (elect_one()) mma_commit(bars + S::kAcc);
    __syncwarp();
  }

  // -------------------------------------------------- partial sums, epilogue --
  // The commit follows every MMA that was issued, also after a timeout, so the
  // wait ends; an aborted CTA goes through the cluster barriers all the same.
  const bool done = drain_wait(ctx, S::kAcc, 0);
  tc_fence_after();
  const bool ok = __syncthreads_and(done && !*abort_flag);
  const uint32_t tcol = tmem + (static_cast<uint32_t>(warp * 32) << 16);

  if constexpr (SPLIT > 1) {
    // Send every rank the slice that it finishes: [rank][token][feature]. All
    // CTAs of the cluster run by now (the barrier that they arrived at first).
    cluster_wait();
    const uint32_t mine = smem_u32(smem + S::kOffPart) + rank * kPer * 512 + threadIdx.x * 4;
#pragma unroll 1
    for (int c = 0; c < NT && t0 + c < p.M; c += 8) {
      uint32_t d[8];
      tmem_ld8(tcol + c, d);
      tmem_ld_wait();
      WF_REG_FENCE8(d, 0);
#pragma unroll
      for (int h = 0; h < 8; h += kG) {                // kG tokens for one rank
        const uint32_t to = map_shared(mine + (c + h) % kPer * 512, static_cast<uint32_t>((c + h) / kPer));
        if (t0 + c + h < p.M)
#pragma unroll
          for (int j = 0; j < kG; ++j) store_cluster_f32(to + j * 512, __uint_as_float(d[h + j]));
      }
    }
    cluster_sync();
  }
  const float *part = reinterpret_cast<const float *>(smem + S::kOffPart) + threadIdx.x;
#pragma unroll 1
  for (int base = 0; base < kPer; base += kHold) {
    if (base > 0 && res) fetch(first + base);
#pragma unroll
    for (int h = 0; h < kHold; h += kG) {
      const int c = base + h;
      if (first + c >= end || !ok) break;
      float v[kG];
      if constexpr (SPLIT == 1) {
        uint32_t d[8];
        tmem_ld8(tcol + c, d);
        tmem_ld_wait();
        WF_REG_FENCE8(d, 0);
#pragma unroll
        for (int j = 0; j < kG; ++j) v[j] = __uint_as_float(d[j]) + bias;
      } else {
#pragma unroll
        for (int j = 0; j < kG; ++j) v[j] = part[(c + j) * 128];
#pragma unroll
        for (int r = 1; r < SPLIT; ++r)
#pragma unroll
          for (int j = 0; j < kG; ++j) v[j] += part[(r * kPer + c + j) * 128];
#pragma unroll
        for (int j = 0; j < kG; ++j) v[j] += bias;
      }
      if (p.act == kGelu) {
#pragma unroll
        for (int j = 0; j < kG; ++j) v[j] = activate(v[j], kGelu);
      } else if (p.act == kSilu) {
#pragma unroll
        for (int j = 0; j < kG; ++j) v[j] = activate(v[j], kSilu);
      }
      if constexpr (!OUT8) {
        if (res) {
#pragma unroll
          for (int j = 0; j < kG; ++j) v[j] += __uint_as_float(static_cast<uint32_t>(held[h + j]) << 16);
        }
      }
#pragma unroll
      for (int j = 0; j < kG; ++j) {
        const int tok = first + c + j;
        if constexpr (OUT8) {
          // N is a multiple of 32: a warp's features are all inside or all outside.
          const float a = fabsf(v[j]);
          const uint32_t m = __reduce_max_sync(0xffffffffu, a == a ? __float_as_uint(a) : 0u);
          const int ex = block_exponent(__uint_as_float(m));
          if (f_on && tok < end) {
            static_cast<uint8_t *>(p.out.data)[static_cast<int64_t>(tok) * p.out.ld + f] =
                static_cast<uint8_t>(pack_e4m3x2(v[j] * block_factor(ex), 0.f) & 0xffu);
            if (lane == 0)
              p.out.scales[scale_offset(tok, f >> 5, g.out_block_tiles)] = static_cast<uint8_t>(ex + 127);
          }
        } else if (f_on && tok < end) {
          static_cast<__nv_bfloat16 *>(p.out.data)[static_cast<int64_t>(tok) * p.out.ld + f] =
              __float2bfloat16_rn(v[j]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

template <bool MX, int NT, int SPLIT, bool OUT8>
cudaError_t run_skinny(const LinearParams &p, cudaStream_t st) {
  using S = Shape<MX, NT>;
  const int elt = MX ? 1 : 2;
  CUtensorMap tx{}, tw{}, tsx{}, tsw{};
  const uint64_t K = static_cast<uint64_t>(p.K), M = static_cast<uint64_t>(p.M), N = static_cast<uint64_t>(p.N);
  const uint64_t xd[2] = {K, M}, wd[2] = {K, N};
  const uint64_t xs[1] = {static_cast<uint64_t>(p.x.ld) * elt}, ws[1] = {static_cast<uint64_t>(p.w.ld) * elt};
  const uint32_t xb[2] = {S::kKElems, NT}, wb[2] = {S::kKElems, 128};
  bool ok = encode_rows_map(&tx, elt, 128, p.x.data, 2, xd, xs, xb) &&
            encode_rows_map(&tw, elt, 128, p.w.data, 2, wd, ws, wb);
  if (MX) {
    const uint64_t kt = (K + 127) / 128;
    const uint64_t sd[3] = {128, kt, (M + 127) / 128}, qd[3] = {128, kt, (N + 127) / 128};
    const uint64_t ss[2] = {512, 512 * kt};
    const uint32_t sb[3] = {128, 1, 1};
    ok = ok && encode_rows_map(&tsx, 4, 0, p.x.scales, 3, sd, ss, sb) &&
         encode_rows_map(&tsw, 4, 0, p.w.scales, 3, qd, ss, sb);
  }
  if (!ok) return cudaErrorInvalidValue;
  // A token tile's scales start at a 32-row column of a scale tile, and the scale
  // operand's TMEM column has to be even.
  if (MX && NT < 64 && p.M > NT) return cudaErrorInvalidValue;
  SkinnyGrid g{};
  const int64_t ft = (static_cast<int64_t>(p.N) + 127) / 128, tt = (static_cast<int64_t>(p.M) + NT - 1) / NT;
  if (ft * tt * SPLIT > 0x7fffffff) return cudaErrorInvalidValue;
  g.t_tiles = static_cast<int>(tt);
  g.n_kb = (p.K + S::kKElems - 1) / S::kKElems;
  g.k_steps = (p.K + S::kKStep - 1) / S::kKStep;
  g.out_block_tiles = (p.N + 127) / 128;
  static std::atomic<uint64_t> allowed;
  const cudaError_t e = allow_shared(linear_skinny_kernel<MX, NT, SPLIT, OUT8>, allowed, p.device, S::kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(linear_skinny_kernel<MX, NT, SPLIT, OUT8>, static_cast<unsigned>(ft * tt * SPLIT), kThreads,
                          S::kSmemBytes, SPLIT, st, p, g, tx, tw, tsx, tsw);
}

template <bool MX, int NT, bool OUT8>
cudaError_t pick_split(const LinearParams &p, int split, cudaStream_t st) {
  switch (split) {
    case 8: return run_skinny<MX, NT, 8, OUT8>(p, st);
    case 4: return run_skinny<MX, NT, 4, OUT8>(p, st);
    case 2: return run_skinny<MX, NT, 2, OUT8>(p, st);
    default: return run_skinny<MX, NT, 1, OUT8>(p, st);
  }
}

template <bool MX, bool OUT8>
cudaError_t pick_skinny(const LinearParams &p, int nt, int split, cudaStream_t st) {
  switch (nt) {
    case 16: return pick_split<MX, 16, OUT8>(p, split, st);
    case 32: return pick_split<MX, 32, OUT8>(p, split, st);
    case 64: return pick_split<MX, 64, OUT8>(p, split, st);
    default: return pick_split<MX, 128, OUT8>(p, split, st);
  }
}

}  // namespace

cudaError_t launch_linear_skinny(const LinearParams &p, bool e4m3, bool out_e4m3, int nt, int split,
                                 cudaStream_t st) {
  if (e4m3) return out_e4m3 ? pick_skinny<true, true>(p, nt, split, st) : pick_skinny<true, false>(p, nt, split, st);
  return out_e4m3 ? pick_skinny<false, true>(p, nt, split, st) : pick_skinny<false, false>(p, nt, split, st);
}

}  // namespace wf
