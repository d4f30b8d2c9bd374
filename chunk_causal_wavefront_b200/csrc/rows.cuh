// Shared by the row operators (norm, E4M3 rows, linear): E4M3 block scales and
// their tiled layout, and the parameters of the launches.
//
// E4M3 rows hold one byte e + 127 per row and block of 32 columns, e the
// smallest integer >= -100 with amax * 2^-e <= 448: the same rule as the E4M3
// pools, on the block size and scale type of the block-scaled tensor-core
// products, so the scales never touch the CUDA cores again.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include <utility>

#include "wf.h"

namespace wf {

// One operand or result, as the kernels see it.
struct RowsView {
  void *data;
  uint8_t *scales;
  int64_t ld;
};

struct NormParams {
  RowsView x, residual, sum, out;   // residual.data / sum.data null if absent
  const float *weight;              // null: ones
  float eps;
  int32_t rows, cols;
};

struct ConvertParams {
  RowsView x, out;
  int32_t rows, cols;
};

struct LinearParams {
  RowsView x, w, residual, out;     // residual.data null if absent
  const float *bias;                // null: zeros
  int32_t act;
  int32_t M, N, K;
  int32_t *status;                  // the device's row-operator status word
  int32_t device, sms;
  // Test hook (wf_rows_debug_next_linear): the k-block at which the products stall (-1: none), and
  // the cycles after which a wait gives up.
  int32_t stall_k_block;
  long long wait_limit;
};

// A launch that may start while the one before it in the stream is leaving (its
// kernel calls grid_wait before it touches global memory), in clusters of `cluster`
// blocks (0: the kernel's own, or none). Calls back to back: 1 x 6144 x 1536 linear
// 6.5 -> 5.3 us, 23400 x 1536 norm 51.4 -> 49.8 us.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), unsigned grid, unsigned threads, uint32_t shared,
                             unsigned cluster, cudaStream_t st, A &&...args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = st;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

enum class RowsType { kBf16, kF32, kE4m3 };

cudaError_t launch_add_rms_norm(const NormParams &p, RowsType in, bool out_e4m3, cudaStream_t st);
cudaError_t launch_quantize_rows(const ConvertParams &p, RowsType in, cudaStream_t st);
cudaError_t launch_dequantize_rows(const ConvertParams &p, RowsType out, cudaStream_t st);
// Large products, on CTA pairs. bn: 192, 256 (bf16 to bf16 only) or 384 features per
// tile, the last for at least kWideMinBlocks k-blocks of 128 bytes. direct: bf16
// output or residual rows are not 16-byte aligned.
constexpr int kWideMinBlocks = 8;
cudaError_t launch_linear_pair(const LinearParams &p, bool e4m3, bool out_e4m3, bool direct, int bn,
                               cudaStream_t st);
// Few rows: features on the MMA's M side, K split
// over a cluster of `split` CTAs, `nt` tokens per tile.
cudaError_t launch_linear_skinny(const LinearParams &p, bool e4m3, bool out_e4m3, int nt,
                                 int split, cudaStream_t st);
// What a launch needs to know of the current device; asked of the runtime once per
// device, since the queries cost as much as a launch.
struct DeviceFacts {
  int device, sms;
  int32_t *status;      // the row-operator status word
};
cudaError_t device_facts(DeviceFacts *facts);

// Raises a kernel's dynamic shared memory limit, once per kernel and device.
template <typename Kernel>
cudaError_t allow_shared(Kernel kernel, std::atomic<uint64_t> &done, int device, uint32_t bytes) {
  if (device < 64 && (done.load(std::memory_order_acquire) >> device & 1)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(bytes));
  if (e == cudaSuccess && device < 64) done.fetch_or(uint64_t(1) << device, std::memory_order_release);
  return e;
}

// Tiled tensor map (rank <= 5, element strides 1) over device memory; `swizzle`
// is the swizzle width in bytes (0, 32, 64 or 128), `elt` the element size in
// bytes (1, 2 or 4). Writes a CUtensorMap (128 bytes) to *map.
bool encode_rows_map(void *map, int elt, int swizzle, const void *base, int rank,
                     const uint64_t *dims, const uint64_t *strides_bytes, const uint32_t *box);

// Byte offset of the scale of (row, block) in the tiles of 128 rows x 4 blocks;
// block_tiles = ceil(blocks / 4).
__host__ __device__ __forceinline__ int64_t scale_offset(int64_t row, int block, int block_tiles) {
  return ((row >> 7) * block_tiles + (block >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
         (block & 3);
}

#ifdef __CUDACC__
// e for a block with largest magnitude amax (>= 0, not NaN; infinity gives 120).
// 448 = 1.75 * 2^8: e is the exponent of amax less 8, plus one if its
// significand is above 1.75.
__device__ __forceinline__ int block_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -100 ? -100 : e;
}
// 2^-e, exact for e in [-100, 120].
__device__ __forceinline__ float block_factor(int e) {
  return __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

constexpr int kGelu = WF_ACT_GELU, kSilu = WF_ACT_SILU;

// v / (1 + exp(-z)) with exp as 2^(-z log2 e): no cancellation for negative v,
// unlike 1 + tanh; both hardware approximations are good to about 2^-22.
__device__ __forceinline__ float gated(float v, float z_log2e) {
  float t, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(-z_log2e));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
  return v * r;
}
__device__ __forceinline__ float activate(float v, int act) {
  if (act == kGelu) {
    constexpr float c1 = 2.30220818f;         // 2 sqrt(2 / pi) log2(e)
    constexpr float c3 = c1 * 0.044715f;
    return gated(v, v * (c1 + c3 * (v * v)));
  }
  if (act == kSilu) return gated(v, v * 1.44269504f);
  return v;
}
#endif

}  // namespace wf
