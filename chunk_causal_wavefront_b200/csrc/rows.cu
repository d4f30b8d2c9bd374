// Residual addition + root-mean-square norm, and E4M3 rows to and from bf16 or
// fp32, for sm_100a.
//
// All three read each element once and write each result once; HBM bounds them.
// Measured, of the 6554 GB/s that a copy reaches: norm with residual, 23400 x 1536
// bf16 48-50 us (88-91 %), fp32 104 us (85 %), 23400 x 5120 bf16 to E4M3 144-146 us
// (88-90 %); without residual 23400 x 1536 bf16 27-28 us (78-81 %: half the bytes in
// flight per row), fp32 51 us (86 %), 23400 x 5120 fp32 212 us (69 %); 23400 x 5120 bf16
// to E4M3 58 us (95 %) and back 60-63 us (88-92 %); a single row 2.7 us, all of it launch
// and latency.
//
// Norm: s = x + residual, out = s / sqrt(mean(s^2) + eps) * weight.
//   A row stays in registers between its one read and its one write: up to 8
//   warps share a row, each lane holds up to four chunks of 8 elements (16-byte
//   loads of bf16), and the next row's loads are issued before this row's sum is
//   reduced. The weight comes from L1 (held in registers it cost occupancy). The
//   sum of squares is fp32 per lane and 64 bits from there: by shuffles, then over
//   the row's warps through shared memory in a fixed order.
//   E4M3 output: a block of 32 columns is four neighbouring lanes' chunks, so its
//   largest magnitude takes two shuffles; the codes are made from the fp32
//   values, not from their bf16 rounding.
//   Rows of odd width go through a like kernel on the aligned chunks that they
//   cover; rows that are too wide (over 8192 columns), or that start at different
//   places within 16 bytes in different operands, through a block per row, element
//   by element.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <new>

#include "f32x2.cuh"
#include "rows.cuh"
#include "sm100.cuh"

namespace wf {
namespace {

using sm100::pack_e4m3x4;

constexpr int kNormThreads = 256;

// Eight consecutive elements as fp32; 16-byte aligned.
struct Raw16 { uint4 a; };
struct Raw32 { float4 a, b; };
template <typename T> struct RawOf;
template <> struct RawOf<__nv_bfloat16> { using type = Raw16; };
template <> struct RawOf<float> { using type = Raw32; };

__device__ __forceinline__ Raw16 load8(const __nv_bfloat16 *p) {
  return {__ldcs(reinterpret_cast<const uint4 *>(p))};
}
__device__ __forceinline__ Raw32 load8(const float *p) {
  return {__ldcs(reinterpret_cast<const float4 *>(p)), __ldcs(reinterpret_cast<const float4 *>(p) + 1)};
}
__device__ __forceinline__ void widen8(const Raw16 &r, float (&v)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen8(const Raw32 &r, float (&v)[8]) {
  v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
  v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&b);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *(reinterpret_cast<float4 *>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ void narrow(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void narrow(float *p, float v) { *p = v; }

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ Raw16 pack8(const __nv_bfloat16 (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __bfloat16_as_ushort(v[2 * i]) | static_cast<uint32_t>(__bfloat16_as_ushort(v[2 * i + 1])) << 16;
  return {make_uint4(w[0], w[1], w[2], w[3])};
}
__device__ __forceinline__ Raw32 pack8(const float (&v)[8]) {
  return {make_float4(v[0], v[1], v[2], v[3]), make_float4(v[4], v[5], v[6], v[7])};
}

// 1 / sqrt(mean + eps), computed in 64 bits and rounded once: a row's elements
// share this factor's error.
__device__ __forceinline__ float norm_factor(double ss, double inv_cols, float eps) {
  return static_cast<float>(rsqrt(ss * inv_cols + static_cast<double>(eps)));
}
// s * factor * w rounded to fp32: twice on the way to bf16 or fp32, once (s * factor
// as a sum of two floats) on the way to E4M3, where every error carries a few values
// over the border between two codes. s * factor is below sqrt(cols), so it never
// overflows, unlike factor * w of a row near zero.
__device__ __forceinline__ float scaled(float s, float factor, float w) { return s * factor * w; }
// The remainder's part, negated on the way in: with an infinite weight or factor it may be
// an infinity of the other sign or a NaN, and t * w is the whole value.
__device__ __forceinline__ float rest_part(float u) { return fminf(fmaxf(-u, -3.402823466e38f), 3.402823466e38f); }
__device__ __forceinline__ float scaled_once(float s, float factor, float w) {
  const float t = s * factor;
  return fmaf(t, w, rest_part(fmaf(s, -factor, t) * w));
}
// The same for a chunk, in packed pairs: element by element it cost 23400 x 5120
// bf16 to E4M3 2 us.
__device__ __forceinline__ void scale8_once(float (&v)[8], float factor, const float (&w)[8]) {
  const uint64_t up = f2(factor, factor), down = f2(-factor, -factor);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint64_t s = f2(v[i], v[i + 1]), t = fmul2(s, up), w2 = f2(w[i], w[i + 1]);
    float a, b;
    unf2(fmul2(ffma2(s, down, t), w2), a, b);
    unf2(ffma2(t, w2, f2(rest_part(a), rest_part(b))), v[i], v[i + 1]);
  }
}

// Largest magnitude; fmaxf leaves NaN out.
__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

// CH chunks of 8 elements per lane; `wpr` warps per row, blockDim / 32 / wpr rows
// per block and pass. The next pass's rows are loaded before this pass's sums
// are reduced, so that loads are in flight at every barrier. Outputs may be the
// inputs: a chunk is stored by the thread that loaded it, and rows do not overlap.
template <typename T, bool OUT8, int CH>
__global__ void __launch_bounds__(kNormThreads, (sizeof(T) == 2 ? 2 : 1) + (CH < 4)) norm_kernel(const NormParams p, const int wpr) {
  __shared__ double part[2][kNormThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp / wpr;                      // row of the block's pass
  const int rows = blockDim.x / 32 / wpr;
  const int t = (warp - sub * wpr) * 32 + lane;    // thread of the row
  const int chunks = p.cols >> 3, stride = 32 * wpr;
  const double inv = 1.0 / p.cols;
  const int block_tiles = (p.cols + 127) >> 7;
  const T *x = static_cast<const T *>(p.x.data), *r = static_cast<const T *>(p.residual.data);
  typename RawOf<T>::type rx[CH] = {}, rr[CH] = {};
  auto load = [&](int64_t row) {
    if (row >= p.rows) return;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = t + c * stride;
      if (k < chunks) {
        rx[c] = load8(x + row * p.x.ld + 8 * k);
        if (r) rr[c] = load8(r + row * p.residual.ld + 8 * k);
      }
    }
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
  int64_t base = static_cast<int64_t>(blockIdx.x) * rows;
  sm100::grid_wait();
  sm100::grid_trigger();
  load(base + sub);
  for (int turn = 0; base < p.rows; base += step, turn ^= 1) {
    const int64_t row = base + sub;
    const bool live = row < p.rows;
    float v[CH][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      widen8(rx[c], v[c]);
      if (r) {
        float u[8];
        widen8(rr[c], u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] += u[i];
      }
      if (t + c * stride < chunks) {
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[c][i], v[c][i], ss);
      }
    }
    load(row + step);
    double sum = warp_sum(static_cast<double>(ss));
    if (wpr > 1) {
      // Two sets of partial sums in turn, so one barrier per pass is enough.
      if (lane == 0) part[turn][warp] = sum;
      __syncthreads();
      sum = 0.0;
      for (int i = 0; i < wpr; ++i) sum += part[turn][sub * wpr + i];
    }
    const float factor = norm_factor(sum, inv, p.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = t + c * stride;
      const bool on = live && k < chunks;
      if (on && p.sum.data) store8(static_cast<T *>(p.sum.data) + row * p.sum.ld + 8 * k, v[c]);
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 1.0f;
      if (p.weight && on) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(p.weight) + 2 * k);
        const float4 b = __ldg(reinterpret_cast<const float4 *>(p.weight) + 2 * k + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
      }
      if constexpr (OUT8) {
        scale8_once(v[c], factor, w);
        float m = amax8(v[c]);
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int e = block_exponent(m);
        const float f = block_factor(e);
        if (on) {
          const uint2 codes = make_uint2(
              pack_e4m3x4(v[c][0] * f, v[c][1] * f, v[c][2] * f, v[c][3] * f),
              pack_e4m3x4(v[c][4] * f, v[c][5] * f, v[c][6] * f, v[c][7] * f));
          *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.out.data) + row * p.out.ld + 8 * k) = codes;
          if ((k & 3) == 0)
            p.out.scales[scale_offset(row, k >> 2, block_tiles)] = static_cast<uint8_t>(e + 127);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = scaled(v[c][i], factor, w[i]);
        if (on) store8(static_cast<T *>(p.out.data) + row * p.out.ld + 8 * k, v[c]);
      }
    }
  }
}

// The same for rows that start anywhere within 16 bytes (odd widths), at the same
// place in every operand. Chunks are those of memory: chunk k of a row holds its
// elements [8 k - mis, 8 k - mis + 8), mis the elements between the aligned address
// and the row's start. A chunk that reaches into the neighbouring rows is loaded whole
// (the strange elements are dropped) unless it leaves the operand, and stored
// element by element. The weight is staged in shared memory: at eight loads of it per
// chunk that no vector load can replace, and a select for each, this bounds the kernel:
// 23400 x 1001 bf16 37-38 us, with residual 47-49 (58-60 % of HBM; element by element 53
// and 70), 23400 x 5119 160-163 and 191-194 us (193 and 352).
template <typename T, int CH>
__global__ void __launch_bounds__(kNormThreads, (sizeof(T) == 2 ? 2 : 1) + (CH < 4)) norm_shift_kernel(const NormParams p, const int wpr) {
  __shared__ double part[2][kNormThreads / 32];
  extern __shared__ float weight[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp / wpr;                      // row of the block's pass
  const int rows = blockDim.x / 32 / wpr;
  const int t = (warp - sub * wpr) * 32 + lane;    // thread of the row
  const int stride = 32 * wpr;
  const double inv = 1.0 / p.cols;
  const T *x = static_cast<const T *>(p.x.data), *r = static_cast<const T *>(p.residual.data);
  typename RawOf<T>::type rx[CH] = {}, rr[CH] = {};
  auto shift_of = [&](int64_t row) {
    return static_cast<int>((reinterpret_cast<uintptr_t>(x + row * p.x.ld) & 15u) / sizeof(T));
  };
  // Element of the row that chunk c of this thread starts at.
  auto start_of = [&](int c, int mis) { return 8 * (t + c * stride) - mis; };
  auto whole = [&](int e) { return e >= 0 && e + 8 <= p.cols; };
  auto fetch = [&](const T *row_data, int64_t row, int e, typename RawOf<T>::type &raw) {
    if (whole(e) || ((e >= 0 || row > 0) && (e + 8 <= p.cols || row + 1 < p.rows))) {
      raw = load8(row_data + e);
    } else {
      T part[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        narrow(part + i, 0.f);
        if (e + i >= 0 && e + i < p.cols) part[i] = row_data[e + i];
      }
      raw = pack8(part);
    }
  };
  auto load = [&](int64_t row) {
    if (row >= p.rows) return;
    const int mis = shift_of(row);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e = start_of(c, mis);
      if (e < p.cols) {
        fetch(x + row * p.x.ld, row, e, rx[c]);
        if (r) fetch(r + row * p.residual.ld, row, e, rr[c]);
      }
    }
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
  int64_t base = static_cast<int64_t>(blockIdx.x) * rows;
  sm100::grid_wait();
  sm100::grid_trigger();
  for (int i = threadIdx.x; i < p.cols; i += blockDim.x) weight[i + (i >> 3)] = p.weight ? p.weight[i] : 1.0f;
  __syncthreads();
  load(base + sub);
  for (int turn = 0; base < p.rows; base += step, turn ^= 1) {
    const int64_t row = base + sub;
    const bool live = row < p.rows;
    const int mis = shift_of(row);
    float v[CH][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      widen8(rx[c], v[c]);
      if (r) {
        float u[8];
        widen8(rr[c], u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] += u[i];
      }
      const int e = start_of(c, mis);
      if (!whole(e)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e + i < 0 || e + i >= p.cols) v[c][i] = 0.f;
      }
      if (e < p.cols) {
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[c][i], v[c][i], ss);
      }
    }
    load(row + step);
    double sum = warp_sum(static_cast<double>(ss));
    if (wpr > 1) {
      // Two sets of partial sums in turn, so one barrier per pass is enough.
      if (lane == 0) part[turn][warp] = sum;
      __syncthreads();
      sum = 0.0;
      for (int i = 0; i < wpr; ++i) sum += part[turn][sub * wpr + i];
    }
    const float factor = norm_factor(sum, inv, p.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e = start_of(c, mis);
      const bool on = live && e < p.cols;
      auto store = [&](T *row_data) {
        if (whole(e)) {
          store8(row_data + e, v[c]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (e + i >= 0 && e + i < p.cols) narrow(row_data + e + i, v[c][i]);
        }
      };
      if (on && p.sum.data) store(static_cast<T *>(p.sum.data) + row * p.sum.ld);
      // Element x of the weight is at x + x / 8 in shared memory, so that lanes 8
      // elements apart do not meet in one bank.
      const float *w = weight + 9 * (t + c * stride) - mis;
      if (whole(e)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = scaled(v[c][i], factor, w[i - (i < mis)]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e + i >= 0 && e + i < p.cols) v[c][i] = scaled(v[c][i], factor, w[i - (i < mis)]);
      }
      if (on) store(static_cast<T *>(p.out.data) + row * p.out.ld);
    }
  }
}

// Any width, alignment and stride: one block per row, element by element. Up to
// 2048 columns the row stays in registers (KEEP), all its loads in flight at once;
// longer rows are read twice, a thread's squares summed in fp32 sixteen at a time and
// in 64 bits from there (a row may have 2^24 columns per thread, and an fp32 sum
// stands still at that many). A thread's elements are the same in both readings, so
// outputs may be the inputs. A block and a barrier per row: 23400 x 33 bf16 36 us; 23400 x
// 8200 bf16 with residual 555 us (42 % of HBM).
constexpr int kAnyThreads = 128;
constexpr int kAnyKeep = 16;

template <typename T, bool OUT8, bool KEEP>
__global__ void __launch_bounds__(kAnyThreads) norm_any_kernel(const NormParams p) {
  __shared__ double part[2][kAnyThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const double inv = 1.0 / p.cols;
  const int block_tiles = (p.cols + 127) >> 7;
  int turn = 0;
  sm100::grid_wait();
  sm100::grid_trigger();
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    const T *x = static_cast<const T *>(p.x.data) + row * p.x.ld;
    const T *r = p.residual.data ? static_cast<const T *>(p.residual.data) + row * p.residual.ld : nullptr;
    float held[KEEP ? kAnyKeep : 1];
    float ss = 0.f;
    double sum = 0.0;
    if constexpr (KEEP) {
      T a[kAnyKeep], b[kAnyKeep];
#pragma unroll
      for (int j = 0; j < kAnyKeep; ++j) {
        const int k = threadIdx.x + j * kAnyThreads;
        if (k < p.cols) a[j] = x[k];
      }
      if (r) {
#pragma unroll
        for (int j = 0; j < kAnyKeep; ++j) {
          const int k = threadIdx.x + j * kAnyThreads;
          if (k < p.cols) b[j] = r[k];
        }
      }
#pragma unroll
      for (int j = 0; j < kAnyKeep; ++j) {
        const bool on = threadIdx.x + j * kAnyThreads < static_cast<unsigned>(p.cols);
        held[j] = on ? widen(a[j]) + (r ? widen(b[j]) : 0.f) : 0.f;
        ss = fmaf(held[j], held[j], ss);
      }
    } else {
      int64_t k = threadIdx.x;
      for (; k + (kAnyKeep - 1) * kAnyThreads < p.cols; k += kAnyKeep * kAnyThreads) {
        float v[kAnyKeep];                             // loads in flight together
#pragma unroll
        for (int j = 0; j < kAnyKeep; ++j) v[j] = widen(x[k + j * kAnyThreads]);
        if (r) {
#pragma unroll
          for (int j = 0; j < kAnyKeep; ++j) v[j] += widen(r[k + j * kAnyThreads]);
        }
        ss = 0.f;
#pragma unroll
        for (int j = 0; j < kAnyKeep; ++j) ss = fmaf(v[j], v[j], ss);
        sum += static_cast<double>(ss);
      }
      ss = 0.f;
      for (; k < p.cols; k += kAnyThreads) {
        const float v = widen(x[k]) + (r ? widen(r[k]) : 0.f);
        ss = fmaf(v, v, ss);
      }
    }
    sum = warp_sum(sum + static_cast<double>(ss));
    if (lane == 0) part[turn][warp] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < kAnyThreads / 32; ++i) sum += part[turn][i];
    const float factor = norm_factor(sum, inv, p.eps);
    // cols is a multiple of 32 for E4M3, so a warp is wholly in or out there.
    auto finish = [&](int64_t k, float s) {
      const float w = p.weight ? __ldg(p.weight + k) : 1.0f;
      const float v = OUT8 ? scaled_once(s, factor, w) : scaled(s, factor, w);
      if (p.sum.data) narrow(static_cast<T *>(p.sum.data) + row * p.sum.ld + k, s);
      if constexpr (OUT8) {
        const float a = fabsf(v);
        const uint32_t m = __reduce_max_sync(0xffffffffu, a == a ? __float_as_uint(a) : 0u);
        const int e = block_exponent(__uint_as_float(m));
        static_cast<uint8_t *>(p.out.data)[row * p.out.ld + k] =
            static_cast<uint8_t>(sm100::pack_e4m3x2(v * block_factor(e), 0.f) & 0xffu);
        if (lane == 0)
          p.out.scales[scale_offset(row, static_cast<int>(k >> 5), block_tiles)] = static_cast<uint8_t>(e + 127);
      } else {
        narrow(static_cast<T *>(p.out.data) + row * p.out.ld + k, v);
      }
    };
    if constexpr (KEEP) {
#pragma unroll
      for (int j = 0; j < kAnyKeep; ++j) {
        const int k = threadIdx.x + j * kAnyThreads;
        if (k < p.cols) finish(k, held[j]);
      }
    } else {
      for (int64_t k = threadIdx.x; k < p.cols; k += kAnyThreads)
        finish(k, widen(x[k]) + (r ? widen(r[k]) : 0.f));
    }
  }
}

// Rows to E4M3: 16 columns per thread, a block of 32 is two neighbouring lanes.
// VEC: 16-byte loads; else element by element.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) quantize_kernel(const ConvertParams p) {
  const uint32_t per_row = static_cast<uint32_t>(p.cols) >> 4;
  const uint32_t total = static_cast<uint32_t>(p.rows) * per_row;   // even, < 2^31 (host check)
  const int block_tiles = (p.cols + 127) >> 7;
  sm100::grid_wait();
  sm100::grid_trigger();
  for (uint32_t i = blockIdx.x * 256u + threadIdx.x; i < total; i += gridDim.x * 256u) {
    const uint32_t row = i / per_row, k = i - row * per_row;
    const T *x = static_cast<const T *>(p.x.data) + static_cast<int64_t>(row) * p.x.ld + 16 * k;
    float v[2][8];
    if constexpr (VEC) {
      const auto a = load8(x), b = load8(x + 8);
      widen8(a, v[0]);
      widen8(b, v[1]);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j >> 3][j & 7] = widen(x[j]);
    }
    float m = fmaxf(amax8(v[0]), amax8(v[1]));
    // The pair's other lane is in the loop too: total is even.
    const uint32_t pair = 3u << (threadIdx.x & 30);
    m = fmaxf(m, __shfl_xor_sync(pair, m, 1));
    const int e = block_exponent(m);
    const float f = block_factor(e);
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float *u = v[j >> 1] + 4 * (j & 1);
      c[j] = pack_e4m3x4(u[0] * f, u[1] * f, u[2] * f, u[3] * f);
    }
    *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out.data) + static_cast<int64_t>(row) * p.out.ld + 16 * k) =
        make_uint4(c[0], c[1], c[2], c[3]);
    if ((k & 1) == 0)
      p.out.scales[scale_offset(row, static_cast<int>(k >> 1), block_tiles)] = static_cast<uint8_t>(e + 127);
  }
}

// E4M3 rows to T: 16 columns per thread. The product with 2^e is exact in fp32.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) dequantize_kernel(const ConvertParams p) {
  const uint32_t per_row = static_cast<uint32_t>(p.cols) >> 4;
  const uint32_t total = static_cast<uint32_t>(p.rows) * per_row;
  const int block_tiles = (p.cols + 127) >> 7;
  sm100::grid_wait();
  sm100::grid_trigger();
  for (uint32_t i = blockIdx.x * 256u + threadIdx.x; i < total; i += gridDim.x * 256u) {
    const uint32_t row = i / per_row, k = i - row * per_row;
    const uint4 c = *reinterpret_cast<const uint4 *>(
        static_cast<const uint8_t *>(p.x.data) + static_cast<int64_t>(row) * p.x.ld + 16 * k);
    const int s = p.x.scales[scale_offset(row, static_cast<int>(k >> 1), block_tiles)];
    // 2^(s - 127); the byte of the smallest exponent, 0, is a subnormal float.
    const float f2 = __uint_as_float(s ? static_cast<uint32_t>(s) << 23 : 0x400000u);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    float v[2][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
          static_cast<__nv_fp8x2_storage_t>(w[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      v[j >> 2][2 * (j & 3)] = f.x * f2;
      v[j >> 2][2 * (j & 3) + 1] = f.y * f2;
    }
    T *out = static_cast<T *>(p.out.data) + static_cast<int64_t>(row) * p.out.ld + 16 * k;
    if constexpr (VEC) {
      store8(out, v[0]);
      store8(out + 8, v[1]);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) narrow(out + j, v[j >> 3][j & 7]);
    }
  }
}

bool aligned(const void *p, int64_t ld, int64_t elt) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * elt) % 16 == 0;
}

// Blocks that the device holds at once: a grid of that size walks the rows with no
// second wave. Asked once per kernel, block size and device.
template <typename K>
cudaError_t resident_blocks(K kernel, int threads, std::atomic<int> (&known)[64], const DeviceFacts &dev, int64_t *blocks) {
  int per_sm = dev.device < 64 ? known[dev.device].load(std::memory_order_relaxed) : 0;
  if (per_sm == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, 0);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) per_sm = 1;
    if (dev.device < 64) known[dev.device].store(per_sm, std::memory_order_relaxed);
  }
  *blocks = static_cast<int64_t>(per_sm) * dev.sms;
  return cudaSuccess;
}

// One launch of norm_kernel or norm_shift_kernel with `shared` dynamic bytes.
template <typename K>
cudaError_t run_norm(K kernel, std::atomic<int> (&known)[9][64], const NormParams &p, int wpr, uint32_t shared,
                     const DeviceFacts &dev, cudaStream_t st) {
  const int rows = kNormThreads / 32 / wpr;        // per block and pass, >= 1
  const int threads = rows * wpr * 32;
  int64_t grid = 0;
  const cudaError_t e = resident_blocks(kernel, threads, known[wpr], dev, &grid);
  if (e != cudaSuccess) return e;
  const int64_t need = (static_cast<int64_t>(p.rows) + rows - 1) / rows;
  return launch_dependent(kernel, static_cast<unsigned>(need < grid ? need : grid), threads, shared, 0, st, p, wpr);
}

template <typename T, bool OUT8, int CH, bool SHIFT>
cudaError_t run_chunks(const NormParams &p, int wpr, const DeviceFacts &dev, cudaStream_t st) {
  static std::atomic<int> known[9][64];
  if constexpr (SHIFT)
    return run_norm(norm_shift_kernel<T, CH>, known, p, wpr, (p.cols + p.cols / 8 + 1) * 4, dev, st);
  else
    return run_norm(norm_kernel<T, OUT8, CH>, known, p, wpr, 0, dev, st);
}

template <typename T, bool OUT8, bool SHIFT>
cudaError_t pick_chunks(const NormParams &p, const DeviceFacts &dev, cudaStream_t st) {
  // Warps per row and chunks per lane that leave the fewest lanes idle; among
  // those the most chunks, for more bytes in flight per lane.
  const int chunks = (p.cols + (SHIFT ? 7 + 15 / static_cast<int>(sizeof(T)) : 0)) / 8;
  int wpr = 8, ch = 4;
  for (int c = 4; c >= 1; --c) {
    const int w = (chunks + 32 * c - 1) / (32 * c);
    if (w <= 8 && w * c < wpr * ch) {
      wpr = w;
      ch = c;
    }
  }
  switch (ch) {
    case 1: return run_chunks<T, OUT8, 1, SHIFT>(p, wpr, dev, st);
    case 2: return run_chunks<T, OUT8, 2, SHIFT>(p, wpr, dev, st);
    case 3: return run_chunks<T, OUT8, 3, SHIFT>(p, wpr, dev, st);
    default: return run_chunks<T, OUT8, 4, SHIFT>(p, wpr, dev, st);
  }
}

template <typename T, bool OUT8>
cudaError_t pick_norm(const NormParams &p, cudaStream_t st) {
  DeviceFacts dev;
  const cudaError_t e = device_facts(&dev);
  if (e != cudaSuccess) return e;
  const int64_t elt = sizeof(T);
  const bool vec = p.cols % 8 == 0 && p.cols <= 8192 && aligned(p.x.data, p.x.ld, elt) &&
                   (!p.residual.data || aligned(p.residual.data, p.residual.ld, elt)) &&
                   (!p.sum.data || aligned(p.sum.data, p.sum.ld, elt)) &&
                   aligned(p.out.data, p.out.ld, OUT8 ? 1 : elt) &&
                   (reinterpret_cast<uintptr_t>(p.weight) & 15u) == 0;
  if (vec) return pick_chunks<T, OUT8, false>(p, dev, st);
  if constexpr (!OUT8) {
    // Every operand's rows start at the same place within 16 bytes.
    const auto like_x = [&](const RowsView &o) {
      return !o.data || ((reinterpret_cast<uintptr_t>(o.data) - reinterpret_cast<uintptr_t>(p.x.data)) % 16 == 0 &&
                         (p.rows == 1 || (o.ld - p.x.ld) * elt % 16 == 0));
    };
    if (p.cols >= 64 && p.cols <= 8192 - 16 && like_x(p.residual) && like_x(p.sum) && like_x(p.out))
      return pick_chunks<T, false, true>(p, dev, st);
  }
  const int64_t most = static_cast<int64_t>(dev.sms) * 16;
  const unsigned grid = static_cast<unsigned>(p.rows < most ? p.rows : most);
  return launch_dependent(p.cols <= kAnyThreads * kAnyKeep ? norm_any_kernel<T, OUT8, true>
                                                           : norm_any_kernel<T, OUT8, false>,
                          grid, kAnyThreads, 0, 0, st, p);
}

unsigned convert_grid(const ConvertParams &p, int sms) {
  const int64_t need = (static_cast<int64_t>(p.rows) * (p.cols / 16) + 255) / 256;
  const int64_t most = static_cast<int64_t>(sms) * 64;
  return static_cast<unsigned>(need < most ? need : most);
}

}  // namespace

// Sticky status of the row operators that wait on barriers: one word per device.
__device__ int32_t g_rows_status;

cudaError_t device_facts(DeviceFacts *facts) {
  static std::atomic<const DeviceFacts *> known[64];   // entries live as long as the process
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64) {
    if (const DeviceFacts *f = known[dev].load(std::memory_order_acquire)) {
      *facts = *f;
      return cudaSuccess;
    }
  }
  void *word = nullptr;
  facts->device = dev;
  e = cudaDeviceGetAttribute(&facts->sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaGetSymbolAddress(&word, g_rows_status);
  if (e != cudaSuccess) return e;
  facts->status = static_cast<int32_t *>(word);
  if (dev < 64) {
    const DeviceFacts *fresh = new (std::nothrow) DeviceFacts(*facts), *none = nullptr;
    if (fresh && !known[dev].compare_exchange_strong(none, fresh, std::memory_order_release)) delete fresh;
  }
  return cudaSuccess;
}

cudaError_t launch_add_rms_norm(const NormParams &p, RowsType in, bool out_e4m3, cudaStream_t st) {
  if (in == RowsType::kBf16)
    return out_e4m3 ? pick_norm<__nv_bfloat16, true>(p, st) : pick_norm<__nv_bfloat16, false>(p, st);
  return out_e4m3 ? pick_norm<float, true>(p, st) : pick_norm<float, false>(p, st);
}

cudaError_t launch_quantize_rows(const ConvertParams &p, RowsType in, cudaStream_t st) {
  DeviceFacts dev;
  const cudaError_t e = device_facts(&dev);
  if (e != cudaSuccess) return e;
  const unsigned grid = convert_grid(p, dev.sms);
  if (in == RowsType::kBf16)
    return launch_dependent(aligned(p.x.data, p.x.ld, 2) ? quantize_kernel<__nv_bfloat16, true>
                                                         : quantize_kernel<__nv_bfloat16, false>,
                            grid, 256, 0, 0, st, p);
  return launch_dependent(aligned(p.x.data, p.x.ld, 4) ? quantize_kernel<float, true> : quantize_kernel<float, false>,
                          grid, 256, 0, 0, st, p);
}

cudaError_t launch_dequantize_rows(const ConvertParams &p, RowsType out, cudaStream_t st) {
  DeviceFacts dev;
  const cudaError_t e = device_facts(&dev);
  if (e != cudaSuccess) return e;
  const unsigned grid = convert_grid(p, dev.sms);
  if (out == RowsType::kBf16)
    return launch_dependent(aligned(p.out.data, p.out.ld, 2) ? dequantize_kernel<__nv_bfloat16, true>
                                                             : dequantize_kernel<__nv_bfloat16, false>,
                            grid, 256, 0, 0, st, p);
  return launch_dependent(aligned(p.out.data, p.out.ld, 4) ? dequantize_kernel<float, true>
                                                           : dequantize_kernel<float, false>,
                          grid, 256, 0, 0, st, p);
}

}  // namespace wf
