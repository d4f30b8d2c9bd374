// Host side of the row operators: checks of arguments and choice of kernel.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "rows.cuh"
#include "wf.h"
#include "wf_internal.h"

namespace wf {
namespace {

constexpr int64_t kMaxDim = 0x7fffff00;        // row and column numbers of any tile fit int32
constexpr int64_t kMaxLd = int64_t(1) << 37;   // keeps a row stride within a tensor map's 2^40 bytes

int element_size(int32_t dtype) {
  return dtype == WF_DTYPE_F32 ? 4 : dtype == WF_DTYPE_BF16 ? 2 : 1;
}

bool multiple_of(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

wf_status check_rows(const wf_rows *r) {
  if (!r) return WF_ERR_INVALID_ARG;
  if (r->dtype != WF_DTYPE_BF16 && r->dtype != WF_DTYPE_F32 && r->dtype != WF_DTYPE_FP8_E4M3)
    return WF_ERR_INVALID_ARG;
  if (r->rows < 0 || r->rows > kMaxDim || r->cols < 1 || r->cols > kMaxDim || r->ld < r->cols ||
      r->ld > kMaxLd)
    return WF_ERR_INVALID_ARG;
  if (r->rows > (int64_t(1) << 60) / (r->ld * element_size(r->dtype))) return WF_ERR_INVALID_ARG;
  if (r->dtype == WF_DTYPE_FP8_E4M3 && (r->cols % 32 != 0 || r->ld % 16 != 0)) return WF_ERR_INVALID_ARG;
  if (r->rows == 0) return WF_OK;              // empty rows may have no memory
  if (!r->data || !multiple_of(r->data, element_size(r->dtype))) return WF_ERR_INVALID_ARG;
  if (r->dtype == WF_DTYPE_FP8_E4M3 &&
      (!multiple_of(r->data, 16) || !r->scales || !multiple_of(r->scales, 16)))
    return WF_ERR_INVALID_ARG;
  return WF_OK;
}

bool same_shape(const wf_rows *a, const wf_rows *b) { return a->rows == b->rows && a->cols == b->cols; }

// The bytes that an operand touches: `count` pieces of `width` bytes, `pitch`
// bytes from one to the next.
struct Span {
  uintptr_t base;
  int64_t width, pitch, count;
};

Span data_span(const wf_rows *r) {
  const int64_t elt = element_size(r->dtype);
  return {reinterpret_cast<uintptr_t>(r->data), r->cols * elt, r->ld * elt, r->rows};
}

Span scale_span(const wf_rows *r) {
  const int64_t n = (r->rows + 127) / 128 * ((r->cols + 127) / 128) * 512;
  return {reinterpret_cast<uintptr_t>(r->scales), n, n, 1};
}

Span vector_span(const float *v, int64_t n) { return {reinterpret_cast<uintptr_t>(v), 4 * n, 4 * n, 1}; }

// Whether two spans share a byte. Two column ranges of one strided buffer do
// not; spans of different pitches are taken as overlapping if their ranges do.
bool overlap(const Span &a, const Span &b) {
  if (a.count == 0 || b.count == 0 || !a.base || !b.base) return false;
  const uintptr_t ae = a.base + (a.count - 1) * a.pitch + a.width, be = b.base + (b.count - 1) * b.pitch + b.width;
  if (ae <= b.base || be <= a.base) return false;
  if (a.pitch != b.pitch) return true;
  const int64_t off = static_cast<int64_t>((b.base - a.base) % static_cast<uint64_t>(a.pitch));
  const int64_t d = b.base >= a.base ? off
                                     : (a.pitch - static_cast<int64_t>((a.base - b.base) % static_cast<uint64_t>(a.pitch))) % a.pitch;
  return d < a.width || d + b.width > a.pitch;
}

bool same_place(const wf_rows *a, const wf_rows *b) {
  return a->data == b->data && a->ld == b->ld && a->dtype == b->dtype;
}

// Whether an output collides with an input or another output. `in_place`: the
// output may be exactly that operand.
bool collides(const wf_rows *out, const wf_rows *other, bool in_place) {
  if (!other) return false;
  if (in_place && same_place(out, other)) return false;
  const Span od = data_span(out), xd = data_span(other);
  if (overlap(od, xd)) return true;
  const bool os = out->dtype == WF_DTYPE_FP8_E4M3, xs = other->dtype == WF_DTYPE_FP8_E4M3;
  if (os && overlap(scale_span(out), xd)) return true;
  if (xs && overlap(od, scale_span(other))) return true;
  return os && xs && overlap(scale_span(out), scale_span(other));
}

bool collides(const wf_rows *out, const float *v, int64_t n) {
  if (!v) return false;
  const Span s = vector_span(v, n);
  return overlap(data_span(out), s) || (out->dtype == WF_DTYPE_FP8_E4M3 && overlap(scale_span(out), s));
}

// An E4M3 output's codes and scales must be apart too.
bool folded(const wf_rows *out) {
  return out->dtype == WF_DTYPE_FP8_E4M3 && overlap(data_span(out), scale_span(out));
}

// The stride of a single row is never used, so it is taken as one that suits
// every access: the next multiple of 16 elements.
int64_t row_stride(const wf_rows *r) { return r->rows == 1 ? (r->cols + 15) / 16 * 16 : r->ld; }

RowsView view(const wf_rows *r) {
  if (!r) return {nullptr, nullptr, 0};
  return {r->data, static_cast<uint8_t *>(r->scales), row_stride(r)};
}

RowsType type_of(int32_t dtype) {
  return dtype == WF_DTYPE_BF16 ? RowsType::kBf16 : dtype == WF_DTYPE_F32 ? RowsType::kF32 : RowsType::kE4m3;
}

wf_status status_of(cudaError_t e) { return e == cudaSuccess ? WF_OK : WF_ERR_CUDA; }

wf_status convert(const wf_rows *x, const wf_rows *out, bool to_e4m3, cudaStream_t st) {
  wf_status s = check_rows(x);
  if (s == WF_OK) s = check_rows(out);
  if (s != WF_OK) return s;
  const wf_rows *wide = to_e4m3 ? x : out, *codes = to_e4m3 ? out : x;
  if (wide->dtype == WF_DTYPE_FP8_E4M3 || codes->dtype != WF_DTYPE_FP8_E4M3) return WF_ERR_INVALID_ARG;
  if (!same_shape(x, out)) return WF_ERR_INVALID_ARG;
  if (x->rows == 0) return WF_OK;
  if (x->rows * (x->cols / 16) > kMaxDim) return WF_ERR_UNSUPPORTED;   // 32-bit indexes
  if (collides(out, x, false) || folded(out)) return WF_ERR_INVALID_ARG;
  ConvertParams p{};
  p.x = view(x);
  p.out = view(out);
  p.rows = static_cast<int32_t>(x->rows);
  p.cols = static_cast<int32_t>(x->cols);
  return status_of(to_e4m3 ? launch_quantize_rows(p, type_of(x->dtype), st)
                           : launch_dequantize_rows(p, type_of(out->dtype), st));
}

// Which kernel a product takes, and its tile: the smallest estimate of the time in
// microseconds, from figures measured on a B200 (large products under its power
// cap, small ones at 1965 MHz with weights in HBM). Where an epilogue is longer than its
// tile's products (K of a few hundred, or rows that TMA cannot reach) the estimate does
// not know it, and 192 features can be faster than the tile taken: 23400 x 1535 x 1536 bf16
// with residual 114 us against 135 (384). Waves of wide clusters cost more than it says:
// 512 x 1536 x 6144 takes 39 us with K split over eight CTAs, 23 over two.
struct Plan {
  bool pair;
  int bn, nt, split;
};

Plan plan_linear(const LinearParams &p, bool e4m3, bool out8, bool direct) {
  const int64_t n_kb = (static_cast<int64_t>(p.K) + (e4m3 ? 127 : 63)) / (e4m3 ? 128 : 64);
  const auto tiles = [](int64_t n, int64_t by) { return (n + by - 1) / by; };
  Plan best{false, 0, 0, 0};
  double least = 0.0;
  const auto offer = [&](double us, const Plan &plan) {
    if (best.nt == 0 && !best.pair) least = us + 1.0;
    if (us < least) {
      least = us;
      best = plan;
    }
  };
  // Waves of CTA pairs: a k-block of 128 bytes, and the part of a tile's epilogue
  // that its neighbours' products do not cover; with SMs to spare the loads meet
  // less traffic.
  for (const int bn : {192, 256, 384}) {
    if (bn == 256 && (e4m3 || out8)) continue;
    if (bn == 384 && n_kb < kWideMinBlocks) continue;
    const int64_t pairs = p.sms / 2, all = tiles(p.M, 256) * tiles(p.N, bn);
    const double k_block = (e4m3 ? (bn == 192 ? 0.376 : 0.70) : bn == 192 ? 0.38 : bn == 256 ? 0.45 : 0.66) *
                           (all <= pairs ? 0.72 : 1.0);
    const double rest = (e4m3 ? (bn == 192 ? 1.3 : 3.6) : bn == 192 ? 0.6 : bn == 256 ? 0.8 : 3.2) +
                        (direct ? 1.5 : 0.0);
    offer(6.0 + tiles(all, pairs) * (n_kb * k_block + rest), Plan{true, bn, 0, 0});
  }
  // Features on the M side: either the chain of k-blocks of a CTA (two CTAs per SM
  // up to 64 tokens) and its epilogue, or the bytes that all tiles read through L2
  // at 11 TB/s, or the weights from HBM.
  for (int nt = 16; nt <= 128; nt *= 2) {
    // Several token tiles need 64-row steps of the E4M3 scale tiles, and 16-token
    // tiles are for a single one.
    if (p.M > nt && (nt == 16 || (e4m3 && nt < 64))) continue;
    const double k_block = nt == 16 ? 0.20 : nt == 32 ? 0.25 : nt == 64 ? 0.33 : 0.40;
    const int64_t all = tiles(p.N, 128) * tiles(p.M, nt);
    const int64_t room = static_cast<int64_t>(p.sms) * (nt <= 64 ? 2 : 1);
    for (int split = 1; split <= 8 && split <= n_kb; split *= 2) {
      const double chain = static_cast<double>(tiles(n_kb, split)) * k_block + 0.05 * nt / split;
      const int64_t waves = tiles(all * split, room);
      double us = waves * chain;
      const double l2 = static_cast<double>(all) * n_kb * (16.0 + nt / 8.0) / 11e3;
      const double hbm = p.N * 128e-3 * n_kb / 6.5e3;
      us = us > l2 ? us : l2;
      us = us > hbm ? us : hbm;
      // What does not overlap: a share of the chain, a start per further wave.
      offer(4.0 + us + 0.25 * waves * chain + 1.5 * (waves - 1), Plan{false, 0, nt, split});
    }
    if (p.M <= nt) break;
  }
  return best;
}

// Whether this product has an instance of the kernel and tile.
bool offers(const Plan &plan, const LinearParams &p, bool e4m3, bool out8) {
  const int64_t n_kb = (static_cast<int64_t>(p.K) + (e4m3 ? 127 : 63)) / (e4m3 ? 128 : 64);
  if (plan.pair)
    return plan.bn == 192 || (plan.bn == 256 && !e4m3 && !out8) || (plan.bn == 384 && n_kb >= kWideMinBlocks);
  const int nt = plan.nt, split = plan.split;
  if ((nt != 16 && nt != 32 && nt != 64 && nt != 128) || (split != 1 && split != 2 && split != 4 && split != 8))
    return false;
  return split <= n_kb && (!e4m3 || nt >= 64 || p.M <= nt);
}

// Test hook, consumed by the thread's next product.
struct NextLinear {
  bool armed = false, forced = false;
  Plan plan{};
  int32_t stall_k_block = -1;
  long long wait_limit = 0;
};
thread_local NextLinear t_next;

constexpr long long kWaitLimit = 2000000000LL;   // ~1 s at 2 GHz

bool rows16(const wf_rows *r) {
  return multiple_of(r->data, 16) && row_stride(r) * element_size(r->dtype) % 16 == 0;
}

}  // namespace
}  // namespace wf

using namespace wf;

extern "C" {

wf_status wf_scale_bytes(int64_t rows, int64_t cols, size_t *bytes) {
  if (!bytes || rows < 0 || rows > kMaxDim || cols < 1 || cols > kMaxDim || cols % 32 != 0)
    return WF_ERR_INVALID_ARG;
  *bytes = static_cast<size_t>((rows + 127) / 128) * static_cast<size_t>((cols + 127) / 128) * 512;
  return WF_OK;
}

wf_status wf_quantize_rows(const wf_rows *x, const wf_rows *out, wf_stream_t stream) {
  return convert(x, out, true, reinterpret_cast<cudaStream_t>(stream));
}

wf_status wf_dequantize_rows(const wf_rows *x, const wf_rows *out, wf_stream_t stream) {
  return convert(x, out, false, reinterpret_cast<cudaStream_t>(stream));
}

wf_status wf_add_rms_norm(const wf_rows *x, const wf_rows *residual, const float *weight, float eps,
                          const wf_rows *sum, const wf_rows *out, wf_stream_t stream) {
  wf_status s = check_rows(x);
  if (s == WF_OK && residual) s = check_rows(residual);
  if (s == WF_OK && sum) s = check_rows(sum);
  if (s == WF_OK) s = check_rows(out);
  if (s != WF_OK) return s;
  if (x->dtype == WF_DTYPE_FP8_E4M3) return WF_ERR_INVALID_ARG;
  if (residual && (residual->dtype != x->dtype || !same_shape(x, residual))) return WF_ERR_INVALID_ARG;
  if (sum && (sum->dtype != x->dtype || !same_shape(x, sum))) return WF_ERR_INVALID_ARG;
  if ((out->dtype != x->dtype && out->dtype != WF_DTYPE_FP8_E4M3) || !same_shape(x, out))
    return WF_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !std::isfinite(eps) || !multiple_of(weight, 4)) return WF_ERR_INVALID_ARG;
  if (x->rows == 0) return WF_OK;
  if (collides(out, x, true) || collides(out, residual, true) || collides(out, sum, false) ||
      collides(out, weight, x->cols) || folded(out))
    return WF_ERR_INVALID_ARG;
  if (sum && (collides(sum, x, true) || collides(sum, residual, true) || collides(sum, weight, x->cols)))
    return WF_ERR_INVALID_ARG;
  NormParams p{};
  p.x = view(x);
  p.residual = view(residual);
  p.sum = view(sum);
  p.out = view(out);
  p.weight = weight;
  p.eps = eps;
  p.rows = static_cast<int32_t>(x->rows);
  p.cols = static_cast<int32_t>(x->cols);
  return status_of(launch_add_rms_norm(p, type_of(x->dtype), out->dtype == WF_DTYPE_FP8_E4M3,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

wf_status wf_linear(const wf_rows *x, const wf_rows *w, const float *bias, int32_t act,
                    const wf_rows *residual, const wf_rows *out, wf_stream_t stream) {
  wf_status s = check_rows(x);
  if (s == WF_OK) s = check_rows(w);
  if (s == WF_OK && residual) s = check_rows(residual);
  if (s == WF_OK) s = check_rows(out);
  if (s != WF_OK) return s;
  if (act != WF_ACT_NONE && act != WF_ACT_GELU && act != WF_ACT_SILU) return WF_ERR_INVALID_ARG;
  if (x->cols != w->cols || out->rows != x->rows || out->cols != w->rows) return WF_ERR_INVALID_ARG;
  if (residual && !same_shape(residual, out)) return WF_ERR_INVALID_ARG;
  if (x->dtype == WF_DTYPE_F32 || w->dtype != x->dtype || out->dtype == WF_DTYPE_F32) return WF_ERR_UNSUPPORTED;
  if (residual && (residual->dtype != WF_DTYPE_BF16 || out->dtype != WF_DTYPE_BF16)) return WF_ERR_UNSUPPORTED;
  if (!multiple_of(bias, 4)) return WF_ERR_INVALID_ARG;
  if (x->rows == 0) return WF_OK;
  if (!rows16(x) || !rows16(w)) return WF_ERR_INVALID_ARG;
  if (collides(out, x, false) || collides(out, w, false) || collides(out, residual, true) ||
      collides(out, bias, out->cols) || folded(out))
    return WF_ERR_INVALID_ARG;
  const bool e4m3 = x->dtype == WF_DTYPE_FP8_E4M3, out8 = out->dtype == WF_DTYPE_FP8_E4M3;
  LinearParams p{};
  p.x = view(x);
  p.w = view(w);
  p.residual = view(residual);
  p.out = view(out);
  p.bias = bias;
  p.act = act;
  p.M = static_cast<int32_t>(x->rows);
  p.N = static_cast<int32_t>(w->rows);
  p.K = static_cast<int32_t>(x->cols);
  DeviceFacts dev;
  if (device_facts(&dev) != cudaSuccess) return WF_ERR_CUDA;
  p.status = dev.status;
  p.device = dev.device;
  p.sms = dev.sms;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool stored_by_tma = rows16(out) && (!residual || rows16(residual));
  p.stall_k_block = -1;
  p.wait_limit = kWaitLimit;
  const NextLinear next = t_next;
  t_next = NextLinear{};
  if (next.armed) {
    p.stall_k_block = next.stall_k_block;
    p.wait_limit = next.wait_limit;
    if (next.forced && !offers(next.plan, p, e4m3, out8)) return WF_ERR_INVALID_ARG;
  }
  const Plan plan = next.forced ? next.plan : plan_linear(p, e4m3, out8, !stored_by_tma);
  return status_of(plan.pair ? launch_linear_pair(p, e4m3, out8, !stored_by_tma, plan.bn, st)
                             : launch_linear_skinny(p, e4m3, out8, plan.nt, plan.split, st));
}

wf_status wf_rows_debug_next_linear(int32_t kernel, int32_t tile, int32_t split, int32_t stall_k_block,
                                    int64_t wait_limit_cycles) {
  if (kernel < 0 || kernel > 2 || stall_k_block < -1 || wait_limit_cycles < 1000 || wait_limit_cycles > kWaitLimit)
    return WF_ERR_INVALID_ARG;
  if (kernel == 1 && tile != 16 && tile != 32 && tile != 64 && tile != 128) return WF_ERR_INVALID_ARG;
  if (kernel == 1 && split != 1 && split != 2 && split != 4 && split != 8) return WF_ERR_INVALID_ARG;
  if (kernel == 2 && tile != 192 && tile != 256 && tile != 384) return WF_ERR_INVALID_ARG;
  t_next.armed = true;
  t_next.forced = kernel != 0;
  t_next.plan = kernel == 2 ? Plan{true, tile, 0, 0} : Plan{false, 0, tile, split};
  t_next.stall_k_block = stall_k_block;
  t_next.wait_limit = wait_limit_cycles;
  return WF_OK;
}

wf_status wf_rows_check_status(wf_stream_t stream) {
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return WF_ERR_CUDA;
  DeviceFacts dev;
  if (device_facts(&dev) != cudaSuccess) return WF_ERR_CUDA;
  int32_t v = 0;
  if (cudaMemcpy(&v, dev.status, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return WF_ERR_CUDA;
  if (v != 0 && cudaMemset(dev.status, 0, 4) != cudaSuccess) return WF_ERR_CUDA;
  return static_cast<wf_status>(v);
}

}  // extern "C"
