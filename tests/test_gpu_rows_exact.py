"""Row operators where their roundings can be told apart, against the float64 oracle or the exact
value.

The norm's error, kernel by kernel: a thread adds the squares of at most T elements in fp32 (T =
32 where rows stay in registers, 16 in the kernel that takes any row), which is off by at most
T 2^-24 of their sum; the threads' sums meet in 64 bits, where the factor is computed and then
rounded once. So the factor is off by (T / 2 + 1) 2^-24 of itself, and by 2^-24 more with a residual, whose
sum is rounded; s has that one rounding, and two more follow in out: (T / 2 + 5) 2^-24 of out,
whatever the width, to fp32 (plus half a step, 2^-8, to bf16).
"""
import numpy as np
import pytest
import torch

from oracle import wf_rows as R

import chunk_causal_wavefront_b200 as wfb

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().double().cpu().numpy()


# 8200 columns do not fit the register kernels, 2^20 + 4 give a thread 8192 elements.
@pytest.mark.parametrize("cols,terms", [(1, 16), (63, 16), (1001, 32), (1536, 32), (8171, 32), (8192, 32), (8200, 16),
                                        (20479, 16), ((1 << 20) + 4, 16)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_error_does_not_grow_with_the_width(cols, terms, residual):
    n = 5
    g = np.random.default_rng([1, cols])
    x = g.standard_normal((n, cols))
    x[0] = 1.1                               # the same rounding at every addition
    x[1] = np.where(np.arange(cols) % 2, 1e-3, 3.0)
    x = torch.from_numpy(x).float().cuda()
    r = torch.from_numpy(0.25 * g.standard_normal((n, cols))).float().cuda() if residual else None
    w = torch.from_numpy(1 + 0.3 * g.standard_normal(cols)).float().cuda()
    out = wfb.add_rms_norm(x, w, residual=r)
    out = out[0] if residual else out
    want, _ = R.add_rms_norm(f64(x), None if r is None else f64(r), f64(w), 1e-6)
    # A sum s near zero has lost its leading digits: s is off by 2^-24 of itself all the same
    # (one rounding), so the bound is relative everywhere.
    off = np.abs(f64(out) - want)
    assert (off <= np.abs(want) * (terms / 2 + 5) * 2.0 ** -24 * 1.01).all(), float((off / np.abs(want)).max() * 2 ** 24)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", [96, 1536, 8224])
def test_norm_to_e4m3_near_the_ends_of_fp32(cols, dtype):
    """Rows near zero, so that the row's factor times a large weight is past fp32's range where the
    result is not, with weights of both signs, and infinite weights. The result is as any other: half
    a step of E4M3 (2^-4 of the value; the block's smallest step is 2^-10 of its scale), and before
    that the fp32 error of this file's bound."""
    n = 40
    g = np.random.default_rng([2, cols])
    x = torch.from_numpy(2.0 ** -14 * g.choice([-1.0, 1.0, 0.5], (n, cols))).to(dtype).cuda()
    w = g.uniform(0.5, 1.0, cols) * 1e37 * np.where(np.arange(cols) % 3 == 0, -1, 1)
    w[:32] = np.where(np.arange(32) % 2, np.inf, -np.inf)             # the first block: infinities alone
    w = torch.from_numpy(w).float().cuda()
    q = wfb.add_rms_norm(x, w, eps=1e-6, out_dtype="e4m3")
    want, _ = R.add_rms_norm(f64(x), None, f64(w), 1e-6)
    assert (np.abs(want[:, 32:]).max() < 2.0 ** 127) and (np.abs(f64(w)[32:]) * 900 > 2.0 ** 128).any()
    got = f64(q.dequantize(dtype=F32))
    np.testing.assert_array_equal(got[:, :32], want[:, :32])          # infinite, with the sign
    _, e = R.quantize(want)
    tol = np.maximum(np.abs(want) * (2.0 ** -4 + 2.0 ** -18), np.repeat(2.0 ** (e - 10.0), 32, axis=1))[:, 32:]
    assert (np.abs(got[:, 32:] - want[:, 32:]) <= tol).all()


def test_norm_to_e4m3_without_eps_near_zero():
    """eps = 0: the factor is as large as the row is small, whatever the weight."""
    x = torch.full((3, 64), 2.0 ** -60, device="cuda")
    w = torch.full((64,), 2.0 ** 70, device="cuda")
    w[::2] = -w[::2]
    got = f64(wfb.add_rms_norm(x, w, eps=0.0, out_dtype="e4m3").dequantize(dtype=F32))
    np.testing.assert_array_equal(got, np.broadcast_to(f64(w), (3, 64)))


def test_norm_to_e4m3_of_an_infinite_factor():
    """Without eps, squares below fp32's range give a mean of zero and an infinite factor; to E4M3 as to
    fp32 the values are infinities of s * weight's sign, and NaN where that is zero."""
    x = torch.full((2, 96), 2.0 ** -80, device="cuda")
    x[1] = -x[1]
    w = torch.linspace(0.5, 3.0, 96, device="cuda")
    w[::2] = -w[::2]
    w[5], x[0, 70] = 0.0, 0.0
    want = f64(wfb.add_rms_norm(x, w, eps=0.0))
    assert np.isinf(np.delete(want, [5, 70], axis=1)).all() and np.isnan(want[0, [5, 70]]).all()
    np.testing.assert_array_equal(f64(wfb.add_rms_norm(x, w, eps=0.0, out_dtype="e4m3").dequantize(dtype=F32)), want)
    x = torch.full((2, 8224), 2.0 ** -80, device="cuda")                     # the kernel for any row
    assert (wfb.add_rms_norm(x, eps=0.0, out_dtype="e4m3").dequantize(dtype=F32) == float("inf")).all()


def factor_of(x, eps=0.0):
    """The rows' factor: computed in 64 bits from the exact sum, rounded once. (The kernel's 64-bit
    reciprocal root may be an ulp of 64 bits away, which changes the fp32 rounding of one row in 2^27.)"""
    s = x.astype(np.float64)
    return (1 / np.sqrt((s * s).sum(1, keepdims=True) * (1.0 / x.shape[1]) + eps)).astype(np.float32)


@pytest.mark.parametrize("cols", [63, 1001, 1536, 8192, 20479])
def test_norm_sums_meet_in_64_bits(cols):
    """Whole numbers whose squares a thread adds without rounding (32 x 700^2 < 2^24), while a row's sum
    needs more than 24 bits: with every later sum in 64 bits, out is s * factor, bit for bit."""
    n = 200
    x = np.random.default_rng([3, cols]).integers(-700, 701, (n, cols)).astype(np.float32)
    x[:, 0] = 1
    out = wfb.add_rms_norm(torch.from_numpy(x).cuda(), eps=0.0)
    np.testing.assert_array_equal(out.cpu().numpy(), x * factor_of(x))


@pytest.mark.parametrize("cols,shift,dtype", [(96, 0, F32), (96, 0, BF16), (1536, 0, BF16), (96, 1, F32), (8224, 0, BF16)])
def test_norm_rounds_once_before_e4m3(cols, shift, dtype):
    """Values beside the borders between codes, where a rounding more ends on the other side.
    s has 4 bits and factor and weight 24 each, so s * factor * weight is exact in float64; one rounding
    to fp32 must give the codes."""
    n = 16
    g = np.random.default_rng([4, cols, shift])
    s = g.integers(1, 16, cols).astype(np.float64)
    x = (s * g.choice([-1.0, 1.0], (n, cols))).astype(np.float32)    # one factor for all rows
    f = factor_of(x)
    assert (f == f[0]).all()
    f = f.astype(np.float64)
    # Midpoints of two codes from 2^-2 to 2^8, and a block's largest value, 448.
    mid = (1 + (2 * g.integers(0, 7, cols) + 1) / 16) * 2.0 ** g.integers(-2, 8, cols)
    mid[::32] = 448
    w = (mid / (s * f[0, 0])).astype(np.float32)
    w = np.nextafter(w, w * (1 + g.integers(-1, 2, cols) * 1.0).astype(np.float32))
    w[::32] = (448 / (s * f[0, 0]))[::32] * 0.99
    t = torch.zeros(n, cols + shift, device="cuda")[:, shift:]
    t.copy_(torch.from_numpy(x))
    q = wfb.add_rms_norm(t.to(dtype) if dtype is BF16 else t, torch.from_numpy(w).cuda(), eps=0.0, out_dtype="e4m3")
    codes, e = R.quantize((x.astype(np.float64) * f * w.astype(np.float64)).astype(np.float32))
    twice, _ = R.quantize((x * f.astype(np.float32)) * w)
    assert (codes != twice).mean() > 0.02                     # these inputs do tell
    np.testing.assert_array_equal(q.codes.view(torch.uint8).cpu().numpy(), codes)
    np.testing.assert_array_equal(R.untile_scales(q.scales.cpu().numpy(), n, cols // 32), e)


@pytest.mark.parametrize("n,features,blocks", [(1, 512, 40), (20, 1000, 24), (120, 1000, 40), (600, 1000, 40),
                                               (4600, 1528, 24)])
def test_linear_with_other_scales_in_every_block(n, features, blocks):
    """Block scales that change by up to 2^12 from one step along K to the next, over many rounds of the
    stages: a scale of another step would show. Products and scales are exact in fp32; K of them
    are added with an error of (K / 16 + 16) 2^-23 of S = sum |x| |w| (the unit may truncate), and one
    rounding to bf16 follows."""
    K = 128 * blocks
    g = np.random.default_rng([5, n, features])

    def operand(rows):
        v = g.standard_normal((rows, K)) * np.repeat(2.0 ** g.integers(-6, 7, (rows, K // 32)), 32, axis=1)
        codes, e = R.quantize(v)
        return (wfb.E4M3Rows(torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn),
                             torch.from_numpy(R.tile_scales(e, fill=255)).cuda()), R.dequantize(codes, e))

    (x, xv), (w, wv) = operand(n), operand(features)
    want, S = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    for _ in range(3):
        got = f64(wfb.linear(x, w))
        assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -8 + (K / 16 + 16) * 2.0 ** -23 * S * (1 + 2.0 ** -8)).all()
    assert wfb.rows_check_status() == 0
