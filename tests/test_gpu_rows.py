"""GPU parity of the row operators against their float64 oracle.

Tolerances, derived from the arithmetic:
  * a rounding to bf16 is off by at most 2^-8 of the value, to fp32 by 2^-24, to
    E4M3 by 2^-4 of the value or 2^-10 of the block's scale (half of the smallest
    step), whichever is larger;
  * norm: the sum of squares has relative error at most (terms per thread + 16)
    2^-24 (fused multiply-adds over a thread's terms, five shuffles, at most
    eight warps), its root half of that, s one rounding, and three more in
    out: (cols / 32 + 24) 2^-24 covers both kernels;
  * linear: products of bf16 or E4M3 values are exact in fp32; adding K of them
    in fp32, 16 or 32 per instruction, is off by at most (K / 16 + 16) 2^-23 of
    S = sum |x| |w| (2^-23: the unit may truncate). GELU's slope is at most 1.13
    and SILU's 1.1; their hardware exponential and reciprocal are good to 2^-20.
"""
import numpy as np
import pytest
import torch

from oracle import wf_rows as R

import chunk_causal_wavefront_b200 as wfb
from chunk_causal_wavefront_b200 import wf as W

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def f64(t):
    return t.detach().double().cpu().numpy()


def rows(n, cols, seed, dtype=BF16, scale=1.0, ld=None, offset=0):
    """Seeded rows with outlier columns on the GPU; strided if ld is given."""
    g = np.random.default_rng([seed, n, cols])
    x = g.standard_normal((n, cols)) * scale * np.where(g.random(cols) < 0.05, 8.0, 1.0)
    t = torch.from_numpy(x).to(dtype).cuda()
    if ld is None:
        return t
    big = torch.full((n * ld + offset,), float("nan"), dtype=dtype, device="cuda")
    v = big[offset:].view(n, ld)[:, :cols] if offset == 0 else big[offset:offset + n * ld].view(n, ld)[:, :cols]
    v.copy_(t)
    return v


def vec(n, seed, about=0.0):
    return torch.from_numpy(about + 0.3 * np.random.default_rng([seed, n]).standard_normal(n)).float().cuda()


def quantized(t):
    """E4M3Rows built by the oracle from t, with 0xFF (NaN) in every unused scale byte."""
    codes, e = R.quantize(f64(t))
    q = wfb.E4M3Rows(torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn),
                     torch.from_numpy(R.tile_scales(e, fill=255)).cuda())
    return q, R.dequantize(codes, e)


def raw(q):
    r, c = q.shape
    return q.codes.view(torch.uint8).cpu().numpy(), R.untile_scales(q.scales.cpu().numpy(), r, c // 32)


def assert_e4m3(q, want, slop):
    """q holds `want` (float64, known to an absolute error `slop`) as E4M3 rows."""
    codes, e = raw(q)
    got = R.dequantize(codes, e)
    we = R.block_exponents(want)
    near = np.abs(np.abs(want).reshape(*we.shape, 32).max(-1) * 2.0 ** -we.astype(float) / 448 - 1) < 2.0 ** -10
    near |= np.abs(np.abs(want).reshape(*we.shape, 32).max(-1) * 2.0 ** -we.astype(float) / 224 - 1) < 2.0 ** -10
    assert ((e == we) | (near & (np.abs(e - we) == 1))).all()
    step = np.repeat(2.0 ** (e - 10.0), 32, axis=1)
    # 2^-4 + 2^-8: half a step of a value that slop may have carried over a power of two
    tol = np.maximum(np.abs(want) * 2.0 ** -4 + slop, step) + slop
    assert (np.abs(got - want) <= tol).all()


# ------------------------------------------------------------------------------- norm --

NORM_COLS = [1, 7, 8, 31, 64, 250, 256, 264, 768, 1001, 1024, 1536, 2048, 2056, 4096, 5120, 8192, 8200, 20480]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", NORM_COLS)
def test_norm(cols, dtype):
    n = 13
    x, r, w = rows(n, cols, 1, dtype), rows(n, cols, 2, dtype, 2.0), vec(cols, 3, 1.0)
    out, s = wfb.add_rms_norm(x, w, residual=r, eps=1e-5)
    want, total = R.add_rms_norm(f64(x), f64(r), f64(w), 1e-5)
    assert torch.equal(s, (x.float() + r.float()).to(dtype))
    tol = np.abs(want) * (HALF[dtype] + (cols / 32 + 24) * 2.0 ** -24) * 1.01
    assert out.dtype == dtype and (np.abs(f64(out) - want) <= tol).all()
    # no residual, no weight
    out = wfb.add_rms_norm(x, eps=1e-5)
    want, _ = R.add_rms_norm(f64(x), None, None, 1e-5)
    tol = np.abs(want) * (HALF[dtype] + (cols / 32 + 24) * 2.0 ** -24) * 1.01
    assert (np.abs(f64(out) - want) <= tol).all()


@pytest.mark.parametrize("n", [1, 2, 129, 1000, 3001])
@pytest.mark.parametrize("cols", [72, 1536, 1537])
def test_norm_row_counts(n, cols):
    x, r, w = rows(n, cols, 4), rows(n, cols, 5), vec(cols, 6, 1.0)
    out, s = wfb.add_rms_norm(x, w, residual=r)
    want, _ = R.add_rms_norm(f64(x), f64(r), f64(w), 1e-6)
    assert torch.equal(s, (x.float() + r.float()).bfloat16())
    assert (np.abs(f64(out) - want) <= np.abs(want) * (HALF[BF16] + (cols / 32 + 24) * 2.0 ** -24) * 1.01).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", [32, 96, 288, 1536, 5120, 8192, 8224])
def test_norm_e4m3(cols, dtype):
    n = 133
    x, r, w = rows(n, cols, 7, dtype), rows(n, cols, 8, dtype), vec(cols, 9, 1.0)
    x[5], r[5] = 0, 0                                        # a row of zeros
    out, s = wfb.add_rms_norm(x, w, residual=r, out_dtype="e4m3")
    assert torch.equal(s, (x.float() + r.float()).to(dtype))
    want, _ = R.add_rms_norm(f64(x), f64(r), f64(w), 1e-6)
    assert_e4m3(out, want, np.abs(want) * (cols / 32 + 24) * 2.0 ** -24)


@pytest.mark.parametrize("ld,offset", [(1536 + 64, 0), (1536 + 8, 8), (1536 + 1, 0), (1536 + 8, 3)])
def test_norm_strided(ld, offset):
    cols, n = 1536, 21
    x, r = rows(n, cols, 10, ld=ld, offset=offset), rows(n, cols, 11, ld=ld + 8)
    out, s = rows(n, cols, 12, ld=ld, offset=offset), rows(n, cols, 13, ld=cols + 2)
    w = vec(cols + 1, 14, 1.0)[1:]                           # not 16-byte aligned
    wfb.add_rms_norm(x, w, residual=r, out=out, sum_out=s)
    want, _ = R.add_rms_norm(f64(x), f64(r), f64(w), 1e-6)
    assert torch.equal(s, (x.float() + r.float()).bfloat16())
    assert (np.abs(f64(out) - want) <= np.abs(want) * (HALF[BF16] + 80 * 2.0 ** -24) * 1.01).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols,ld,offset,n", [(65, 65, 1, 40), (250, 250, 5, 3), (1001, 1001, 0, 57), (1001, 1004, 3, 57),
                                              (1001, 1009, 7, 1), (4099, 4107, 2, 9), (8171, 8171, 1, 2), (2049, 2049, 0, 600)])
def test_norm_rows_at_any_place(cols, ld, offset, n, dtype):
    """Rows that start anywhere, with NaN before, between and behind them that must neither leak in
    nor change, in and out of place."""
    def buffer(seed):
        flat = torch.full((offset + n * ld + 16,), float("nan"), dtype=dtype, device="cuda")
        v = flat[offset:offset + n * ld].view(n, ld)[:, :cols]
        v.copy_(rows(n, cols, seed, dtype))
        return flat, v

    def gaps(flat):
        f = flat.clone()
        f[offset:offset + n * ld].view(n, ld)[:, :cols] = 0
        return f

    (fx, x), (fr, r), (fo, o), (fs, s) = (buffer(i) for i in range(120, 124))
    w = vec(cols, 124, 1.0)
    want, _ = R.add_rms_norm(f64(x), f64(r), f64(w), 1e-6)
    total = (x.float() + r.float()).to(dtype)
    tol = np.abs(want) * (HALF[dtype] + (cols / 32 + 24) * 2.0 ** -24) * 1.01
    wfb.add_rms_norm(x, w, residual=r, out=o, sum_out=s)
    assert torch.equal(s, total) and (np.abs(f64(o) - want) <= tol).all()
    kept = o.clone()
    wfb.add_rms_norm(x, w, residual=r, out=x, sum_out=r)
    assert torch.equal(r, total) and torch.equal(x, kept)
    for flat in (fx, fr, fo, fs):
        g = gaps(flat)
        assert torch.equal(g.isnan(), gaps(torch.full_like(flat, float("nan"))).isnan())


@pytest.mark.parametrize("cols", [1536, 1001, 8200])
def test_norm_in_place(cols):
    x0, r0, w = rows(300, cols, 15), rows(300, cols, 16), vec(cols, 17, 1.0)
    out0, s0 = wfb.add_rms_norm(x0, w, residual=r0)
    x, r = x0.clone(), r0.clone()
    out, s = wfb.add_rms_norm(x, w, residual=r, sum_out=r)   # the residual stream
    assert s is r and torch.equal(r, s0) and torch.equal(out, out0) and torch.equal(x, x0)
    x, r = x0.clone(), r0.clone()
    wfb.add_rms_norm(x, w, residual=r, sum_out=x, out=r)
    assert torch.equal(x, s0) and torch.equal(r, out0)
    x = x0.clone()
    wfb.add_rms_norm(x, w, out=x)
    assert torch.equal(x, wfb.add_rms_norm(x0, w))


def test_norm_leaves_other_rows_and_columns():
    big = torch.full((40, 128), 3.0, dtype=BF16, device="cuda")
    x = rows(7, 64, 18)
    wfb.add_rms_norm(x, out=big[5:12, 32:96])
    keep = big.clone()
    keep[5:12, 32:96] = 3.0
    assert (keep == 3.0).all()
    q = wfb.E4M3Rows(torch.zeros(40, 96, device="cuda").to(torch.float8_e4m3fn),
                     torch.full((512,), 77, dtype=torch.uint8, device="cuda"))
    wfb.add_rms_norm(x, out=wfb.E4M3Rows(q.codes[:7, :64], q.scales))
    assert (q.codes[7:].view(torch.uint8) == 0).all() and (q.codes[:, 64:].view(torch.uint8) == 0).all()
    s = q.scales.cpu().numpy()
    touched = {(r % 32) * 16 + (r // 32) * 4 + b for r in range(7) for b in range(2)}
    assert all(s[i] == 77 for i in range(512) if i not in touched)


def test_norm_non_finite_rows_stay_apart():
    x = rows(6, 256, 19)
    clean = wfb.add_rms_norm(x)
    x[1, 3], x[4, 200] = float("nan"), float("inf")
    out = wfb.add_rms_norm(x)
    assert out[1].isnan().all()
    assert out[4, 200].isnan() and (out[4, :200] == 0).all()   # inf / inf, finite / inf
    for i in (0, 2, 3, 5):
        assert torch.equal(out[i], clean[i])
    q = wfb.add_rms_norm(x, out_dtype="e4m3").dequantize()
    assert q[1].isnan().all() and not q[0].isnan().any()


# ------------------------------------------------------------------------- E4M3 rows --

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,cols", [(1, 32), (3, 64), (128, 128), (129, 160), (1000, 1536), (257, 5120)])
def test_quantize_bit_exact(n, cols, dtype):
    x = rows(n, cols, 20, dtype) * torch.exp2(torch.randint(-30, 30, (n, 1), device="cuda").float()).to(dtype)
    x[0, :32] = 0
    q = wfb.quantize_rows(x)
    codes, e = R.quantize(f64(x))
    gc, ge = raw(q)
    np.testing.assert_array_equal(ge, e)
    np.testing.assert_array_equal(gc, codes)
    for out in (q.dequantize(), q.dequantize(dtype=F32)):
        np.testing.assert_array_equal(f64(out), R.dequantize(codes, e))


def test_quantize_edges():
    x = torch.zeros(8, 64, device="cuda")
    x[0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1.0])
    x[1, :2] = torch.tensor([448.0, -448.0])
    x[2, 0] = float(np.nextafter(np.float32(448.0), np.float32(1e9)))
    x[3, :3] = torch.tensor([3.4028234663852886e38, 1.0, -1e38])
    x[4, :2] = torch.tensor([1e-45, -3e-39])                   # subnormal
    x[5, :] = float("nan")
    x[6, :3] = torch.tensor([1.0, 2.0 ** -9, 3 * 2.0 ** -11])  # subnormal codes, a tie
    codes, e = R.quantize(f64(x))
    gc, ge = raw(wfb.quantize_rows(x))
    np.testing.assert_array_equal(ge, e)
    np.testing.assert_array_equal(np.where((gc & 0x7F) == 0x7F, 0x7F, gc), codes)
    back = wfb.quantize_rows(x).dequantize(dtype=F32)
    assert back[0, 0].isnan() and back[0, 1] == float("inf") and back[0, 2] == -float("inf")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_strided(dtype):
    x = rows(50, 96, 21, dtype, ld=101, offset=1)
    codes, e = R.quantize(f64(x))
    buf = torch.zeros(50, 160, device="cuda").to(torch.float8_e4m3fn)
    q = wfb.E4M3Rows(buf[:, 16:112], torch.empty(512, dtype=torch.uint8, device="cuda"))
    wfb.quantize_rows(x, out=q)
    gc, ge = raw(q)
    np.testing.assert_array_equal(gc, codes)
    np.testing.assert_array_equal(ge, e)
    assert (buf[:, :16].view(torch.uint8) == 0).all() and (buf[:, 112:].view(torch.uint8) == 0).all()
    out = torch.full((50, 103), 7.0, dtype=dtype, device="cuda")
    q.dequantize(out=out[:, 3:99])
    np.testing.assert_array_equal(f64(out[:, 3:99]), R.dequantize(codes, e))
    assert (out[:, :3] == 7).all() and (out[:, 99:] == 7).all()


# ----------------------------------------------------------------------------- linear --

def check_linear(x, w, bias, act, residual, got, xv=None, wv=None):
    """xv, wv: the float64 operands where x and w are E4M3 rows."""
    xv, wv = f64(x) if xv is None else xv, f64(w) if wv is None else wv
    want = R.linear(xv, wv, None if bias is None else f64(bias), act, None if residual is None else f64(residual))
    K = xv.shape[1]
    S = np.abs(xv) @ np.abs(wv).T + (0 if bias is None else np.abs(f64(bias)))
    inner = want if residual is None else np.abs(want) + np.abs(f64(residual))
    slop = 1.13 * (K / 16 + 16) * 2.0 ** -23 * S + 2.0 ** -20 * np.abs(inner)
    if isinstance(got, wfb.E4M3Rows):
        assert_e4m3(got, want, slop)
    else:
        err = np.abs(f64(got) - want)
        bad = err > np.abs(want) * 2.0 ** -8 + slop * (1 + 2.0 ** -8)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(err.max()))


SKINNY = [(1, 8, 1), (1, 64, 1536), (1, 1536, 512), (5, 200, 72), (16, 128, 2048), (17, 129, 264),
          (33, 1000, 64), (64, 96, 8), (65, 384, 1544), (100, 77, 128), (128, 130, 640), (150, 33, 200)]


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("n,features,k", SKINNY)
def test_linear_few_rows_bf16(n, features, k, act):
    k8 = -(-k // 8) * 8                                        # K itself may be odd: only the stride counts
    x, w = rows(n, k8, 30)[:, :k], rows(features, k8, 31, scale=k ** -0.5)[:, :k]
    b, r = vec(features, 32), rows(n, features, 33)
    check_linear(x, w, b, act, r, wfb.linear(x, w, b, act=act, residual=r))
    check_linear(x, w, None, act, None, wfb.linear(x, w, act=act))
    assert wfb.rows_check_status() == 0


# Shapes that wf_linear's choice sends to every tile width of its many-row kernel (192, 256 and,
# for long K, 384 features), ragged in every dimension.
PAIR = [(512, 1536, 512), (1111, 1000, 1544), (2000, 2048, 72), (2340, 1800, 200), (700, 5000, 64),
        (4600, 1528, 3000), (4601, 1000, 1032),
        # output rows that TMA cannot store
        (2340, 1801, 200), (4600, 1527, 3000), (4601, 1001, 1032), (1500, 4999, 64)]


@pytest.mark.parametrize("n,features,k", PAIR)
def test_linear_many_rows_bf16(n, features, k):
    x, w = rows(n, k, 34), rows(features, k, 35, scale=k ** -0.5)
    b, r = vec(features, 36), rows(n, features, 37)
    check_linear(x, w, b, "none", r, wfb.linear(x, w, b, residual=r))
    check_linear(x, w, b, "gelu", None, wfb.linear(x, w, b, act="gelu"))
    check_linear(x, w, None, "silu", r, wfb.linear(x, w, act="silu", residual=r))
    assert wfb.rows_check_status() == 0


SKINNY8 = [(1, 64, 32), (1, 1536, 1536), (3, 96, 128), (16, 130, 160), (20, 1000, 512), (40, 128, 2048),
           (64, 256, 96), (90, 544, 288), (129, 100, 1024), (200, 33, 64)]


@pytest.mark.parametrize("n,features,k", SKINNY8)
def test_linear_few_rows_e4m3(n, features, k):
    x, xv = quantized(rows(n, k, 40))
    w, wv = quantized(rows(features, k, 41, scale=k ** -0.5))
    b, r = vec(features, 42), rows(n, features, 43)
    check_linear(x, w, b, "gelu", r, wfb.linear(x, w, b, act="gelu", residual=r), xv, wv)
    check_linear(x, w, None, "none", None, wfb.linear(x, w), xv, wv)
    assert wfb.rows_check_status() == 0


PAIR8 = [(512, 1536, 512), (1111, 1000, 1184), (2000, 2048, 32), (2340, 1800, 224), (700, 5000, 96),
         (4600, 1528, 3008), (4601, 1496, 1056),
         (2340, 1801, 224), (4600, 1527, 3008), (2000, 2047, 32)]


@pytest.mark.parametrize("n,features,k", PAIR8)
def test_linear_many_rows_e4m3(n, features, k):
    x, xv = quantized(rows(n, k, 44))
    w, wv = quantized(rows(features, k, 45, scale=k ** -0.5))
    b, r = vec(features, 46), rows(n, features, 47)
    check_linear(x, w, b, "none", r, wfb.linear(x, w, b, residual=r), xv, wv)
    check_linear(x, w, None, "silu", None, wfb.linear(x, w, act="silu"), xv, wv)
    assert wfb.rows_check_status() == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,features,k", [(1, 96, 128), (30, 544, 288), (300, 64, 64), (1500, 1504, 320), (600, 6144, 128),
                                          (4600, 1504, 3008)])
def test_linear_e4m3_output(n, features, k, e4m3):
    x, w, b = rows(n, k, 50), rows(features, k, 51, scale=k ** -0.5), vec(features, 52)
    xv = wv = None
    if e4m3:
        (x, xv), (w, wv) = quantized(x), quantized(w)
    check_linear(x, w, b, "gelu", None, wfb.linear(x, w, b, act="gelu", out_dtype="e4m3"), xv, wv)
    assert wfb.rows_check_status() == 0


@pytest.mark.parametrize("n", [40, 1300])
@pytest.mark.parametrize("ldo", [1504, 1544, 1601])
def test_linear_strides_and_untouched_memory(n, ldo):
    k, features = 192, 1504
    x, w = rows(n, k, 53, ld=k + 8), rows(features, k, 54, ld=k + 64, scale=k ** -0.5)
    r = rows(n, features, 55, ld=ldo)
    big = torch.full((n + 6, ldo), 5.0, dtype=BF16, device="cuda")
    out = big[2:n + 2, :features]
    wfb.linear(x, w, residual=r, out=out)
    check_linear(x, w, None, "none", r, out)
    assert (big[:2] == 5).all() and (big[n + 2:] == 5).all() and (big[:, features:] == 5).all()


@pytest.mark.parametrize("n,features", [(9, 130), (1300, 1536), (2600, 1535)])
def test_linear_in_place_on_the_residual(n, features):
    x, w, r = rows(n, 256, 56), rows(features, 256, 57, scale=1 / 16), rows(n, features, 58)
    want = wfb.linear(x, w, residual=r)
    got = wfb.linear(x, w, residual=r, out=r)
    assert got is r and torch.equal(r, want)


@pytest.mark.parametrize("n,features", [(7, 512), (300, 1536), (1300, 1536)])
def test_linear_is_repeatable_and_row_local(n, features):
    x, w = rows(n, 512, 59), rows(features, 512, 60, scale=0.05)
    a = wfb.linear(x, w)
    for _ in range(3):
        assert torch.equal(a, wfb.linear(x, w))
    x2 = x.clone()
    x2[n // 2] = float("nan")
    b = wfb.linear(x2, w)
    assert b[n // 2].isnan().all()
    b[n // 2] = a[n // 2]
    assert torch.equal(a, b)


def test_linear_prefix_of_e4m3_rows():
    x, xv = quantized(rows(400, 128, 61))
    w, wv = quantized(rows(256, 128, 62, scale=0.1))
    check_linear(x.first(150), w, None, "none", None, wfb.linear(x.first(150), w), xv[:150], wv)


def test_linear_nd_shapes():
    x, w = rows(12, 64, 63).view(3, 4, 64), rows(40, 64, 64)
    y = wfb.linear(x, w)
    assert y.shape == (3, 4, 40)
    assert torch.equal(y.view(12, 40), wfb.linear(x.view(12, 64), w))
    out, s = wfb.add_rms_norm(x, residual=x)
    assert out.shape == s.shape == x.shape


# ------------------------------------------------------------------ together, streams --

def feed_forward(x, r, p, e4m3):
    to = "e4m3" if e4m3 else None
    y, s = wfb.add_rms_norm(x, p["weight"], residual=r, out_dtype=to)
    h = wfb.linear(y, p["w1"], p["b1"], act="gelu", out_dtype=to)
    return wfb.linear(h, p["w2"], p["b2"], residual=s), s


def ff_params(hidden, ffn, e4m3):
    w1, w2 = rows(ffn, hidden, 70, scale=hidden ** -0.5), rows(hidden, ffn, 71, scale=ffn ** -0.5)
    p = dict(weight=vec(hidden, 72, 1.0), b1=vec(ffn, 73), b2=vec(hidden, 74), w1=w1, w2=w2)
    if e4m3:
        p["w1"], p["w2"] = wfb.quantize_rows(w1), wfb.quantize_rows(w2)
    return p


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [1, 77, 1400])
def test_feed_forward(n, e4m3):
    hidden, ffn = 512, 2048
    p = ff_params(hidden, ffn, e4m3)
    x, r = rows(n, hidden, 75), rows(n, hidden, 76)
    got, s = feed_forward(x, r, p, e4m3)
    y, total = R.add_rms_norm(f64(x), f64(r), f64(p["weight"]), 1e-6)

    def held(v):
        return R.dequantize(*R.quantize(v)) if e4m3 else f64(torch.from_numpy(v).bfloat16())

    wv = [f64(w.dequantize()) if e4m3 else f64(w) for w in (p["w1"], p["w2"])]
    yh = held(y)
    h = R.linear(yh, wv[0], f64(p["b1"]), "gelu", None)
    want = R.linear(held(h), wv[1], f64(p["b2"]), "none", f64(s))
    # An fp32 error may flip a rounding of y or h on a tie's edge; a flip moves a value by
    # one step (2^-3 or 2^-7 of it) and is rare, so the whole is held to its own
    # rounding plus a thousandth of the products' root sum of squares.
    half = 2.0 ** -8
    q = np.sqrt((np.abs(held(h)) ** 2) @ (np.abs(wv[1]) ** 2).T)
    assert (np.abs(f64(got) - want) <= np.abs(want) * half + 1e-3 * q + 1e-3 * half).mean() > 0.999
    assert np.linalg.norm(f64(got) - want) <= 2.0 ** -8 * np.linalg.norm(want)


def test_streams_and_graphs():
    """Another stream than the current one, and a captured chain replayed on new inputs; two
    captured graphs of the same calls take turns."""
    p = ff_params(512, 1024, True)
    xs = [rows(300, 512, 80 + i) for i in range(3)]
    r = rows(300, 512, 83)
    want = [feed_forward(x, r, p, True) for x in xs]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = wfb.add_rms_norm(xs[0], p["weight"], residual=r, out_dtype="e4m3", stream=st)
    h = wfb.linear(y[0], p["w1"], p["b1"], act="gelu", out_dtype="e4m3", stream=st)
    got = wfb.linear(h, p["w2"], p["b2"], residual=y[1], stream=st)
    deq = y[0].dequantize(stream=st)
    st.synchronize()
    assert torch.equal(got, want[0][0])
    assert torch.equal(deq, y[0].dequantize())
    assert wfb.rows_check_status(stream=st) == 0
    graphs = []
    for _ in range(2):
        x = xs[0].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = feed_forward(x, r, p, True)
        graphs.append((g, x, out))
    for i in (1, 2, 0):
        for g, x, out in graphs:
            x.copy_(xs[i])
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[0], want[i][0]) and torch.equal(out[1], want[i][1])


FIRST_CALL = """
import torch, chunk_causal_wavefront_b200 as wf
x = torch.ones(40, 256, device="cuda").bfloat16()
w = torch.ones(512, 256, device="cuda").bfloat16()
big, wide = torch.ones(2600, 256, device="cuda").bfloat16(), torch.ones(2048, 256, device="cuda").bfloat16()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y, s = wf.add_rms_norm(x, residual=x, out_dtype="e4m3")
    z = wf.linear(y, wf.quantize_rows(w))
    v = wf.linear(big, wide, act="silu")
g.replay()
torch.cuda.synchronize()
assert (s == 2).all() and (z == 256).all() and (v == 256).all() and wf.rows_check_status() == 0
print("first calls captured")
"""


def test_first_calls_of_a_process_can_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "first calls captured" in r.stdout, r.stderr[-2000:]


def test_two_streams_at_once():
    """Few-row and many-row products and norms interleaved on two streams give what they give alone."""
    x, w = rows(1400, 512, 94), rows(1536, 512, 95, scale=0.05)
    few = [rows(n, 512, 96) for n in (1, 20, 90)]
    x8, _ = quantized(x)
    w8, _ = quantized(w)
    calls = [lambda: wfb.linear(x, w), lambda: wfb.linear(few[0], w), lambda: wfb.linear(x8, w8),
             lambda: wfb.linear(few[1], w, act="gelu"), lambda: wfb.add_rms_norm(x),
             lambda: wfb.linear(few[2], w, out_dtype="e4m3").dequantize()]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for rep in range(6):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                order = range(len(calls)) if k == 0 else reversed(range(len(calls)))
                got += [(i, calls[i]()) for i in order]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i, y in got)
    assert wfb.rows_check_status() == 0


def test_offsets_past_32_bits():
    """Over 2^31 elements: the last rows match the same rows alone."""
    n, cols = 425000, 5120
    assert n * cols > 2 ** 31
    x = torch.empty(n, cols, dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(7)
    tail = torch.randn(256, cols, generator=g, device="cuda").bfloat16()
    x[:256], x[-256:] = tail, tail
    x[256:-256] = 1.0
    out, s = wfb.add_rms_norm(x, residual=x)
    want, ws = wfb.add_rms_norm(tail, residual=tail)
    for a, b in ((out, want), (s, ws)):
        assert torch.equal(a[-256:], b) and torch.equal(a[:256], b)
    del out, s
    q = wfb.quantize_rows(x)
    wq = wfb.quantize_rows(tail).dequantize()
    back = q.dequantize()
    assert torch.equal(back[-256:], wq) and torch.equal(back[:256], wq) and (back[300:-300] == 1).all()
    del back
    w = rows(64, cols, 97, scale=cols ** -0.5)
    want = wfb.linear(tail, w)
    for got in (wfb.linear(x, w), wfb.linear(x, w[:63])):      # stored by TMA, and not
        k = got.shape[1]
        err = (got[-256:].float() - want[:, :k].float()).abs().max()
        assert err <= 2 ** -7 * want.abs().max() and torch.equal(got[:256], got[-256:])
    w8 = wfb.quantize_rows(w)
    got = wfb.linear(q, w8)
    assert torch.equal(got[:256], got[-256:])
    del x, q
    small, wide = rows(110000, 64, 98), rows(20480, 64, 99, scale=0.125)
    y = wfb.linear(small, wide)
    assert y.numel() > 2 ** 31
    want = R.linear(f64(small[-64:]), f64(wide), None, "none", None)
    assert (np.abs(f64(y[-64:]) - want) <= np.abs(want) * 2.0 ** -8 + 1e-4).all()
    assert wfb.rows_check_status() == 0


def test_operands_may_share_memory():
    x = rows(300, 256, 100)
    check_linear(x, x, None, "none", None, wfb.linear(x, x))
    q, v = quantized(x)
    check_linear(q, q, None, "none", None, wfb.linear(q, q), v, v)
    buf = rows(200, 768, 101)
    a, b = buf[:, :256], buf[:, 256:768]
    w = rows(512, 256, 102, scale=1 / 16)
    want = wfb.linear(a, w)
    wfb.linear(a, w, out=b)                                   # a column range beside its input
    assert torch.equal(b, want)
    with pytest.raises(wfb.WfError):
        wfb.linear(a, w, out=buf[:, 128:640])
    out, s = wfb.add_rms_norm(x, residual=x)
    assert torch.equal(s, (2 * x.float()).bfloat16())


def test_compiled_calls_are_the_python_calls(monkeypatch):
    """The compiled common case gives the bits of the Python path, and leaves it what it does not take."""
    from chunk_causal_wavefront_b200 import rows as PR
    assert PR._fast is not None, "_rows_bind.so is not built"
    x, r, w = rows(37, 256, 110), rows(37, 256, 111), rows(96, 256, 112, scale=1 / 16)
    wt, b, r2 = vec(256, 113, 1.0), vec(96, 114), rows(37, 96, 115)
    nd = x.view(37, 4, 64)
    x8, w8 = wfb.quantize_rows(x), wfb.quantize_rows(w)
    calls = [
        lambda: wfb.add_rms_norm(x), lambda: wfb.add_rms_norm(x.float(), wt, residual=r.float(), eps=1e-3),
        lambda: wfb.add_rms_norm(x, wt, residual=r, out_dtype="e4m3"), lambda: wfb.add_rms_norm(x, out_dtype="e4m3"),
        lambda: wfb.add_rms_norm(nd), lambda: wfb.add_rms_norm(x[:, :128]), lambda: wfb.add_rms_norm(x[:0], residual=x[:0]),
        lambda: wfb.linear(x, w), lambda: wfb.linear(x, w, b, act="gelu", residual=r2),
        lambda: wfb.linear(x, w, out_dtype="e4m3"), lambda: wfb.linear(x8, w8, b, act="silu", residual=r2),
        lambda: wfb.linear(x8, w8, out_dtype="e4m3"), lambda: wfb.linear(nd, w[:, :64].contiguous()),
        lambda: wfb.linear(x[:, :128], w[:, :128]), lambda: wfb.linear(x, w, out_dtype=torch.bfloat16),
        lambda: wfb.linear(x[0], w), lambda: wfb.linear(x[:0], w), lambda: wfb.linear(x8.first(9), w8),
        lambda: wfb.quantize_rows(nd), lambda: x8.dequantize(), lambda: x8.dequantize(dtype=F32),
    ]
    bad = [lambda: wfb.linear(x, w[:, :64]), lambda: wfb.linear(x, w, b[:5]), lambda: wfb.linear(x, w8),
           lambda: wfb.linear(x8, w), lambda: wfb.linear(x, w, residual=r), lambda: wfb.linear(x.float(), w.float()),
           lambda: wfb.linear(x, w, residual=r2, out_dtype="e4m3"), lambda: wfb.linear(x, w[:33], out_dtype="e4m3"),
           lambda: wfb.add_rms_norm(x, b), lambda: wfb.add_rms_norm(x, residual=r2), lambda: wfb.add_rms_norm(x, eps=-1.0),
           lambda: wfb.add_rms_norm(x, eps=float("nan")), lambda: wfb.add_rms_norm(x.half()), lambda: wfb.linear(x.cpu(), w),
           lambda: wfb.quantize_rows(x[:, :40].contiguous()), lambda: wfb.linear(x.clone().requires_grad_(), w),
           lambda: wfb.linear(x, None), lambda: wfb.add_rms_norm(x, "w"), lambda: x8.dequantize(dtype=torch.float16)]

    def flat(v):
        if isinstance(v, tuple):
            return [t for u in v for t in flat(u)]
        return [v.codes.view(torch.uint8), v.dequantize()] if isinstance(v, wfb.E4M3Rows) else [v]

    fast, fast_errors = [flat(c()) for c in calls], []
    for c in bad:
        with pytest.raises(Exception) as e:
            c()
        fast_errors.append((type(e.value), str(e.value)))
    monkeypatch.setattr(PR, "_fast", None)
    for c, want in zip(calls, fast):
        got = flat(c())
        assert len(got) == len(want)
        for g, v in zip(got, want):
            assert g.shape == v.shape and g.dtype == v.dtype and torch.equal(g, v)
    for c, want in zip(bad, fast_errors):
        with pytest.raises(Exception) as e:
            c()
        assert (type(e.value), str(e.value)) == want


def test_refusals_on_device():
    x, w = rows(4, 64, 90), rows(8, 64, 91)
    with pytest.raises(ValueError, match="one device"):
        wfb.linear(x, w.cpu())
    with pytest.raises(ValueError, match="bias"):
        wfb.linear(x, w, vec(9, 92))
    with pytest.raises(ValueError, match="bias"):
        wfb.linear(x, w, vec(8, 92).bfloat16())
    with pytest.raises(ValueError, match="weight"):
        wfb.add_rms_norm(x, vec(63, 92))
    with pytest.raises(ValueError, match="out"):
        wfb.linear(x, w, out=torch.empty(4, 9, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError, match="out_dtype"):
        wfb.linear(x, w, out_dtype=torch.float32)
    with pytest.raises(ValueError, match="gradients"):
        wfb.linear(x.clone().requires_grad_(), w)
    with torch.no_grad():
        wfb.linear(x.clone().requires_grad_(), w)
    with pytest.raises(wfb.WfError) as e:
        wfb.linear(x.float(), w.float())
    assert e.value.status == W.WF_ERR_UNSUPPORTED
    with pytest.raises(wfb.WfError) as e:
        wfb.linear(wfb.quantize_rows(x), w)
    assert e.value.status == W.WF_ERR_UNSUPPORTED
    with pytest.raises(ValueError, match="32"):
        wfb.quantize_rows(rows(4, 48, 93))
    shared = wfb.E4M3Rows(torch.zeros(1, 64, device="cuda").to(torch.float8_e4m3fn).expand(4, 64),
                          torch.zeros(512, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="share"):
        shared.dequantize()
    y = wfb.linear(x[:0], w)
    assert y.shape == (0, 8)
    assert wfb.add_rms_norm(x[:0]).shape == (0, 64)
