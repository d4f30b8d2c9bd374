"""Pins of the row operators' float64 oracle: against PyTorch's float64 library
routines, and of the E4M3 row rule against its definition."""
import numpy as np
import pytest
import torch

from oracle import wf_rows as R


def test_norm_and_activations_match_library_routines():
    g = np.random.default_rng(0)
    x, r, w = g.standard_normal((5, 96)), g.standard_normal((5, 96)), g.standard_normal(96)
    out, s = R.add_rms_norm(x, r, w, 1e-3)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x + r), (96,), torch.from_numpy(w), 1e-3)
    np.testing.assert_allclose(out, want.numpy(), rtol=1e-13)
    np.testing.assert_array_equal(s, x + r)
    v = torch.linspace(-12, 12, 1001, dtype=torch.float64)
    np.testing.assert_allclose(R.activate(v.numpy(), "gelu"),
                               torch.nn.functional.gelu(v, approximate="tanh").numpy(), atol=1e-15)
    np.testing.assert_allclose(R.activate(v.numpy(), "silu"), torch.nn.functional.silu(v).numpy(), atol=1e-15)
    b = g.standard_normal(7)
    w2 = g.standard_normal((7, 96))
    want = torch.nn.functional.linear(torch.from_numpy(x), torch.from_numpy(w2), torch.from_numpy(b))
    np.testing.assert_allclose(R.linear(x, w2, b, "none", None), want.numpy(), atol=1e-12)


def test_block_exponent_is_the_smallest():
    g = np.random.default_rng(1)
    amax = np.concatenate([2.0 ** g.uniform(-90, 100, 500), 448 * 2.0 ** np.arange(-90, 100.0),
                           np.nextafter(448 * 2.0 ** np.arange(-90, 100.0), np.inf)])
    x = np.zeros((amax.size, 32))
    x[:, 5] = -amax
    e = R.block_exponents(x)[:, 0].astype(np.float64)
    assert (amax * 2.0 ** -e <= 448).all() and (amax * 2.0 ** -(e - 1) > 448).all()
    assert (R.block_exponents(np.zeros((1, 32))) == -100).all()
    assert (R.block_exponents(np.full((1, 32), np.nan)) == -100).all()


def test_rows_round_trip_and_edges():
    g = np.random.default_rng(2)
    x = g.standard_normal((9, 96)) * 2.0 ** g.integers(-20, 20, (9, 1))
    codes, e = R.quantize(x)
    y = R.dequantize(codes, e)
    # half a step: 2^-4 of the value, or half of the smallest step of the block
    assert (np.abs(y - x) <= np.maximum(np.abs(x) * 2.0 ** -4, np.repeat(2.0 ** (e - 10.0), 32, 1))).all()
    ref = torch.from_numpy(x * np.repeat(2.0 ** -e.astype(float), 32, 1)).float().to(torch.float8_e4m3fn)
    np.testing.assert_array_equal(codes, ref.view(torch.uint8).numpy())
    bad = np.zeros((1, 32))
    bad[0, :4] = [np.nan, np.inf, -np.inf, 1.0]
    codes, e = R.quantize(bad)
    assert list(codes[0, :4]) == [0x7F, 0x7E, 0xFE, 0] and e[0, 0] == 120


@pytest.mark.parametrize("rows,blocks", [(1, 1), (128, 4), (129, 5), (300, 12)])
def test_scale_tiles(rows, blocks):
    e = np.random.default_rng(3).integers(-100, 121, (rows, blocks))
    t = R.tile_scales(e)
    assert t.size == -(-rows // 128) * -(-blocks // 4) * 512
    np.testing.assert_array_equal(R.untile_scales(t, rows, blocks), e)
    # a prefix of the rows reads the same bytes
    np.testing.assert_array_equal(R.untile_scales(t, max(1, rows // 2), blocks), e[:max(1, rows // 2)])
