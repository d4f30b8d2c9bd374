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
