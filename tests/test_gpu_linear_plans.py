"""Every instance of the two product kernels, whatever wf_linear's estimate would choose, and their
bounded waits, through wf_rows_debug_next_linear. Tolerances: check_linear's."""
import time

import pytest
import torch

from test_gpu_rows import check_linear, quantized, rows, vec

import chunk_causal_wavefront_b200 as wfb
from chunk_causal_wavefront_b200 import wf as W

pytestmark = pytest.mark.gpu

FEW, PAIRS = 1, 2


def force(kernel, tile, split=0, **kw):
    assert W.wf_rows_debug_next_linear(kernel, tile, split, **kw) == W.WF_OK


def operands(n, features, k, e4m3, seed):
    x, w = rows(n, k, seed), rows(features, k, seed + 1, scale=k ** -0.5)
    if not e4m3:
        return x, w, None, None
    (x, xv), (w, wv) = quantized(x), quantized(w)
    return x, w, xv, wv


# Ragged token and feature tiles, eight k-blocks and a rest; with more than one token tile where that
# exists (E4M3 operands have tiles of 16 and 32 tokens for a single one). 128 tokens unsplit fetch
# their residual in two parts.
@pytest.mark.parametrize("split", [1, 2, 4, 8])
@pytest.mark.parametrize("tile", [16, 32, 64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
def test_few_row_instances(e4m3, tile, split):
    k = 128 * 9 + 32 if e4m3 else 64 * 9 + 24
    n = tile - 3 if e4m3 and tile < 64 else 2 * tile - 5
    x, w, xv, wv = operands(n, 133, k, e4m3, 200)
    b, r = vec(133, 202), rows(n, 133, 203)
    force(FEW, tile, split)
    check_linear(x, w, b, "gelu", r, wfb.linear(x, w, b, act="gelu", residual=r), xv, wv)
    force(FEW, tile, split)
    check_linear(x, w, None, "none", None, wfb.linear(x, w), xv, wv)
    x, w, xv, wv = operands(n, 160, k, e4m3, 204)
    b = vec(160, 206)
    force(FEW, tile, split)
    check_linear(x, w, b, "silu", None, wfb.linear(x, w, b, act="silu", out_dtype="e4m3"), xv, wv)
    assert wfb.rows_check_status() == 0


# One pair's tile alone, and more tiles than pairs, so that each walks several; 3000 features have
# rows that TMA reaches, 2999 do not, 2976 are whole blocks for an E4M3 output.
@pytest.mark.parametrize("n,wide", [(130, False), (2590, True)])
@pytest.mark.parametrize("tile", [192, 256, 384])
@pytest.mark.parametrize("e4m3", [False, True])
def test_pair_instances(e4m3, tile, n, wide):
    if e4m3 and tile == 256:
        pytest.skip("two accumulators of 256 columns leave no room for scales")
    k = 128 * 9 + 32 if e4m3 else 64 * 9 + 24
    for features in ((3000, 2999) if wide else (200, 97)):
        x, w, xv, wv = operands(n, features, k, e4m3, 210)
        b, r = vec(features, 212), rows(n, features, 213)
        force(PAIRS, tile)
        check_linear(x, w, b, "silu", r, wfb.linear(x, w, b, act="silu", residual=r), xv, wv)
        force(PAIRS, tile)
        check_linear(x, w, None, "none", None, wfb.linear(x, w), xv, wv)
    assert wfb.rows_check_status() == 0
    if tile == 256:
        return
    features = 2976 if wide else 96
    x, w, xv, wv = operands(n, features, k, e4m3, 214)
    b = vec(features, 216)
    force(PAIRS, tile)
    check_linear(x, w, b, "gelu", None, wfb.linear(x, w, b, act="gelu", out_dtype="e4m3"), xv, wv)
    assert wfb.rows_check_status() == 0


def test_products_without_an_instance_are_refused():
    x, w, _, _ = operands(40, 64, 64, False, 220)
    x8, w8, _, _ = operands(40, 64, 64, True, 222)
    for (a, b, out), plan in (((x, w, None), (FEW, 64, 2)),             # one k-block
                              ((x, w, None), (PAIRS, 384)),
                              ((x8, w8, None), (PAIRS, 256)), ((x, w, "e4m3"), (PAIRS, 256)),
                              ((x8, w8, None), (FEW, 32, 1))):           # two token tiles
        force(*plan)
        with pytest.raises(wfb.WfError) as e:
            wfb.linear(a, b, out_dtype=out)
        assert e.value.status == W.WF_ERR_INVALID_ARG
        wfb.linear(a, b, out_dtype=out)                                  # the hook is used up
    assert wfb.rows_check_status() == 0


# Products that stall at a k-block: every wait behind it runs out after about a millisecond, the call
# reports it, and the next call is as before. Early and late blocks, of the first and a later CTA of a
# cluster; one tile and several per pair.
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,features,plan,block", [(5, 300, (FEW, 16, 1), 0), (60, 300, (FEW, 64, 4), 5),
                                                   (128, 300, (FEW, 128, 8), 8), (200, 300, (FEW, 128, 1), 7),
                                                   (130, 200, (PAIRS, 192), 0), (2590, 3000, (PAIRS, 192), 7),
                                                   (2590, 3000, (PAIRS, 384), 6), (2590, 2999, (PAIRS, 384), 9)])
def test_waits_run_out(n, features, plan, block, e4m3):
    k = 128 * 10 if e4m3 else 64 * 10
    x, w, _, _ = operands(n, features, k, e4m3, 230)
    r = rows(n, features, 232)
    force(*plan)
    want = wfb.linear(x, w, residual=r)
    torch.cuda.synchronize()
    for _ in range(2):
        force(*plan, stall_k_block=block, wait_limit_cycles=2000000)
        t0 = time.monotonic()
        wfb.linear(x, w, residual=r)
        assert wfb.rows_check_status() == W.WF_ERR_TIMEOUT
        assert time.monotonic() - t0 < 1.0
        assert wfb.rows_check_status() == 0
        force(*plan)
        assert torch.equal(wfb.linear(x, w, residual=r), want)
        assert torch.equal(wfb.linear(x, w), wfb.linear(x, w))
    assert wfb.rows_check_status() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_layer_reports_both_status_words(kv):
    from test_gpu_layer import config, make_pool, stream, weights
    cfg = config()
    layer, w = wfb.LayerRound(make_pool(cfg, kv), 512), weights(256, 512, 1, kv == "fp8")
    layer.run(0, stream(cfg, 0), w)
    assert layer.check_status() == 0
    assert W.wf_rows_debug_next_linear(0, stall_k_block=0, wait_limit_cycles=2000000) == W.WF_OK
    layer.run(0, stream(cfg, 0), w)
    assert layer.check_status() == W.WF_ERR_TIMEOUT
    assert layer.check_status() == 0
    layer.pool.advance()
    layer.attend_slot(0, 0, stream(cfg, 1), w)               # nothing of this round is published
    assert layer.check_status() == W.WF_ERR_NOT_READY
    assert layer.check_status() == 0
