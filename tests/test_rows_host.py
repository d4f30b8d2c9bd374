"""Refusals of the row operators at the C ABI and in the binding, without a GPU.

Addresses here are made up: every call must be answered by the host's checks, so
no kernel could ever see them."""
import ctypes
import math

import pytest
import torch

import chunk_causal_wavefront_b200 as wfb
from chunk_causal_wavefront_b200 import wf as W
from chunk_causal_wavefront_b200 import rows as PR

BF16, F32, E4M3 = W.WF_DTYPE_BF16, W.WF_DTYPE_F32, W.WF_DTYPE_FP8_E4M3
INVALID, UNSUPPORTED = W.WF_ERR_INVALID_ARG, W.WF_ERR_UNSUPPORTED


def R(base, rows, cols, dtype=BF16, ld=None, scales=None):
    if dtype == E4M3 and scales is None:
        scales = base + (1 << 36)
    return W.WfRows(base, scales, rows, cols, cols if ld is None else ld, dtype)


A, B, C, D, E = (k << 40 for k in range(1, 6))   # far apart


def test_scale_bytes():
    assert W.wf_scale_bytes(1, 32) == 512
    assert W.wf_scale_bytes(129, 160) == 4 * 512
    assert W.wf_scale_bytes(0, 64) == 0
    assert W.wf_scale_bytes(23400, 5120) == 183 * 40 * 512
    for rows, cols in ((-1, 32), (1, 0), (1, 33), (1, -32), (1 << 31, 32)):
        with pytest.raises(wfb.WfError):
            W.wf_scale_bytes(rows, cols)
    assert W.lib().wf_scale_bytes(1, 32, None) == INVALID


def test_empty_rows_do_nothing():
    x = W.WfRows(None, None, 0, 64, 64, BF16)
    q = W.WfRows(None, None, 0, 64, 64, E4M3)
    assert W.wf_quantize_rows(x, q, 0) == W.WF_OK
    assert W.wf_dequantize_rows(q, x, 0) == W.WF_OK
    assert W.wf_add_rms_norm(x, None, None, 1e-6, None, x, 0) == W.WF_OK
    assert W.wf_linear(x, R(A, 8, 64), None, 0, None, W.WfRows(None, None, 0, 8, 8, BF16), 0) == W.WF_OK


BAD_ROWS = [
    W.WfRows(None, None, 4, 64, 64, BF16),                 # no memory
    R(A + 1, 4, 64),                                       # not aligned to an element
    R(A, -1, 64), R(A, 4, 0), R(A, 4, 64, ld=63), R(A, 1 << 31, 64), R(A, 4, 64, dtype=7),
    R(A, 1 << 30, 64, ld=1 << 37),                         # extent past 2^60 bytes
]
BAD_E4M3 = [R(A, 4, 48, E4M3), R(A, 4, 64, E4M3, ld=72), R(A + 8, 4, 64, E4M3),
            R(A, 4, 64, E4M3, scales=B + 8), W.WfRows(A, None, 4, 64, 64, E4M3)]


@pytest.mark.parametrize("bad", BAD_ROWS)
def test_bad_rows(bad):
    cols = bad.cols
    out = R(B, 4, 64, E4M3)
    assert W.wf_quantize_rows(bad, out, 0) == INVALID
    assert W.wf_add_rms_norm(bad, None, None, 1e-6, None, R(C, 4, 64), 0) == INVALID
    assert W.wf_add_rms_norm(R(C, 4, 64), None, None, 1e-6, None, bad, 0) == INVALID
    assert W.wf_add_rms_norm(R(C, 4, 64), bad, None, 1e-6, None, R(D, 4, 64), 0) == INVALID
    assert W.wf_linear(bad, R(C, 8, 64), None, 0, None, R(D, 4, 8), 0) == INVALID
    assert W.wf_linear(R(C, 4, 64), R(D, 64, 64), None, 0, bad, R(E, 4, 64), 0) == INVALID


@pytest.mark.parametrize("bad", BAD_E4M3)
def test_bad_e4m3_rows(bad):
    assert W.wf_quantize_rows(R(C, 4, 64), bad, 0) == INVALID
    assert W.wf_dequantize_rows(bad, R(C, 4, 64), 0) == INVALID
    assert W.wf_add_rms_norm(R(C, 4, 64), None, None, 1e-6, None, bad, 0) == INVALID
    assert W.wf_linear(R(C, 4, 64, E4M3), R(D, 64, 64, E4M3), None, 0, None, bad, 0) == INVALID
    assert W.wf_linear(bad, R(D, 64, 64, E4M3), None, 0, None, R(E, 4, 64), 0) == INVALID


def test_null_structs():
    r = R(A, 4, 64)
    assert W.wf_quantize_rows(None, R(B, 4, 64, E4M3), 0) == INVALID
    assert W.wf_quantize_rows(r, None, 0) == INVALID
    assert W.wf_add_rms_norm(r, None, None, 1e-6, None, None, 0) == INVALID
    assert W.wf_linear(r, None, None, 0, None, R(B, 4, 8), 0) == INVALID


def test_convert_types_and_shapes():
    assert W.wf_quantize_rows(R(A, 4, 64), R(B, 4, 64), 0) == INVALID           # out not E4M3
    assert W.wf_quantize_rows(R(A, 4, 64, E4M3), R(B, 4, 64, E4M3), 0) == INVALID
    assert W.wf_dequantize_rows(R(A, 4, 64), R(B, 4, 64), 0) == INVALID
    assert W.wf_quantize_rows(R(A, 5, 64), R(B, 4, 64, E4M3), 0) == INVALID
    assert W.wf_quantize_rows(R(A, 4, 96), R(B, 4, 64, E4M3), 0) == INVALID
    assert W.wf_quantize_rows(R(A, 1 << 22, 1 << 14), R(B, 1 << 22, 1 << 14, E4M3, scales=D), 0) == UNSUPPORTED
    # overlaps: codes over the input, scales over the input, codes over their scales
    assert W.wf_quantize_rows(R(A, 4, 64), R(A + 256, 4, 64, E4M3), 0) == INVALID
    assert W.wf_quantize_rows(R(A, 4, 64), R(B, 4, 64, E4M3, scales=A + 128), 0) == INVALID
    assert W.wf_quantize_rows(R(A, 4, 64), R(B, 4, 64, E4M3, scales=B + 128), 0) == INVALID
    assert W.wf_dequantize_rows(R(A, 4, 64, E4M3, scales=B), R(B + 256, 4, 64), 0) == INVALID


def test_norm_refusals():
    x, out = R(A, 4, 64), R(B, 4, 64)

    def norm(x=x, residual=None, weight=None, eps=1e-6, s=None, out=out):
        return W.wf_add_rms_norm(x, residual, weight, eps, s, out, 0)

    assert norm(x=R(A, 4, 64, E4M3)) == INVALID
    assert norm(out=R(B, 4, 64, F32)) == INVALID
    assert norm(out=R(B, 4, 32)) == INVALID
    assert norm(residual=R(C, 4, 64, F32)) == INVALID
    assert norm(residual=R(C, 3, 64)) == INVALID
    assert norm(s=R(C, 4, 64, F32)) == INVALID
    assert norm(s=R(C, 4, 65)) == INVALID
    for eps in (-1e-6, math.inf, math.nan):
        assert norm(eps=eps) == INVALID
    assert norm(weight=D + 2) == INVALID
    # aliases: only whole operands, and never two outputs
    assert norm(out=R(A, 4, 64, ld=72)) == INVALID
    assert norm(out=R(A + 2, 4, 64)) == INVALID
    assert norm(residual=R(C, 4, 64), s=R(B, 4, 64)) == INVALID                # sum is out
    assert norm(residual=R(C, 4, 64), s=x, out=x) == INVALID
    assert norm(residual=R(C, 4, 64), s=R(A + 64, 4, 64)) == INVALID
    assert norm(weight=B + 64) == INVALID
    assert norm(residual=R(C, 4, 64), s=R(D, 4, 64), weight=D + 4) == INVALID
    assert norm(out=R(B, 4, 64, E4M3, scales=A)) == INVALID


def test_linear_refusals():
    x, w, out = R(A, 4, 64), R(B, 96, 64), R(C, 4, 96)

    def lin(x=x, w=w, bias=None, act=0, residual=None, out=out):
        return W.wf_linear(x, w, bias, act, residual, out, 0)

    assert lin(act=3) == INVALID and lin(act=-1) == INVALID
    assert lin(w=R(B, 96, 72)) == INVALID
    assert lin(out=R(C, 5, 96)) == INVALID and lin(out=R(C, 4, 95)) == INVALID
    assert lin(residual=R(D, 4, 95)) == INVALID
    assert lin(bias=D + 1) == INVALID
    assert lin(x=R(A, 4, 64, F32), w=R(B, 96, 64, F32)) == UNSUPPORTED
    assert lin(x=R(A, 4, 64, E4M3)) == UNSUPPORTED                              # mixed operands
    assert lin(out=R(C, 4, 96, F32)) == UNSUPPORTED
    assert lin(residual=R(D, 4, 96, F32)) == UNSUPPORTED
    assert lin(residual=R(D, 4, 96), out=R(C, 4, 96, E4M3)) == UNSUPPORTED
    # operands that TMA cannot take
    assert lin(x=R(A + 2, 4, 64)) == INVALID and lin(x=R(A, 4, 64, ld=65)) == INVALID
    assert lin(w=R(B, 96, 64, ld=66)) == INVALID
    # overlaps
    assert lin(out=R(A, 4, 96)) == INVALID and lin(out=R(B + 32, 4, 96)) == INVALID
    assert lin(residual=R(C + 2, 4, 96)) == INVALID
    assert lin(residual=R(C, 4, 96, ld=104)) == INVALID
    assert lin(bias=C + 64) == INVALID


def test_column_slices_of_one_buffer_do_not_overlap():
    # x and out are column ranges of the same strided rows: not refused by the
    # overlap check, so the call gets as far as the (missing) device.
    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    x, out = R(A, 4, 64, ld=256), R(A + 128, 4, 96, ld=256)
    assert W.wf_linear(x, R(B, 96, 64), None, 0, None, out, 0) == W.WF_ERR_CUDA
    assert W.wf_linear(x, R(B, 96, 64), None, 0, None, R(A + 126, 4, 96, ld=256), 0) == INVALID
    # the next row's head
    assert W.wf_linear(x, R(B, 96, 64), None, 0, None, R(A + 2 * 161, 4, 96, ld=256), 0) == INVALID
    assert W.wf_linear(x, R(B, 96, 64), None, 0, None, R(A + 2 * 160, 4, 96, ld=256), 0) == W.WF_ERR_CUDA


def test_binding_refusals_on_cpu_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        wfb.linear(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        wfb.add_rms_norm(x)
    with pytest.raises(ValueError, match="CUDA"):
        wfb.quantize_rows(x)
    with pytest.raises(ValueError, match="act"):
        wfb.linear(x, w, act="relu")
    with pytest.raises(ValueError, match="shapes"):
        wfb.linear(x, torch.zeros(8, 32, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="residual"):
        wfb.linear(x, w, residual=torch.zeros(4, 9))
    with pytest.raises(ValueError, match="residual"):
        wfb.add_rms_norm(x, residual=x[:3])
    with pytest.raises(ValueError, match="sum_out"):
        wfb.add_rms_norm(x, sum_out=x)


def test_row_descriptions():
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    r = W.WfRows.from_buffer_copy(PR._rows(x))
    assert (r.rows, r.cols, r.ld, r.dtype) == (6, 64, 64, BF16)
    r = W.WfRows.from_buffer_copy(PR._rows(torch.zeros(5, 96)[:, :64]))
    assert (r.rows, r.cols, r.ld, r.dtype) == (5, 64, 96, F32)
    r = W.WfRows.from_buffer_copy(PR._rows(torch.zeros(64, dtype=torch.bfloat16)))
    assert (r.rows, r.cols) == (1, 64)
    for bad in (torch.zeros(4, 64).t(), torch.zeros(2, 3, 64)[:, :, ::2], torch.zeros(1, 64).expand(4, 64),
                torch.zeros(4, 0), torch.zeros(()), torch.zeros(4, 64, dtype=torch.float16)):
        with pytest.raises(ValueError):
            PR._rows(bad)


def test_live_rows_and_layer_refusals():
    def pool(dtype="bf16"):
        return wfb.KVPool(wfb.make_config(num_stages=2, chunk_tokens=128, num_heads=2, head_dim=128,
                                          anchor_chunks=1, history_chunks=1, page_tokens=128, dtype=dtype))
    p = pool()
    seen = []
    for _ in range(4):
        live = [r[2] for r in p.layout() if r[2] is not None]
        assert sorted(live) == list(range(len(live)))          # a prefix of the slots
        assert p.live_rows == 128 * len(live)
        seen.append(p.live_rows)
        p.advance()
    assert seen == [128, 256, 384, 384]
    with pytest.raises(ValueError, match="bf16 and FP8"):
        wfb.LayerRound(pool("f32"), 256)


def test_e4m3_rows_checks():
    codes = torch.zeros(130, 96, dtype=torch.float8_e4m3fn)
    q = wfb.E4M3Rows(codes, torch.zeros(1024, dtype=torch.uint8))
    assert q.first(3).shape == (3, 96)
    s = q.span(128, 130)
    assert s.shape == (2, 96) and s.scales.data_ptr() == q.scales.data_ptr() + 512
    for start, stop in ((1, 2), (128, 131), (128, 0), (-128, 0)):
        with pytest.raises(ValueError):
            q.span(start, stop)
    with pytest.raises(ValueError):
        wfb.E4M3Rows(codes, torch.zeros(1023, dtype=torch.uint8))
    with pytest.raises(ValueError):
        wfb.E4M3Rows(codes, torch.zeros(1024, dtype=torch.int8))
    with pytest.raises(ValueError):
        wfb.E4M3Rows(codes.view(torch.uint8), torch.zeros(1024, dtype=torch.uint8))
    with pytest.raises(ValueError):
        wfb.E4M3Rows(codes[:, :40], torch.zeros(1024, dtype=torch.uint8))
    with pytest.raises(ValueError):
        wfb.E4M3Rows(codes.view(-1), torch.zeros(1024, dtype=torch.uint8))
