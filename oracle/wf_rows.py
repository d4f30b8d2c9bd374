"""Row operators of a layer around its round attention: float64 CPU oracle.

TEST INFRASTRUCTURE ONLY, like ``wf_oracle``. Definitions:
  * add_rms_norm: s = x + residual, out = s / sqrt(mean(s^2) + eps) * weight;
  * linear: act(x w^T + bias) + residual, GELU in its tanh form;
  * E4M3 rows: blocks of 32 columns with a scale 2^e, e the smallest integer
    >= -100 with amax * 2^-e <= 448 over the block's values that are not NaN
    (e = 120 with an infinity), codes rounded to nearest even and saturating.
"""
from __future__ import annotations

import numpy as np

from .wf_fp8 import e4m3_decode, e4m3_encode

__all__ = ["add_rms_norm", "activate", "linear", "block_exponents", "quantize", "dequantize",
           "tile_scales", "untile_scales"]


def add_rms_norm(x, residual, weight, eps):
    """(out, s) in float64."""
    s = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    out = s / np.sqrt(np.mean(s * s, axis=-1, keepdims=True) + eps)
    return (out if weight is None else out * np.asarray(weight, np.float64)), s


def activate(v, act):
    if act == "gelu":
        return 0.5 * v * (1 + np.tanh(np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)))
    if act == "silu":
        return v / (1 + np.exp(-v))
    assert act == "none"
    return v


def linear(x, w, bias, act, residual):
    v = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    if bias is not None:
        v = v + np.asarray(bias, np.float64)
    v = activate(v, act)
    return v if residual is None else v + np.asarray(residual, np.float64)


def block_exponents(x):
    """e of every (row, block of 32 columns)."""
    x = np.asarray(x, np.float64)
    a = np.abs(x).reshape(x.shape[0], -1, 32)
    amax = np.where(np.isnan(a), 0.0, a).max(axis=-1)
    m, p = np.frexp(np.where(np.isinf(amax) | (amax == 0), 1.0, amax))   # amax = m 2^p, 1/2 <= m < 1
    e = np.where(m <= 448 / 512, p - 9, p - 8)
    e = np.where(amax == 0, -100, np.maximum(e, -100))
    return np.where(np.isinf(amax), 120, e)


def quantize(x):
    """(codes uint8 [rows][cols], e [rows][cols / 32])."""
    x = np.asarray(x, np.float64)
    e = block_exponents(x)
    scaled = x * np.repeat(2.0 ** (-e.astype(np.float64)), 32, axis=1)
    fin = np.where(np.isfinite(scaled), scaled, 0.0)
    codes = e4m3_encode(np.clip(fin, -448, 448))
    codes = np.where(np.isposinf(scaled), 0x7E, np.where(np.isneginf(scaled), 0xFE, codes))
    return np.where(np.isnan(scaled), 0x7F, codes).astype(np.uint8), e


def dequantize(codes, e):
    return e4m3_decode(codes) * np.repeat(2.0 ** np.asarray(e, np.float64), 32, axis=1)


def tile_scales(e, fill=0):
    """Exponents as the bytes e + 127 in tiles of 128 rows x 4 blocks."""
    rows, blocks = e.shape
    kt = -(-blocks // 4)
    out = np.full(-(-rows // 128) * kt * 512, fill, np.uint8)
    for r in range(rows):
        for b in range(blocks):
            out[((r // 128) * kt + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4] = e[r, b] + 127
    return out


def untile_scales(tiles, rows, blocks):
    r, b = np.arange(rows)[:, None], np.arange(blocks)[None, :]
    at = ((r // 128) * -(-blocks // 4) + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4
    return np.asarray(tiles)[at].astype(np.int64) - 127
