"""What LayerRound refuses before it computes anything, without a GPU: a pool that is host
bookkeeping only, and tensors in host memory, which the first kernel call would refuse."""
import dataclasses

import pytest
import torch

import chunk_causal_wavefront_b200 as wfb

HIDDEN, FFN = 256, 320


@pytest.fixture
def layer():
    pool = wfb.KVPool(wfb.make_config(num_stages=2, chunk_tokens=128, num_heads=2, head_dim=128,
                                      anchor_chunks=1, history_chunks=1, page_tokens=128))
    return wfb.LayerRound(pool, FFN)


def stream(**kw):
    return torch.zeros(3, 128, HIDDEN, dtype=torch.bfloat16, **kw)


def weights():
    m = lambda n, k: torch.zeros(n, k, dtype=torch.bfloat16)
    v = lambda n: torch.zeros(n)
    return wfb.LayerWeights(w_qkv=m(3 * HIDDEN, HIDDEN), w_out=m(HIDDEN, HIDDEN), w_up=m(FFN, HIDDEN),
                            w_down=m(HIDDEN, FFN), norm1=v(HIDDEN), norm2=v(HIDDEN), b_out=v(HIDDEN),
                            b_up=v(FFN), b_down=v(HIDDEN))


def refuses(layer, match, h=None, **change):
    w = dataclasses.replace(weights(), **change)
    h = stream() if h is None else h
    for call in (lambda: layer.run(0, h, w), lambda: layer.publish_slot(0, 0, h, w),
                 lambda: layer.attend_slot(0, 0, h, w)):
        with pytest.raises(ValueError, match=match):
            call()


def passes(layer, **change):
    """Nothing is refused before the first kernel call, which wants device memory."""
    with pytest.raises(ValueError, match="CUDA"):
        layer.run(0, stream(), dataclasses.replace(weights(), **change))


# The projection takes the weight's address: fewer rows, other columns or wider elements
# would be read past their end.
@pytest.mark.parametrize("name,shape", [("w_qkv", (3 * HIDDEN - 1, HIDDEN)), ("w_qkv", (HIDDEN, HIDDEN)),
                                        ("w_qkv", (3 * HIDDEN, HIDDEN // 2)), ("w_qkv", (HIDDEN, 3 * HIDDEN)),
                                        ("w_out", (HIDDEN, HIDDEN + 8)), ("w_up", (FFN, HIDDEN + 8)),
                                        ("w_down", (HIDDEN, FFN + 8)), ("w_down", (HIDDEN + 1, FFN))])
def test_shapes_of_weights(layer, name, shape):
    refuses(layer, name, **{name: torch.zeros(shape, dtype=torch.bfloat16)})


@pytest.mark.parametrize("name", ["w_qkv", "w_out", "w_up", "w_down"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.float8_e4m3fn])
def test_types_of_weights(layer, name, dtype):
    refuses(layer, name, **{name: getattr(weights(), name).to(dtype)})


def test_e4m3_weights(layer):
    empty = lambda n, k: wfb.E4M3Rows.empty(n, k, "cpu")
    w = dict(w_qkv=empty(3 * HIDDEN, HIDDEN), w_out=empty(HIDDEN, HIDDEN), w_up=empty(FFN, HIDDEN),
             w_down=empty(HIDDEN, FFN))
    passes(layer, **w)
    refuses(layer, "w_qkv", **{**w, "w_qkv": empty(2 * HIDDEN, HIDDEN)})
    refuses(layer, "all bf16 or all", **{**w, "w_up": weights().w_up})


# What the products would refuse, one of them after h has been changed.
@pytest.mark.parametrize("name,shape", [("w_out", (HIDDEN, HIDDEN)), ("w_up", (FFN, HIDDEN)), ("w_down", (HIDDEN, FFN))])
def test_rows_of_weights(layer, name, shape):
    n, k = shape
    bf16 = dict(dtype=torch.bfloat16)
    for bad in (torch.zeros(n * k + 1, **bf16)[1:].view(n, k), torch.zeros(n, k + 1, **bf16)[:, :k],
                torch.zeros(k, n, **bf16).t(), torch.zeros(1, k, **bf16).expand(n, k)):
        refuses(layer, name, **{name: bad})
    passes(layer, **{name: torch.zeros(n, k + 8, **bf16)[:, :k]})             # strided rows are fine


def test_odd_feed_forward(layer):
    wide = torch.zeros(HIDDEN, FFN, dtype=torch.bfloat16)[:, :FFN - 3]
    refuses(layer, "multiple of 8", w_up=torch.zeros(FFN - 3, HIDDEN, dtype=torch.bfloat16), w_down=wide,
            b_up=torch.zeros(FFN - 3))


@pytest.mark.parametrize("name,n", [("norm1", HIDDEN), ("norm2", HIDDEN), ("b_out", HIDDEN), ("b_up", FFN),
                                    ("b_down", HIDDEN)])
def test_vectors(layer, name, n):
    for bad in (torch.zeros(n + 1), torch.zeros(n, dtype=torch.bfloat16), torch.zeros(2 * n)[::2]):
        refuses(layer, name, **{name: bad})


def test_devices_and_gradients(layer):
    refuses(layer, "w_qkv is on meta", w_qkv=weights().w_qkv.to("meta"))
    refuses(layer, "b_down is on meta", b_down=weights().b_down.to("meta"))
    refuses(layer, "h is on meta", h=stream(device="meta"))
    refuses(layer, "no_grad", w_qkv=weights().w_qkv.requires_grad_())
    refuses(layer, "no_grad", h=stream().requires_grad_())
    with torch.no_grad():
        passes(layer, w_qkv=weights().w_qkv.requires_grad_())
