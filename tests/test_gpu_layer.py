"""LayerRound: whole layers through pipeline fill into steady rounds, in bf16 and 8 bits, on
bf16 and FP8 pools, against the float64 oracle and bit for bit against the same calls made
one by one; one slot at a time as under Wave Parallelism.

Tolerances against the oracle, which rounds nothing in between (its operands are the bf16
inputs and weights, or the values that the E4M3 weights stand for): every value that the
layer stores is off by at most half a step of its type, 2^-8 of itself in bf16 and 2^-4 in
E4M3. In bf16 seven such roundings follow one another (norm, q/k/v, attention with
its own 1e-2 rel-L2 bound, stream, norm, hidden, stream): 6 x 2^-8 + 1e-2 < 4e-2 of the
layer's change of h. In E4M3 the norm outputs, q/k/v, probabilities, attention output and
hidden are rounded so too: six times 2^-4, independent of one another, add up to
sqrt(6) 2^-4 < 0.16 of the change. Weights of unit gain keep errors from growing.
"""
import numpy as np
import pytest
import torch

import wf_inputs
from oracle import wf_oracle as O
from oracle import wf_rows as R
from wf_test_utils import min_pages, pool_config

import chunk_causal_wavefront_b200 as wfb

pytestmark = pytest.mark.gpu


def config(heads=2, chunk=2 * 8 * 20):
    return wf_inputs.CONFIGS["wan13b_bf16"].replace(
        num_stages=2, chunk_tokens=chunk, num_heads=heads, history_chunks=1,
        frames_per_chunk=2, grid_h=8, grid_w=chunk // 16)


def make_pool(cfg, dtype, layers=1):
    return wfb.KVPool(pool_config(cfg, num_layers=layers, num_pages=0, dtype=dtype), device="cuda",
                      page_order=wf_inputs.draw_page_order(min_pages(cfg), 3))


def weights(hidden, ffn, seed, e4m3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    m = lambda n, k: (torch.randn(n, k, generator=g, device="cuda") / k ** 0.5).bfloat16()
    v = lambda n, about: about + 0.2 * torch.randn(n, generator=g, device="cuda")
    w = wfb.LayerWeights(w_qkv=m(3 * hidden, hidden), w_out=m(hidden, hidden), w_up=m(ffn, hidden),
                         w_down=m(hidden, ffn), norm1=v(hidden, 1.0), norm2=v(hidden, 1.0),
                         b_out=v(hidden, 0.0), b_up=v(ffn, 0.0), b_down=v(hidden, 0.0))
    return w.to_e4m3() if e4m3 else w


def f64(t):
    return (t.dequantize(dtype=torch.float32) if isinstance(t, wfb.E4M3Rows) else t).double().cpu().numpy()


def stream(cfg, rnd):
    hidden = cfg.num_heads * cfg.head_dim
    g = torch.Generator(device="cuda").manual_seed(100 + rnd)
    return torch.randn(cfg.num_slots, cfg.chunk_tokens, hidden, generator=g, device="cuda").bfloat16()


class Oracle:
    """The layer in float64 over the same rounds."""

    def __init__(self, cfg, w):
        self.cfg, self.w, self.stored = cfg, {k: None if t is None else f64(t) for k, t in vars(w).items()}, {}

    def run(self, rnd, h):
        c, w = self.cfg, self.w
        D = c.num_heads * c.head_dim
        lay = O.round_layout(c.num_stages, c.anchor_chunks, c.history_chunks, rnd)
        qr, keys, vals = {}, {}, {}
        rope = lambda x, ch: O.rope_3d(x, ch, c.frames_per_chunk, c.grid_h, c.grid_w)
        for p in lay:
            if p.slot is None:
                keys[p.chunk], vals[p.chunk] = self.stored[p.chunk]
                continue
            y, _ = R.add_rms_norm(h[p.slot], None, w["norm1"], 1e-6)
            q, k, v = (np.split(y @ w["w_qkv"].T, 3, axis=1)[i].reshape(-1, c.num_heads, c.head_dim)
                       for i in range(3))
            qr[p.slot], keys[p.chunk], vals[p.chunk] = rope(q, p.chunk), rope(k, p.chunk), v
            if p.kind == "store":
                self.stored[p.chunk] = (keys[p.chunk], vals[p.chunk])
        out = O.attention_slot_prefix(qr, keys, vals, lay)
        new = {}
        for s, a in out.items():
            x = R.linear(a.reshape(-1, D), w["w_out"], w["b_out"], "none", h[s])
            y, _ = R.add_rms_norm(x, None, w["norm2"], 1e-6)
            new[s] = R.linear(R.linear(y, w["w_up"], w["b_up"], "gelu", None), w["w_down"], w["b_down"], "none", x)
        return new


@pytest.mark.parametrize("kv,e4m3,heads,chunk", [("bf16", False, 2, 320), ("bf16", False, 1, 320),
                                                 ("bf16", True, 2, 320), ("fp8", False, 2, 160),
                                                 ("fp8", True, 2, 320)])
def test_layer_against_the_oracle(kv, e4m3, heads, chunk):
    cfg = config(heads, chunk)
    hidden = heads * cfg.head_dim
    pool = make_pool(cfg, kv)
    w = weights(hidden, 4 * hidden, 1, e4m3)
    layer, oracle = wfb.LayerRound(pool, 4 * hidden), Oracle(cfg, w)
    bound = 0.16 if e4m3 or kv == "fp8" else 4e-2
    for rnd in range(cfg.steady_round() + 2):
        h = stream(cfg, rnd)
        h0 = f64(h)
        assert layer.run(0, h, w) is h
        assert pool.check_status() == 0 and wfb.rows_check_status() == 0
        got, want = f64(h), oracle.run(rnd, h0)
        for s in range(cfg.num_slots):
            if s not in want:
                np.testing.assert_array_equal(got[s], h0[s])          # not live: untouched
                continue
            off = np.linalg.norm(got[s] - want[s]) / np.linalg.norm(want[s] - h0[s])
            assert off <= bound, (rnd, s, off)
        pool.advance()


@pytest.mark.parametrize("kv,e4m3", [("bf16", False), ("fp8", True)])
def test_layer_is_its_calls(kv, e4m3):
    """Two layers on one pool give the bits of the public calls made one by one."""
    cfg = config()
    hidden, ffn = 256, 640
    ws = [weights(hidden, ffn, s, e4m3) for s in (5, 6)]
    a, b = make_pool(cfg, kv, 2), make_pool(cfg, kv, 2)
    layer = wfb.LayerRound(a, ffn)
    to = "e4m3" if e4m3 else None
    shape = (cfg.num_slots, cfg.chunk_tokens, cfg.num_heads, cfg.head_dim)
    for rnd in range(4):
        h = stream(cfg, rnd)
        g = h.clone()
        n = b.live_rows
        for i, w in enumerate(ws):
            layer.run(i, h, w)
            x = g.view(-1, hidden)[:n]
            q_rot = torch.empty(shape, dtype=b.dtype, device="cuda")
            att = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
            y = wfb.add_rms_norm(x, w.norm1, out_dtype=to)
            if e4m3:
                q, k, v = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(3))
                for j, t in enumerate((q, k, v)):
                    t.view(-1, hidden)[:n] = wfb.linear(y, w.w_qkv.span(j * hidden, (j + 1) * hidden))
                b.publish(i, q, k, v, q_rot)
            else:
                full = torch.zeros(cfg.num_slots, cfg.chunk_tokens, hidden, dtype=torch.bfloat16, device="cuda")
                full.view(-1, hidden)[:n] = y
                b.project_publish(i, full, w.w_qkv, q_rot)
            b.attention(i, q_rot, att)
            o = att.view(-1, hidden)[:n].contiguous()
            x = wfb.linear(wfb.quantize_rows(o) if e4m3 else o, w.w_out, w.b_out, residual=x)
            y = wfb.add_rms_norm(x, w.norm2, out_dtype=to)
            x = wfb.linear(wfb.linear(y, w.w_up, w.b_up, act="gelu", out_dtype=to), w.w_down, w.b_down, residual=x)
            g.view(-1, hidden)[:n] = x
        assert torch.equal(h, g)
        a.advance()
        b.advance()


def test_layer_one_slot_at_a_time():
    """Wave Parallelism on one device: each slot's rank publishes, delivers and attends."""
    cfg = config()
    hidden, ffn, slots = 256, 512, cfg.num_slots
    w = weights(hidden, ffn, 9, True)                    # linears and publication in both paths
    whole = make_pool(cfg, "bf16")
    ranks = [make_pool(cfg, "bf16") for _ in range(slots)]
    layer, layers = wfb.LayerRound(whole, ffn), [wfb.LayerRound(p, ffn) for p in ranks]
    for rnd in range(5):
        h = stream(cfg, rnd)
        g = h.clone()
        layer.run(0, h, w)
        live = [r[2] for r in whole.layout() if r[2] is not None]
        for s in live:
            layers[s].publish_slot(0, s, g, w)
        for s in live:
            for r in range(slots):
                if r != s:
                    ranks[s].deliver(0, s, ranks[r])
        for s in live:
            layers[s].attend_slot(0, s, g, w)
        assert torch.equal(h, g)
        for p in (whole, *ranks):
            assert p.check_status() == 0
            p.advance()


def test_layer_refusals():
    cfg = config()
    layer, w, w8 = wfb.LayerRound(make_pool(cfg, "bf16"), 512), weights(256, 512, 1, False), weights(256, 512, 1, True)
    h = stream(cfg, 0)
    for bad in (h.float(), h[:2], h.transpose(0, 1)):
        with pytest.raises(ValueError):
            layer.run(0, bad, w)
    w.w_up = w8.w_up
    with pytest.raises(ValueError, match="all bf16 or all"):
        layer.run(0, h, w)
