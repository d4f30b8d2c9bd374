"""Cases and plain forms of the row operators that stand around a layer's round attention.

Rows are tokens. A steady round has S + 1 = 5 slots of C = 4680 tokens, 23400 rows in all;
a rank that owns one slot has 4680; small row counts are last chunks, previews and single
tokens. Hidden sizes are those of the round workloads (1536 and 5120) with a feed-forward
of four times as many features.

Four kinds of case:
  norm      s = x + residual, out = s / sqrt(mean(s^2) + eps) * weight
  quantize  rows to E4M3 codes with a power-of-two scale for each 32 elements, and back
  linear    out = act(x w^T + bias) + residual
  ffn       norm -> linear (GELU) -> linear (+ s), the half of a layer behind attention

E4M3 rows are codes [rows][cols] and one byte e + 127 for each block of 32 columns, e the
smallest integer >= -100 with amax * 2^-e <= 448. The bytes are kept in tiles of 128 rows
x 4 blocks: [rows / 128][blocks / 4][row % 32][row / 32 % 4][block % 4].
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------------------ cases --

def listed():
    return [
        # A single token's norm between two layers: latency alone.
        dict(name="norm_token", op="norm", rows=1, cols=1536, dtype="bf16", to="same", residual=True),
        # Every token of a steady round at hidden 1536, in the residual stream's type.
        dict(name="norm_round", op="norm", rows=23400, cols=1536, dtype="bf16", to="same", residual=True),
        # The same at hidden 5120, handed to 8-bit products.
        dict(name="norm_round_e4m3", op="norm", rows=23400, cols=5120, dtype="bf16", to="e4m3", residual=True),
        # Rows of an fp32 pool with an odd width: no vector loads.
        dict(name="norm_odd_f32", op="norm", rows=771, cols=1001, dtype="f32", to="same", residual=False),
        # One head group's worth of attention output, small.
        dict(name="quantize_small", op="quantize", rows=333, cols=1536, dtype="bf16"),
        # All tokens of a round before an 8-bit output projection.
        dict(name="quantize_round", op="quantize", rows=23400, cols=5120, dtype="bf16"),
        # One token through the first feed-forward product: the weights' bytes bound it.
        dict(name="linear_token", op="linear", rows=1, k=1536, n=6144, dtype="bf16", act="gelu", bias=True, residual=False),
        # A few tokens against 8-bit weights.
        dict(name="linear_few_e4m3", op="linear", rows=24, k=5120, n=5120, dtype="e4m3", act="none", bias=True, residual=True),
        # A ragged middle size: neither rows nor features fill tiles.
        dict(name="linear_ragged", op="linear", rows=1111, k=1544, n=1000, dtype="bf16", act="silu", bias=True, residual=True),
        # The output projection behind a round's attention, into the residual stream.
        dict(name="linear_out", op="linear", rows=23400, k=1536, n=1536, dtype="bf16", act="none", bias=True, residual=True),
        # One rank's chunk through the wide feed-forward product.
        dict(name="linear_wide", op="linear", rows=4680, k=5120, n=20480, dtype="bf16", act="gelu", bias=True, residual=False),
        # A round's feed-forward half in 8 bits.
        dict(name="ffn_round_e4m3", op="ffn", rows=23400, k=1536, n=6144, dtype="e4m3"),
    ]


_MOST = 4680 * 5120 * 20480   # products of the largest listed case


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "linear", "linear", "ffn"])
    rows = _log(rng, 1, 23400)
    if op == "norm":
        to = rng.choice(["same", "e4m3"])
        cols = 32 * _log(rng, 2, 160) if to == "e4m3" else _log(rng, 17, 5200)
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "f32"]), to=to, residual=rng.random() < 0.7)
    if op == "quantize":
        return dict(op=op, rows=rows, cols=32 * _log(rng, 2, 200), dtype=rng.choice(["bf16", "f32"]))
    if op == "linear":
        dtype = rng.choice(["bf16", "e4m3"])
        k = 8 * _log(rng, 8, 640) if dtype == "bf16" else 32 * _log(rng, 2, 160)
        n = _log(rng, 33, 20480)
        rows = max(1, min(rows, _MOST // (k * n)))
        return dict(op=op, rows=rows, k=k, n=n, dtype=dtype, act=rng.choice(["none", "gelu", "silu"]), bias=rng.random() < 0.7, residual=rng.random() < 0.5)
    k, n = 32 * _log(rng, 4, 64), 32 * _log(rng, 4, 256)
    rows = max(1, min(rows, _MOST // (2 * k * n)))
    return dict(op=op, rows=rows, k=k, n=n, dtype=rng.choice(["bf16", "e4m3"]))


# ----------------------------------------------------------------------------- inputs --

_T = {"bf16": torch.bfloat16, "f32": torch.float32}


def _activations(g, rows, cols, scale=1.0):
    """N(0, 1) rows with one feature in twenty eight times as large, as activations have."""
    x = torch.randn(rows, cols, generator=g, device="cuda") * scale
    big = torch.rand(cols, generator=g, device="cuda") < 0.05
    return x * torch.where(big, 8.0, 1.0)


def _tile(e):
    """Block exponents [rows][blocks] as the tiled bytes e + 127."""
    rows, blocks = e.shape
    rt, kt = -(-rows // 128), -(-blocks // 4)
    s = torch.zeros(rt * 128, kt * 4, dtype=torch.uint8, device=e.device)
    s[:rows, :blocks] = (e + 127).to(torch.uint8)
    return s.view(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _untile(s, rows, cols):
    """Tiled bytes as the factors 2^e, [rows][blocks] in 32 bits."""
    blocks = cols // 32
    rt, kt = -(-rows // 128), -(-blocks // 4)
    b = s.view(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:rows, :blocks]
    return torch.ldexp(torch.ones(1, device=s.device), b.to(torch.int32) - 127)


def _codes(v):
    """E4M3 codes and block exponents of rows in 32 bits."""
    rows, cols = v.shape
    b = v.view(rows, cols // 32, 32)
    m, p = torch.frexp(b.abs().amax(-1))
    e = torch.where(m <= 0.875, p - 9, p - 8).clamp_min(-100)
    return torch.ldexp(b, -e.unsqueeze(-1)).to(torch.float8_e4m3fn).view(rows, cols), e


def _params(g, n, scale=0.1, about=0.0):
    return about + scale * torch.randn(n, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, op, rows = dict(case), case["op"], case["rows"]
    if op == "norm":
        t = _T[c["dtype"]]
        return dict(c, x=_activations(g, rows, c["cols"]).to(t), weight=_params(g, c["cols"], about=1.0),
                    r=_activations(g, rows, c["cols"], 2.0).to(t) if c["residual"] else None)
    if op == "quantize":
        return dict(c, x=_activations(g, rows, c["cols"]).to(_T[c["dtype"]]))
    k, n = c["k"], c["n"]

    def operand(v):
        v = v.to(torch.bfloat16)
        if c["dtype"] == "bf16":
            return v
        codes, e = _codes(v.float())
        return codes, _tile(e)

    def weights(features, terms):
        return operand(torch.randn(features, terms, generator=g, device="cuda") / math.sqrt(terms))

    if op == "linear":
        return dict(c, x=operand(_activations(g, rows, k)), w=weights(n, k),
                    b=_params(g, n) if c["bias"] else None,
                    r=torch.randn(rows, n, generator=g, device="cuda").bfloat16() if c["residual"] else None)
    return dict(c, x=_activations(g, rows, k).bfloat16(), r=_activations(g, rows, k, 2.0).bfloat16(),
                weight=_params(g, k, about=1.0), w1=weights(n, k), b1=_params(g, n), w2=weights(k, n), b2=_params(g, k))


# ------------------------------------------------------------------- the framework's --

def _run_own(s):
    import chunk_causal_wavefront_b200 as wf

    op = s["op"]
    if op == "norm":
        to = "e4m3" if s["to"] == "e4m3" else None
        if s["r"] is None:
            y, total = wf.add_rms_norm(s["x"], s["weight"], eps=EPS, out_dtype=to), None
        else:
            y, total = wf.add_rms_norm(s["x"], s["weight"], residual=s["r"], eps=EPS, out_dtype=to)
        return {"y": y.dequantize() if to else y, "sum": total}
    if op == "quantize":
        return {"y": wf.quantize_rows(s["x"]).dequantize()}
    e4m3 = s["dtype"] == "e4m3"

    def operand(t):
        return wf.E4M3Rows(*t) if e4m3 else t

    if op == "linear":
        return {"y": wf.linear(operand(s["x"]), operand(s["w"]), s["b"], act=s["act"], residual=s["r"])}
    to = "e4m3" if e4m3 else None
    y, total = wf.add_rms_norm(s["x"], s["weight"], residual=s["r"], eps=EPS, out_dtype=to)
    hidden = wf.linear(y, operand(s["w1"]), s["b1"], act="gelu", out_dtype=to)
    return {"y": wf.linear(hidden, operand(s["w2"]), s["b2"], residual=total), "sum": total}


# ------------------------------------------------------------------------ plain forms --

def _norm(x, r, weight):
    total = x.float() if r is None else x.float() + r.float()
    return total, total * torch.rsqrt((total * total).mean(-1, keepdim=True) + EPS) * weight


def _values(codes, e):
    rows, cols = codes.shape
    return torch.ldexp(codes.float().view(rows, cols // 32, 32), e.unsqueeze(-1)).view(rows, cols)


def _wide(t):
    if isinstance(t, tuple):
        codes, s = t
        rows, cols = codes.shape
        return (codes.float().view(rows, cols // 32, 32) * _untile(s, rows, cols).unsqueeze(-1)).view(rows, cols)
    return t.float()


def _act(v, act):
    if act == "gelu":
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v / (1 + torch.exp(-v)) if act == "silu" else v


def _linear(x, w, b, act, r):
    v = x @ w.t()
    if b is not None:
        v = v + b
    v = _act(v, act)
    return v if r is None else v + r.float()


def run(state):
    if own:
        return _run_own(state)
    s, op = state, state["op"]
    if op == "norm":
        total, y = _norm(s["x"], s["r"], s["weight"])
        y = _values(*_codes(y)).bfloat16() if s["to"] == "e4m3" else y.to(s["x"].dtype)
        return {"y": y, "sum": None if s["r"] is None else total.to(s["x"].dtype)}
    if op == "quantize":
        return {"y": _values(*_codes(s["x"].float())).bfloat16()}
    if op == "linear":
        return {"y": _linear(_wide(s["x"]), _wide(s["w"]), s["b"], s["act"], s["r"]).bfloat16()}
    total, y = _norm(s["x"], s["r"], s["weight"])
    total = total.bfloat16()
    y = _values(*_codes(y)) if s["dtype"] == "e4m3" else y.bfloat16().float()
    h = _linear(y, _wide(s["w1"]), s["b1"], "gelu", None)
    h = _values(*_codes(h)) if s["dtype"] == "e4m3" else h.bfloat16().float()
    return {"y": _linear(h, _wide(s["w2"]), s["b2"], "none", total).bfloat16(), "sum": total}


# ------------------------------------------------------------------------------- work --

def work(case):
    c, rows = case, case["rows"]
    if c["op"] in ("norm", "quantize"):
        each = rows * c["cols"]
        size = 4 if c["dtype"] == "f32" else 2
        back = 1 + 1 / 32
        if c["op"] == "quantize":
            # the rows read, codes and scales written
            return {"bytes": each * (size + back), "flops": 2 * each}
        moved = size * (3 if c["residual"] else 1) + (back if c["to"] == "e4m3" else size)
        return {"bytes": each * moved + 4 * c["cols"], "flops": 5 * each}
    k, n = c["k"], c["n"]
    one = 2 if c["dtype"] == "bf16" else 1 + 1 / 32
    if c["op"] == "linear":
        out = 2 * rows * n * (2 if c["residual"] else 1) + (4 * n if c["bias"] else 0)
        return {"bytes": one * k * (rows + n) + out, "flops": 2 * rows * k * n}
    # x, residual in; sum and y out; both weights; what passes between the products stays inside
    return {"bytes": 2 * 4 * rows * k + one * 2 * k * n + 4 * (2 * k + n), "flops": 4 * rows * k * n}


# ------------------------------------------------------------------- exact, in 64 bits --

def _e4m3_64(v):
    """The values that E4M3 codes with block scales stand for, by their definition."""
    blocks = v.reshape(v.shape[0], -1, 32)
    top = blocks.abs().amax(dim=2, keepdim=True)
    # the smallest power of two that brings the largest value to 448 or below
    step = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448)) - 1)
    for _ in range(3):
        step = torch.where(top > 448 * step, step * 2, step)
    step = torch.where(top > 0, step, torch.zeros_like(step)).clamp_min(2.0 ** -100)
    a = blocks / step
    # three bits behind the leading one, subnormal below 2^-6
    grain = torch.exp2(torch.floor(torch.log2(a.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(a / grain) * grain * step).reshape(v.shape)


def _held_64(t):
    if not isinstance(t, tuple):
        return t.double()
    codes, s = t
    rows, cols = codes.shape
    i = torch.arange(rows, device=s.device).view(-1, 1)
    j = torch.arange(cols // 32, device=s.device).view(1, -1)
    tiles = -(-(cols // 32) // 4)
    at = (((i // 128) * tiles + j // 4) * 32 + i % 32) * 16 + (i % 128 // 32) * 4 + j % 4
    scale = torch.exp2(s[at].double() - 127)
    return codes.double() * scale.repeat_interleave(32, dim=1)


def exact(case, seed):
    s = prepare(case, seed)

    def norm(v, weight):
        return v / torch.sqrt(v.square().sum(1, keepdim=True) / v.shape[1] + EPS) * weight.double()

    def gelu(v):
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))

    def total():
        return s["x"].double() + (0 if s["r"] is None else s["r"].double())

    if s["op"] == "norm":
        y = norm(total(), s["weight"])
        return {"y": _e4m3_64(y) if s["to"] == "e4m3" else y, "sum": None if s["r"] is None else total()}
    if s["op"] == "quantize":
        return {"y": _e4m3_64(s["x"].double())}
    if s["op"] == "linear":
        v = torch.mm(_held_64(s["x"]), _held_64(s["w"]).T)
        v = v if s["b"] is None else v + s["b"].double()
        v = gelu(v) if s["act"] == "gelu" else v * torch.sigmoid(v) if s["act"] == "silu" else v
        return {"y": v if s["r"] is None else v + s["r"].double()}
    held = _e4m3_64 if s["dtype"] == "e4m3" else lambda v: v.bfloat16().double()
    y = held(norm(total(), s["weight"]))
    h = held(gelu(torch.mm(y, _held_64(s["w1"]).T) + s["b1"].double()))
    # the residual stream is held in its own type between the two halves
    return {"y": torch.mm(h, _held_64(s["w2"]).T) + s["b2"].double() + total().bfloat16().double(), "sum": total()}
