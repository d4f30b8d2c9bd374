"""Tensors that want gradients are refused on the GPU by the compiled calls and the Python ones."""
import pytest
import torch
from torch.autograd import forward_ad as fw

import chunk_causal_wavefront_b200 as wfb
from chunk_causal_wavefront_b200 import rows as PR

pytestmark = pytest.mark.gpu


def operands():
    g = torch.Generator(device="cuda").manual_seed(1)
    t = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return dict(x=t(8, 64).bfloat16(), w=t(96, 64).bfloat16(), r=t(8, 96).bfloat16(), s=t(8, 64).bfloat16(),
                bias=t(96), weight=t(64))


CALLS = {
    "linear": (lambda o: wfb.linear(o["x"], o["w"], o["bias"], residual=o["r"]), ("x", "w", "bias", "r")),
    "linear out": (lambda o: wfb.linear(o["x"], o["w"], o["bias"], out=torch.empty_like(o["r"])), ("x", "w", "bias")),
    "norm": (lambda o: wfb.add_rms_norm(o["x"], o["weight"], residual=o["s"]), ("x", "weight", "s")),
    "norm e4m3": (lambda o: wfb.add_rms_norm(o["x"], o["weight"], out_dtype="e4m3"), ("x", "weight")),
    "quantize": (lambda o: wfb.quantize_rows(o["x"]), ("x",)),
}


@pytest.mark.parametrize("compiled", [True, False])
@pytest.mark.parametrize("name", CALLS)
def test_dual_tensors_are_refused(name, compiled, monkeypatch):
    if not compiled:
        monkeypatch.setattr(PR, "_fast", None)
    call, names = CALLS[name]
    with fw.dual_level():
        call(operands())                                       # nothing dual among them
        for n in names:
            o = operands()
            o[n] = fw.make_dual(o[n], torch.ones_like(o[n]))
            for mode in (torch.enable_grad, torch.no_grad):
                with mode(), pytest.raises(ValueError, match="tangents"):
                    call(o)
    call(o)                                                    # the level has ended: a plain tensor again


@pytest.mark.parametrize("compiled", [True, False])
def test_function_transforms_are_refused(compiled, monkeypatch):
    if not compiled:
        monkeypatch.setattr(PR, "_fast", None)
    o = operands()
    f = lambda x: wfb.linear(x, o["w"])
    with pytest.raises(Exception):
        torch.func.jvp(f, (o["x"],), (torch.ones_like(o["x"]),))
    with pytest.raises(Exception):
        torch.func.grad(lambda x: f(x).float().sum())(o["x"])
    with pytest.raises(Exception):
        torch.func.vmap(f)(torch.stack([o["x"], o["x"]]))
