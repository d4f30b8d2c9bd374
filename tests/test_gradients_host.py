"""What the row operators and layers say to tensors that want gradients, without a GPU."""
import pytest
import torch
from torch.autograd import forward_ad as fw

import chunk_causal_wavefront_b200 as wfb
from chunk_causal_wavefront_b200.rows import refuse_gradients
from test_layer_host import layer, stream, weights  # noqa: F401  (layer: a fixture)


def test_recording_tensors_and_tangents():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = wfb.E4M3Rows.empty(4, 64, "cpu")
    refuse_gradients("calls", x, None, q)
    wants = x.clone().requires_grad_()
    with pytest.raises(ValueError, match="calls compute no gradients"):
        refuse_gradients("calls", x, wants)
    with torch.no_grad():
        refuse_gradients("calls", x, wants)
    with fw.dual_level():
        refuse_gradients("calls", x, None, q)
        dual = fw.make_dual(x, torch.ones_like(x))
        assert not dual.requires_grad
        for mode in (torch.enable_grad, torch.no_grad):        # neither switches forward mode off
            with mode(), pytest.raises(ValueError, match="tangents"):
                refuse_gradients("calls", None, x, dual)
        refuse_gradients("calls", fw.unpack_dual(dual).primal)
    refuse_gradients("calls", dual)                            # its level has ended


def test_layers_refuse_tangents(layer):  # noqa: F811
    with fw.dual_level():
        w = weights()
        w.w_qkv = fw.make_dual(w.w_qkv, torch.ones_like(w.w_qkv))
        with pytest.raises(ValueError, match="layers compute no tangents"):
            layer.run(0, stream(), w)
        h = fw.make_dual(stream(), torch.ones_like(stream()))
        with pytest.raises(ValueError, match="layers compute no tangents"):
            layer.attend_slot(0, 0, h, weights())
