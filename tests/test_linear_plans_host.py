"""Arguments of the products' test hook, without a GPU."""
import pytest

from chunk_causal_wavefront_b200 import wf as W


@pytest.mark.parametrize("args", [
    dict(kernel=-1), dict(kernel=3), dict(kernel=1, tile=0, split=1), dict(kernel=1, tile=48, split=1),
    dict(kernel=1, tile=64, split=3), dict(kernel=1, tile=64, split=16), dict(kernel=2, tile=128),
    dict(kernel=0, stall_k_block=-2), dict(kernel=0, wait_limit_cycles=999),
    dict(kernel=0, wait_limit_cycles=2000000001)])
def test_hook_arguments(args):
    assert W.wf_rows_debug_next_linear(**args) == W.WF_ERR_INVALID_ARG
