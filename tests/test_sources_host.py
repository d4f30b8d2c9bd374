"""The kernels' headers hold nothing that no kernel uses."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunk_causal_wavefront_b200", "csrc")


def test_every_device_helper_is_used():
    text = {f: re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read()) for f in os.listdir(CSRC)}
    everything = "\n".join(text.values())
    for f, src in text.items():
        if not f.endswith(".cuh"):
            continue
        for name in re.findall(r"__device__[^;{}()]*?\b(\w+)\(", src):
            assert len(re.findall(rf"\b{name}\b", everything)) > 1, (f, name)
