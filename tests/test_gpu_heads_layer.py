"""The example layer with grouped heads: append, attend, read, offload and prefix reuse together, every result within the example's
BOUND of 64 bits.

BOUND: the result's rounding to bf16 is 2^-8 of it at most, a weight's to fp16 2^-11; scores are sums of up to 128 products of about
normal numbers, times dim^-0.5: magnitudes below 30, errors below (128 / 16 + 16) 2^-23 30 < 2^-13; sums and exponentials are below
2^-16.  2^-8 + 2^-11 + 2 * 2^-13 + ... < 2^-8 + 2^-10."""
import importlib.util
import os

import pytest

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "grouped_heads_layer.py")


@pytest.mark.parametrize("kw", [{}, {"prompts": (64, 1, 200), "chunk": 100, "kv": 3, "group": 1, "dim": 64, "seed": 1},
                                {"prompts": (700, 640), "chunk": 333, "kv": 1, "group": 7, "seed": 2, "steps": 3, "drafts": 2},
                                {"prompts": (129, 63, 65, 128), "chunk": 64, "kv": 2, "group": 16, "dim": 64, "seed": 3, "drafts": 1}])
def test_layer(kw):
    spec = importlib.util.spec_from_file_location("grouped_heads_layer", PATH)
    layer = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(layer)
    worst = layer.run(**kw)
    assert all(0 < x < layer.BOUND for x in worst.values()), worst
