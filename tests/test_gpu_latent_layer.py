"""The example layer (append, expanded and absorbed attention with the resolver and the offload) against 64 bits.

Tolerance, set before any run: every result is off by at most (2^-7 + 2 es + 2^-18 + n 2^-27) A with A = sum_k w |v|
(tests/test_gpu_latent.py); here es < 2^-12, and A, a mean of the values' magnitudes, is at most the largest |v|.  The
values are about normal, |v| < 5.5, and a layer's largest result exceeds 0.35, so an error is below
5.5 / 0.35 * (2^-7 + 2^-11) < 0.14 of it; a wrong row, mask or head changes results by as much as they are."""
import importlib.util
import os

import pytest

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sparse_mla_layer.py")


@pytest.mark.parametrize("kw", [{}, {"prompts": (64, 1, 200), "offloaded": (2,), "heads": 5, "topk": 32, "seed": 1},
                                {"prompts": (500, 129), "offloaded": (0, 1), "heads": 64, "topk": 128, "seed": 2, "steps": 3}])
def test_layer(kw):
    spec = importlib.util.spec_from_file_location("sparse_mla_layer", PATH)
    layer = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(layer)
    worst = layer.run(**kw)
    called = {"attend_expanded", "attend_rows"} | ({"attend_pages"} if len(kw.get("offloaded", (0, 2))) < len(kw.get("prompts", "abc")) else set())
    for name in called:
        assert 0 < worst[name] < 0.14, worst
