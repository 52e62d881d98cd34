"""The example layer element by element: every result within the example's BOUND of 64 bits, and mistakes of a single row
beyond it.

BOUND is the tolerance of tests/test_gpu_latent.py relative to A = sum_k w |v|: (2^-7 + 2 es + 2^-18 + n 2^-27) with
es = 52 * 2^-23 * scale * max_k sum |q||k|.  Queries and keys are about normal (absorbed queries 0.5 normal over 512 dimensions), so
that scale * sum |q||k| stays below 30, es below 2^-12 and the whole below 2^-7 + 2^-10.  A row of another token in a
reference changes it by w_k |v' - v|: with up to 334 rows, w_k reaches 0.01 in some head and |v' - v| 3 in some dimension, some four
times BOUND where A is about 0.8."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sparse_mla_layer.py")


def example():
    spec = importlib.util.spec_from_file_location("sparse_mla_layer", PATH)
    layer = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(layer)
    return layer


@pytest.mark.parametrize("kw", [{}, {"prompts": (64, 1, 200), "offloaded": (2,), "heads": 5, "topk": 32, "seed": 1},
                                {"prompts": (500, 129), "offloaded": (0, 1), "heads": 64, "topk": 128, "seed": 2, "steps": 3},
                                {"prompts": (128, 300), "offloaded": (0,), "heads": 16, "topk": 128, "seed": 3}])
def test_every_element_is_within_the_bound(kw):
    layer = example()
    worst = layer.run(**kw)
    assert all(x < layer.BOUND for x in worst.values()), worst
    assert worst["attend_expanded"] > 0 and worst["attend_rows"] > 0


@pytest.mark.parametrize("mistake", ["another row", "a row less", "another head"])
def test_mistakes_of_a_single_row_are_beyond_the_bound(mistake):
    layer = example()
    right = layer.plain

    def wrong(q, k, v, scale, seen=None):
        if mistake == "another row":      # the reference reads its first row in the place of its middle one
            k, v = k.clone(), v.clone()
            k[len(k) // 2], v[len(v) // 2] = k[0], v[0]
        elif mistake == "a row less":     # and does not see the last row
            seen = torch.ones((len(q), len(k)), dtype=torch.bool, device=q.device) if seen is None else seen.clone()
            seen[-1, -1] = False
        else:
            q = q.roll(1, 1)
        return right(q, k, v, scale, seen)

    layer.plain = wrong
    worst = layer.run()
    assert all(x > layer.BOUND for x in worst.values()), worst
