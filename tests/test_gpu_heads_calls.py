"""Calls of the operators on pages of grouped heads that the header allows and that are all edge (no requests at all), and some that it does not."""
import math

import pytest

torch = pytest.importorskip("torch")
import sparse_mla_kv_gb300 as hs  # noqa: E402
from test_gpu_heads import gen, i32, make, normal, same  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 63, 64, 1000])
def test_tokens_that_no_request_has_because_there_is_none(n):
    """Offsets of no request: the call does nothing, however many tokens the tensors have."""
    g = gen(41)
    kv, dim = 2, 128
    pool, cache, _ = make(g, [200], kv, dim)
    was = cache.clone()
    none, cu, status = torch.empty((0, 4), dtype=torch.int32, device="cuda"), i32([0]), i32([0])
    k, v = normal(g, n, kv, dim), normal(g, n, kv, dim)
    hs.append_heads(pool, none, i32([]), k, v, cu=cu, status=status)
    same(cache, was)
    a, b = k.clone(), v.clone()
    hs.read_heads(pool, none, i32([]), cu, n, dim, k=a, v=b, status=status)
    hs.read_heads(pool, none, None, cu, n, dim, k=a, v=b, status=status)
    same(a, k)
    same(b, v)
    assert int(status) == 0


def test_scales_that_are_refused():
    """Those whose product with log2(e) is not a finite number of 32 bits, with nothing launched; the largest is taken."""
    g = gen(42)
    pool, _, table = make(g, [70], 1, 64)
    q = normal(g, 1, 1, 64)
    before = hs.launch_count()
    for scale in (math.inf, -math.inf, math.nan, 2.0 ** 127 * 1.001, -3e38):
        with pytest.raises(hs.HSError):
            hs.attend_heads(pool, table, i32([70]), q, scale)
    assert hs.launch_count() == before
    out, lse = hs.attend_heads(pool, table, i32([70]), q * 2.0 ** -100, 2.0 ** 127)
    assert bool(out.isfinite().all()) and bool(lse.isfinite().all())
