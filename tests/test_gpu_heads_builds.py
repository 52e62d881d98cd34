"""The operators on pages of grouped heads and read_rows in two other builds of the library.

The bounds-checked build: every case must give its usual results, and no kernel may record a violation (checked after every test by
the fixture in conftest.py).  The build whose bounded waits give up at once (see tests/test_gpu_latent_timeout.py): attend_heads then
runs to its end, reports HS_ERR_TIMEOUT and leaves the device usable; what it writes stays within its outputs."""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import torch
import sparse_mla_kv_gb300 as hs

g = torch.Generator(device="cuda")
g.manual_seed(1)

def normal(*shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()

def guarded(*shape, dtype=torch.bfloat16):
    whole = torch.full((shape[0] + 2, *shape[1:]), 7.0, dtype=dtype, device="cuda")
    return whole, whole[1:-1]

def kept(whole):
    return bool((whole[0] == 7).all()) and bool((whole[-1] == 7).all())

for dim in (64, 128):
    for kv, group, ctx, new in ((2, 4, [900, 70], [1, 1]), (1, 16, [3000], [2]), (8, 8, [500] * 20, [1] * 20), (2, 4, [700, 300], [300, 80]),
                                (1, 1, [5000], [900]), (2, 16, [64, 0, 999], [4, 0, 4]), (4, 2, [50] * 40, [40] * 40),
                                (8, 8, [6000] * 64, [1] * 64)):
        pages = max(-(-c // 64) for c in ctx)
        cache = torch.zeros((len(ctx) * pages, 64, hs.heads_row_bytes(kv, dim)), dtype=torch.uint8, device="cuda")
        cache.view(len(ctx) * pages, -1)[:, kv * 2 * dim * 64:].view(torch.float32)[:] = 1.0
        pool = hs.Pool([cache])
        table = torch.arange(len(ctx) * pages, device="cuda").int().reshape(len(ctx), pages)
        lens = torch.tensor(ctx, device="cuda").int()
        cu = torch.tensor([0, *new], device="cuda").cumsum(0).int()
        n = sum(new)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        wo, out = guarded(n, kv * group, dim)
        wl, lse = guarded(n, kv * group, dtype=torch.float32)
        hs.attend_heads(pool, table, lens, normal(n, kv * group, dim), 0.1, cu_q=cu, out=out, lse=lse, status=status)
        torch.cuda.synchronize()
        # (a copy that has landed when its wait first looks is no wait: few pages a worker may all have, beside the queries)
        sure = max(new) * group > 64 or len(ctx) == 64
        assert int(status) in ((7,) if sure else (0, 7)) and kept(wo) and kept(wl), (dim, kv, group, int(status))
x = torch.ones(1000, device="cuda")
assert float((x + x).sum()) == 2000.0
print("all gave up")
"""


def test_waits_that_run_out_are_reported_and_leave_the_device_usable():
    from sparse_mla_kv_gb300 import _build

    _build.build(variant="timeout")
    p = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=dict(os.environ, HS_LIB_VARIANT="timeout"),
                       capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stdout[-2000:] + p.stderr[-3000:]
    assert "all gave up" in p.stdout


def test_operators_in_the_checked_build():
    from sparse_mla_kv_gb300 import _build

    _build.build(variant="checked")
    p = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "-k", "not past_32_bits",
                        "tests/test_gpu_heads.py"], cwd=ROOT, env=dict(os.environ, HS_LIB_VARIANT="checked"), capture_output=True,
                       text=True, timeout=900)
    assert p.returncode == 0, p.stdout[-3000:] + p.stderr[-2000:]
    assert " passed" in p.stdout and "failed" not in p.stdout
