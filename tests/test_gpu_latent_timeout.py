"""Bounded waits of the attention kernels that run out.

libhs_timeout.so is the library with a limit of zero: a wait that is not over at its first look gives up, as one would after
two seconds of a copy or a product that does not end.  The kernels then run to their end (their own copies and products in
flight are waited for with the usual limit), report HS_ERR_TIMEOUT and leave the device usable; what they write stays within
their outputs.  In a child process, because the library is chosen when it is loaded."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import sys
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

for fmt, size in (("fp8", 656), ("bf16", 1152)):
    pool = hs.Pool([torch.zeros((40, 64, size), dtype=torch.uint8, device="cuda")])
    for n, K, H in ((1, 64, 8), (40, 600, 64), (3, 2000, 24)):
        rows = torch.randint(-1, 2560, (n, K), generator=g, device="cuda").int()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        wo, out = guarded(n, H, 512)
        wl, lse = guarded(n, H, dtype=torch.float32)
        hs.attend_rows(pool, rows, normal(n, H, 512), normal(n, H, 64), 0.07, out=out, lse=lse, status=status)
        torch.cuda.synchronize()
        assert int(status) == 7 and kept(wo) and kept(wl), (fmt, n, int(status))
    table = torch.arange(40, device="cuda").int().reshape(4, 10)
    ctx = torch.tensor([640, 1, 300, 65], device="cuda").int()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    wo, out = guarded(4, 3, 30, 512)
    hs.attend_pages(pool, table, ctx, normal(4, 3, 30, 512), normal(4, 3, 30, 64), 0.07, out=out, status=status)
    torch.cuda.synchronize()
    assert int(status) == 7 and kept(wo)
for qn, kn, causal in (([1], [1], True), ([300, 40, 700], [300, 900, 700], True), ([500], [900], False), ([20] * 200, [90] * 200, True)):
    H = 5
    cu = [torch.tensor([0, *x], device="cuda").cumsum(0).int() for x in (qn, kn)]
    Tq, Tk = sum(qn), sum(kn)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    wo, out = guarded(Tq, H, 128)
    wl, lse = guarded(Tq, H, dtype=torch.float32)
    hs.attend_expanded(normal(Tq, H, 128), normal(Tq, H, 64), normal(Tk, H, 128), normal(Tk, 64), normal(Tk, H, 128), *cu, 0.07,
                       causal=causal, out=out, lse=lse, status=status)
    torch.cuda.synchronize()
    assert int(status) == 7 and kept(wo) and kept(wl), (qn, int(status))
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
