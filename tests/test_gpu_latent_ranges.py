"""The latent-row operators where magnitudes, signs and lengths range widely, against their formulas in 64 bits.

Tolerances: those of tests/test_gpu_latent.py.  They hold for every row format: the operands keep their values (scales are
powers of two within a row's range of the product's type), so only sums, weights and results round."""
import pytest

torch = pytest.importorskip("torch")
import sparse_mla_kv_gb300 as hs  # noqa: E402
import test_gpu_latent as base  # noqa: E402
from test_gpu_latent import D, RD, SCALE, gen, normal  # noqa: E402

pytestmark = pytest.mark.gpu


def powers(g, lo, hi, *shape):
    return torch.exp2(torch.randint(lo, hi + 1, shape, generator=g, device="cuda").double())


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("H", [4, 24, 64])
@pytest.mark.parametrize("order", ["mixed", "growing", "falling"])
def test_rows_of_every_magnitude(fmt, H, order):
    """Keys, groups of a key, rotated parts and queries of 2^-12 .. 2^12 times the usual size: the factors that bring
    operands into range move within a unit and differ between its columns."""
    g = gen(H * 3 + len(order))
    blocks, K = 12, 700
    n = blocks * 64
    key = powers(g, -6, 6, n)
    if order != "mixed":
        key = torch.sort(key, descending=order == "falling").values
    lat = normal(g, n, 4, 128).double() * (key[:, None] * powers(g, -4, 4, n, 4))[..., None]
    rope = normal(g, n, RD).double() * (key * powers(g, -6, 6, n))[:, None]
    t = base.rows_bytes(lat.reshape(n, D), rope, fmt).reshape(blocks, 64, -1)
    pool = hs.Pool([t])
    rows = torch.sort(torch.randperm(n, generator=g, device="cuda")[:K]).values.int()[None].repeat(2, 1).contiguous()
    q = normal(g, 2, H, D + RD).double() * powers(g, -12, 6, 2, H)[..., None]
    ql, qr = q[..., :D].bfloat16(), q[..., D:].bfloat16()
    out, lse = hs.attend_rows(pool, rows, ql, qr, SCALE / 64)
    base.check_rows([t], fmt, rows, ql, qr, SCALE / 64, out, lse)


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
def test_rows_of_a_negative_scale(fmt):
    g = gen(5)
    pool, tensors = base.make_pool(g, 8, fmt)
    rows = torch.randint(0, 512, (3, 200), generator=g, device="cuda").int()
    ql, qr = normal(g, 3, 9, D), normal(g, 3, 9, RD)
    out, lse = hs.attend_rows(pool, rows, ql, qr, -SCALE)
    base.check_rows(tensors, fmt, rows, -ql, -qr, SCALE, out, lse)
    out, lse = hs.attend_rows(pool, rows, ql, qr, 0.0)
    base.check_rows(tensors, fmt, rows, ql, qr, 0.0, out, lse)


@pytest.mark.parametrize("fmt,ctx,P,H", [("fp8", [70001], 2, 16), ("fp8", [40000, 1, 3, 129], 4, 64), ("bf16", [50003], 1, 33)])
def test_long_pages(fmt, ctx, P, H):
    g = gen(P + H)
    pages = -(-max(ctx) // 64)
    pool, tensors = base.make_pool(g, pages + 7, fmt)
    table = torch.stack([torch.randperm(pages + 7, generator=g, device="cuda")[:pages] for _ in ctx]).int()
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    ql, qr = normal(g, len(ctx), P, H, D), normal(g, len(ctx), P, H, RD)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = hs.attend_pages(pool, table, c, ql, qr, SCALE, status=status)
    assert int(status) == 0
    base.check_pages(tensors, fmt, table, ctx, ql, qr, SCALE, out, lse)


@pytest.mark.parametrize("n", [1, 63, 152, 153, 500])
@pytest.mark.parametrize("H", [7, 48, 200])
def test_units_and_runs_of_every_shape(n, H):
    """One tile a unit, units of one CTA and of several, more column groups than one: the shared places of queries, weights
    and sums change hands at every unit."""
    g = gen(n + H)
    pool, tensors = base.make_pool(g, 8, "fp8")
    K = 40 if n > 60 else 1000
    rows = torch.randint(-20, 512, (n, K), generator=g, device="cuda").clamp(min=-1).int()
    ql, qr = normal(g, n, H, D), normal(g, n, H, RD)
    out, lse = hs.attend_rows(pool, rows, ql, qr, SCALE)
    base.check_rows(tensors, "fp8", rows, ql, qr, SCALE, out, lse)


def expanded_inputs(g, Tq, Tk, H):
    kv, q = normal(g, Tk, H, 256), normal(g, Tq, H, 192)
    return q[..., :128], q[..., 128:], kv[..., :128], normal(g, Tk, RD), kv[..., 128:]


@pytest.mark.parametrize("scale", [-SCALE, 0.0])
@pytest.mark.parametrize("causal", [True, False])
def test_expanded_of_other_signs(scale, causal):
    qn, kn = [130, 7], [300, 140]
    a = expanded_inputs(gen(3), sum(qn), sum(kn), 3)
    out, lse = hs.attend_expanded(*a, base.cum(qn), base.cum(kn), scale, causal=causal)
    b = (-a[0], -a[1], *a[2:]) if scale < 0 else a
    base.check_expanded(*b, base.cum(qn).tolist(), base.cum(kn).tolist(), abs(scale), causal, out, lse)


@pytest.mark.parametrize("seqs,H", [(33, 1), (70, 2), (300, 1)])
def test_expanded_of_many_sequences(seqs, H):
    g = gen(seqs)
    qn = torch.randint(0, 40, (seqs,), generator=g, device="cuda").tolist()
    kn = [n + e for n, e in zip(qn, torch.randint(0, 30, (seqs,), generator=g, device="cuda").tolist())]
    qn[seqs // 2], kn[seqs // 2] = 300, 310
    a = expanded_inputs(g, sum(qn), sum(kn), H)
    out, lse = hs.attend_expanded(*a, base.cum(qn), base.cum(kn), SCALE)
    base.check_expanded(*a, base.cum(qn).tolist(), base.cum(kn).tolist(), SCALE, True, out, lse)


def test_expanded_shared_heads():
    """Keys and values that all heads share (a stride of 0 between heads)."""
    g = gen(9)
    q = normal(g, 70, 4, 192)
    k, v, kr = (normal(g, 200, 1, 128).expand(-1, 4, -1) for _ in range(2)), None, normal(g, 200, RD)
    k, v = k
    a = (q[..., :128], q[..., 128:], k, kr, v)
    out, lse = hs.attend_expanded(*a, base.cum([70]), base.cum([200]), SCALE)
    base.check_expanded(*a, [0, 70], [0, 200], SCALE, True, out, lse)


def test_more_refusals():
    g = gen(1)
    pool, _ = base.make_pool(g, 4, "fp8")
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    before = hs.launch_count()

    def refused(f, *a, **k):
        with pytest.raises(hs.HSError) as e:
            f(*a, **k)
        assert e.value.code == 1

    q, qr, kn, kr, v = expanded_inputs(g, 8, 8, 2)
    cu = base.cum([8])
    for i in range(5):  # one row for all tokens
        a = [q, qr, kn, kr, v]
        a[i] = a[i][:1].expand(8, *a[i].shape[1:])
        refused(hs.attend_expanded, *a, cu, cu, SCALE)
    # more pages than 2^30 tokens, and more tiles of a request than 32 bits count
    ql, qrr = normal(g, 1, 1, 1, D), normal(g, 1, 1, 1, RD)
    refused(hs.attend_pages, pool, one.reshape(1, 1).expand(1, 2 ** 24 + 1).contiguous(), one, ql, qrr, SCALE)
    q9, r9 = normal(g, 1, 1, 1, D).expand(1, 513, 1024, D), normal(g, 1, 1, 1, RD).expand(1, 513, 1024, RD)
    out = torch.empty((1, 513, 1024, D), dtype=torch.bfloat16, device="cuda")
    refused(hs.attend_pages, pool, one.reshape(1, 1).expand(1, 2 ** 18).contiguous(), one, q9, r9, SCALE, out=out)
    assert hs.launch_count() == before


def test_own_buffers_on_another_stream():
    """Outputs and workspaces made by calls on a side stream: many in flight, while the current stream keeps allocating,
    writing and freeing memory of the same sizes."""
    g = gen(21)
    pool, tensors = base.make_pool(g, 16, "fp8")
    n, K, H = 32, 500, 16
    rows = torch.randint(0, 1024, (n, K), generator=g, device="cuda").int()
    ql, qr = normal(g, n, H, D), normal(g, n, H, RD)
    want = hs.attend_rows(pool, rows, ql, qr, SCALE)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, held = [], []
    for _ in range(20):
        got.append(hs.attend_rows(pool, rows, ql, qr, SCALE, stream=side))
        churn = [torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0),
                 torch.full((hs.alloc_attend_workspace().numel(),), 255, dtype=torch.uint8, device="cuda")]
        held.append(churn[0].clone())
        del churn
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(x, want[1]) for o, x in got)
    assert all(bool((x == 7).all()) for x in held)
