"""The latent-row operators at the edges of their inputs: rows of very different sizes, rows and groups of zeros, values that
are not finite where a token does not see them, query tokens of no sequence, values near the end of fp32's range.

Tolerances, set before any run, as in tests/test_gpu_latent.py.  A key of no weight needs more than that: its score may be so
large that the bound on a score's error, taken over all keys, says nothing.  Its own score is off by at most es_k = 52 * 2^-23
of its sum of magnitudes; where it lies below the log of the sum by more than es_k + 60, its weight is below e^-60 in the
kernel as in the formula, and es is the largest over the other keys."""
import math

import pytest

torch = pytest.importorskip("torch")
import sparse_mla_kv_gb300 as hs  # noqa: E402
import test_gpu_latent as base  # noqa: E402
from test_gpu_latent import D, RD, SCALE, gen, normal  # noqa: E402

pytestmark = pytest.mark.gpu


def expect(q, k, v, mask, scale):
    """base.expect with the score errors of the keys that have weight."""
    n = k.shape[0]
    s = ((q @ k.T) * scale).masked_fill(~mask, -math.inf)
    lse = torch.logsumexp(s, 1)
    low = torch.where(lse == -math.inf, 0, lse)[:, None]
    w = torch.exp(s - low)
    es_k = 52 * 2.0 ** -23 * abs(scale) * (q.abs() @ k.abs().T)
    none = (s + es_k < low - 60) | ~mask
    es = es_k.masked_fill(none, 0).amax(1)
    a = w @ v.abs()
    tol_o = (2.0 ** -7 + 2 * es + 2.0 ** -18 + n * 2.0 ** -27)[:, None] * a
    return w @ v, lse, tol_o, es + 2.0 ** -18 + n * 2.0 ** -27 + 2.0 ** -22 * low[:, 0].abs()


def check(flat, fmt, at, ql, qr, scale, out, lse, seen=None):
    """One token's heads over the rows `at` of a pool's bytes."""
    c, k = base.row_values(flat[at.long()], fmt)
    q = torch.cat([ql, qr], -1).double()
    seen = torch.ones((q.shape[0], len(at)), dtype=torch.bool, device="cuda") if seen is None else seen
    base.close(out, lse, expect(q, k, c, seen, scale))


# --------------------------------------------------------------------------------------------------------------------
# rows of different sizes


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("H", [16, 32, 64])
@pytest.mark.parametrize("power", [20, 24, 30, 40])
@pytest.mark.parametrize("where", [0, 350, 699])
def test_a_large_row_without_weight(fmt, H, power, where):
    """One row 2^power times the size of the others, with a score far below theirs: first, in the middle and last."""
    g = gen(power + where)
    K = 700
    lat, rope = normal(g, 704, D, dtype=torch.float32), normal(g, 704, RD)
    lat[where] *= 2.0 ** power
    lat[where, 3] = -6 * 2.0 ** power
    t = base.rows_bytes(lat, rope, fmt).reshape(11, 64, -1)
    pool = hs.Pool([t])
    rows = torch.arange(K, device="cuda").int()[None].repeat(2, 1).contiguous()
    ql, qr = normal(g, 2, H, D, scale=0.1), normal(g, 2, H, RD)
    ql[:, :, 3] = 8
    out, lse = hs.attend_rows(pool, rows, ql, qr, SCALE)
    flat = t.reshape(704, -1)
    for i in range(2):
        check(flat, fmt, rows[i], ql[i], qr[i], SCALE, out[i], lse[i])
    table, ctx = torch.arange(11, device="cuda").int()[None], torch.tensor([K], device="cuda").int()
    out, lse = hs.attend_pages(pool, table, ctx, ql[:1, None], qr[:1, None], SCALE)
    check(flat, fmt, rows[0], ql[0], qr[0], SCALE, out[0, 0], lse[0, 0])


@pytest.mark.parametrize("H", [8, 40])
@pytest.mark.parametrize("order", ["mixed", "growing", "falling"])
def test_weights_against_sizes(H, order):
    """Row sizes of 2^-16 .. 2^24 with weights that fall with the size, as its 0th to 1.5th power: large rows of small
    weight, small rows that have nearly all of it, and both with equal shares of the result."""
    g = gen(H)
    n = 640
    a = torch.randint(-16, 25, (n,), generator=g, device="cuda").double()
    if order != "mixed":
        a = torch.sort(a, descending=order == "falling").values
    lat = normal(g, n, D).double() * torch.exp2(a)[:, None]
    rope = normal(g, n, RD).double()
    rope[:, 0] = -a * math.log(2)
    t = base.rows_bytes(lat, rope, "fp8").reshape(10, 64, 656)
    pool = hs.Pool([t])
    rows = torch.arange(n, device="cuda").int()[None].repeat(3, 1).contiguous()
    ql, qr = torch.zeros((3, H, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((3, H, RD), dtype=torch.bfloat16, device="cuda")
    qr[:, :, 0] = torch.linspace(0, 1.5, H, device="cuda").bfloat16()
    out, lse = hs.attend_rows(pool, rows, ql, qr, 1.0)
    for i in range(3):
        check(t.reshape(n, 656), "fp8", rows[i], ql[i], qr[i], 1.0, out[i], lse[i])


@pytest.mark.parametrize("H", [8, 64])
@pytest.mark.parametrize("power", [-24, -40])
def test_rows_and_groups_of_zeros(H, power):
    """Appended rows of small values, some of them zero altogether or in one group, whose scale is 1 by definition: what is
    zero has no size.  (A row of zeros takes part in the softmax like any other.)"""
    g = gen(H - power)
    n = 300
    lat, rope = normal(g, n, D, dtype=torch.float32, scale=2.0 ** power), normal(g, n, RD, dtype=torch.float32, scale=2.0 ** power)
    for r in (0, 70, 299):
        lat[r], rope[r] = 0, 0
    lat[5:60:2, 128:256] = 0
    lat[200:230, :384] = 0
    lat[100], rope[101] = 0, 0
    t = torch.zeros((5, 64, 656), dtype=torch.uint8, device="cuda")
    pool = hs.Pool([t])
    turn = torch.cat([torch.ones(1, 32), torch.zeros(1, 32)], 1).cuda()
    at = torch.arange(n, device="cuda").int()
    hs.append_rows(pool, at, lat, rope, torch.zeros(n, dtype=torch.int32, device="cuda"), turn)
    flat = t.reshape(-1, 656)
    assert bool((flat[0, 512:528].view(torch.float32) == 1).all())
    ql, qr = normal(g, 2, H, D, scale=2.0 ** -power), normal(g, 2, H, RD, scale=2.0 ** -power)
    rows = at[None].repeat(2, 1).contiguous()
    out, lse = hs.attend_rows(pool, rows, ql, qr, SCALE)
    for i in range(2):
        check(flat, "fp8", rows[i], ql[i], qr[i], SCALE, out[i], lse[i])
    ctx = torch.tensor([n], device="cuda").int()
    out, lse = hs.attend_pages(pool, torch.arange(5, device="cuda").int()[None], ctx, ql[:1, None], qr[:1, None], SCALE)
    check(flat, "fp8", at, ql[0], qr[0], SCALE, out[0, 0], lse[0, 0])


@pytest.mark.parametrize("K", [1, 5, 70])
def test_fp8_rows_weights_keep_eleven_bits(K):
    """Weights are rounded to fp16 there, 2^-11 of each, so that |out - ref| <= 2^-8 |ref| (its rounding to bf16)
    + (1 + 2^-8) (2^-11 + 2 es + 2^-18 + n 2^-27) A.  The bound that bf16 weights need, 2^-7 A, is up to 14 times as wide
    where terms cancel."""
    g = gen(K)
    pool, tensors = base.make_pool(g, 8, "fp8")
    rows = torch.randint(0, 512, (40, K), generator=g, device="cuda").int()
    ql, qr = normal(g, 40, 64, D), normal(g, 40, 64, RD)
    out, lse = hs.attend_rows(pool, rows, ql, qr, SCALE)
    flat = tensors[0].reshape(-1, 656)
    caught = False
    for i in range(40):
        c, k = base.row_values(flat[rows[i].long()], "fp8")
        q = torch.cat([ql[i], qr[i]], -1).double()
        seen = torch.ones((64, K), dtype=torch.bool, device="cuda")
        ref, _, wide, _ = base.expect(q, k, c, seen, SCALE)
        s = q @ k.T * SCALE
        w = torch.softmax(s, 1)
        a = w @ c.abs()
        tol = 2.0 ** -8 * ref.abs() + (1 + 2.0 ** -8) * (wide - (2.0 ** -7 - 2.0 ** -11) * a)
        assert bool(((out[i].double() - ref).abs() <= tol).all())
        caught |= bool(((w.bfloat16().double() @ c - ref).abs() > tol).any())
    assert caught == (K > 1)   # the check would see weights of 8 bits


# --------------------------------------------------------------------------------------------------------------------
# values that are not finite


@pytest.mark.parametrize("fmt,bad", [("fp8", math.nan), ("bf16", math.nan), ("bf16", math.inf)])
@pytest.mark.parametrize("ctx,P,H", [([130, 65, 64, 5], 4, 16), ([67], 3, 64), ([5000, 700], 4, 20), ([70], 70, 2)])
def test_pages_rows_that_a_position_does_not_see(fmt, bad, ctx, P, H):
    """Values that are not finite in one of the last rows: only the positions that see the row may notice."""
    g = gen(sum(ctx) + P)
    pages = -(-max(ctx) // 64)
    pool, tensors = base.make_pool(g, pages * len(ctx), fmt)
    flat = tensors[0].reshape(-1, base.FMT[fmt])
    first = []   # the first position of each request that sees the bad row
    for r, n in enumerate(ctx):
        p = 1 + r % (P - 1)
        first.append(p)
        lat = normal(g, 1, D, dtype=torch.float32)
        lat[0, 7 + 128 * (r % 4)] = bad
        row = base.rows_bytes(lat, normal(g, 1, RD), fmt, scales=torch.full((1, 4), 1 / 64, device="cuda") if fmt == "fp8" else None)
        flat[r * pages * 64 + n - P + p] = row[0]
    table = torch.arange(pages * len(ctx), device="cuda").int().reshape(len(ctx), pages)
    cl = torch.tensor(ctx, device="cuda").int()
    ql, qr = normal(g, len(ctx), P, H, D), normal(g, len(ctx), P, H, RD)
    out, lse = hs.attend_pages(pool, table, cl, ql, qr, SCALE)
    for r, n in enumerate(ctx):
        for p in range(P):
            if p < first[r]:
                at = r * pages * 64 + torch.arange(n - P + 1 + p, device="cuda")
                check(flat, fmt, at, ql[r, p], qr[r, p], SCALE, out[r, p], lse[r, p])
            elif math.isnan(bad):
                assert bool(torch.isnan(out[r, p]).all()) and bool(torch.isnan(lse[r, p]).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("qn,kn", [([300], [300]), ([40, 200], [170, 456]), ([1, 130, 5], [64, 130, 300]), ([700], [700])])
def test_expanded_values_under_the_causal_mask(qn, kn, bad):
    """Values that are not finite in single dimensions of a few keys: queries before those keys do not notice, and the
    others only in that dimension."""
    H = 2
    g = gen(sum(qn) + sum(kn))
    q, kv, kr = normal(g, sum(qn), H, 192), normal(g, sum(kn), H, 256), normal(g, sum(kn), RD)
    cq, ck = base.cum(qn).tolist(), base.cum(kn).tolist()
    v = kv[..., 128:]
    clean = v.clone()
    marks = []
    for b in range(len(qn)):
        for i, back in enumerate((0, qn[b] // 3, qn[b] // 2, qn[b] - 1)):
            key = max(kn[b] - 1 - back, 0)
            d = (31 * i + 5) % 128
            v[ck[b] + key, i % H, d] = bad
            clean[ck[b] + key, i % H, d] = 0
            marks.append((b, key, i % H, d))
    a = (q[..., :128], q[..., 128:], kv[..., :128], kr)
    out, lse = hs.attend_expanded(*a, v, base.cum(qn), base.cum(kn), SCALE)
    repaired = out.clone()
    for b, key, h, d in marks:
        sees = torch.arange(qn[b], device="cuda") + kn[b] - qn[b] >= key
        at = out[cq[b]:cq[b + 1], h, d]
        assert not bool(torch.isfinite(at[sees]).any())
        if math.isinf(bad):
            assert bool((at[sees] == bad).all())
    want, _ = hs.attend_expanded(*a, clean, base.cum(qn), base.cum(kn), SCALE)
    for b, key, h, d in marks:   # what sees a mark is checked above; the rest against the formula
        sees = torch.arange(qn[b], device="cuda") + kn[b] - qn[b] >= key
        part = repaired[cq[b]:cq[b + 1], h, d]
        part[sees] = want[cq[b]:cq[b + 1], h, d][sees]
    base.check_expanded(*a, clean, cq, ck, SCALE, True, repaired, lse)


def test_expanded_keys_under_the_causal_mask():
    """Keys that are NaN: queries before them do not notice."""
    g = gen(77)
    n, H = 300, 2
    q, kv, kr = normal(g, n, H, 192), normal(g, n, H, 256), normal(g, n, RD)
    kv[200, 0, 5], kr[290, 3] = math.nan, math.nan
    a = [q[..., :128], q[..., 128:], kv[..., :128], kr, kv[..., 128:]]
    out, lse = hs.attend_expanded(*a, base.cum([n]), base.cum([n]), SCALE)
    for h, first in ((0, 200), (1, 290)):
        assert bool(torch.isnan(out[first:, h]).all()) and bool(torch.isnan(lse[first:, h]).all())
        part = [x[:first, h:h + 1] for x in a[:3]] + [kr[:first], a[4][:first, h:h + 1]]
        base.check_expanded(*part, [0, first], [0, first], SCALE, True, out[:first, h:h + 1], lse[:first, h:h + 1])


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
def test_infinite_queries_stay_in_their_head(fmt):
    """An infinite query element makes every score infinite (or NaN), some of them +infinity: NaN by the formula."""
    g = gen(30)
    pool, tensors = base.make_pool(g, 4, fmt)
    rows = torch.randint(0, 256, (2, 200), generator=g, device="cuda").int()
    ql, qr = normal(g, 2, 20, D), normal(g, 2, 20, RD)
    clean = ql.clone()
    ql[0, 3, 100], ql[1, 7, 0], qr[1, 19, 5] = math.inf, -math.inf, math.inf
    out, lse = hs.attend_rows(pool, rows, ql, qr, SCALE)
    bad = torch.zeros((2, 20), dtype=torch.bool, device="cuda")
    bad[0, 3] = bad[1, 7] = bad[1, 19] = True
    assert bool(torch.isnan(out[bad]).all())
    ref, ref_l = hs.attend_rows(pool, rows, clean, qr.where(torch.isfinite(qr), torch.zeros_like(qr)), SCALE)
    assert torch.equal(out[~bad], ref[~bad]) and torch.equal(lse[~bad], ref_l[~bad])


# --------------------------------------------------------------------------------------------------------------------
# values near the end of the range


@pytest.mark.parametrize("order", ["rising", "falling"])
def test_expanded_large_values_and_rising_scores(order):
    """Values of 2^90 and scores that rise by 40 over the keys: no weight may carry a sum past fp32's range."""
    g = gen(91)
    n, H = 500, 2
    ramp = torch.linspace(0, 40, n, device="cuda") if order == "rising" else torch.linspace(40, 0, n, device="cuda")
    qn, qr, kn = normal(g, n, H, 128), normal(g, n, H, RD, scale=0.1), normal(g, n, H, 128, scale=0.05)
    qr[..., 0] = 1
    kr = normal(g, n, RD, scale=0.1)
    kr[:, 0] = ramp.bfloat16()
    v = (normal(g, n, H, 128).double() * 2.0 ** 90).bfloat16()
    for causal in (True, False):
        out, lse = hs.attend_expanded(qn, qr, kn, kr, v, base.cum([n]), base.cum([n]), 1.0, causal=causal)
        base.check_expanded(qn, qr, kn, kr, v, [0, n], [0, n], 1.0, causal, out, lse)


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_rows_large_values_and_rising_scores(fmt, order):
    g = gen(92)
    n, H = 700, 20
    ramp = torch.linspace(0, 40, n, device="cuda") if order == "rising" else torch.linspace(40, 0, n, device="cuda")
    rope = normal(g, n, RD)
    rope[:, 0] = ramp.bfloat16()
    lat = normal(g, n, D).double() * 2.0 ** 90
    t = torch.zeros((11, 64, base.FMT[fmt]), dtype=torch.uint8, device="cuda")
    t.reshape(704, -1)[:n] = base.rows_bytes(lat, rope, "bf16") if fmt == "bf16" else base.rows_bytes(lat, rope * 2.0 ** 80, "fp8")
    pool = hs.Pool([t])
    T = 160   # tokens enough that a CTA has a unit's tiles one after the other
    rows = torch.arange(n, device="cuda").int()[None].repeat(T, 1).contiguous()
    ql, qr = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, H, RD), dtype=torch.bfloat16, device="cuda")
    qr[:, :, 0] = 1.0 if fmt == "bf16" else 2.0 ** -80
    out, lse = hs.attend_rows(pool, rows, ql, qr, 1.0)
    for i in range(0, T, 13):
        check(t.reshape(704, -1), fmt, rows[i], ql[i], qr[i], 1.0, out[i], lse[i])


# --------------------------------------------------------------------------------------------------------------------
# query tokens of no sequence


@pytest.mark.parametrize("cq,ck,covered", [
    ([0, 30, 50], [0, 30, 64], [(0, 50)]),                 # tokens after the last sequence
    ([3, 30, 64], [0, 30, 64], [(3, 64)]),                 # and before the first
    ([0, 32, 64], [0, 40, 65], [(0, 32)]),                 # a sequence whose keys are out of range
    ([0, 40, 30], [0, 40, 64], [(0, 40)]),                 # or whose queries are
    ([0, 20, 20, 64], [0, -3, 20, 64], [(20, 64)]),
    ([70, 80], [0, 64], []),
    ([0], [0], []),                                        # no sequence at all
    ([0, 0, 0], [0, 10, 64], []),                          # only empty ones
])
@pytest.mark.parametrize("H", [1, 3])
def test_expanded_tokens_of_no_sequence(cq, ck, covered, H):
    """They get zeros and -infinity, like a token that sees nothing."""
    g = gen(53)
    n = 64
    q, kv = normal(g, n, H, 192), normal(g, n, H, 256)
    a = (q[..., :128], q[..., 128:], kv[..., :128], normal(g, n, RD), kv[..., 128:])
    out = torch.full((H, n, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, H), 7.0, device="cuda")
    o, _ = hs.attend_expanded(*a, torch.tensor(cq, device="cuda").int(), torch.tensor(ck, device="cuda").int(), SCALE,
                              out=out.transpose(0, 1)[..., :128], lse=lse)
    there = torch.zeros(n, dtype=torch.bool, device="cuda")
    for x, y in covered:
        there[x:y] = True
    assert bool((o[~there] == 0).all()) and bool((lse[~there] == -math.inf).all())
    assert bool(torch.isfinite(o[there]).all()) and bool(torch.isfinite(lse[there]).all())
    assert bool((out[..., 128:] == 7).all())


def test_expanded_many_tokens_of_no_sequence():
    g = gen(54)
    n, H = 5000, 5
    q, kv = normal(g, n, H, 192), normal(g, 100, H, 256)
    a = (q[..., :128], q[..., 128:], kv[..., :128], normal(g, 100, RD), kv[..., 128:])
    cq = [0] + [1000 + 3 * i for i in range(40)]
    cq[1] = 0
    ck = [min(i, 100) for i in range(41)]
    out = torch.full((n, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    c = torch.tensor(cq, device="cuda").int()
    out, lse = hs.attend_expanded(*a, c, torch.tensor(ck, device="cuda").int(), SCALE, out=out, causal=False)
    assert bool((out[cq[-1]:] == 0).all()) and bool((lse[cq[-1]:] == -math.inf).all())
    base.check_expanded(*a, cq, ck, SCALE, False, out, lse)
