"""The latent-row operators (append, absorbed and expanded attention) against their formulas in 64 bits.

Tolerances, set before any run.  Scores are sums of 576 (192) products of bf16 values accumulated in fp32 in steps of
16: at most 36 + 16 additions, each off by at most 2^-23 of the sum of magnitudes, so
es = 52 * 2^-23 * scale * max_k sum |q||c| bounds a score's error.  A softmax weight is then off by a factor of 1 +- 2 es
(its own score and the sum's), by 2^-20 for the exponential, and by 2^-8 for its rounding to bf16 (8 significant bits:
half a unit in the last place is up to 2^-8 of the value); the sums over n keys add at most n / 16 * 2^-23; the result is
rounded to bf16 once (2^-8).  With A = sum_k w |c|:
|out - ref| <= (2^-7 + 2 es + 2^-18 + n 2^-27) A, and |lse - ref| <= es + 2^-18 + n 2^-27 + 2^-22 |lse|."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import sparse_mla_kv_gb300 as hs  # noqa: E402

pytestmark = pytest.mark.gpu

D, RD = 512, 64
FMT = {"fp8": 656, "bf16": 1152}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def pow2_scale(lat):
    """Definition, from the exponent of amax: the smallest 2^k >= 2^-126 with finite amax <= 448 * 2^k; 1 for zeros."""
    x = lat.double().reshape(*lat.shape[:-1], 4, 128)
    amax = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1).cpu().numpy()
    k = np.full(amax.shape, -126)
    for _ in range(260):
        k = np.where(amax > 448.0 * np.exp2(k.astype(np.float64)), k + 1, k)
    s = np.where(amax == 0, 1.0, np.exp2(k.astype(np.float64)))
    return torch.from_numpy(s).cuda()


def rows_bytes(lat, rope, fmt, scales=None):
    """Row bytes of latents and rotated keys (both any float type), built from the format's description."""
    n = lat.shape[0]
    out = torch.empty((n, FMT[fmt]), dtype=torch.uint8, device="cuda")
    if fmt == "fp8":
        s = pow2_scale(lat) if scales is None else scales.double()
        code = (lat.double().reshape(n, 4, 128) / s[..., None]).reshape(n, D).float().to(torch.float8_e4m3fn)
        out[:, :512] = code.view(torch.uint8)
        out[:, 512:528] = s.float().view(torch.uint8)
        out[:, 528:] = rope.to(torch.bfloat16).contiguous().view(torch.uint8)
    else:
        out[:, :1024] = lat.to(torch.bfloat16).contiguous().view(torch.uint8)
        out[:, 1024:] = rope.to(torch.bfloat16).contiguous().view(torch.uint8)
    return out


def row_values(b, fmt):
    """(latent as the attention reads it, key) of row bytes, in 64 bits."""
    if fmt == "fp8":
        c = b[:, :512].contiguous().view(torch.float8_e4m3fn).float()
        s = b[:, 512:528].contiguous().view(torch.float32)
        c = (c * s.repeat_interleave(128, 1)).to(torch.bfloat16).double()
        return c, torch.cat([c, b[:, 528:].contiguous().view(torch.bfloat16).double()], 1)
    v = b.contiguous().view(torch.bfloat16).double()
    return v[:, :D], v


def make_pool(g, blocks, fmt, page=64, layers=1, lat_scale=1.0):
    tensors = []
    for _ in range(layers):
        n = blocks * page
        t = rows_bytes(normal(g, n, D, dtype=torch.float32, scale=lat_scale), normal(g, n, RD), fmt)
        tensors.append(t.reshape(blocks, page, -1))
    return hs.Pool(tensors), tensors


def expect(q, k, v, mask, scale):
    """q [m, d], k [n, d], v [n, e], mask [m, n] (True: seen) -> out, lse and their tolerances, in 64 bits."""
    n = k.shape[0]
    if n == 0:
        m = q.shape[0]
        z = torch.zeros((m, v.shape[1]), dtype=torch.float64, device="cuda")
        return z, torch.full((m,), -math.inf, dtype=torch.float64, device="cuda"), z, torch.zeros(m, device="cuda").double()
    s = (q @ k.T) * scale
    es = 52 * 2.0 ** -23 * scale * (q.abs() @ k.abs().T).masked_fill(~mask, 0).amax(1)
    s = s.masked_fill(~mask, -math.inf)
    lse = torch.logsumexp(s, 1)
    w = torch.exp(s - torch.where(lse == -math.inf, 0, lse)[:, None])
    a = w @ v.abs()
    tol_o = (2.0 ** -7 + 2 * es + 2.0 ** -18 + n * 2.0 ** -27)[:, None] * a
    tol_l = es + 2.0 ** -18 + n * 2.0 ** -27 + 2.0 ** -22 * torch.where(lse == -math.inf, 0, lse).abs()
    return w @ v, lse, tol_o, tol_l


def close(got, lse, ref):
    o, l, to, tl = ref
    empty = l == -math.inf
    assert torch.equal(lse.double() == -math.inf, empty)
    assert bool((got[empty] == 0).all())
    assert bool(((got.double() - o).abs() <= to).all()), float(((got.double() - o).abs() - to).max())
    d = (lse.double() - l).abs()[~empty]
    assert bool((d <= tl[~empty]).all()), (float(d.max()), float(tl.max()))


def check_rows(tensors, fmt, rows, ql, qr, scale, out, lse, layer=0):
    """Every token of a rows call against the formula."""
    flat = tensors[layer].reshape(-1, FMT[fmt])
    for t in range(rows.shape[0]):
        at = rows[t][(rows[t] >= 0) & (rows[t] < flat.shape[0])].long()
        c, k = row_values(flat[at], fmt)
        q = torch.cat([ql[t], qr[t]], -1).double()
        close(out[t], lse[t], expect(q, k, c, torch.ones((q.shape[0], len(at)), dtype=torch.bool, device="cuda"), scale))


def check_pages(tensors, fmt, table, ctx, ql, qr, scale, out, lse):
    flat = tensors[0].reshape(-1, FMT[fmt])
    page = tensors[0].shape[1]
    R, P, H = ql.shape[:3]
    for r in range(R):
        n = min(int(ctx[r]), table.shape[1] * page)
        j = torch.arange(n, device="cuda")
        b = table[r].long()[j // page] if n else j
        ok = (b >= 0) & (b < tensors[0].shape[0])
        c, k = row_values(flat[(b * page + j % page)[ok]], fmt)
        seen = (j[ok][None] < (int(ctx[r]) - P + 1 + torch.arange(P, device="cuda"))[:, None]).repeat_interleave(H, 0)
        q = torch.cat([ql[r], qr[r]], -1).double().reshape(P * H, -1)
        close(out[r].reshape(P * H, -1), lse[r].reshape(-1), expect(q, k, c, seen, scale))


SCALE = 192 ** -0.5


# --------------------------------------------------------------------------------------------------------------------
# append


def rotated(x, cs, inter):
    """Rotation of [..., 64] in 64 bits and the sum of magnitudes behind each element."""
    c, s = cs[..., :32].double(), cs[..., 32:].double()
    x = x.double()
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :32], x[..., 32:])
    u, v = a * c - b * s, b * c + a * s
    mu, mv = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    join = (lambda p, q: torch.stack([p, q], -1).flatten(-2)) if inter else (lambda p, q: torch.cat([p, q], -1))
    return join(u, v), join(mu, mv)


def check_turned(got, x, cs, inter):
    """One rounding of the type (2^-8, 2^-11 or 2^-23 of the result, half an ulp) and three of fp32 in the magnitudes;
    fp16 results below its normals are off by at most 2^-25."""
    ref, mag = rotated(x, cs, inter)
    half_ulp = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -23}[got.dtype]
    floor = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    assert bool(((got.double() - ref).abs() <= half_ulp * ref.abs() + 4 * 2.0 ** -24 * mag + floor).all())


def table(n):
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(32, device="cuda").double() / 32)
    return torch.cat([a.cos(), a.sin()], 1).float()


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,heads,inter,page", [(1, 1, False, 64), (1, 0, True, 64), (7, 16, True, 16), (64, 64, False, 64),
                                                (333, 9, False, 48), (1000, 128, True, 64)])
def test_append(fmt, dtype, n, heads, inter, page):
    g = gen(n + heads)
    blocks = n // page + 3
    pool, tensors = make_pool(g, blocks, fmt, page, layers=2)
    before = [t.clone() for t in tensors]
    rows = torch.randperm(blocks * page, generator=g, device="cuda")[:n].int()
    if n > 3:
        rows[n // 2] = -1
    lat = normal(g, n, 512 + 64, dtype=dtype)[:, :512]        # a strided view, as a fused projection leaves it
    lat[0, :128] = 0
    if n > 1:
        lat[1] *= 2.0 ** -10
    rope = normal(g, n, RD, dtype=dtype)
    pos = torch.randint(0, 5000, (n,), generator=g, device="cuda").int()
    cs = table(5000)
    q = normal(g, n, heads, 192, dtype=dtype)[..., 128:] if heads else None
    q0 = None if q is None else q.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = hs.append_rows(pool, rows, lat, rope, pos, cs, layer=1, q_rope=q, interleaved=inter, status=status)
    assert int(status) == 0
    assert torch.equal(tensors[0], before[0])
    flat, old = tensors[1].reshape(-1, FMT[fmt]), before[1].reshape(-1, FMT[fmt])
    untouched = torch.ones(len(flat), dtype=torch.bool, device="cuda")
    untouched[rows[rows >= 0].long()] = False
    assert torch.equal(flat[untouched], old[untouched])
    keep = rows >= 0
    new = flat[rows[keep].long()]
    want = rows_bytes(lat[keep], rope[keep], fmt)
    cut = 528 if fmt == "fp8" else 1024
    assert torch.equal(new[:, :cut], want[:, :cut])            # codes and scales (or the latents) exactly
    check_turned(new[:, cut:].contiguous().view(torch.bfloat16), rope[keep], cs[pos[keep].long()], inter)
    if heads:
        assert torch.equal(q, q0)
        check_turned(got, q, cs[pos.long()][:, None], inter)
        hs.append_rows(pool, rows, lat, rope, pos, cs, layer=1, q_rope=q, q_out=q, interleaved=inter)   # in place
        assert torch.equal(q, got)


def test_append_edges_of_the_type():
    """Powers of two and 448 * 2^k on the border of a scale, infinities and NaN, subnormal and huge fp32 groups."""
    vals = [448.0, 449.0, 447.9, 1.75, 1.7500001, 3.5, 2.0 ** -126, 2.0 ** -140, 3.0e38, 1e-30, 0.0]
    lat = torch.zeros((len(vals) + 2, D), device="cuda")
    g = gen(3)
    for i, v in enumerate(vals):
        for grp in range(4):
            lat[i, 128 * grp:128 * grp + 128] = torch.rand(128, generator=g, device="cuda") * (v * 0.9)
            lat[i, 128 * grp + 7 * grp] = -v if grp & 1 else v
    lat[-2] = torch.randn(D, generator=g, device="cuda")
    lat[-2, 5], lat[-2, 200], lat[-2, 300] = math.inf, -math.inf, math.nan
    lat[-1, :128] = math.nan
    n = len(lat)
    pool, tensors = make_pool(g, 1, "fp8")
    rope = torch.zeros((n, RD), device="cuda")
    hs.append_rows(pool, torch.arange(n, device="cuda").int(), lat, rope, torch.zeros(n, device="cuda").int(), table(2))
    b = tensors[0].reshape(-1, 656)[:n]
    s = b[:, 512:528].contiguous().view(torch.float32)
    assert torch.equal(s.double(), pow2_scale(lat))
    code = b[:, :512].contiguous().view(torch.float8_e4m3fn).float()
    finite = torch.isfinite(lat)
    assert torch.equal(torch.isnan(code), ~finite)
    want = (lat.double() / s.double().repeat_interleave(128, 1)).float().to(torch.float8_e4m3fn).float()
    assert torch.equal(code[finite], want[finite])


def test_append_bad_rows_and_positions():
    g = gen(5)
    pool, tensors = make_pool(g, 2, "fp8")
    before = tensors[0].clone()
    n = 4
    lat, rope, q = normal(g, n, D), normal(g, n, RD), normal(g, n, 2, RD)
    for rows, pos, bad_q in (([1, 128, 3, -2], [0, 1, 2, 3], []), ([1, 2, 3, 4], [0, -1, 10, 3], [1, 2])):
        tensors[0].copy_(before)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = hs.append_rows(pool, torch.tensor(rows, device="cuda").int(), lat, rope, torch.tensor(pos, device="cuda").int(),
                             table(10), q_rope=q, status=status)
        assert int(status) == 2
        ok = [t for t in range(n) if 0 <= rows[t] < 128 and 0 <= pos[t] < 10]
        changed = (tensors[0].reshape(-1, 656) != before.reshape(-1, 656)).any(1).nonzero().flatten().tolist()
        assert changed == sorted(rows[t] for t in ok)
        for t in range(n):
            assert bool((got[t] == 0).all()) == (t in bad_q)


# --------------------------------------------------------------------------------------------------------------------
# absorbed, over row ids


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("n,K,H,fill", [(1, 1, 1, 1.0), (1, 127, 16, 1.0), (1, 129, 17, 1.0), (4, 256, 16, 1.0),
                                        (3, 2048, 128, 1.0), (5, 1000, 96, 0.9), (7, 333, 20, 0.5), (300, 130, 8, 0.97),
                                        (2, 5000, 64, 1.0), (200, 640, 64, 1.0), (40, 2048, 32, 0.99), (1, 8192, 8, 1.0),
                                        (160, 96, 128, 0.8), (3, 64, 1024, 1.0)])
def test_rows(fmt, n, K, H, fill):
    g = gen(n * K + H)
    pool, tensors = make_pool(g, 100, fmt)
    rows = torch.randint(0, 6400, (n, K), generator=g, device="cuda").int()
    rows = torch.where(torch.rand((n, K), generator=g, device="cuda") < fill, rows, -1)
    ql, qr = normal(g, n, H, D), normal(g, n, H, RD)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = hs.attend_rows(pool, rows, ql, qr, SCALE, status=status)
    assert int(status) == 0
    check_rows(tensors, fmt, rows, ql, qr, SCALE, out, lse)
    again, lse2 = hs.attend_rows(pool, rows, ql, qr, SCALE)
    assert torch.equal(out, again) and torch.equal(lse, lse2)    # the same bits every time


@pytest.mark.parametrize("K", [0, 1, 128, 1300])
def test_rows_that_see_nothing(K):
    g = gen(K)
    pool, tensors = make_pool(g, 4, "fp8")
    rows = torch.full((5, K), -1, dtype=torch.int32, device="cuda")
    if K > 1:
        rows[1, K - 1] = 7          # only the last id
        rows[3, 0] = 9              # only the first
    ql, qr = normal(g, 5, 40, D), normal(g, 5, 40, RD)
    out = torch.full((5, 40, D), 3.0, dtype=torch.bfloat16, device="cuda")
    out, lse = hs.attend_rows(pool, rows, ql, qr, SCALE, out=out)
    check_rows(tensors, "fp8", rows, ql, qr, SCALE, out, lse)
    none = torch.empty((0, K), dtype=torch.int32, device="cuda")
    o, l = hs.attend_rows(pool, none, ql[:0], qr[:0], SCALE)
    assert o.shape == (0, 40, D) and l.shape == (0, 40)


@pytest.mark.parametrize("H", [16, 32, 64])
@pytest.mark.parametrize("order", ["up", "down", "spike", "low"])
def test_rows_whose_scores_range_widely(H, order):
    """Scores over some hundreds, rising (the running maximum moves far many times), falling, with one peak, and all far
    below zero: rescaling and ranges."""
    g = gen(11)
    K = 1500
    lat = normal(g, K, D, dtype=torch.float32, scale=0.05)
    ramp = {"up": torch.linspace(-400, 400, K), "down": torch.linspace(400, -400, K),
            "spike": torch.where(torch.arange(K) == 901, 380.0, 0.0), "low": torch.full((K,), -390.0)}[order]
    lat[:, 3] = ramp.cuda()
    b = rows_bytes(lat, normal(g, K, RD), "bf16")
    pad = torch.zeros((1536 - K, 1152), dtype=torch.uint8, device="cuda")
    t = torch.cat([b, pad]).reshape(24, 64, 1152)
    pool = hs.Pool([t])
    rows = torch.arange(K, device="cuda").int()[None].repeat(2, 1)
    ql, qr = normal(g, 2, H, D, scale=0.1), normal(g, 2, H, RD)
    ql[:, :, 3] = torch.linspace(0.0, 4.0, H, device="cuda").to(torch.bfloat16)
    out, lse = hs.attend_rows(pool, rows, ql, qr, 0.5)
    check_rows([t], "bf16", rows, ql, qr, 0.5, out, lse)


def test_rows_scales_that_are_no_powers_of_two():
    g = gen(13)
    n = 640
    s = torch.rand((n, 4), generator=g, device="cuda") * 0.03 + 0.02   # codes of values up to 6 fit
    t = rows_bytes(normal(g, n, D, dtype=torch.float32), normal(g, n, RD), "fp8", scales=s).reshape(10, 64, 656)
    pool = hs.Pool([t])
    rows = torch.randperm(n, generator=g, device="cuda")[:600].reshape(2, 300).int()
    ql, qr = normal(g, 2, 64, D), normal(g, 2, 64, RD)
    out, lse = hs.attend_rows(pool, rows, ql, qr, SCALE)
    check_rows([t], "fp8", rows, ql, qr, SCALE, out, lse)


def test_rows_layers_strides_streams_and_repeats():
    """The second layer, head-major and padded queries and outputs, ids that repeat, another stream than the tensors' own,
    and rows full of NaN that no list names."""
    g = gen(17)
    pool, tensors = make_pool(g, 20, "fp8", page=32, layers=2)
    tensors[1].reshape(-1, 656)[600:] = 0xFF
    n, K, H = 6, 700, 24
    rows = torch.randint(0, 600, (n, K), generator=g, device="cuda").int()
    rows[0] = 5
    ql = normal(g, H, n, D + 64).transpose(0, 1)[..., :D]
    qr = normal(g, H, n, RD + 8).transpose(0, 1)[..., :RD]
    out = torch.zeros((H, n, D + 8), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    ws = hs.alloc_attend_workspace()
    o, lse = hs.attend_rows(pool, rows, ql, qr, SCALE, layer=1, out=out.transpose(0, 1)[..., :D], workspace=ws, stream=st)
    st.synchronize()
    check_rows(tensors, "fp8", rows, ql, qr, SCALE, o, lse, layer=1)
    assert bool((out[..., D:] == 0).all())


def test_rows_bad_ids():
    g = gen(19)
    pool, tensors = make_pool(g, 4, "fp8")
    rows = torch.randint(0, 256, (3, 200), generator=g, device="cuda").int()
    rows[1, 17], rows[1, 190], rows[2, 0] = 256, -5, 2 ** 31 - 1
    ql, qr = normal(g, 3, 16, D), normal(g, 3, 16, RD)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = hs.attend_rows(pool, rows, ql, qr, SCALE, status=status)
    assert int(status) == 2
    check_rows(tensors, "fp8", rows, ql, qr, SCALE, out, lse)


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
def test_rows_beyond_32_bit_byte_offsets(fmt):
    """A pool of over 4 GiB: rows at its far end."""
    blocks = (5 << 30) // (64 * FMT[fmt])
    t = torch.empty((blocks, 64, FMT[fmt]), dtype=torch.uint8, device="cuda")
    g = gen(23)
    far = rows_bytes(normal(g, 6400, D, dtype=torch.float32), normal(g, 6400, RD), fmt)
    t[-100:] = far.reshape(100, 64, -1)
    pool = hs.Pool([t])
    rows = (blocks * 64 - 1 - torch.randperm(6400, generator=g, device="cuda")[:900].reshape(3, 300)).int()
    ql, qr = normal(g, 3, 64, D), normal(g, 3, 64, RD)
    out, lse = hs.attend_rows(pool, rows, ql, qr, SCALE)
    check_rows([t], fmt, rows, ql, qr, SCALE, out, lse)
    tab = torch.arange(blocks - 100, blocks, device="cuda").int()[None]
    ctx = torch.tensor([6333], device="cuda").int()
    out, lse = hs.attend_pages(pool, tab, ctx, ql[None], qr[None], SCALE)
    check_pages([t], fmt, tab, ctx, ql[None], qr[None], SCALE, out, lse)


def test_rows_nan_and_infinite_queries_stay_in_their_head():
    g = gen(29)
    pool, tensors = make_pool(g, 4, "fp8")
    rows = torch.randint(0, 256, (2, 200), generator=g, device="cuda").int()
    ql, qr = normal(g, 2, 20, D), normal(g, 2, 20, RD)
    clean = ql.clone()
    ql[0, 3, 100], ql[1, 7, 0] = math.nan, math.nan
    out, lse = hs.attend_rows(pool, rows, ql, qr, SCALE)
    assert bool(torch.isnan(out[0, 3]).all()) and bool(torch.isnan(out[1, 7]).all()) and bool(torch.isnan(lse[0, 3]))
    ref, ref_l = hs.attend_rows(pool, rows, clean, qr, SCALE)
    ok = torch.ones((2, 20), dtype=torch.bool, device="cuda")
    ok[0, 3] = ok[1, 7] = False
    assert torch.equal(out[ok], ref[ok]) and torch.equal(lse[ok], ref_l[ok])


# --------------------------------------------------------------------------------------------------------------------
# absorbed, over pages


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("ctx,P,H,page", [([1], 1, 1, 64), ([0, 1, 2, 3], 3, 8, 64), ([63, 64, 65, 127, 128, 129], 1, 16, 64),
                                          ([1000, 17, 256], 4, 64, 64), ([511, 3000], 2, 20, 48), ([4096], 5, 128, 16),
                                          ([20000], 1, 16, 64), ([7] * 200, 1, 32, 64), ([129] * 3, 7, 9, 1),
                                          ([5000, 1, 0, 64, 800], 1, 128, 1024)])
def test_pages(fmt, ctx, P, H, page):
    g = gen(sum(ctx) + P + H)
    R = len(ctx)
    mp = -(-max(max(ctx), 1) // page) + 1
    blocks = R * mp + 2
    pool, tensors = make_pool(g, blocks, fmt, page)
    tab = torch.randperm(blocks, generator=g, device="cuda")[:R * mp].reshape(R, mp).int()
    for r in range(R):
        tab[r, -(-ctx[r] // page):] = -1                        # pages beyond the context
    cl = torch.tensor(ctx, device="cuda").int()
    ql, qr = normal(g, R, P, H, D), normal(g, R, P, H, RD)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = hs.attend_pages(pool, tab, cl, ql, qr, SCALE, status=status)
    assert int(status) == 0
    check_pages(tensors, fmt, tab, cl, ql, qr, SCALE, out, lse)
    again, lse2 = hs.attend_pages(pool, tab, cl, ql, qr, SCALE)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_pages_rows_past_the_context_do_not_matter():
    """NaN in the rows of the last page that lie past the context."""
    g = gen(31)
    pool, tensors = make_pool(g, 8, "fp8")
    tab = torch.arange(8, device="cuda").int().reshape(2, 4)
    tensors[0][1, 6:] = 0xFF
    tensors[0][2:4] = 0xFF
    tensors[0][7, 63] = 0xFF
    cl = torch.tensor([70, 255], device="cuda").int()
    ql, qr = normal(g, 2, 2, 16, D), normal(g, 2, 2, 16, RD)
    out, lse = hs.attend_pages(pool, tab, cl, ql, qr, SCALE)
    check_pages(tensors, "fp8", tab, cl, ql, qr, SCALE, out, lse)


def test_pages_bad_entries_and_lengths():
    g = gen(37)
    pool, tensors = make_pool(g, 10, "fp8")
    tab = torch.arange(9, device="cuda").int().reshape(3, 3)
    ql, qr = normal(g, 3, 1, 16, D), normal(g, 3, 1, 16, RD)
    for entry, ctx in ((10, [100, 192, 5]), (-1, [100, 192, 5]), (4, [100, 193, -3])):
        t = tab.clone()
        t[1, 1] = entry
        cl = torch.tensor(ctx, device="cuda").int()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = hs.attend_pages(pool, t, cl, ql, qr, SCALE, status=status)
        assert int(status) == 8
        check_pages(tensors, "fp8", t, cl.clamp_min(0), ql, qr, SCALE, out, lse)


# --------------------------------------------------------------------------------------------------------------------
# expanded


def check_expanded(qn, qr, kn, kr, v, cq, ck, scale, causal, out, lse):
    for b in range(len(cq) - 1):
        n, m = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        i, j = torch.arange(n, device="cuda")[:, None], torch.arange(m, device="cuda")[None]
        seen = (j <= i + m - n) if causal else (j >= 0).expand(n, m)
        for h in range(qn.shape[1]):
            q = torch.cat([qn[cq[b]:cq[b + 1], h], qr[cq[b]:cq[b + 1], h]], 1).double()
            k = torch.cat([kn[ck[b]:ck[b + 1], h], kr[ck[b]:ck[b + 1]]], 1).double()
            close(out[cq[b]:cq[b + 1], h], lse[cq[b]:cq[b + 1], h], expect(q, k, v[ck[b]:ck[b + 1], h].double(), seen, scale))


def cum(v):
    return torch.tensor([0] + list(v), device="cuda").cumsum(0).int()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("qn,kn,H", [([1], [1], 1), ([127], [127], 2), ([128, 129], [128, 129], 3), ([300, 0, 5, 1], [300, 0, 5, 1], 2),
                                     ([1, 1, 1], [1000, 513, 64], 4), ([200, 64], [1500, 64], 2), ([50], [20], 2),
                                     ([3, 257], [0, 600], 5), ([1024], [1024], 2), ([40] * 30, [90] * 30, 8)])
def test_expanded(qn, kn, H, causal):
    g = gen(sum(qn) * 7 + sum(kn))
    Tq, Tk = sum(qn), sum(kn)
    kv = normal(g, Tk, H, 256)
    q = normal(g, Tq, H, 192)
    kr = normal(g, Tk, RD)
    a = (q[..., :128], q[..., 128:], kv[..., :128], kr, kv[..., 128:])
    cq, ck = cum(qn), cum(kn)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = hs.attend_expanded(*a, cq, ck, SCALE, causal=causal, status=status)
    assert int(status) == 0
    check_expanded(*a, cq.tolist(), ck.tolist(), SCALE, causal, out, lse)
    again, lse2 = hs.attend_expanded(*a, cq, ck, SCALE, causal=causal)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_expanded_neighbours_and_hidden_keys_do_not_matter():
    """NaN in the other sequences' keys and values, and in the tensors' rows past the last sequence."""
    g = gen(41)
    H, qn, kn = 2, [70, 130, 90], [200, 130, 333]
    Tk = sum(kn) + 100
    kv, q, kr = normal(g, Tk, H, 256), normal(g, sum(qn), H, 192), normal(g, Tk, RD)
    kv[sum(kn):], kr[sum(kn):] = math.nan, math.nan
    kv[200:330], kr[200:330] = math.nan, math.nan            # the whole middle sequence
    a = (q[..., :128], q[..., 128:], kv[..., :128], kr, kv[..., 128:])
    out, lse = hs.attend_expanded(*a, cum(qn), cum(kn), SCALE)
    assert bool(torch.isnan(out[70:200]).all())
    for q0, q1, k0, k1 in ((0, 70, 0, 200), (200, 290, 330, 663)):
        part = [q[q0:q1, :, :128], q[q0:q1, :, 128:], kv[k0:k1, :, :128], kr[k0:k1], kv[k0:k1, :, 128:]]
        check_expanded(*part, [0, q1 - q0], [0, k1 - k0], SCALE, True, out[q0:q1], lse[q0:q1])


@pytest.mark.parametrize("order", ["up", "down", "spike", "low"])
def test_expanded_scores_that_range_widely(order):
    g = gen(43)
    n, H = 700, 2
    kn = normal(g, n, H, 128, scale=0.05)
    ramp = {"up": torch.linspace(-400, 400, n), "down": torch.linspace(400, -400, n),
            "spike": torch.where(torch.arange(n) == 333, 380.0, 0.0), "low": torch.full((n,), -390.0)}[order]
    kn[:, :, 3] = ramp.cuda()[:, None].to(torch.bfloat16)
    qn = normal(g, n, H, 128, scale=0.1)
    qn[:, :, 3] = torch.linspace(0.0, 4.0, n, device="cuda").to(torch.bfloat16)[:, None]
    a = (qn, normal(g, n, H, RD), kn, normal(g, n, RD), normal(g, n, H, 128))
    out, lse = hs.attend_expanded(*a, cum([n]), cum([n]), 0.5)
    check_expanded(*a, [0, n], [0, n], 0.5, True, out, lse)


def test_expanded_strides_and_a_stream():
    """Head-major tensors, and one key and value head broadcast to all by a stride of zero."""
    g = gen(47)
    H, n, m = 3, 150, 260
    q, qr = normal(g, H, n, 128).transpose(0, 1), normal(g, H, n, 72).transpose(0, 1)[..., :64]
    kn, v = normal(g, m, 1, 128).expand(m, H, 128), normal(g, H, m, 136).transpose(0, 1)[..., :128]
    kr = normal(g, m, 192)[:, 64:128]
    out = torch.zeros((H, n, 128), dtype=torch.bfloat16, device="cuda")
    cq, ck = cum([n]), cum([m])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    o, lse = hs.attend_expanded(q, qr, kn, kr, v, cq, ck, SCALE, out=out.transpose(0, 1), stream=st)
    st.synchronize()
    check_expanded(q, qr, kn, kr, v, [0, n], [0, m], SCALE, True, o, lse)


def test_expanded_bad_offsets():
    g = gen(53)
    H, n = 1, 64
    a = (normal(g, n, H, 128), normal(g, n, H, 64), normal(g, n, H, 128), normal(g, n, 64), normal(g, n, H, 128))
    for cq, ck in (([0, 32, 64], [0, 40, 65]), ([0, 32, 70], [0, 32, 64]), ([0, 32, 64], [0, -3, 64]), ([0, 40, 30], [0, 32, 64])):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        hs.attend_expanded(*a, torch.tensor(cq, device="cuda").int(), torch.tensor(ck, device="cuda").int(), SCALE, status=status)
        assert int(status) == 2, (cq, ck)


# --------------------------------------------------------------------------------------------------------------------
# together


def test_merge_of_prefix_and_chunk_by_lse():
    """A chunk's expanded attention over itself and its attention over the prefix join by their lse."""
    g = gen(59)
    H, pre, n = 4, 500, 130
    Tk = pre + n
    kv, q, kr = normal(g, Tk, H, 256), normal(g, n, H, 192), normal(g, Tk, RD)
    qn, qr = q[..., :128], q[..., 128:]
    whole, wl = hs.attend_expanded(qn, qr, kv[..., :128], kr, kv[..., 128:], cum([n]), cum([Tk]), SCALE)
    a, al = hs.attend_expanded(qn, qr, kv[:pre, :, :128], kr[:pre], kv[:pre, :, 128:], cum([n]), cum([pre]), SCALE, causal=False)
    b, bl = hs.attend_expanded(qn, qr, kv[pre:, :, :128], kr[pre:], kv[pre:, :, 128:], cum([n]), cum([n]), SCALE)
    l = torch.logaddexp(al, bl)
    o = a.float() * torch.exp(al - l)[..., None] + b.float() * torch.exp(bl - l)[..., None]
    # both sides carry the two bf16 roundings of the tolerance above: (2^-7 + 2^-7) of the sum of magnitudes, which is at
    # most the largest |v|; half of that is asked for
    assert float((l - wl).abs().max()) < 1e-4
    assert float((o - whole.float()).abs().max()) <= 2.0 ** -7 * float(kv[..., 128:].abs().max())


def test_calls_in_a_graph():
    g = gen(61)
    pool, tensors = make_pool(g, 40, "fp8")
    rows = torch.randint(0, 2560, (9, 500), generator=g, device="cuda").int()
    ql, qr = normal(g, 9, 16, D), normal(g, 9, 16, RD)
    ws = hs.alloc_attend_workspace()
    out, lse = torch.empty((9, 16, D), dtype=torch.bfloat16, device="cuda"), torch.empty((9, 16), device="cuda")
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        hs.attend_rows(pool, rows, ql, qr, SCALE, out=out, lse=lse, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            hs.attend_rows(pool, rows, ql, qr, SCALE, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    for seed in (1, 2):
        rows.copy_(torch.randint(0, 2560, (9, 500), generator=gen(seed), device="cuda").int())
        out.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        check_rows(tensors, "fp8", rows, ql, qr, SCALE, out, lse)


# --------------------------------------------------------------------------------------------------------------------
# refusals


def test_refusals():
    g = gen(67)
    pool, _ = make_pool(g, 4, "fp8")
    other = hs.Pool([torch.zeros((4, 64, 640), dtype=torch.uint8, device="cuda")])
    rows = torch.zeros((2, 8), dtype=torch.int32, device="cuda")
    ql, qr = normal(g, 2, 4, D), normal(g, 2, 4, RD)
    tab, ctx = torch.zeros((2, 1), dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    lat, rope, pos, cs = normal(g, 2, D), normal(g, 2, RD), torch.zeros(2, dtype=torch.int32, device="cuda"), table(4)
    before = hs.launch_count()

    def refused(code, f, *a, **k):
        with pytest.raises((hs.HSError, TypeError, ValueError)) as e:
            f(*a, **k)
        if code:
            assert isinstance(e.value, hs.HSError) and e.value.code == code

    refused(1, hs.attend_rows, other, rows, ql, qr, SCALE)                                # not a latent row size
    refused(1, hs.attend_rows, pool, rows, ql, qr, SCALE, layer=1)
    refused(1, hs.attend_rows, pool, rows, ql, qr, SCALE, layer=-1)
    refused(1, hs.attend_rows, pool, rows, ql, qr, float("nan"))
    refused(1, hs.attend_rows, pool, rows, ql, qr, SCALE, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    refused(1, hs.attend_rows, pool, rows, normal(g, 2, 4, D + 4)[..., 4:], qr, SCALE)    # 8 bytes off
    refused(1, hs.attend_rows, pool, rows, normal(g, 2, 4, D + 4)[..., :D], qr, SCALE)    # strides of 8 bytes
    refused(1, hs.attend_rows, pool, rows, normal(g, 2, 1025, D), normal(g, 2, 1025, RD), SCALE)
    refused(0, hs.attend_rows, pool, rows.long(), ql, qr, SCALE)
    refused(0, hs.attend_rows, pool, rows, ql.float(), qr, SCALE)
    refused(0, hs.attend_rows, pool, rows, ql[..., :256], qr, SCALE)
    refused(0, hs.attend_rows, pool, rows, ql, qr[:1], SCALE)
    refused(0, hs.attend_rows, pool, rows, ql.transpose(1, 2).contiguous().transpose(1, 2), qr, SCALE)
    refused(0, hs.attend_rows, pool, rows, ql, qr, SCALE, lse=torch.empty((2, 5), device="cuda"))
    refused(1, hs.attend_rows, pool, rows, ql, qr, SCALE, out=torch.empty((2, 1, D), dtype=torch.bfloat16, device="cuda").expand(2, 4, D))
    refused(1, hs.attend_pages, other, tab, ctx, ql[:, None], qr[:, None], SCALE)
    refused(0, hs.attend_pages, pool, tab[:1], ctx, ql[:, None], qr[:, None], SCALE)
    refused(0, hs.attend_pages, pool, tab, ctx, ql, qr, SCALE)
    refused(1, hs.append_rows, other, pos, lat, rope, pos, cs)
    refused(0, hs.append_rows, pool, pos, lat, rope[:1], pos, cs)
    refused(0, hs.append_rows, pool, pos, lat, rope.float(), pos, cs)
    refused(0, hs.append_rows, pool, pos, lat.double(), rope.double(), pos, cs)
    refused(0, hs.append_rows, pool, pos, lat, rope, pos, cs[:, :32])
    refused(0, hs.append_rows, pool, pos, lat, rope, pos[:1], cs)
    refused(1, hs.append_rows, pool, pos, lat, normal(g, 2, RD + 4)[:, 4:], pos, cs)
    refused(1, hs.append_rows, pool, pos, lat, rope, pos, cs, q_rope=normal(g, 2, 1, RD), q_out=normal(g, 1, 1, RD).expand(2, 1, RD))
    q, k = normal(g, 8, 2, 128), normal(g, 8, 64)
    qr8 = normal(g, 8, 2, 64)
    refused(0, hs.attend_expanded, q, qr8, q, k, q, cum([8]), cum([4, 4]), SCALE)
    refused(0, hs.attend_expanded, q, qr8, q[:, :1], k, q, cum([8]), cum([8]), SCALE)
    refused(1, hs.attend_expanded, q, qr8, q, normal(g, 8, 68)[:, 4:], q, cum([8]), cum([8]), SCALE)
    refused(1, hs.attend_expanded, q, qr8, q, k, q, cum([8]), cum([8]), SCALE,
            out=torch.empty((8, 1, 128), dtype=torch.bfloat16, device="cuda").expand(8, 2, 128))
    assert hs.launch_count() == before


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("H", [16, 20, 32, 64])
def test_rows_same_bits_with_cold_caches(fmt, H):
    """Runs that follow a flush of the caches, with units cut between CTAs: slots and tiles are reused while loads are
    late, and every run gives the same bits."""
    g = gen(71)
    pool, tensors = make_pool(g, 100, fmt)
    rows = torch.randint(0, 6400, (40, 2048), generator=g, device="cuda").int()
    ql, qr = normal(g, 40, H, D), normal(g, 40, H, RD)
    ws = hs.alloc_attend_workspace()
    flush = torch.empty(1 << 29, dtype=torch.uint8, device="cuda")
    first = None
    for i in range(25):
        flush.fill_(i)
        out, lse = hs.attend_rows(pool, rows, ql, qr, SCALE, workspace=ws)
        if first is None:
            first = (out.clone(), lse.clone())
            check_rows(tensors, fmt, rows, ql, qr, SCALE, out, lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
