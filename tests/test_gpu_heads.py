"""The operators on pages of grouped heads (append, read, attention) and read_rows, against their formulas in 64 bits.

Quantising and reading are compared bit by bit: scales are powers of two, so that x / scale, code * scale and code * old / new are
exact but for the one rounding that the definition has.

Attention: tolerances, set before any run.  For a query q over keys k[j] = codes * sk, values v[j] = codes * sv:
 - a score is a sum of D products in fp32, in steps of 16 (D / 16 + 16 additions, 2^-23 of the magnitudes each); q in fp16 keeps its
   bits but for 2^-23 of its largest value: es = scale ((D / 16 + 16) 2^-23 sum |q||k| + 2^-23 max|q| sum |k|), at most over j;
 - in log2 units, t = s log2(e) + log2(sv) - R is made by a product and a sum: 5 roundings (three factors, fma, the log) of numbers
   up to T = max |s| log2(e) + max |log2 sv| + 32, 2^-24 each: et = 5 T 2^-24.  The sum of weights goes through one more
   exponential of a difference of such numbers: twice that;
 - exponentials are off by 2^-21; a weight in fp16 by 2^-11 of itself, or, below 2^-14, by 2^-25 where the largest is at least 2^7:
   2^-32 of the largest w sv, times a code of up to 448;
 - sums over n tokens in fp32 add (n / 16 + 32) 2^-23 of the magnitudes;
 - the result is rounded to its type once (2^-8 or 2^-11 of it; fp16 has steps of 2^-24 at the low end).
With A = sum_j w |v|, all errors of exponents counted twice (the weight's and the sum's):
|out - ref| <= (2^-11 + 2 (es + 3 et ln 2) + 2^-19 + (n / 8 + 64) 2^-23) A + n 2^-32 448 max(w sv) + rounding,
|lse - ref| <= es + 3 et ln 2 + 2^-19 + (n / 16 + 32) 2^-23 + 2^-22 |lse|."""
import math

import pytest

torch = pytest.importorskip("torch")
import sparse_mla_kv_gb300 as hs  # noqa: E402

pytestmark = pytest.mark.gpu

PAGE = 64
F8 = torch.float8_e4m3fn


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets(n):
    return i32([0, *n]).cumsum(0).int()


def empty_pool(blocks, kv, dim, fill=0xA5, layers=1):
    row = 2 * kv * dim + 16
    t = [torch.full((blocks, PAGE, row), fill, dtype=torch.uint8, device="cuda") for _ in range(layers)]
    return hs.Pool(t), t


def parts(cache, kv, dim):
    """Key codes [block][head][dim / 64][token][64], value codes [block][head][dim / 64][64][token] as bytes, scales [block][2][kv]."""
    flat = cache.view(cache.shape[0], -1)
    codes = flat[:, :kv * 2 * dim * PAGE].unflatten(1, (kv, 2, dim // 64, 64, 64))
    scales = flat[:, kv * 2 * dim * PAGE:].view(torch.float32)[:, :2 * kv].unflatten(1, (2, kv))
    return codes[:, :, 0], codes[:, :, 1], scales


def values(cache, kv, dim, table, n):
    """Keys and values of the first n tokens of a table's row in 64 bits: [n][kv][dim], and their scales [n][kv]."""
    k, v, s = parts(cache, kv, dim)
    j = torch.arange(n, device="cuda")
    b = table.long()[j // PAGE] if n else j
    key = k[b, :, :, j % PAGE].view(F8).double().flatten(2)
    val = v[b, :, :, :, j % PAGE].view(F8).double().flatten(2)
    sk, sv = s[b, 0].double(), s[b, 1].double()
    return key * sk[..., None], val * sv[..., None], sv


def power(x):
    """The smallest 2^k >= 2^-126 with |x| <= 448 * 2^k for the finite x, by search."""
    x = x.double()
    a = float(torch.where(torch.isfinite(x), x.abs(), 0.0).max()) if x.numel() else 0.0
    k = -126
    while a > 448.0 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def append_plain(cache, kv, dim, table, ctx, new, k, v):
    """The definition, page by page, head by head."""
    kc, vc, s = parts(cache, kv, dim)
    t0 = 0
    for r, n in enumerate(new):
        first = ctx[r] - n
        for page in range(first // PAGE, -(-ctx[r] // PAGE) if n else first // PAGE):
            lo, hi = max(first - page * PAGE, 0), min(ctx[r] - page * PAGE, PAGE)
            b = int(table[r, page])
            rows = slice(t0 + page * PAGE + lo - first, t0 + page * PAGE + hi - first)
            for h in range(kv):
                for side, (codes, x) in enumerate(((kc[b, h], k[rows, h]), (vc[b, h].transpose(1, 2), v[rows, h]))):
                    old = float(s[b, side, h])
                    scale = max(power(x), old) if lo else power(x)
                    if lo and scale > old:
                        was = codes[:, :lo].contiguous().view(F8).double() * (old / scale)
                        codes[:, :lo] = was.float().to(F8).view(torch.uint8)
                    y = torch.where(torch.isfinite(x.double()), x.double() / scale, math.nan).float().to(F8)
                    codes[:, lo:hi] = y.view(torch.uint8).unflatten(1, (dim // 64, 64)).transpose(0, 1)
                    s[b, side, h] = scale
        t0 += n


def same(a, b):
    bad = (a != b).nonzero()
    assert len(bad) == 0, (len(bad), bad[:5].tolist(), a[tuple(bad[0])].item(), b[tuple(bad[0])].item())


def make(g, ctx, kv, dim, spread=0.0, spare=3, order="random", scale=1.0):
    """A filled cache of requests with these contexts: the pool, its bytes, the table.  spread: of the pages' sizes, in powers of 2."""
    pages = [-(-c // PAGE) for c in ctx]
    most = max([1, *pages])
    blocks = len(ctx) * most + spare
    pool, (cache,) = empty_pool(blocks, kv, dim)
    kc, vc, s = parts(cache, kv, dim)
    for side, codes in enumerate((kc, vc)):
        x = torch.randn((blocks, kv, dim // 64, 64, 64), generator=g, device="cuda") * scale
        x = x * torch.exp2(torch.round(spread * (torch.rand((blocks, kv, 1, 1, 1), generator=g, device="cuda") - 0.5)))
        m, e = torch.frexp(x.abs().amax((2, 3, 4)))
        sc = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875))
        codes.copy_((x / sc[:, :, None, None, None]).to(F8).view(torch.uint8))
        s[:, side] = sc
    ids = torch.randperm(blocks, generator=g, device="cuda")[:len(ctx) * most].reshape(len(ctx), most).int()
    return pool, cache, ids


# --------------------------------------------------------------------------------------------------------------------
# append and read


APPENDS = [
    # kv, dim, dtype, old tokens, new tokens
    (1, 64, torch.bfloat16, [0], [1]),
    (2, 128, torch.bfloat16, [63, 64, 0, 1], [1, 1, 64, 63]),
    (8, 128, torch.float16, [5, 200, 0, 127], [130, 1, 65, 2]),
    (3, 64, torch.float32, [10, 0, 62], [300, 0, 3]),
    (5, 128, torch.float32, [1, 33], [62, 95]),
    (128, 64, torch.bfloat16, [30], [40]),
    (1, 128, torch.bfloat16, [3 * i for i in range(300)], [1 + i % 5 for i in range(300)]),
]


@pytest.mark.parametrize("kv,dim,dtype,old,new", APPENDS)
def test_append_writes_what_its_definition_says(kv, dim, dtype, old, new):
    g = gen(1)
    ctx = [a + b for a, b in zip(old, new)]
    pool, cache, table = make(g, ctx, kv, dim, spread=4)
    k, v = (normal(g, sum(new), kv, dim, dtype=torch.float32) * torch.exp2(
        torch.randint(-3, 4, (sum(new), 1, 1), generator=g, device="cuda")) for _ in range(2))
    k, v = k.to(dtype), v.to(dtype)
    want = cache.clone()
    append_plain(want, kv, dim, table.cpu(), ctx, new, k, v)
    status = i32([0])
    hs.append_heads(pool, table, i32(ctx), k, v, cu=offsets(new), status=status)
    same(cache, want)
    assert int(status) == 0
    hs.append_heads(pool, table, i32(ctx), k, v, cu=offsets(new))  # once more: nothing changes
    same(cache, want)


def test_append_by_single_tokens_and_even_batches():
    g = gen(2)
    kv, dim, R = 2, 128, 5
    pool, cache, table = make(g, [200] * R, kv, dim)
    want = cache.clone()
    ctx = [60, 64, 1, 127, 30]
    for step in range(6):
        n = 1 + step % 3
        ctx = [c + n for c in ctx]
        k, v = (normal(g, R * n, kv, dim, scale=2.0 ** (step - 2)) for _ in range(2))
        append_plain(want, kv, dim, table.cpu(), ctx, [n] * R, k, v)
        hs.append_heads(pool, table, i32(ctx), k, v)
        same(cache, want)


def test_append_of_extreme_values():
    g = gen(3)
    kv, dim = 4, 64
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        pool, cache, table = make(g, [64, 64, 64], kv, dim)
        k, v = (normal(g, 3 * 40, kv, dim, dtype=torch.float32) for _ in range(2))
        big = torch.finfo(dtype).max
        k[:40, 0] = 0                                         # a page of zeros
        k[:40, 1] = torch.where(torch.rand(40, dim, generator=g, device="cuda") < 0.1, math.inf, k[:40, 1])
        v[:40, 1, 3] = math.nan
        v[:40, 2] = math.nan                                  # nothing finite
        k[40:80, 0], v[40:80, 3] = big, -big
        k[40:80, 1] *= 1e-6
        v[40:80, 1] *= 2.0 ** -140                            # below the smallest scale's range
        k[80:, 2] = 448.0 * 2.0 ** -3                         # the largest value of a scale, and the next one
        v[80:, 2] = 449.0 * 2.0 ** -3
        k, v = k.to(dtype), v.to(dtype)
        want = cache.clone()
        for new, old in (([40, 40, 40], [0, 0, 0]), ([20, 20, 20], [40, 40, 40])):
            x, y = k[:sum(new)], v[:sum(new)]
            if old[0]:
                x, y = x.flip(0).contiguous(), y.flip(0).contiguous()
            ctx = [a + b for a, b in zip(old, new)]
            append_plain(want, kv, dim, table.cpu(), ctx, new, x, y)
            hs.append_heads(pool, table, i32(ctx), x, y, cu=offsets(new))
            same(cache, want)


def test_append_takes_strided_keys_and_values():
    g = gen(4)
    kv, dim, n = 3, 128, 100
    pool, cache, table = make(g, [150], kv, dim)
    both = normal(g, n, 2 * kv + 1, dim)  # as a joint projection leaves them
    want = cache.clone()
    append_plain(want, kv, dim, table.cpu(), [150], [n], both[:, :kv], both[:, kv:2 * kv])
    hs.append_heads(pool, table, i32([150]), both[:, :kv], both[:, kv:2 * kv])
    same(cache, want)
    one = normal(g, n, 1, dim)  # all heads alike, by a stride of zero
    append_plain(want, kv, dim, table.cpu(), [150], [n], one.expand(-1, kv, -1), both[:, 1:1 + kv])
    hs.append_heads(pool, table, i32([150]), one.expand(-1, kv, -1), both[:, 1:1 + kv])
    same(cache, want)


def test_append_of_bad_data_writes_nothing_of_it():
    g = gen(5)
    kv, dim = 2, 64
    pool, cache, table = make(g, [200, 200, 200], kv, dim)
    new = [10, 70, 5]
    k, v = normal(g, 85, kv, dim), normal(g, 85, kv, dim)

    def run(table, ctx, cu, code, ok):
        want = cache.clone()
        for r in ok:
            t0 = sum(new[:r])
            append_plain(want, kv, dim, table[r:r + 1].cpu(), [ctx[r]], [new[r]], k[t0:t0 + new[r]], v[t0:t0 + new[r]])
        status = i32([0])
        hs.append_heads(pool, table, i32(ctx), k, v, cu=i32(cu), status=status)
        same(cache, want)
        assert int(status) == code

    run(table, [50, 60, 150], [0, 10, 80, 85], 2, [0, 2])         # fewer tokens than are new
    run(table, [50, -3, 150], [0, 10, 80, 85], 2, [0, 2])
    run(table, [50, 100, 150], [0, 10, 8, 85], 2, [])             # offsets that do not ascend
    run(table, [50, 100, 150], [0, 10, 80, 86], 2, [])
    run(table, [50, 100, 150], [-1, 10, 80, 85], 2, [])
    for bad in (-1, cache.shape[0], 2 ** 31 - 1):                 # a page that is not there
        t = table.clone()
        t[0, 0], t[2, 2] = bad, bad
        run(t, [50, 100, 150], [0, 10, 80, 85], 8, [1])
    run(table, [50, 100, 64 * table.shape[1] + 5], [0, 10, 80, 85], 8, [0, 1])  # past the table


READS = [
    # kv, dim, dtype, start, tokens
    (1, 64, torch.bfloat16, [0], [1]),
    (8, 128, torch.bfloat16, [0, 63, 1, 100], [64, 2, 200, 0]),
    (3, 64, torch.float32, [5, 70], [60, 129]),
    (5, 128, torch.float16, [64, 0, 33], [64, 300, 31]),
    (2, 128, torch.float32, [7 * i for i in range(290)], [i % 4 for i in range(290)]),
]


@pytest.mark.parametrize("kv,dim,dtype,start,n", READS)
def test_read_gives_code_times_scale(kv, dim, dtype, start, n):
    g = gen(6)
    ends = [a + b for a, b in zip(start, n)]
    pool, cache, table = make(g, ends, kv, dim, spread=4)
    status = i32([0])
    k, v = hs.read_heads(pool, table, i32(start), offsets(n), sum(n), dim, dtype=dtype, status=status)
    assert k.dtype == v.dtype == dtype and int(status) == 0
    t0 = 0
    for r, (a, m) in enumerate(zip(start, n)):
        wk, wv, _ = values(cache, kv, dim, table[r], a + m)
        same(k[t0:t0 + m], wk[a:].to(dtype))
        same(v[t0:t0 + m], wv[a:].to(dtype))
        t0 += m


def test_read_into_strided_tensors_evenly_and_of_bad_data():
    g = gen(7)
    kv, dim = 3, 128
    pool, cache, table = make(g, [200, 200], kv, dim)
    whole = torch.full((105, 2 * kv, dim), 9.0, dtype=torch.bfloat16, device="cuda")
    k, v = whole[:100, :kv], whole[:100, kv:]
    hs.read_heads(pool, table, None, None, 100, dim, k=k, v=v)
    for r in range(2):
        wk, wv, _ = values(cache, kv, dim, table[r], 50)
        same(k[50 * r:50 * r + 50], wk.bfloat16())
        same(v[50 * r:50 * r + 50], wv.bfloat16())
    assert bool((whole[100:] == 9).all())
    # rows that no request has keep what they hold; pages that are not there give zeros
    t = table.clone()
    t[1, 0] = cache.shape[0]
    status = i32([0])
    k, v = (torch.full((105, kv, dim), 9.0, device="cuda") for _ in range(2))
    hs.read_heads(pool, t, i32([3, 60]), i32([2, 52, 102]), 105, dim, k=k, v=v, status=status)
    assert int(status) == 8
    wk, wv, _ = values(cache, kv, dim, table[0], 53)
    same(k[2:52], wk[3:].float())
    assert bool((k[52:56] == 0).all()) and bool((v[52:56] == 0).all())
    wk, wv, _ = values(cache, kv, dim, table[1], 110)
    same(v[56:102], wv[64:].float())
    for x in (k, v):
        assert bool((x[:2] == 9).all()) and bool((x[102:] == 9).all())
    for start, cu in (([-1, 0], [0, 50, 100]), ([2 ** 31 - 10, 0], [0, 50, 100]), ([0, 0], [0, 60, 50]), ([0, 0], [0, 50, 106])):
        status.zero_()
        k, v = (torch.full((105, kv, dim), 9.0, device="cuda") for _ in range(2))
        hs.read_heads(pool, table, i32(start), i32(cu), 105, dim, k=k, v=v, status=status)
        assert int(status) == 2
        done = start[0] != 0
        assert bool((k[:50] == 9).all()) and bool((k[50:100] != 9).any()) == done and bool((v[100:] == 9).all())


@pytest.mark.parametrize("fmt", [656, 1152])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n", [1, 7, 64, 1001])
def test_read_rows(fmt, dtype, n):
    g = gen(8)
    cache = torch.zeros((20, 16, fmt), dtype=torch.uint8, device="cuda")
    pool = hs.Pool([cache, cache.clone()])
    rope = normal(g, 320, 64)
    if fmt == 656:
        codes = (torch.randn((320, 512), generator=g, device="cuda") * 50).to(F8)
        scale = torch.exp2(torch.randint(-9, 3, (320, 4), generator=g, device="cuda").float())
        scale[5] = 0.3
        lat = codes.float() * scale.repeat_interleave(128, 1)
        raw = torch.cat([codes.view(torch.uint8), scale.view(torch.uint8), rope.view(torch.uint8)], 1)
    else:
        b = normal(g, 320, 512)
        lat, raw = b.float(), torch.cat([b.view(torch.uint8), rope.view(torch.uint8)], 1)
    cache.view(320, fmt).copy_(raw)
    rows = torch.randint(-1, 320, (n,), generator=g, device="cuda").int()
    status = i32([0])
    latent, key = hs.read_rows(pool, rows, dtype=dtype, status=status)
    there = (rows >= 0)[:, None]
    same(latent, torch.where(there, lat[rows.long()], 0.0).to(dtype))
    same(key, torch.where(there, rope[rows.long()].float(), 0.0).to(dtype))
    assert int(status) == 0
    hs.read_rows(pool, rows, layer=1, latent=latent, rope=key)
    assert bool((latent == 0).all()) and bool((key == 0).all())
    rows[n // 2], rows[0] = 320, -2
    wide = torch.full((n + 1, 1024), 3.0, dtype=dtype, device="cuda")
    hs.read_rows(pool, rows, latent=wide[:n, 256:768], rope=wide[:n, 768:832], status=status)
    assert int(status) == 2 and bool((wide[n // 2, 256:832] == 0).all()) and bool((wide[0, 256:832] == 0).all())
    ok = (rows >= 0) & (rows < 320)
    same(wide[:n, 256:768][ok], lat[rows[ok].long()].to(dtype))
    assert bool((wide[n] == 3).all()) and bool((wide[:, :256] == 3).all()) and bool((wide[:, 832:] == 3).all())


# --------------------------------------------------------------------------------------------------------------------
# attention


def expect(q, k, v, sv, seen, scale, dtype):
    """One query head: q [m][D], k and v [n][D], sv [n], seen bool [m][n] -> out, lse, tolerances, in 64 bits."""
    m, n, D = q.shape[0], k.shape[0], q.shape[1]
    if n == 0:
        z = torch.zeros((m, D), dtype=torch.float64, device="cuda")
        return z, torch.full((m,), -math.inf, device="cuda").double(), z, z[:, 0]
    s = (q @ k.T) * scale
    mag = abs(scale) * ((D / 16 + 16) * 2.0 ** -23 * (q.abs() @ k.abs().T) + 2.0 ** -23 * q.abs().amax(1)[:, None] * k.abs().sum(1)[None])
    es = mag.masked_fill(~seen, 0).amax(1)
    T = s.masked_fill(~seen, 0).abs().amax(1) * math.log2(math.e) + sv.log2().abs().max() + 32
    et = 5 * T * 2.0 ** -24 * math.log(2)
    s = s.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, 1)
    w = torch.exp(s - torch.where(lse == -math.inf, 0, lse)[:, None])
    out, a = w @ v, w @ v.abs()
    tol = (2.0 ** -11 + 2 * (es + 3 * et) + 2.0 ** -19 + (n / 8 + 64) * 2.0 ** -23)[:, None] * a
    tol = tol + n * 2.0 ** -32 * 448 * (w * sv).amax(1)[:, None]
    tol = tol + torch.finfo(dtype).eps / 2 * (out.abs() + tol) + (2.0 ** -25 if dtype is torch.float16 else 0)
    return out, lse, tol, es + 3 * et + 2.0 ** -19 + (n / 16 + 32) * 2.0 ** -23 + 2.0 ** -22 * torch.where(lse == -math.inf, 0, lse).abs()


def check(cache, kv, dim, table, ctx, new, q, scale, out, lse, causal=True, room=None):
    t0 = 0
    group = q.shape[1] // kv
    for r, n in enumerate(new):
        m = max(0, min(ctx[r], PAGE * table.shape[1]))
        b = table[r].long()
        there = (b >= 0) & (b < cache.shape[0])
        k, v, sv = values(cache, kv, dim, torch.where(there, b, 0), m)
        j = torch.arange(m, device="cuda")
        ok = there[j // PAGE] if m else j.bool()
        last = ctx[r] - n + 1 + torch.arange(n, device="cuda") if causal else torch.full((n,), ctx[r], device="cuda")
        seen = (j[None] < last[:, None]) & ok[None]
        x = q[t0:t0 + n].double()
        for h in range(kv * group):
            o, l, to, tl = expect(x[:, h], k[:, h // group], v[:, h // group], sv[:, h // group], seen, scale, q.dtype)
            got, gl = out[t0:t0 + n, h].double(), lse[t0:t0 + n, h].double()
            none = l == -math.inf
            assert torch.equal(gl == -math.inf, none), (r, h)
            assert bool((got[none] == 0).all())
            off = (got - o).abs()
            assert bool((off <= to).all()), (r, h, float((off / to.clamp_min(1e-300)).max()), float(off.max()))
            d = (gl - l).abs()[~none]
            assert bool((d <= tl[~none]).all()), (r, h, float((d / tl[~none]).max()))
        t0 += n


STEPS = [
    # kv, dim, group, dtype, contexts, new tokens (None: one each)
    (1, 64, 1, torch.bfloat16, [1], None),
    (2, 128, 4, torch.bfloat16, [1, 63, 64, 65, 0, 500], None),
    (8, 128, 8, torch.bfloat16, [700, 129, 1300], None),
    (3, 64, 5, torch.float16, [64, 128, 2000], None),
    (1, 128, 16, torch.float16, [9000], None),
    (2, 64, 12, torch.bfloat16, [300, 3, 77], [2, 2, 2]),
    (2, 128, 7, torch.bfloat16, [300, 3, 64], [4, 4, 4]),
    (4, 128, 16, torch.bfloat16, [1000, 5], [4, 4]),
    (1, 128, 3, torch.bfloat16, [100 + i for i in range(300)], None),
    (2, 64, 2, torch.float16, [4, 130, 70, 64, 200, 0], [3, 0, 70, 1, 9, 0]),
    (1, 128, 64, torch.bfloat16, [333, 200], [1, 3]),
]


@pytest.mark.parametrize("kv,dim,group,dtype,ctx,new", STEPS)
@pytest.mark.parametrize("causal", [True, False])
def test_attend(kv, dim, group, dtype, ctx, new, causal):
    g = gen(9)
    pool, cache, table = make(g, ctx, kv, dim, spread=4)
    even = new is None
    new = new or [1] * len(ctx)
    q = normal(g, sum(new), kv * group, dim, dtype=dtype)
    status = i32([0])
    out, lse = hs.attend_heads(pool, table, i32(ctx), q, dim ** -0.5, cu_q=None if even else offsets(new), causal=causal,
                               status=status)
    assert int(status) == 0
    check(cache, kv, dim, table, ctx, new, q, dim ** -0.5, out, lse, causal)
    again, lse2 = hs.attend_heads(pool, table, i32(ctx), q, dim ** -0.5, cu_q=None if even else offsets(new), causal=causal)
    same(out, again)
    same(lse, lse2)


PROMPTS = [
    (2, 128, 4, torch.bfloat16, [700, 300], [700, 300]),
    (1, 64, 8, torch.float16, [5000], [130]),
    (4, 128, 1, torch.bfloat16, [1500, 200, 0, 90], [300, 200, 0, 65]),
    (3, 128, 7, torch.bfloat16, [2000], [77]),
    (2, 64, 2, torch.bfloat16, [100 + 3 * i for i in range(600)], [i % 37 for i in range(600)]),
    (1, 128, 2, torch.bfloat16, [50, 128, 129, 256, 300], [200, 128, 129, 128, 257]),
    (2, 64, 1, torch.float16, [1300], [1300]),
    (1, 128, 128, torch.bfloat16, [64, 640], [3, 1]),
    # items of one query tile and of two in turn, with parts of a run, short and long
    (2, 128, 1, torch.bfloat16, [3000, 500, 4000, 260, 900, 2100], [100, 400, 70, 256, 300, 128]),
    (2, 64, 1, torch.bfloat16, [3000, 500, 4000, 260, 900, 2100], [100, 400, 70, 256, 300, 128]),
    (4, 128, 4, torch.float16, [4000, 64, 130, 5000], [20, 64, 30, 25]),
    (4, 64, 4, torch.float16, [4000, 64, 130, 5000], [20, 64, 30, 25]),
    # items of many parts, beside some of few
    (1, 128, 8, torch.bfloat16, [20000, 900], [40, 17]),
    (2, 64, 5, torch.float16, [17001, 13], [27, 13]),
]


@pytest.mark.parametrize("kv,dim,group,dtype,ctx,new", PROMPTS)
@pytest.mark.parametrize("causal", [True, False])
def test_attend_prompts(kv, dim, group, dtype, ctx, new, causal):
    test_attend(kv, dim, group, dtype, ctx, new, causal)


@pytest.mark.parametrize("causal", [True, False])
def test_attend_even_prompts(causal):
    g = gen(20)
    kv, dim, group, ctx, n = 2, 128, 4, [400, 90, 333], 80
    pool, cache, table = make(g, ctx, kv, dim)
    q = normal(g, 3 * n, kv * group, dim)
    out, lse = hs.attend_heads(pool, table, i32(ctx), q, 0.1, causal=causal)
    check(cache, kv, dim, table, ctx, [n] * 3, q, 0.1, out, lse, causal)


@pytest.mark.parametrize("spread", [20, 90])
@pytest.mark.parametrize("kv,dim,group,ctx,new", [(2, 128, 4, [900, 70], [1, 1]), (1, 64, 8, [5000], [40])])
def test_attend_pages_of_very_different_sizes(spread, kv, dim, group, ctx, new):
    g = gen(10)
    pool, cache, table = make(g, ctx, kv, dim, spread=spread)
    parts(cache, kv, dim)[2][:, 0] = 2.0 ** -8  # keys of one size
    q = normal(g, sum(new), kv * group, dim)
    out, lse = hs.attend_heads(pool, table, i32(ctx), q, 0.1, cu_q=offsets(new))
    check(cache, kv, dim, table, ctx, new, q, 0.1, out, lse)


def test_attend_values_that_are_zero_do_not_spoil_the_sum_of_weights():
    g = gen(11)
    kv, dim, ctx = 2, 128, [640, 300]
    pool, cache, table = make(g, ctx, kv, dim)
    k, v, s = parts(cache, kv, dim)
    for r, pages in enumerate(([0, 3, 4], [1, 4])):  # pages of zeros, as append_heads writes them: the smallest scale
        for p in pages:
            b = int(table[r, p])
            v[b], s[b, 1] = 0, 2.0 ** -126
    q = normal(g, 2, 8, dim)
    out, lse = hs.attend_heads(pool, table, i32(ctx), q, 0.3)
    check(cache, kv, dim, table, ctx, [1, 1], q, 0.3, out, lse)
    v[:], s[:, 1] = 0, 2.0 ** -126
    out, lse = hs.attend_heads(pool, table, i32(ctx), q, 0.3)
    assert bool((out == 0).all())
    check(cache, kv, dim, table, ctx, [1, 1], q, 0.3, out, lse)


@pytest.mark.parametrize("new", [[1, 1], [3, 9], [90, 70]])
@pytest.mark.parametrize("dim", [64, 128])
def test_what_a_query_does_not_see_has_no_part(new, dim):
    g = gen(12)
    kv, group, ctx = 2, 4, [150, 300]
    pool, cache, table = make(g, ctx, kv, dim)
    k, v, s = parts(cache, kv, dim)
    q = normal(g, sum(new), kv * group, dim)
    run = lambda: hs.attend_heads(pool, table, i32(ctx), q, 0.1, cu_q=offsets(new))  # noqa: E731
    out, lse = run()
    for r in range(2):  # behind the contexts, and pages of nobody
        b, place = int(table[r, ctx[r] // PAGE]), ctx[r] % PAGE
        k[b, :, :, place:], v[b, :, :, :, place:] = 0x7F, 0xFF
    used = set(table.flatten().tolist())
    for b in range(cache.shape[0]):
        if b not in used:
            cache[b] = 0xFF
    got, glse = run()
    same(out, got)
    same(lse, glse)
    # a NaN value of the last token: only the queries that see it, and only there
    for r in range(2):
        j = ctx[r] - 1
        v[int(table[r, j // PAGE]), 1, 0, 5, j % PAGE] = 0x7F
    got, glse = run()
    last = offsets(new)[1:].long() - 1
    want = out.clone()
    want[last, group:, 5] = math.nan
    assert torch.equal(got.isnan(), want.isnan())
    same(torch.nan_to_num(got), torch.nan_to_num(want))
    same(lse, glse)
    # a NaN key of the last token: all of those queries' results
    for r in range(2):
        j = ctx[r] - 1
        k[int(table[r, j // PAGE]), 0, 0, j % PAGE, 7] = 0xFF
    got, glse = run()
    want[last, :group] = math.nan
    assert torch.equal(got.isnan(), want.isnan())
    same(torch.nan_to_num(got), torch.nan_to_num(want))
    assert bool(glse[last, :group].isnan().all()) and int(glse.isnan().sum()) == 2 * group


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0, 1e-30, -1e30])
def test_attend_scales_of_either_sign(scale):
    g = gen(13)
    kv, dim, ctx, new = 2, 128, [200, 90], [1, 2]
    pool, cache, table = make(g, ctx, kv, dim)
    q = normal(g, 3, 8, dim)
    if abs(scale) > 1e3:  # one token takes all: scores that differ by more than their errors
        out, lse = hs.attend_heads(pool, table, i32(ctx), q, scale, cu_q=offsets(new))
        assert bool(torch.isfinite(out).all())
        return
    out, lse = hs.attend_heads(pool, table, i32(ctx), q, scale, cu_q=offsets(new))
    check(cache, kv, dim, table, ctx, new, q, scale, out, lse)


@pytest.mark.parametrize("size", [1e4, 1e8, 1e20])
@pytest.mark.parametrize("new", [[1, 1], [3, 2], [130, 66]])
def test_attend_scores_of_any_size(size, new):
    """One token's score passes all others by far: its value is the result, whatever the scores' size and sign."""
    g = gen(19)
    kv, dim, group, ctx = 2, 64, 4, [900, 300]
    pool, cache, table = make(g, ctx, kv, dim, spread=6)
    k, v, s = parts(cache, kv, dim)
    s[:, 0] = 1.0
    k.copy_(torch.full(k.shape, -1.0, device="cuda").to(F8).view(torch.uint8))
    best = [17, 130]
    for r, j in enumerate(best):
        k[int(table[r, j // PAGE]), :, :, j % PAGE] = torch.tensor(0.5, device="cuda").to(F8).view(torch.uint8)
    q = torch.full((sum(new), kv * group, dim), size, device="cuda").bfloat16()
    for sign in (1, -1):
        if sign < 0:
            k ^= 0x80
        out, lse = hs.attend_heads(pool, table, i32(ctx), q, sign * 0.25, cu_q=offsets(new))
        for r, j in enumerate(best):
            t0 = sum(new[:r])
            _, val, _ = values(cache, kv, dim, table[r], j + 1)
            same(out[t0:t0 + new[r]], val[j].repeat_interleave(group, 0).bfloat16().expand(new[r], -1, -1))
        want = float(q[0, 0, 0]) * 0.5 * dim * 0.25
        assert bool(((lse.double() - want).abs() <= 2.0 ** -20 * want).all())


def test_attend_queries_of_any_size_and_strides():
    g = gen(14)
    kv, dim, group, ctx, new = 2, 64, 3, [500, 64, 129], [1, 2, 30]
    pool, cache, table = make(g, ctx, kv, dim, scale=2.0 ** -10)
    wide = normal(g, 33, 20, dim)
    q = wide[:, 3:3 + kv * group]
    q *= torch.exp2(torch.randint(-60, 60, (33, 1, 1), generator=g, device="cuda").float()).bfloat16() * 2.0 ** -30
    q[4] = 0
    res = torch.full((35, 9, dim), 5.0, dtype=torch.bfloat16, device="cuda")
    out = res[1:34, 2:2 + kv * group]
    lse = torch.full((33, kv * group), 5.0, device="cuda")
    hs.attend_heads(pool, table, i32(ctx), q, 0.5, cu_q=offsets(new), out=out, lse=lse)
    check(cache, kv, dim, table, ctx, new, q, 0.5, out, lse)
    for x in (res[0], res[34], res[:, :2], res[:, 8:]):
        assert bool((x == 5).all())
    q[:] = wide[:1, 3:4]
    one = wide[:1, 3:4].expand(33, kv * group, -1)  # by strides of zero
    same(hs.attend_heads(pool, table, i32(ctx), one, 0.5, cu_q=offsets(new))[0],
         hs.attend_heads(pool, table, i32(ctx), q, 0.5, cu_q=offsets(new))[0])


@pytest.mark.parametrize("new", [[1, 1, 1], [2, 40, 5], [200, 1, 80]])
def test_attend_of_bad_data(new):
    g = gen(15)
    kv, dim, group, ctx = 2, 128, 4, [400, 260, 330]
    pool, cache, table = make(g, ctx, kv, dim)
    q = normal(g, sum(new), kv * group, dim)
    n = sum(new)

    def run(table, ctx, cu, code):
        status = i32([0])
        out, lse = (torch.full((n, kv * group, d), 7.0, dtype=t, device="cuda") for d, t in ((dim, q.dtype), (1, torch.float32)))
        hs.attend_heads(pool, table, i32(ctx), q, 0.1, cu_q=cu, out=out, lse=lse[..., 0], status=status)
        assert int(status) == code
        return out, lse[..., 0]

    for bad in (-1, cache.shape[0], -2 ** 31):  # pages that are not there are skipped
        t = table.clone()
        t[0, 2], t[2, 0], t[1, 4] = bad, bad, bad
        out, lse = run(t, ctx, offsets(new), 8)
        check(cache, kv, dim, t, ctx, new, q, 0.1, out, lse)
    longer = [400, 64 * table.shape[1] + 3, 330]  # a context past the table
    out, lse = run(table, longer, offsets(new), 8)
    check(cache, kv, dim, table, longer, new, q, 0.1, out, lse)
    out, lse = run(table, [400, -5, 0], offsets(new), 0)
    check(cache, kv, dim, table, [400, -5, 0], new, q, 0.1, out, lse)
    for cu in ([0, new[0], 0, n], [0, new[0], n + 1, n], [-1, 0, 0, n]):  # offsets that do not ascend
        out, lse = run(table, ctx, i32(cu), 2)
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_attend_query_tokens_that_no_request_has():
    g = gen(16)
    kv, dim, group, ctx, new = 1, 128, 8, [90, 200], [1, 20]
    pool, cache, table = make(g, ctx, kv, dim)
    q = normal(g, 30, group, dim)
    out, lse = (torch.full((30, group, d), 7.0, dtype=t, device="cuda") for d, t in ((dim, q.dtype), (1, torch.float32)))
    lse = lse[..., 0].contiguous()
    hs.attend_heads(pool, table, i32(ctx), q, 0.1, cu_q=i32([4, 5, 25]), out=out, lse=lse)
    rest = torch.tensor([t for t in range(30) if not 4 <= t < 25], device="cuda")
    assert bool((out[rest] == 0).all()) and bool((lse[rest] == -math.inf).all())
    check(cache, kv, dim, table, ctx, new, q[4:25], 0.1, out[4:25], lse[4:25])
    none = torch.empty((0, 2), dtype=torch.int32, device="cuda")  # no requests at all
    hs.attend_heads(pool, none, i32([]), q, 0.1, cu_q=i32([0]), out=out, lse=lse)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    z = torch.empty((0, group, dim), dtype=torch.bfloat16, device="cuda")
    assert hs.attend_heads(pool, table, i32(ctx), z, 0.1)[0].shape == z.shape
    no_pages = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    out, lse = hs.attend_heads(pool, no_pages, i32([0, 0]), q, 0.1)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_captured_calls_and_calls_on_other_streams():
    g = gen(17)
    kv, dim, group, R = 2, 128, 4, 3
    pool, cache, table = make(g, [400] * R, kv, dim)
    ctx, q, k, v = i32([250, 63, 330]), normal(g, R, kv * group, dim), normal(g, R, kv, dim), normal(g, R, kv, dim)
    ws = [hs.alloc_heads_workspace() for _ in range(2)]
    out = [torch.zeros_like(q) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            hs.append_heads(pool, table, ctx, k, v)
            hs.attend_heads(pool, table, ctx, q, 0.1, out=out[i], workspace=ws[i])
        graphs.append(graph)
    for step in range(3):
        ctx += 1
        for x in (q, k, v):
            x.copy_(normal(g, *x.shape))
        for i in range(2):
            graphs[i].replay()
        torch.cuda.synchronize()
        got, lse = hs.attend_heads(pool, table, ctx, q, 0.1)
        same(out[0], got)
        same(out[1], got)
        check(cache, kv, dim, table, ctx.tolist(), [1] * R, q, 0.1, got, lse)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    a = hs.attend_heads(pool, table, ctx, q, 0.1, stream=other)[0]
    b = hs.read_heads(pool, table, None, None, 3 * 60, dim, stream=other)[0]
    other.synchronize()
    same(a, got)
    same(b, hs.read_heads(pool, table, None, None, 3 * 60, dim)[0])


def test_two_calls_at_once():
    """Prompts on one stream and single tokens among prompts on another, over the same pages: each has the bits that it has alone."""
    g = gen(23)
    kv, dim, group = 2, 128, 4
    ctx = [1500, 130, 700, 2000]
    pool, _, table = make(g, ctx, kv, dim)
    news = [[300, 130, 500, 64], [1, 40, 1, 900]]
    args = [(i32(ctx), normal(g, sum(new), kv * group, dim), offsets(new)) for new in news]
    alone = [hs.attend_heads(pool, table, lens, q, 0.1, cu_q=cu) for lens, q, cu in args]
    ws = [hs.alloc_heads_workspace() for _ in news]
    status = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in news]
    streams = [torch.cuda.Stream() for _ in news]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [hs.attend_heads(pool, table, lens, q, 0.1, cu_q=cu, workspace=w, status=st, stream=s)
               for (lens, q, cu), w, st, s in zip(args, ws, status, streams)]
    torch.cuda.synchronize()
    for (out, lse), (o, l), st in zip(got, alone, status):
        same(out, o)
        same(lse, l)
        assert int(st) == 0


def test_layers_and_offsets_past_32_bits():
    g = gen(18)
    kv, dim, group = 128, 128, 1  # 2 MB a page: block 1100 begins past 2^31
    blocks = 1100
    pool, (cache,) = empty_pool(blocks, kv, dim, fill=0)
    table = i32([[blocks - 1, 3], [7, blocks - 2]])
    k, v = normal(g, 150, kv, dim), normal(g, 150, kv, dim)
    hs.append_heads(pool, table, i32([70, 80]), k, v, cu=i32([0, 70, 150]))
    rk, rv = hs.read_heads(pool, table, None, i32([0, 70, 150]), 150, dim, dtype=torch.float32)
    for got, x in ((rk, k), (rv, v)):  # a code is within half a step of 4 significant bits, or of the smallest step
        top = x.float().abs().amax()
        assert bool(((got - x.float()).abs() <= (2.0 ** -4 * x.float().abs()).clamp_min(float(top) * 2.0 ** -17)).all())
    q = normal(g, 2, kv, dim)
    out, lse = hs.attend_heads(pool, table, i32([70, 80]), q, 0.1)
    check(cache, kv, dim, table, [70, 80], [1, 1], q, 0.1, out, lse)
    assert bool((cache[100:blocks - 2] == 0).all())


def test_refusals():
    """What the library refuses by itself, with nothing launched."""
    kv, dim = 2, 128
    pool, (cache,) = empty_pool(4, kv, dim)
    table, ctx = i32([[0, 1], [2, 3]]), i32([70, 80])
    q, k = torch.zeros((2, 4, dim), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, kv, dim), dtype=torch.bfloat16, device="cuda")
    small = hs.Pool([torch.zeros((4, 32, 2 * kv * dim + 16), dtype=torch.uint8, device="cuda")])  # pages of another size
    latent = hs.Pool([torch.zeros((4, 64, 656), dtype=torch.uint8, device="cuda")])
    before = hs.launch_count()

    def refused(call):
        with pytest.raises((hs.HSError, ValueError, TypeError)):
            call()

    for other in (small, latent):
        refused(lambda: hs.attend_heads(other, table, ctx, q, 1.0))
        refused(lambda: hs.append_heads(other, table, ctx, k, k))
        refused(lambda: hs.read_heads(other, table, None, None, 2, dim))
    refused(lambda: hs.read_rows(pool, i32([0])))
    refused(lambda: hs.attend_heads(pool, table, ctx, q[:, :3], 1.0))                         # heads that are no multiple
    refused(lambda: hs.attend_heads(pool, table, ctx, q[:, :1], 1.0))
    refused(lambda: hs.attend_heads(pool, table, ctx, q, float("nan")))
    refused(lambda: hs.attend_heads(pool, table, ctx, q, 1.0, layer=1))
    refused(lambda: hs.append_heads(pool, table, ctx, k, k, layer=-1))
    refused(lambda: hs.attend_heads(pool, table, ctx, q, 1.0, workspace=torch.zeros(1000, dtype=torch.uint8, device="cuda")))
    refused(lambda: hs.attend_heads(pool, table, ctx, q, 1.0, workspace=hs.alloc_heads_workspace()[8:]))  # not aligned
    refused(lambda: hs.attend_heads(pool, table, ctx, q, 1.0, out=q[:1].expand(2, -1, -1)))    # results on top of one another
    flat = torch.zeros(4096, dtype=torch.bfloat16, device="cuda")
    refused(lambda: hs.attend_heads(pool, table, ctx, flat[4:4 + 1024].view(2, 4, dim), 1.0))  # 8 bytes off
    refused(lambda: hs.append_heads(pool, table, ctx, flat[:2 * 260].view(2, 260)[:, :256].view(2, kv, dim), k))  # rows of 520 bytes
    refused(lambda: hs.read_heads(pool, table, None, None, 2, dim, k=flat[:256].view(1, kv, dim).expand(2, -1, -1)))
    refused(lambda: hs.read_rows(latent, i32([0, 1]), latent=flat[:512].view(1, 512).expand(2, -1)))
    refused(lambda: hs.append_heads(pool, i32([[0, 1]] * 3), i32([70] * 3), k, k))             # two tokens for three requests
    refused(lambda: hs.attend_heads(pool, torch.empty((0, 2), dtype=torch.int32, device="cuda"), i32([]), q, 1.0))
    assert hs.launch_count() == before
