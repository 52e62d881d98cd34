"""attend_heads where scores are not finite: queries and keys that hold NaN, queries that hold an infinity.

By the formulas, over the scores s of the tokens that a query sees:
  one is NaN                     out and lse are NaN
  else one is +infinity          out is NaN (infinity / infinity), lse is +infinity
  else all are -infinity         out is NaN (0 / 0), lse is -infinity
  it sees no token               out is zero, lse is -infinity
and everything else is finite, within the tolerances of test_gpu_heads.py.  An infinite element times a code is an infinity, or NaN where the
code is zero, in 16 bits as in 64; scores are made in 64 bits here, so that which case it is needs no tolerance.

The contexts lie within one worker's run of pages or are cut over many: either must give the same."""
import math

import pytest

torch = pytest.importorskip("torch")
import sparse_mla_kv_gb300 as hs  # noqa: E402
from test_gpu_heads import F8, PAGE, gen, i32, make, normal, offsets, parts, values  # noqa: E402

pytestmark = pytest.mark.gpu


def key_nan(cache, kv, dim, table, r, token, head):
    parts(cache, kv, dim)[0][int(table[r, token // PAGE]), head, :, token % PAGE, 7] = 0xFF


def expect(q, k, v, sv, seen, scale, dtype):
    """test_gpu_heads.expect for all query heads of a request at once: q [H][n][D], k and v [H][m][D], sv [H][m], seen [n][m], with
    the scores, of which those that are not finite are left out."""
    m, D = k.shape[1:]
    s = (q @ k.transpose(1, 2)) * scale
    shown = seen & s.isfinite()
    q, k = q.nan_to_num(0, 0, 0), k.nan_to_num()
    mag = abs(scale) * ((D / 16 + 16) * 2.0 ** -23 * (q.abs() @ k.abs().transpose(1, 2)) +
                        2.0 ** -23 * q.abs().amax(2)[..., None] * k.abs().sum(2)[:, None])
    es = mag.masked_fill(~shown, 0).amax(2)
    T = s.masked_fill(~shown, 0).abs().amax(2) * math.log2(math.e) + sv.log2().abs().amax(1)[:, None] + 32
    et = 5 * T * 2.0 ** -24 * math.log(2)
    z = s.masked_fill(~shown, -math.inf)
    lse = torch.logsumexp(z, 2)
    w = torch.exp(z - torch.where(lse == -math.inf, 0, lse)[..., None])
    out, a = w @ v.nan_to_num(), w @ v.nan_to_num().abs()
    tol = (2.0 ** -11 + 2 * (es + 3 * et) + 2.0 ** -19 + (m / 8 + 64) * 2.0 ** -23)[..., None] * a
    tol = tol + m * 2.0 ** -32 * 448 * (w * sv[:, None]).amax(2)[..., None]
    tol = tol + torch.finfo(dtype).eps / 2 * (out.abs() + tol) + (2.0 ** -25 if dtype is torch.float16 else 0)
    return s, out, lse, tol, es + 3 * et + 2.0 ** -19 + (m / 16 + 32) * 2.0 ** -23 + 2.0 ** -22 * torch.where(lse == -math.inf, 0, lse).abs()


def check(cache, kv, dim, table, ctx, new, q, scale, out, lse, causal):
    """Compares, and returns how many (query, head) there are of each of the four cases and of finite ones."""
    t0, group, kinds = 0, q.shape[1] // kv, 0
    for r, n in enumerate(new):
        m = max(ctx[r], 0)
        if m == 0:
            assert bool(out[t0:t0 + n].eq(0).all() & lse[t0:t0 + n].eq(-math.inf).all()), r
            t0 += n
            continue
        k, v, sv = (x.repeat_interleave(group, 1).transpose(0, 1) for x in values(cache, kv, dim, table[r], m))
        last = ctx[r] - n + 1 + torch.arange(n, device="cuda") if causal else torch.full((n,), ctx[r], device="cuda")
        seen = torch.arange(m, device="cuda")[None] < last[:, None]
        s, o, l, to, tl = expect(q[t0:t0 + n].double().transpose(0, 1), k, v, sv, seen, scale, q.dtype)
        nan = (s.isnan() & seen).any(2)
        up = (s.eq(math.inf) & seen).any(2) & ~nan
        some = seen.any(1).expand_as(nan)
        down = some & ~nan & ~up & (s.eq(-math.inf) | ~seen).all(2)
        fine = some & ~nan & ~up & ~down
        # (a NaN value that is seen: that element; the tests put them only where all keys are NaN too)
        got, gl = out[t0:t0 + n].double().transpose(0, 1), lse[t0:t0 + n].double().T
        ok = torch.stack([got[nan | up | down].isnan().all(), gl[nan].isnan().all(), gl[up].eq(math.inf).all(),
                          gl[down | ~some].eq(-math.inf).all(), got[~some].eq(0).all(),
                          ((got - o).abs() <= to)[fine].all(), ((gl - l).abs() <= tl)[fine].all()]).tolist()
        assert all(ok), (r, ctx[r], n, ok)
        kinds = kinds + torch.stack([x.sum() for x in (nan, up, down, ~some, fine)])
        t0 += n
    return kinds.tolist()


def poison_queries(g, q, group):
    """A third of the query rows each: a NaN; an infinity in dimension 5; as they were.  Infinities of both signs."""
    kind = torch.randint(0, 3, q.shape[:2], generator=g, device="cuda")
    sign = torch.where(torch.rand(q.shape[:2], generator=g, device="cuda") < 0.5, -math.inf, math.inf).to(q.dtype)
    q[..., 9] = torch.where(kind == 0, math.nan, q[..., 9])
    q[..., 5] = torch.where(kind == 1, sign, q[..., 5])


def signed_codes(cache, kv, dim):
    """Dimension 5 of all keys is 1 in even heads: infinite queries give scores of one sign there."""
    one = int(torch.ones(1).to(F8).view(torch.uint8))
    parts(cache, kv, dim)[0][:, ::2, 0, :, 5] = one


# kv, dim, group, dtype, contexts, new tokens
STEPS = [
    (2, 128, 4, torch.bfloat16, [1, 40, 64, 0, 65, 700], [1] * 6),
    (8, 64, 8, torch.float16, [1 + i % 64 for i in range(300)], [1] * 300),         # whole units
    (1, 128, 16, torch.bfloat16, [9000], [1]),                                      # cut into many
    (2, 64, 5, torch.float16, [3000, 17, 640], [2, 2, 2]),
    (2, 128, 8, torch.bfloat16, [40, 4, 5000, 2], [4, 4, 4, 4]),                    # two warps a worker, queries that see nothing
    (8, 128, 8, torch.bfloat16, [200 + i for i in range(200)], [1 + i % 4 for i in range(200)]),
]
PROMPTS = [
    (2, 128, 4, torch.bfloat16, [300, 40, 9, 700], [300, 40, 20, 100]),
    (2, 64, 4, torch.float16, [300, 40, 9, 700], [300, 40, 20, 100]),
    (1, 128, 8, torch.bfloat16, [9000], [30]),                                      # cut into many
    (1, 64, 8, torch.float16, [9000], [30]),
    (2, 128, 8, torch.bfloat16, [10 + i for i in range(300)], [5 + i % 20 for i in range(300)]),  # whole items, some of more than they see
    (2, 64, 8, torch.bfloat16, [10 + i for i in range(300)], [5 + i % 20 for i in range(300)]),
]


def queries_case(kv, dim, group, dtype, ctx, new, causal):
    g = gen(31)
    pool, cache, table = make(g, ctx, kv, dim, spread=2)
    signed_codes(cache, kv, dim)
    q = normal(g, sum(new), kv * group, dim, dtype=dtype)
    poison_queries(g, q, group)
    args = pool, table, i32(ctx), q, 0.1
    out, lse = hs.attend_heads(*args, cu_q=offsets(new), causal=causal)
    kinds = check(cache, kv, dim, table, ctx, new, q, 0.1, out, lse, causal)
    assert kinds[0] and kinds[4] and (kinds[1] and kinds[2] or sum(new) < 6)
    if len(set(new)) == 1:
        out2, lse2 = hs.attend_heads(*args, causal=causal)
        check(cache, kv, dim, table, ctx, new, q, 0.1, out2, lse2, causal)


def all_keys_case(kv, dim, group, dtype, ctx, new, causal):
    """Every second request has nothing but NaN keys in head 0, and NaN values with them."""
    g = gen(32)
    pool, cache, table = make(g, ctx, kv, dim)
    k, v, _ = parts(cache, kv, dim)
    for r in range(0, len(ctx), 2):
        b = table[r].long()
        k[b, 0], v[b, 0] = 0x7F, 0xFF
    q = normal(g, sum(new), kv * group, dim, dtype=dtype)
    out, lse = hs.attend_heads(pool, table, i32(ctx), q, 0.1, cu_q=offsets(new), causal=causal)
    kinds = check(cache, kv, dim, table, ctx, new, q, 0.1, out, lse, causal)
    assert kinds[0]


@pytest.mark.parametrize("kv,dim,group,dtype,ctx,new", STEPS)
@pytest.mark.parametrize("causal", [True, False])
def test_steps_with_queries_that_are_not_finite(kv, dim, group, dtype, ctx, new, causal):
    queries_case(kv, dim, group, dtype, ctx, new, causal)


@pytest.mark.parametrize("kv,dim,group,dtype,ctx,new", STEPS)
@pytest.mark.parametrize("causal", [True, False])
def test_steps_with_nothing_but_nan_keys(kv, dim, group, dtype, ctx, new, causal):
    all_keys_case(kv, dim, group, dtype, ctx, new, causal)


def one_key_case(dim, place, full, n, group, kv, many):
    """The newest token's key is NaN, at some place of its page: its page begins with it, or a thread's tokens do."""
    g = gen(33)
    ctx, new = [PAGE * full + place + 1] * many, [n] * many
    pool, cache, table = make(g, ctx, kv, dim)
    for r in range(0, many, 2):
        key_nan(cache, kv, dim, table, r, ctx[r] - 1, kv - 1)
    q = normal(g, sum(new), kv * group, dim)
    out, lse = hs.attend_heads(pool, table, i32(ctx), q, 0.1, cu_q=offsets(new))
    kinds = check(cache, kv, dim, table, ctx, new, q, 0.1, out, lse, True)
    assert kinds[0] == group * -(-many // 2)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("place", [0, 15, 16, 32, 48, 63])
def test_steps_with_a_nan_key_in_the_newest_token(dim, place):
    for full, kv, many in ((0, 2, 1), (1, 32, 80), (5, 2, 2), (90, 2, 1)):
        one_key_case(dim, place, full, 1, 4, kv, many)
        one_key_case(dim, place, full, 3, 8, kv, many)


@pytest.mark.parametrize("kv,dim,group,dtype,ctx,new", PROMPTS)
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_with_queries_that_are_not_finite(kv, dim, group, dtype, ctx, new, causal):
    queries_case(kv, dim, group, dtype, ctx, new, causal)


@pytest.mark.parametrize("kv,dim,group,dtype,ctx,new", PROMPTS)
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_with_nothing_but_nan_keys(kv, dim, group, dtype, ctx, new, causal):
    all_keys_case(kv, dim, group, dtype, ctx, new, causal)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("place", [0, 1, 31, 63])
def test_prompts_with_a_nan_key_in_the_newest_token(dim, place):
    for full, kv, n, many in ((0, 2, 40, 1), (1, 16, 20, 40), (2, 16, 20, 40), (5, 2, 150, 2), (90, 2, 70, 1), (91, 1, 40, 1)):
        one_key_case(dim, place, full, n, 4, kv, many)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("ctx", [[200], [33] * 200, [3000]])
def test_prompts_with_a_nan_key_in_the_first_token(dim, ctx):
    """Every query sees it; the first of a prompt sees nothing else."""
    g = gen(34)
    kv, group = 2, 4
    pool, cache, table = make(g, ctx, kv, dim)
    for r in range(len(ctx)):
        key_nan(cache, kv, dim, table, r, 0, 1)
    q = normal(g, sum(ctx), kv * group, dim)
    out, lse = hs.attend_heads(pool, table, i32(ctx), q, 0.1, cu_q=offsets(ctx))
    kinds = check(cache, kv, dim, table, ctx, ctx, q, 0.1, out, lse, True)
    assert kinds[0] == group * sum(ctx) and kinds[4] == group * sum(ctx)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [[1, 1, 1], [3, 40, 1]])
@pytest.mark.parametrize("scale", [0.0, -0.0])
def test_a_scale_of_zero_does_not_hide_queries_that_are_not_finite(dim, new, scale):
    """Zero times an infinity is NaN."""
    g = gen(35)
    kv, group, ctx = 2, 4, [700, 90, 64]
    pool, cache, table = make(g, ctx, kv, dim)
    signed_codes(cache, kv, dim)
    q = normal(g, sum(new), kv * group, dim)
    poison_queries(g, q, group)
    out, lse = hs.attend_heads(pool, table, i32(ctx), q, scale, cu_q=offsets(new))
    kinds = check(cache, kv, dim, table, ctx, new, q, scale, out, lse, True)
    assert kinds[0] and kinds[4] and not kinds[1] and not kinds[2]
