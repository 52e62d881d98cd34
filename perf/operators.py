"""Cases of the latent-cache operators: appending rows with the position rotation, absorbed attention over row ids and
over pages, and expanded attention for prompts.  `own` selects the framework's kernels; otherwise `run` computes
the same in elementary torch operations in 32 bits."""
import math
import random

import torch

own = False

LATENT, ROPE, NOPE, VDIM, GROUP, PAGE = 512, 64, 128, 128, 128, 64
E4M3_MAX = 448.0
POSITIONS = 131072 + 64


def listed():
    return [
        # one decode step of 64 requests: a row each, 64 query heads to rotate; latency counts
        dict(name="append_decode", op="append", n=64, heads=64, row="fp8", pairs="halves", dtype="bf16"),
        # one prompt chunk of the largest scheduled batch (32768 tokens), 16 heads on this rank
        dict(name="append_prompt", op="append", n=32768, heads=16, row="fp8", pairs="interleaved", dtype="bf16"),
        # the tiny decode batch (4 requests, K = 256): latency
        dict(name="rows_tiny", op="rows", requests=4, positions=1, k=256, heads=16, row="fp8", ctx=4096, fill=1.0),
        # the mixed-residency batch (64 requests, K = 2048)
        dict(name="rows_batch", op="rows", requests=64, positions=1, k=2048, heads=64, row="fp8", ctx=16384, fill=1.0),
        # the largest batch with three speculative positions: 256 requests x 4 positions, lists that share nine tenths
        dict(name="rows_verify", op="rows", requests=256, positions=4, k=2048, heads=64, row="fp8", ctx=8192, fill=1.0),
        # all 128 heads on one rank, an odd list length, a tenth of the ids padding
        dict(name="rows_wide", op="rows", requests=96, positions=1, k=1000, heads=128, row="fp8", ctx=8192, fill=0.9),
        # fully resident decode of a ragged batch, 16 heads on this rank
        dict(name="pages_decode", op="pages", requests=48, positions=1, heads=16, row="fp8", ctx=16384, low=1),
        # two long contexts with four verify positions
        dict(name="pages_long", op="pages", requests=2, positions=4, heads=64, row="fp8", ctx=131072, low=131001),
        # a cache kept in bf16, all 128 heads
        dict(name="pages_bf16", op="pages", requests=32, positions=1, heads=128, row="bf16", ctx=4096, low=3000),
        # a batch of ragged prompts
        dict(name="expanded_prompts", op="expanded", seqs=6, q=2500, low=37, prefix=0, heads=16, causal=True),
        # one long prompt
        dict(name="expanded_long", op="expanded", seqs=1, q=16384, low=16384, prefix=0, heads=8, causal=True),
        # chunked prefill: ragged chunks of up to 512 tokens over a long prefix
        dict(name="expanded_chunk", op="expanded", seqs=4, q=512, low=300, prefix=16000, heads=16, causal=True),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "rows", "rows", "pages", "pages", "expanded", "expanded"])
    row = rng.choice(["fp8", "fp8", "bf16"])
    if op == "append":
        n = _spread(rng, 1, 32768)
        heads = min(rng.choice([8, 16, 24, 32, 64, 128]), 524288 // n)
        return dict(op=op, n=n, heads=max(1, heads), row=row, pairs=rng.choice(["halves", "interleaved"]),
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op == "rows":
        requests, positions = _spread(rng, 1, 200), rng.choice([1, 1, 2, 4])
        return dict(op=op, requests=requests, positions=positions, k=_spread(rng, 33, 2048),
                    heads=rng.choice([4, 8, 16, 20, 32, 64, 64, 96, 128]) if requests * positions <= 400 else rng.choice([8, 16, 32]),
                    row=row, ctx=_spread(rng, 3000, 10000), fill=rng.choice([1.0, 1.0, 0.97, 0.5]))
    if op == "pages":
        ctx = _spread(rng, 50, 131072)
        requests = _spread(rng, 1, max(1, min(160, 262144 // ctx)))
        return dict(op=op, requests=requests, positions=rng.choice([1, 1, 2, 3, 4]), heads=rng.choice([4, 8, 16, 32, 48, 64]),
                    row=row, ctx=ctx, low=rng.choice([1, ctx // 2 + 1, ctx]))
    heads, seqs, causal = rng.choice([4, 8, 16]), rng.choice([1, 2, 3, 5]), rng.random() < 0.8
    if rng.random() < 0.5:
        q, prefix = _spread(rng, 60, 5000 if causal else 3500), 0
    else:
        q, prefix = _spread(rng, 1, 500), _spread(rng, 100, 16000)
    return dict(op=op, seqs=seqs, q=q, low=rng.choice([1, q // 2 + 1, q]), prefix=prefix, heads=heads, causal=causal)


_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _scales(x):
    """Power-of-two scale of each group of 128: the smallest 2^k with amax <= 448 * 2^k, 1 for a group of zeros."""
    amax = x.reshape(*x.shape[:-1], -1, GROUP).abs().amax(-1)
    m, e = torch.frexp(amax)
    k = (e - 9 + (m > 0.875)).clamp_min(-126)
    return torch.where(amax == 0, torch.ones_like(amax), torch.ldexp(torch.ones_like(amax), k))


def _parts(cache, row):
    """Typed views of a byte cache [rows, row_bytes]."""
    if row == "fp8":
        return [cache[:, :512].view(torch.float8_e4m3fn), cache[:, 512:528].view(torch.float32), cache[:, 528:].view(torch.bfloat16)]
    return [cache[:, :1024].view(torch.bfloat16), cache[:, 1024:].view(torch.bfloat16)]


def _store(cache, row, at, latent, rope):
    """Writes rows `at` of a byte cache from latents (32 bits) and rotated keys (bf16)."""
    if row == "fp8":
        s = _scales(latent)
        code = (latent.reshape(-1, 4, GROUP) / s[:, :, None]).reshape(-1, LATENT).to(torch.float8_e4m3fn)
        cache[at, :512] = code.view(torch.uint8)
        cache[at, 512:528] = s.view(torch.uint8)
        cache[at, 528:] = rope.contiguous().view(torch.uint8)
    else:
        cache[at, :1024] = latent.to(torch.bfloat16).view(torch.uint8)
        cache[at, 1024:] = rope.contiguous().view(torch.uint8)


def _make_cache(g, blocks, row):
    """A filled cache: every row holds a normed latent vector with a few larger channels, and a rotated key."""
    cache = torch.empty((blocks * PAGE, 656 if row == "fp8" else 1152), dtype=torch.uint8, device="cuda")
    gain = torch.exp(0.3 * torch.randn(LATENT, generator=g, device="cuda"))
    for a in range(0, blocks * PAGE, 1 << 18):
        n = min(1 << 18, blocks * PAGE - a)
        lat = torch.randn((n, LATENT), generator=g, device="cuda") * gain
        _store(cache, row, slice(a, a + n), lat, _normal(g, n, ROPE))
    return cache


def _handle(state, cache, n, heads):
    if own:
        import sparse_mla_kv_gb300 as hs
        state["pool"] = hs.Pool([cache.view(-1, PAGE, cache.shape[1])])
        if heads:
            state["workspace"] = hs.alloc_attend_workspace("cuda")
    return state


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    state = dict(case)
    if op == "append":
        n, dt = case["n"], _TYPES[case["dtype"]]
        blocks = -(-n // PAGE) + 64
        cache = _make_cache(g, blocks, case["row"])
        freq = 10000.0 ** (-torch.arange(32, device="cuda", dtype=torch.float64) / 32)
        angle = torch.arange(POSITIONS, device="cuda", dtype=torch.float64)[:, None] * freq
        state.update(cache=cache, rotation=torch.cat([angle.cos(), angle.sin()], 1).float(),
                     rows=torch.randperm(blocks * PAGE, generator=g, device="cuda")[:n].int(),
                     positions=torch.randint(0, POSITIONS, (n,), generator=g, device="cuda").int(),
                     latent=_normal(g, n, LATENT, dtype=dt), rope=_normal(g, n, ROPE, dtype=dt),
                     q_rope=_normal(g, n, case["heads"], ROPE, dtype=dt))
        return _handle(state, cache, n, 0)
    if op == "rows":
        R, P, K, H, ctx = case["requests"], case["positions"], case["k"], case["heads"], case["ctx"]
        pages = -(-ctx // PAGE)
        cache = _make_cache(g, R * pages, case["row"])
        table = torch.randperm(R * pages, generator=g, device="cuda").reshape(R, pages)
        # a list per request, of distinct ids; later positions keep nine tenths of it
        ids = torch.rand((R, ctx), generator=g, device="cuda").argsort(1)[:, :min(ctx, K + (P - 1) * (K // 10))]
        keep = K - K // 10
        lists = [ids[:, :K]] + [torch.cat([ids[:, :keep], ids[:, K + p * (K // 10):K + (p + 1) * (K // 10)]], 1)
                                for p in range(P - 1)]
        tok = torch.stack(lists, 1)
        rows = torch.gather(table, 1, (tok // PAGE).reshape(R, -1)).reshape(tok.shape) * PAGE + tok % PAGE
        if case["fill"] < 1:
            rows = torch.where(torch.rand(rows.shape, generator=g, device="cuda") < case["fill"], rows, -1)
        n = R * P
        state.update(cache=cache, rows=rows.reshape(n, K).int().contiguous(), scale=(NOPE + ROPE) ** -0.5,
                     q_latent=_normal(g, n, H, LATENT), q_rope=_normal(g, n, H, ROPE))
        return _handle(state, cache, n, H)
    if op == "pages":
        R, P, H, ctx = case["requests"], case["positions"], case["heads"], case["ctx"]
        lens = torch.randint(min(case["low"], ctx), ctx + 1, (R,), generator=g, device="cuda")
        pages = -(-ctx // PAGE)
        cache = _make_cache(g, R * pages, case["row"])
        state.update(cache=cache, table=torch.randperm(R * pages, generator=g, device="cuda").reshape(R, pages).int(),
                     ctx_len=lens.int(), scale=(NOPE + ROPE) ** -0.5,
                     q_latent=_normal(g, R, P, H, LATENT), q_rope=_normal(g, R, P, H, ROPE))
        return _handle(state, cache, R * P, H)
    B, H = case["seqs"], case["heads"]
    qn, kn = _lengths(case)
    Tq, Tk = sum(qn), sum(kn)
    cu = lambda v: torch.tensor([0] + v, device="cuda").cumsum(0).int()  # noqa: E731
    kv = _normal(g, Tk, H, NOPE + VDIM)  # as the up-projection leaves it: keys and values of a head side by side
    q = _normal(g, Tq, H, NOPE + ROPE)
    state.update(q_nope=q[..., :NOPE], q_rope=q[..., NOPE:].contiguous(), k_nope=kv[..., :NOPE], v=kv[..., NOPE:],
                 k_rope=_normal(g, Tk, ROPE), cu_q=cu(qn), cu_k=cu(kn), qn=qn, kn=kn, scale=(NOPE + ROPE) ** -0.5)
    return state


def _lengths(case):
    """Query and key lengths of an expanded case, the same for every seed; the first sequence has the full length."""
    r = random.Random(str(sorted((k, v) for k, v in case.items() if k != "name")))
    qn = [case["q"]] + [r.randint(min(case["low"], case["q"]), case["q"]) for _ in range(case["seqs"] - 1)]
    kn = [n + (r.randint(case["prefix"] // 2, case["prefix"]) if i else case["prefix"]) for i, n in enumerate(qn)]
    return qn, kn


# ---------------------------------------------------------------------------------------------------------------------
# one pass


def run(s):
    if own:
        return _run_own(s)
    return {"append": _plain_append, "rows": _plain_rows, "pages": _plain_pages, "expanded": _plain_expanded}[s["op"]](s)


def _run_own(s):
    import sparse_mla_kv_gb300 as hs
    if s["op"] == "append":
        q = hs.append_rows(s["pool"], s["rows"], s["latent"], s["rope"], s["positions"], s["rotation"], q_rope=s["q_rope"],
                           interleaved=s["pairs"] == "interleaved")
        return _parts(s["cache"], s["row"]) + [q]
    if s["op"] == "rows":
        return hs.attend_rows(s["pool"], s["rows"], s["q_latent"], s["q_rope"], s["scale"], workspace=s["workspace"])
    if s["op"] == "pages":
        return hs.attend_pages(s["pool"], s["table"], s["ctx_len"], s["q_latent"], s["q_rope"], s["scale"],
                               workspace=s["workspace"])
    return hs.attend_expanded(s["q_nope"], s["q_rope"], s["k_nope"], s["k_rope"], s["v"], s["cu_q"], s["cu_k"], s["scale"],
                              causal=s["causal"])


def _rotate(x, cs, pairs):
    x = x.float()
    cos, sin = cs[..., :32], cs[..., 32:]
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs == "interleaved" else (x[..., :32], x[..., 32:])
    u, v = a * cos - b * sin, b * cos + a * sin
    return torch.stack([u, v], -1).flatten(-2) if pairs == "interleaved" else torch.cat([u, v], -1)


def _plain_append(s):
    cs = s["rotation"][s["positions"].long()]
    _store(s["cache"], s["row"], s["rows"].long(), s["latent"].float(), _rotate(s["rope"], cs, s["pairs"]).to(torch.bfloat16))
    return _parts(s["cache"], s["row"]) + [_rotate(s["q_rope"], cs[:, None], s["pairs"]).to(s["q_rope"].dtype)]


def _values(cache, row, at):
    """Rows `at` in 32 bits: latents [..., 512] and keys [..., 576]."""
    got = cache[at]
    if row == "fp8":
        lat = got[..., :512].view(torch.float8_e4m3fn).float().unflatten(-1, (4, GROUP))
        lat = (lat * got[..., 512:528].view(torch.float32)[..., None]).flatten(-2)
        rope = got[..., 528:].view(torch.bfloat16).float()
    else:
        lat, rope = got[..., :1024].view(torch.bfloat16).float(), got[..., 1024:].view(torch.bfloat16).float()
    return lat, torch.cat([lat, rope], -1)


def _softmax_product(scores, values):
    """Normalised sums of values [B, n, d] under scores [B, m, n] (-inf: masked; a row of nothing gives zeros), and the
    log of the sums."""
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, values) / torch.where(total == 0, torch.ones_like(total), total)
    return out, (top + torch.log(total))[..., 0]


def _plain_rows(s):
    lat, key = _values(s["cache"], s["row"], s["rows"].long().clamp_min(0))
    q = torch.cat([s["q_latent"], s["q_rope"]], -1).float()
    scores = torch.matmul(q, key.transpose(1, 2)) * s["scale"]
    out, lse = _softmax_product(scores.masked_fill((s["rows"] < 0)[:, None], -math.inf), lat)
    return out.to(torch.bfloat16), lse


def _plain_pages(s):
    R, P, H = s["q_latent"].shape[:3]
    j = torch.arange(s["table"].shape[1] * PAGE, device="cuda")
    lat, key = _values(s["cache"], s["row"], s["table"].long()[:, j // PAGE] * PAGE + j % PAGE)
    q = torch.cat([s["q_latent"], s["q_rope"]], -1).float().reshape(R, P * H, -1)
    scores = torch.matmul(q, key.transpose(1, 2)) * s["scale"]
    seen = s["ctx_len"].long()[:, None] - P + 1 + torch.arange(P, device="cuda")  # keys that a position sees
    hidden = j >= seen.repeat_interleave(H, 1)[..., None]
    out, lse = _softmax_product(scores.masked_fill(hidden, -math.inf), lat)
    return out.to(torch.bfloat16).reshape(R, P, H, LATENT), lse.reshape(R, P, H)


def _plain_expanded(s):
    # padded to the longest sequence: [seqs, heads, length, dim]
    B, mq, mk = len(s["qn"]), max(s["qn"]), max(s["kn"])
    iq, ik = torch.arange(mq, device="cuda"), torch.arange(mk, device="cuda")
    lq, lk = (s[c][1:] - s[c][:-1] for c in ("cu_q", "cu_k"))
    at = (s["cu_k"][:-1, None] + ik).clamp_max(s["k_rope"].shape[0] - 1).long()
    key = torch.cat([s["k_nope"], s["k_rope"][:, None].expand(-1, s["heads"], -1)], -1).float()[at].transpose(1, 2)
    value = s["v"].float()[at].transpose(1, 2)
    aq = (s["cu_q"][:-1, None] + iq).clamp_max(s["q_rope"].shape[0] - 1).long()
    q = torch.cat([s["q_nope"], s["q_rope"]], -1).float()[aq].transpose(1, 2)
    scores = torch.matmul(q, key.transpose(2, 3)) * s["scale"]
    hidden = (ik >= lk[:, None])[:, None, None]
    if s["causal"]:
        hidden = hidden | (ik > (iq + (lk - lq)[:, None])[..., None])[:, None]
    out, lse = _softmax_product(scores.masked_fill(hidden, -math.inf), value)
    there = iq < lq[:, None]
    return out.transpose(1, 2)[there].to(torch.bfloat16), lse.transpose(1, 2)[there]


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    op = case["op"]
    rb = 656 if case.get("row") == "fp8" else 1152
    if op == "append":
        s = 4 if case["dtype"] == "fp32" else 2
        per = (LATENT + ROPE) * s + rb + 2 * case["heads"] * ROPE * s + 256 + 8
        return {"bytes": case["n"] * per, "flops": case["n"] * (LATENT * 3 + (case["heads"] + 1) * ROPE * 3)}
    if op == "rows":
        n, K, H, P = case["requests"] * case["positions"], case["k"], case["heads"], case["positions"]
        distinct = case["requests"] * (K + (P - 1) * (K // 10)) * case["fill"]
        return {"bytes": distinct * rb + n * (4 * K + H * (2 * 576 + 2 * 512 + 4)),
                "flops": 2 * n * K * case["fill"] * H * (576 + 512)}
    if op == "pages":
        P, H = case["positions"], case["heads"]
        keys = case["requests"] * (min(case["low"], case["ctx"]) + case["ctx"]) / 2
        return {"bytes": keys * (rb + 4 / PAGE) + case["requests"] * P * H * (2 * 576 + 2 * 512 + 4),
                "flops": 2 * keys * P * H * (576 + 512)}
    H, (qn, kn) = case["heads"], _lengths(case)
    pairs = sum(q * k - (q * (q - 1) // 2 if case["causal"] else 0) for q, k in zip(qn, kn))
    return {"bytes": sum(qn) * H * (2 * (192 + 128) + 4) + sum(kn) * (2 * H * 256 + 2 * 64), "flops": 2 * pairs * H * (192 + 128)}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    op = case["op"]
    if op == "append":
        at = s["rows"].long()
        old = [p.double() for p in _parts(s["cache"], s["row"])]
        x = s["latent"].double()
        turn = torch.complex(*(t.double() for t in s["rotation"][s["positions"].long()].split(32, 1)))

        def turned(v):
            v = v.double()
            if s["pairs"] == "interleaved":
                w = torch.view_as_complex(v.unflatten(-1, (32, 2)).contiguous())
                return torch.view_as_real(w * turn.view(len(turn), *[1] * (v.dim() - 2), 32)).flatten(-2)
            w = torch.complex(v[..., :32].contiguous(), v[..., 32:].contiguous()) * turn.view(len(turn), *[1] * (v.dim() - 2), 32)
            return torch.cat([w.real, w.imag], -1)

        if s["row"] == "fp8":
            top = x.unflatten(1, (4, GROUP)).abs().amax(-1)
            scale = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX) - 1e-12).clamp_min(-126)), 1.0)
            old[0][at] = x / scale.repeat_interleave(GROUP, 1)
            old[1][at] = scale
        else:
            old[0][at] = x
        old[-1][at] = turned(s["rope"])
        return old + [turned(s["q_rope"])]
    if op == "rows":
        got = [_attend_exact(s, s["rows"][i][s["rows"][i] >= 0].long(), s["q_latent"][i], s["q_rope"][i])
               for i in range(len(s["rows"]))]
        return torch.stack([o for o, _ in got]), torch.stack([l for _, l in got])
    if op == "pages":
        R, P = s["q_latent"].shape[:2]
        outs, lses = [], []
        for r, length in enumerate(s["ctx_len"].tolist()):
            for p in range(P):
                j = torch.arange(max(0, length - P + 1 + p), device="cuda")
                o, l = _attend_exact(s, s["table"][r].long()[j // PAGE] * PAGE + j % PAGE, s["q_latent"][r, p], s["q_rope"][r, p])
                outs.append(o)
                lses.append(l)
        return torch.stack(outs).unflatten(0, (R, P)), torch.stack(lses).unflatten(0, (R, P))
    outs, lses, a, b = [], [], 0, 0
    for n, m in zip(s["qn"], s["kn"]):
        o, l = [], []
        for h in range(s["heads"]):
            z = s["q_nope"][a:a + n, h].double() @ s["k_nope"][b:b + m, h].double().T
            z = (z + s["q_rope"][a:a + n, h].double() @ s["k_rope"][b:b + m].double().T) * s["scale"]
            if s["causal"]:
                z = z + torch.full((n, m), -math.inf, device="cuda", dtype=torch.float64).triu(m - n + 1)
            l.append(torch.logsumexp(z, 1))
            o.append(torch.softmax(z, 1) @ s["v"][b:b + m, h].double())
        outs.append(torch.stack(o, 1))
        lses.append(torch.stack(l, 1))
        a, b = a + n, b + m
    return torch.cat(outs), torch.cat(lses)


def _attend_exact(s, at, q_latent, q_rope):
    """One query token [heads, ...] over the cache rows `at`, in 64 bits."""
    H = q_latent.shape[0]
    if not len(at):
        return (torch.zeros((H, LATENT), device="cuda", dtype=torch.float64),
                torch.full((H,), -math.inf, device="cuda", dtype=torch.float64))
    b = s["cache"].index_select(0, at)
    if s["row"] == "fp8":
        c = b[:, :512].contiguous().view(torch.float8_e4m3fn).double()
        c = c * b[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(GROUP, 1)
        r = b[:, 528:].contiguous().view(torch.bfloat16).double()
    else:
        b = b.view(torch.bfloat16).double()
        c, r = b[:, :512], b[:, 512:]
    z = (q_latent.double() @ c.T + q_rope.double() @ r.T) * s["scale"]
    return torch.softmax(z, 1) @ c, torch.logsumexp(z, 1)
