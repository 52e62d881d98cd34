"""Cases of the operators on pages of grouped heads in 8 bits, and of reading rows back: quantising keys and values as they are
written, with a scale for each page and head; reading them back; attention over them from single tokens to prompts; and
reading latent rows back.  `own` selects the framework's kernels; otherwise `run` computes the same in elementary torch
operations in 32 bits.

A page holds 64 tokens of one layer.  Of each head: the keys' e4m3 codes, [dim / 64][token][64 dims], then the values' codes,
[dim / 64][64 dims][token].  Behind the heads: a float for each head's keys, then one for each head's values; value = code x
scale."""
import math
import random

import torch

own = False

PAGE, LATENT, ROPE, GROUP = 64, 512, 64, 128
E4M3_MAX = 448.0


def listed():
    return [
        # one decode step of the mixed-residency batch (64 requests): a token each; latency counts
        dict(name="append_step", op="append", seqs=64, q=1, low=1, prefix=16383, kv=8, dim=128, dtype="bf16"),
        # a verify step of the largest batch: 256 requests, four positions each, which often cross into a new page
        dict(name="append_verify", op="append", seqs=256, q=4, low=4, prefix=8000, kv=4, dim=64, dtype="fp16"),
        # prompt chunks of the largest scheduled batch (32768 tokens in all), behind prefixes that end inside a page
        dict(name="append_prompt", op="append", seqs=5, q=8192, low=4001, prefix=1000, kv=8, dim=128, dtype="bf16"),
        # a short prefix of three requests, handed to a layer that runs on fp32
        dict(name="read_heads_short", op="read_heads", seqs=3, n=700, low=1, start=90, kv=3, dim=64, dtype="fp32"),
        # the prefixes of 16 requests that share none
        dict(name="read_heads_prefix", op="read_heads", seqs=16, n=8000, low=500, start=0, kv=8, dim=128, dtype="bf16"),
        # the rows that the resolver hands back for the tiny decode batch (4 requests, K = 256)
        dict(name="read_rows_tiny", op="read_rows", n=1024, row="fp8", fill=0.9, dtype="bf16"),
        # a reused prefix of 131072 tokens, read back to be expanded
        dict(name="read_rows_prefix", op="read_rows", n=131072, row="fp8", fill=1.0, dtype="bf16"),
        # the tiny decode batch (4 requests): latency
        dict(name="attend_tiny", op="attend", seqs=4, q=1, low=1, prefix=4095, ragged=False, kv=8, group=4, dim=128, dtype="bf16",
             causal=True),
        # one decode step of the mixed-residency batch, ragged contexts
        dict(name="attend_batch", op="attend", seqs=64, q=1, low=1, prefix=16383, ragged=True, kv=8, group=8, dim=128, dtype="bf16",
             causal=True),
        # two long contexts with four verify positions, two heads of keys and values on this rank
        dict(name="attend_long", op="attend", seqs=2, q=4, low=4, prefix=131000, ragged=False, kv=2, group=16, dim=128,
             dtype="bf16", causal=True),
        # chunked prefill: ragged chunks of up to 512 tokens over a long prefix
        dict(name="attend_chunk", op="attend", seqs=4, q=512, low=300, prefix=16000, ragged=True, kv=4, group=8, dim=128,
             dtype="bf16", causal=True),
        # one long prompt with narrow heads
        dict(name="attend_prompt", op="attend", seqs=1, q=12000, low=12000, prefix=0, ragged=False, kv=4, group=3, dim=64,
             dtype="fp16", causal=True),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "read_heads", "read_rows", "attend", "attend", "attend", "attend"])
    dim, dtype = rng.choice([64, 128, 128]), rng.choice(["bf16", "bf16", "fp16", "fp32"])
    kv = rng.choice([1, 2, 3, 4, 5, 8, 8])
    if op == "append":
        q = _spread(rng, 1, 8192)
        return dict(op=op, seqs=_spread(rng, 1, max(1, min(300, 32768 // q))), q=q, low=rng.choice([1, q // 2 + 1, q]),
                    prefix=rng.choice([0, _spread(rng, 1, 4000)]), kv=kv, dim=dim, dtype=dtype)
    if op == "read_heads":
        n = _spread(rng, 1, 16000)
        return dict(op=op, seqs=_spread(rng, 1, max(1, min(64, 64000 // n))), n=n, low=rng.choice([1, n // 2 + 1, n]),
                    start=rng.choice([0, 0, _spread(rng, 1, 1000)]), kv=kv, dim=dim, dtype=dtype)
    if op == "read_rows":
        return dict(op=op, n=_spread(rng, 1, 131072), row=rng.choice(["fp8", "fp8", "bf16"]), fill=rng.choice([1.0, 1.0, 0.9, 0.4]),
                    dtype=dtype)
    dtype, ragged = rng.choice(["bf16", "bf16", "fp16"]), rng.random() < 0.7
    kind = rng.choice(["step", "step", "verify", "chunk", "prompt"])
    if kind in ("step", "verify"):
        prefix = _spread(rng, 1, 130000)
        return dict(op=op, seqs=_spread(rng, 1, max(1, min(128, 400000 // prefix))), q=1 if kind == "step" else rng.choice([2, 3, 4]),
                    low=1, prefix=prefix, ragged=ragged, kv=kv, group=rng.choice([1, 2, 4, 5, 7, 8, 8, 12, 16]), dim=dim, dtype=dtype,
                    causal=rng.random() < 0.9)
    group = rng.choice([1, 2, 4, 8]) if kv <= 4 else rng.choice([1, 2, 4])
    if kind == "chunk":
        q = _spread(rng, 5, 512)
        return dict(op=op, seqs=rng.choice([1, 2, 3, 4]), q=q, low=rng.choice([1, q // 2 + 1, q]), prefix=_spread(rng, 100, 16000),
                    ragged=ragged, kv=kv, group=group, dim=dim, dtype=dtype, causal=rng.random() < 0.9)
    q = _spread(rng, 60, 4000)
    return dict(op=op, seqs=rng.choice([1, 2, 3]), q=q, low=rng.choice([1, q // 2 + 1, q]), prefix=0, ragged=ragged, kv=kv, group=group,
                dim=dim, dtype=dtype, causal=rng.random() < 0.8)


_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _power(amax):
    """The smallest power of two, at least 2^-126, that brings amax to 448 or less."""
    m, e = torch.frexp(amax)
    return torch.ldexp(torch.ones_like(amax), (e - 9 + (m > 0.875)).clamp_min(-126))


def _lengths(case):
    """New tokens and contexts (those included) of each request, the same for every seed; the first has the full lengths."""
    r = random.Random(str(sorted((k, v) for k, v in case.items() if k != "name")))
    q = [case["q"]] + [r.randint(min(case["low"], case["q"]), case["q"]) for _ in range(case["seqs"] - 1)]
    even = not case.get("ragged", True)  # every request has the same number of tokens
    if even:
        q = [case["q"]] * case["seqs"]
    old = [case["prefix"]] + [r.randint(case["prefix"] // 8, case["prefix"]) for _ in range(case["seqs"] - 1)]
    return q, [a + b for a, b in zip(q, old)]


def _spans(case):
    """First token and number of tokens that each request reads."""
    r = random.Random(str(sorted((k, v) for k, v in case.items() if k != "name")))
    n = [case["n"]] + [r.randint(min(case["low"], case["n"]), case["n"]) for _ in range(case["seqs"] - 1)]
    return [r.randint(0, case["start"]) for _ in n], n


def _views(cache, kv, dim):
    """Codes of the keys [block][head][dim / 64][token][64], of the values [block][head][dim / 64][64][token], scales
    [block][2][head], as views of a byte cache [block][64][row bytes]."""
    flat = cache.view(cache.shape[0], -1)
    codes = flat[:, :kv * 2 * dim * PAGE].unflatten(1, (kv, 2, dim // 64, 64, 64)).view(torch.float8_e4m3fn)
    scales = flat[:, kv * 2 * dim * PAGE:].view(torch.float32)[:, :2 * kv].unflatten(1, (2, kv))
    return codes[:, :, 0], codes[:, :, 1], scales


def _codes(codes, *index):
    """Codes picked by an index, in 32 bits."""
    return codes.view(torch.uint8)[index].view(torch.float8_e4m3fn).float()


def _make_heads(g, blocks, kv, dim):
    """A filled cache: keys with a few larger channels, values without, every page and head of its own size."""
    cache = torch.zeros((blocks, PAGE, 2 * kv * dim + 16), dtype=torch.uint8, device="cuda")
    k, v, scales = _views(cache, kv, dim)
    gain = torch.exp(0.5 * torch.randn((kv, dim // 64, 1, 64), generator=g, device="cuda"))
    step = max(1, (1 << 27) // (kv * dim * PAGE))
    for a in range(0, blocks, step):
        n = min(step, blocks - a)
        for at, (codes, by) in enumerate(((k, gain), (v, torch.ones((kv, dim // 64, 64, 1), device="cuda")))):
            x = torch.randn((n, kv, dim // 64, 64, 64), generator=g, device="cuda") * by
            x *= torch.exp(0.2 * torch.randn((n, kv, 1, 1, 1), generator=g, device="cuda"))
            s = _power(x.abs().amax((2, 3, 4)))
            codes[a:a + n] = (x / s[:, :, None, None, None]).to(torch.float8_e4m3fn)
            scales[a:a + n, at] = s
    return cache


def _make_rows(g, n, row):
    """Latent rows: 512 values (e4m3 with a scale for each 128, or bf16), then 64 rotated key values in bf16."""
    cache = torch.empty((n, 656 if row == "fp8" else 1152), dtype=torch.uint8, device="cuda")
    gain = torch.exp(0.3 * torch.randn(LATENT, generator=g, device="cuda"))
    for a in range(0, n, 1 << 18):
        m = min(1 << 18, n - a)
        x = torch.randn((m, LATENT), generator=g, device="cuda") * gain
        if row == "fp8":
            s = _power(x.unflatten(1, (4, GROUP)).abs().amax(-1))
            cache[a:a + m, :512] = (x / s.repeat_interleave(GROUP, 1)).to(torch.float8_e4m3fn).view(torch.uint8)
            cache[a:a + m, 512:528] = s.view(torch.uint8)
        else:
            cache[a:a + m, :1024] = x.to(torch.bfloat16).view(torch.uint8)
        cache[a:a + m, -128:] = _normal(g, m, ROPE).view(torch.uint8)
    return cache


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    state = dict(case, dtype=_TYPES[case["dtype"]])
    if op == "read_rows":
        blocks = case["n"] // PAGE + 64
        cache = _make_rows(g, blocks * PAGE, case["row"]).view(blocks, PAGE, -1)
        rows = torch.randperm(blocks * PAGE, generator=g, device="cuda")[:case["n"]].int()
        if case["fill"] < 1:
            rows = torch.where(torch.rand(rows.shape, generator=g, device="cuda") < case["fill"], rows, -1)
        state.update(rows=rows)
    else:
        kv, dim = case["kv"], case["dim"]
        cu = lambda v: torch.tensor([0] + v, device="cuda").cumsum(0).int()  # noqa: E731
        if op == "read_heads":
            start, n = _spans(case)
            longest = max(a + b for a, b in zip(start, n))
            state.update(start=torch.tensor(start, device="cuda").int(), cu=cu(n), tokens=sum(n), n=n, first=start)
        else:
            qn, kn = _lengths(case)
            longest = max(kn)
            state.update(ctx_len=torch.tensor(kn, device="cuda").int(), cu=cu(qn), qn=qn, kn=kn)
        pages = -(-longest // PAGE)
        cache = _make_heads(g, case["seqs"] * pages, kv, dim)
        state["table"] = torch.randperm(case["seqs"] * pages, generator=g, device="cuda").reshape(-1, pages).int()
        if op == "append":
            # some new tokens are larger than what their page holds, so that its scale has to grow
            size = torch.exp(0.5 * torch.randn((2, sum(qn), 1, 1), generator=g, device="cuda"))
            state["k"], state["v"] = ((_normal(g, sum(qn), kv, dim) * s).to(state["dtype"]) for s in size)
        if op == "attend":
            state.update(q=_normal(g, sum(qn), kv * case["group"], dim, dtype=state["dtype"]), scale=dim ** -0.5)
            if not case["ragged"]:
                state["cu"] = None
    state["cache"] = cache
    if own:
        import sparse_mla_kv_gb300 as hs
        state["pool"] = hs.Pool([cache])
        if op == "attend":
            state["workspace"] = hs.alloc_heads_workspace("cuda")
    return state


# ---------------------------------------------------------------------------------------------------------------------
# one pass


def run(s):
    if own:
        return _run_own(s)
    return {"append": _plain_append, "read_heads": _plain_read_heads, "read_rows": _plain_read_rows, "attend": _plain_attend}[s["op"]](s)


def _run_own(s):
    import sparse_mla_kv_gb300 as hs
    if s["op"] == "append":
        hs.append_heads(s["pool"], s["table"], s["ctx_len"], s["k"], s["v"], cu=s["cu"])
        return _views(s["cache"], s["kv"], s["dim"])
    if s["op"] == "read_heads":
        return hs.read_heads(s["pool"], s["table"], s["start"], s["cu"], s["tokens"], s["dim"], dtype=s["dtype"])
    if s["op"] == "read_rows":
        return hs.read_rows(s["pool"], s["rows"], dtype=s["dtype"])
    return hs.attend_heads(s["pool"], s["table"], s["ctx_len"], s["q"], s["scale"], cu_q=s["cu"], causal=s["causal"],
                           workspace=s["workspace"])


def _places(table, cu, first):
    """Block and place in it of every token, for requests whose tokens are cu[r] .. cu[r + 1] - 1 and begin at first[r]."""
    n = (cu[1:] - cu[:-1]).long()
    r = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n)
    pos = torch.arange(len(r), device="cuda") - cu.long()[r] + first.long()[r]
    return table.long()[r, pos // PAGE], pos % PAGE


def _plain_append(s):
    k, v, scales = _views(s["cache"], s["kv"], s["dim"])
    block, place = _places(s["table"], s["cu"], s["ctx_len"] - (s["cu"][1:] - s["cu"][:-1]))
    touched, at = torch.unique(block, return_inverse=True)
    lowest = torch.full((len(touched),), PAGE, device="cuda").scatter_reduce(0, at, place, "amin")
    older = torch.arange(PAGE, device="cuda") < lowest[:, None]  # tokens that the page holds already
    for i, (codes, new) in enumerate(((k, s["k"].float()), (v, s["v"].float()))):
        amax = torch.zeros((len(touched), s["kv"]), device="cuda")
        amax = amax.scatter_reduce(0, at[:, None].expand(-1, s["kv"]), new.abs().amax(-1), "amax")
        old = torch.where((lowest > 0)[:, None], scales[touched, i], 0.0)
        scale = torch.maximum(old, _power(amax))
        page = _codes(codes, touched)  # [page][head][dim / 64][token][64], or [64][token] for the values
        shown = older[:, None, None, :, None] if i == 0 else older[:, None, None, None, :]
        page = torch.where(shown, page * (old / scale)[:, :, None, None, None], page)
        value = (new / scale[at][:, :, None]).unflatten(2, (-1, 64))  # [token][head][dim / 64][64]
        if i == 0:
            page[at, :, :, place] = value
        else:
            page[at, :, :, :, place] = value
        codes.view(torch.uint8)[touched] = page.to(torch.float8_e4m3fn).view(torch.uint8)
        scales[touched, i] = scale
    return k, v, scales


def _tokens(s, block, place):
    """Keys and values [token][head][dim] in 32 bits."""
    k, v, scales = _views(s["cache"], s["kv"], s["dim"])
    keys = _codes(k, block, slice(None), slice(None), place).flatten(2) * scales[block, 0][..., None]
    values = _codes(v, block, slice(None), slice(None), slice(None), place).flatten(2) * scales[block, 1][..., None]
    return keys, values


def _plain_read_heads(s):
    k, v = _tokens(s, *_places(s["table"], s["cu"], s["start"]))
    return k.to(s["dtype"]), v.to(s["dtype"])


def _plain_read_rows(s):
    rows = s["cache"].view(-1, s["cache"].shape[2])[s["rows"].long().clamp_min(0)]
    if s["row"] == "fp8":
        x = rows[:, :512].view(torch.float8_e4m3fn).float().unflatten(1, (4, GROUP))
        x = (x * rows[:, 512:528].view(torch.float32)[..., None]).flatten(1)
    else:
        x = rows[:, :1024].view(torch.bfloat16).float()
    none = (s["rows"] < 0)[:, None]
    rope = rows[:, -128:].view(torch.bfloat16).float()
    return x.masked_fill(none, 0).to(s["dtype"]), rope.masked_fill(none, 0).to(s["dtype"])


def _plain_attend(s):
    R, kv, group, dim = s["table"].shape[0], s["kv"], s["group"], s["dim"]
    cu = torch.tensor([0] + s["qn"], device="cuda").cumsum(0) if s["cu"] is None else s["cu"].long()
    most, ctx = max(s["qn"]), s["ctx_len"].long()
    k, v, scales = _views(s["cache"], kv, dim)
    iq, ik = torch.arange(most, device="cuda"), torch.arange(s["table"].shape[1] * PAGE, device="cuda")
    lq = cu[1:] - cu[:-1]
    rows = (cu[:-1, None] + iq).clamp_max(len(s["q"]) - 1)
    out, lse = [], []
    for h in range(kv):
        block = s["table"].long()
        # [request][page][dim / 64][token][64] -> [request][key][dim]
        key = (_codes(k, block, h) * scales[block, 0, h][:, :, None, None, None]).permute(0, 1, 3, 2, 4).reshape(R, -1, dim)
        value = (_codes(v, block, h) * scales[block, 1, h][:, :, None, None, None]).permute(0, 1, 4, 2, 3).reshape(R, -1, dim)
        q = s["q"][:, h * group:(h + 1) * group].float()[rows]  # [request][token][group][dim]
        x = torch.matmul(q.reshape(R, most * group, dim), key.transpose(1, 2)).view(R, most, group, -1) * s["scale"]
        seen = ctx[:, None].expand(R, most)
        if s["causal"]:
            seen = seen - lq[:, None] + 1 + iq
        x = x.masked_fill((ik >= seen[..., None])[:, :, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        p = torch.exp(x - top)
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p.view(R, most * group, -1), value).view(R, most, group, dim)
        out.append(o / torch.where(total == 0, torch.ones_like(total), total))
        lse.append((top + torch.log(total))[..., 0])
    there = iq < lq[:, None]
    return torch.cat(out, 2)[there].to(s["dtype"]), torch.cat(lse, 2)[there]


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    op = case["op"]
    s = 4 if case["dtype"] == "fp32" else 2
    if op == "read_rows":
        n = case["n"]
        return {"bytes": n * (4 + case["fill"] * (656 if case["row"] == "fp8" else 1152) + 576 * s), "flops": n * LATENT}
    kv, dim = case["kv"], case["dim"]
    if op == "append":
        qn, kn = _lengths(case)
        n = sum(qn)
        return {"bytes": n * 2 * kv * dim * (s + 1) + sum(-(-k // PAGE) - (k - q) // PAGE for q, k in zip(qn, kn)) * (8 * kv + 4),
                "flops": n * 2 * kv * dim * 2}
    if op == "read_heads":
        start, n = _spans(case)
        pages = sum(-(-(a + b) // PAGE) - a // PAGE for a, b in zip(start, n))
        return {"bytes": sum(n) * 2 * kv * dim * (s + 1) + pages * (8 * kv + 4), "flops": sum(n) * 2 * kv * dim}
    qn, kn = _lengths(case)
    pairs = sum(q * k - (q * (q - 1) // 2 if case["causal"] else 0) for q, k in zip(qn, kn))
    H = kv * case["group"]
    return {"bytes": sum(kn) * 2 * kv * dim + sum(-(-k // PAGE) for k in kn) * (8 * kv + 4) + sum(qn) * H * (2 * dim * s + 4),
            "flops": 4 * pairs * H * dim}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    if case["op"] == "read_rows":
        out = torch.zeros((case["n"], LATENT + ROPE), dtype=torch.float64, device="cuda")
        at = s["rows"] >= 0
        b = s["cache"].flatten(0, 1).index_select(0, s["rows"][at].long())
        if case["row"] == "fp8":
            c = b[:, :512].contiguous().view(torch.float8_e4m3fn).double()
            c *= b[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(GROUP, 1)
            out[at] = torch.cat([c, b[:, 528:].contiguous().view(torch.bfloat16).double()], 1)
        else:
            out[at] = b.contiguous().view(torch.bfloat16).double()
        return out[:, :LATENT], out[:, LATENT:]
    kv, dim = case["kv"], case["dim"]
    if case["op"] == "append":
        k, v, scales = (t.double() for t in _views(s["cache"], kv, dim))
        a = 0
        for r, (n, length) in enumerate(zip(s["qn"], s["kn"])):
            for page in range((length - n) // PAGE, -(-length // PAGE)):
                lo, hi = max(length - n - page * PAGE, 0), min(length - page * PAGE, PAGE)
                t0 = a + page * PAGE + lo - (length - n)
                b = int(s["table"][r, page])
                for i, (codes, new) in enumerate(((k[b], s["k"]), (v[b].transpose(2, 3), s["v"]))):
                    x = new[t0:t0 + hi - lo].double()  # [token][head][dim]
                    need = torch.exp2(torch.ceil(torch.log2(x.abs().amax((0, 2)) / E4M3_MAX) - 1e-12).clamp_min(-126))
                    scale = torch.maximum(need, scales[b, i]) if lo else need
                    if lo:
                        codes[:, :, :lo] *= (scales[b, i] / scale)[:, None, None, None]
                    codes[:, :, lo:hi] = (x / scale[:, None]).unflatten(2, (-1, 64)).permute(1, 2, 0, 3)
                    scales[b, i] = scale
            a += n
        return k, v, scales
    views = _views(s["cache"], kv, dim)

    def tokens(r, start, n):
        pages = s["table"][r, start // PAGE:-(-(start + n) // PAGE)].long()
        off = start % PAGE
        k, v = (views[i].view(torch.uint8).index_select(0, pages).view(torch.float8_e4m3fn).double() for i in (0, 1))
        k, v = (x * views[2][pages, i].double()[:, :, None, None, None] for i, x in enumerate((k, v)))
        k = k.permute(0, 3, 1, 2, 4).reshape(-1, kv, dim)
        return k[off:off + n], v.permute(0, 4, 1, 2, 3).reshape(-1, kv, dim)[off:off + n]

    if case["op"] == "read_heads":
        got = [tokens(r, a, n) for r, (a, n) in enumerate(zip(s["first"], s["n"]))]
        return torch.cat([k for k, _ in got]), torch.cat([v for _, v in got])
    group, outs, lses, a = case["group"], [], [], 0
    for r, (n, length) in enumerate(zip(s["qn"], s["kn"])):
        k, v = tokens(r, 0, length)
        q, a = s["q"][a:a + n].double(), a + n
        o, l = [], []
        for h in range(kv * group):
            z = (q[:, h] @ k[:, h // group].T) * s["scale"]
            if case["causal"]:
                z += torch.full((n, length), -math.inf, device="cuda", dtype=torch.float64).triu(length - n + 1)
            l.append(torch.logsumexp(z, 1))
            o.append(torch.softmax(z, 1) @ v[:, h // group])
        outs.append(torch.stack(o, 1))
        lses.append(torch.stack(l, 1))
    return torch.cat(outs), torch.cat(lses)
