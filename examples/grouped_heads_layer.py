"""One attention layer with grouped heads, its keys and values in 8 bits in the paged pool: a layer beside the sparse ones, or that of a
model that drafts the verify positions.

    python examples/grouped_heads_layer.py

Random queries, keys and values stand for the layer's projections; every other step is the library's:
  prompts  go in by chunks: append_heads quantises a chunk's keys and values into the requests' pages, attend_heads attends over
           them and over the chunks before; offload_pages copies the completed pages to the host pool, their scales with them.
  reuse    the first request ends, and its blocks are given to another one that begins with the same prefix: its pages come back
           from the host pool, and only the rest of its prompt is appended.
  decode   each step drafts some tokens, appends and attends to all of them, and keeps a part: the next step's tokens go over the
           rejected ones.
run() returns, for every kind of call, the largest difference of a result's element from the same attention in 64 bits over the
tokens that read_heads gives, relative to the weighted sum of the values' magnitudes there.  The result's rounding allows 2^-8 of it,
the weights' 2^-11, the scores' errors (below 2^-14) and the sums less: BOUND.  It also checks that read_heads gives what was
appended, within what e4m3 and a page's scale leave of it."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_mla_kv_gb300 as hs  # noqa: E402

PAGE = 64
BOUND = 2.0 ** -8 + 2.0 ** -10


def plain(q, k, v, scale, seen):
    """Attention in 64 bits: q [n][H][d], k and v [m][kv][d], seen bool [n][m] -> the results, and the weighted sums of the values'
    magnitudes."""
    group = q.shape[1] // k.shape[1]
    k, v = (x.double().repeat_interleave(group, 1) for x in (k, v))
    s = (torch.einsum("nhd,mhd->hnm", q.double(), k) * scale).masked_fill(~seen, float("-inf"))
    w = s.softmax(-1)
    return torch.einsum("hnm,mhe->nhe", w, v), torch.einsum("hnm,mhe->nhe", w, v.abs())


def run(prompts=(300, 70, 129), chunk=128, steps=5, drafts=4, kv=2, group=4, dim=128, seed=0, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=device).bfloat16()

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=device)

    R, H, scale = len(prompts), kv * group, dim ** -0.5
    pages = (max(prompts) + chunk + steps * drafts + PAGE - 1) // PAGE
    cache = torch.zeros((R * pages, PAGE, hs.heads_row_bytes(kv, dim)), dtype=torch.uint8, device=device)
    host = torch.zeros((R * pages, PAGE, cache.shape[2]), dtype=torch.uint8).pin_memory()
    pool = hs.Pool([cache], [host])
    table = torch.randperm(R * pages, generator=g, device=device).reshape(R, pages).int()
    workspace = hs.alloc_heads_workspace(device)
    given = [[torch.zeros((0, kv, dim), device=device) for _ in range(2)] for _ in range(R)]  # what was appended, for comparison
    ctx = [0] * R
    worst = {"chunk": 0.0, "reuse": 0.0, "decode": 0.0}

    def forward(new, kind):
        """Appends new[r] tokens to each request and attends from them."""
        n = sum(new)
        cu = i32([0, *new]).cumsum(0).int()
        k, v, q = normal(n, kv, dim), normal(n, kv, dim), normal(n, H, dim)
        for r in range(R):
            ctx[r] += new[r]
        lens = i32(ctx)
        hs.append_heads(pool, table, lens, k, v, cu=cu)
        out, _ = hs.attend_heads(pool, table, lens, q, scale, cu_q=cu, workspace=workspace)
        stored = hs.read_heads(pool, table, None, i32([0, *ctx]).cumsum(0).int(), sum(ctx), dim, dtype=torch.float32)
        t0 = s0 = 0
        for r in range(R):
            m = ctx[r]
            for x, side in ((k, 0), (v, 1)):
                given[r][side] = torch.cat([given[r][side][:m - new[r]], x[t0:t0 + new[r]].float()])
            have = [x[s0:s0 + m] for x in stored]
            for x, side in zip(have, given[r]):
                # a code is within half a step of 4 bits, or of the smallest step of its page's scale: 2^-10 of a scale that is at most
                # 1 / 224 of the page's largest value; each time the scale rises, codes are rounded once more
                largest = float(side.abs().max()) if m else 0.0
                assert bool(((x - side).abs() <= 3 * (2.0 ** -4 * side.abs()).clamp_min(largest * 2.0 ** -17)).all()), kind
            if new[r]:
                seen = torch.arange(m, device=device)[None] <= (m - new[r] + torch.arange(new[r], device=device))[:, None]
                ref, size = plain(q[t0:t0 + new[r]], *have, scale, seen)
                worst[kind] = max(worst[kind], float(((out[t0:t0 + new[r]].double() - ref).abs() / size).max()))
            t0, s0 = t0 + new[r], s0 + m

    # prompts, a chunk of each at a time; the completed pages go to the host
    while any(c < n for c, n in zip(ctx, prompts)):
        forward([min(chunk, n - c) for c, n in zip(ctx, prompts)], "chunk")
    home = {(r, j): r * pages + j for r in range(R) for j in range(ctx[r] // PAGE)}
    hs.offload_pages(pool, torch.stack([table[r, j] for r, j in home]) if home else i32([]), i32(list(home.values())))
    torch.cuda.synchronize()

    # request 0 ends; another takes its blocks, in another order, and its prefix from the host
    prefix = ctx[0] // PAGE
    cache[table[0].long()] = 0xFF
    table[0] = table[0].flip(0)
    for j in range(prefix):
        cache[int(table[0, j])].copy_(host[home[0, j]])
    ctx[0] = prefix * PAGE
    given[0] = [x[:ctx[0]] for x in given[0]]
    forward([chunk // 2 + 1] + [0] * (R - 1), "reuse")

    # decode: of each step's drafts some are rejected
    for step in range(steps):
        forward([drafts] * R, "decode")
        ctx = [c - (step + r) % drafts for r, c in enumerate(ctx)]
    return worst


if __name__ == "__main__":
    for name, value in run().items():
        print(f"{name:8} largest difference from 64 bits: {value:.5f} of the weighted sum of magnitudes")
