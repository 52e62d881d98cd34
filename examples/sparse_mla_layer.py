"""One sparse-MLA attention layer served through the library: prompts, then decode steps over offloaded contexts.

    python examples/sparse_mla_layer.py

Random weights and latents stand for the layer's projections; every other step is the library's:
  prompt   append_rows writes the prompts' rows into the paged pool and rotates the queries; read_rows reads them back, and
           attend_expanded attends over the keys and values expanded from them; offload_pages copies the completed pages
           to the host pool.
  decode   per step append_rows writes the new token; the requests whose pages left the GPU attend over the top-K rows
           that resolve_topk hands back (attend_rows), the others over their whole context (attend_pages), both with the
           up-projections absorbed into the queries and the results.
run() returns, for every call, the largest difference of a result's element from the same attention in 64 bits, relative to
the weighted sum of the values' magnitudes there.  bf16 weights and results allow BOUND of it: 2^-7 for the two roundings, and
2^-10 for the scores' errors and the sums (a score is off by less than 2^-12)."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_mla_kv_gb300 as hs  # noqa: E402

PAGE, LATENT, ROPE, NOPE, VALUE = 64, 512, 64, 128, 128
ROW = 656
BOUND = 2.0 ** -7 + 2.0 ** -10


def stored(cache, rows):
    """Latents and rotated keys of pool rows, as the attention reads them."""
    b = cache.reshape(-1, ROW)[rows.long()]
    code = b[:, :512].contiguous().view(torch.float8_e4m3fn).float()
    scale = b[:, 512:528].contiguous().view(torch.float32)
    return (code * scale.repeat_interleave(128, 1)).bfloat16(), b[:, 528:].contiguous().view(torch.bfloat16)


def plain(q, k, v, scale, seen=None):
    """Attention in 64 bits: q [n][H][d], k [m][H or 1][d], v [m][H or 1][e], seen bool [n][m] -> the results, and the
    weighted sums of the values' magnitudes."""
    s = torch.einsum("nhd,mhd->hnm", q.double(), k.double().expand(-1, q.shape[1], -1)) * scale
    if seen is not None:
        s = s.masked_fill(~seen, float("-inf"))
    w, v = s.softmax(-1), v.double().expand(-1, q.shape[1], -1)
    return torch.einsum("hnm,mhe->nhe", w, v), torch.einsum("hnm,mhe->nhe", w, v.abs())


def off(got, plain):
    ref, size = plain
    return float(((got.double() - ref).abs() / size).max())


def run(prompts=(150, 70, 333), offloaded=(0, 2), steps=4, heads=16, topk=64, seed=0, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=device) * scale).bfloat16()

    R, H = len(prompts), heads
    scale = (NOPE + ROPE) ** -0.5
    w_k = normal(H, NOPE, LATENT, scale=LATENT ** -0.5)   # latent -> a head's key without position
    w_v = normal(H, VALUE, LATENT, scale=LATENT ** -0.5)  # latent -> a head's value
    angles = torch.arange(4096, device=device)[:, None] / 10000.0 ** (torch.arange(32, device=device) / 32)
    rotation = torch.cat([angles.cos(), angles.sin()], 1).float().contiguous()

    # the pool: a block per page of every request, then the leased hot buffers of twice K rows
    pages = (max(prompts) + steps + PAGE - 1) // PAGE
    hot_pages = 2 * topk // PAGE
    cache = torch.zeros((R * (pages + hot_pages), PAGE, ROW), dtype=torch.uint8, device=device)
    host = torch.zeros((R * pages, PAGE, ROW), dtype=torch.uint8).pin_memory()
    pool = hs.Pool([cache], [host])
    table = torch.arange(R * pages, dtype=torch.int32, device=device).reshape(R, pages)
    hot_blocks = (R * pages + torch.arange(R * hot_pages, dtype=torch.int32, device=device)).reshape(R, hot_pages)
    hot = hs.HotState.allocate(1, hot_blocks, hot_pages * PAGE)
    hs.hot_reset(pool, hot)
    workspace = hs.alloc_attend_workspace(device)
    worst = {"attend_expanded": 0.0, "attend_rows": 0.0, "attend_pages": 0.0}

    # prompts
    owner = torch.cat([torch.full((n,), r) for r, n in enumerate(prompts)]).to(device)
    pos = torch.cat([torch.arange(n) for n in prompts]).to(device, torch.int32)
    rows = table[owner, (pos // PAGE).long()] * PAGE + pos % PAGE
    T = len(owner)
    q_nope, q_rope = normal(T, H, NOPE), normal(T, H, ROPE)
    q_rope = hs.append_rows(pool, rows, normal(T, LATENT), normal(T, ROPE), pos, rotation, q_rope=q_rope)
    latent, k_rope = hs.read_rows(pool, rows)
    k_nope = torch.einsum("tl,hdl->thd", latent, w_k).contiguous()
    v = torch.einsum("tl,hel->the", latent, w_v).contiguous()
    cu = torch.tensor([0, *prompts], device=device).cumsum(0).int()
    out, _ = hs.attend_expanded(q_nope, q_rope, k_nope, k_rope, v, cu, cu, scale)
    for r in range(R):
        at = slice(int(cu[r]), int(cu[r + 1]))
        k = torch.cat([k_nope[at], k_rope[at, None].expand(-1, H, -1)], -1)
        n = k.shape[0]
        seen = torch.ones((n, n), dtype=torch.bool, device=device).tril()
        ref = plain(torch.cat([q_nope[at], q_rope[at]], -1), k, v[at], scale, seen)
        worst["attend_expanded"] = max(worst["attend_expanded"], off(out[at], ref))

    # the completed pages go to the host; those of the requests in `offloaded` leave the GPU
    full = [(r, j) for r in range(R) for j in range(prompts[r] // PAGE)]
    blocks = torch.tensor([r * pages + j for r, j in full], dtype=torch.int32, device=device)
    hs.offload_pages(pool, blocks, blocks)
    host_table = torch.full_like(table, -1)
    resident = table.clone()
    for r, j in full:
        host_table[r, j] = r * pages + j
        if r in offloaded:
            resident[r, j] = -1
    history = stored(cache, (table[:, :, None] * PAGE + torch.arange(PAGE, device=device, dtype=torch.int32)).reshape(-1))
    history = [x.reshape(R, pages * PAGE, -1).clone() for x in history]  # for the comparison only
    for r in offloaded:
        cache[table[r, :prompts[r] // PAGE].long()] = 0xFF

    # decode
    away = torch.tensor(offloaded, dtype=torch.int64, device=device)
    here = torch.tensor([r for r in range(R) if r not in offloaded], dtype=torch.int64, device=device)
    for step in range(steps):
        ctx = torch.tensor([n + step + 1 for n in prompts], dtype=torch.int32, device=device)
        pos = ctx - 1
        rows = (resident.gather(1, (pos // PAGE).long()[:, None])[:, 0]) * PAGE + pos % PAGE
        q_nope, q_rope = normal(R, H, NOPE), normal(R, H, ROPE)
        q_rope = hs.append_rows(pool, rows, normal(R, LATENT), normal(R, ROPE), pos, rotation, q_rope=q_rope)
        for x, new in zip(history, stored(cache, rows)):
            x[torch.arange(R, device=device), pos.long()] = new
        q_latent = torch.einsum("rhd,hdl->rhl", q_nope, w_k)
        q = torch.cat([q_latent, q_rope], -1)
        keys = torch.cat(history, -1)
        # the indexer's part: the K keys of largest total score
        score = torch.einsum("rhd,rkd->rk", q.float(), keys.float())
        score.masked_fill_(torch.arange(pages * PAGE, device=device)[None] >= ctx[:, None], float("-inf"))
        best = score.topk(min(topk, pages * PAGE), 1).indices.int()
        best = torch.where(score.gather(1, best.long()) == float("-inf"), -1, best)
        ids, _ = hs.resolve_topk(pool, best[None, :, None].contiguous(), resident, host_table, ctx, hot, step)
        sparse, _ = hs.attend_rows(pool, ids[0, away, 0].contiguous(), q_latent[away], q_rope[away], scale, workspace=workspace)
        whole, _ = hs.attend_pages(pool, resident[here].contiguous(), ctx[here], q_latent[here, None], q_rope[here, None],
                                   scale, workspace=workspace)
        layer_out = torch.empty((R, H, VALUE), dtype=torch.bfloat16, device=device)
        layer_out[away] = torch.einsum("rhl,hel->rhe", sparse, w_v)
        layer_out[here] = torch.einsum("rhl,hel->rhe", whole[:, 0], w_v)
        for i, r in enumerate(offloaded):
            k = keys[r, best[r][best[r] >= 0].long()]
            ref = plain(q[r:r + 1], k[:, None], k[:, None, :LATENT], scale)
            worst["attend_rows"] = max(worst["attend_rows"], off(sparse[i:i + 1], ref))
        for i, r in enumerate(here.tolist()):
            k = keys[r, :int(ctx[r])]
            ref = plain(q[r:r + 1], k[:, None], k[:, None, :LATENT], scale)
            worst["attend_pages"] = max(worst["attend_pages"], off(whole[i], ref))
        assert bool(torch.isfinite(layer_out).all())
    return worst


if __name__ == "__main__":
    for name, value in run().items():
        print(f"{name:16} largest difference from 64 bits: {value:.4f} of the weighted sum of magnitudes")
