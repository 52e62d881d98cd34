"""Where the CTAs of attend_heads' kernel for prompts begin: against the same numbering in Python's whole numbers, for calls whose key tiles
(or whose columns) do not fit 31 bits.  Such calls take many seconds or most of the memory, so the search is run alone."""
import bisect
import ctypes
import subprocess

import pytest

torch = pytest.importorskip("torch")
import os  # noqa: E402

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
COLS, KEYS, ITEM_COST, MIN_RUN, LIMIT, CTAS = 256, 128, 3, 4, 32, 152  # as in heads_prompt.cu


@pytest.fixture(scope="module")
def starts(tmp_path_factory):
    from sparse_mla_kv_gb300 import _build

    so = str(tmp_path_factory.mktemp("starts") / "starts.so")
    subprocess.check_call([_build.NVCC, *_build.ARCH, *_build.FLAGS, "-shared", os.path.join(HERE, "heads_prompt_starts.cu"), "-o", so])
    f = ctypes.CDLL(so).heads_prompt_starts
    i, p = ctypes.c_int, ctypes.c_void_p
    f.argtypes = [i, i, i, i, i, i, ctypes.c_int64, p, p, i, p, p]

    def run(kv, group, causal, ctx, new, max_pages):
        lens = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, *new]).cumsum(0).int().cuda()
        out = torch.zeros((CTAS, 32), dtype=torch.uint8, device="cuda")
        header = torch.zeros(2, dtype=torch.int64, device="cuda")
        torch.cuda.synchronize()
        assert f(kv, group, int(causal), LIMIT, len(ctx), max_pages, sum(new), lens.data_ptr(), cu.data_ptr(), CTAS, out.data_ptr(),
                 header.data_ptr()) == 0
        out = out.cpu()
        return (out[:, :16].contiguous().view(torch.int32).tolist(), out[:, 16:].contiguous().view(torch.int64).tolist(), header.tolist())

    return run


def units_before(group, causal, ctx, n, max_pages):
    """Key tiles (and ITEM_COST a block) of one head before each block of 256 columns of a request, and in all."""
    cols = n * group
    if cols <= LIMIT:
        return [0]
    keys = max(0, min(ctx, max_pages * 64))
    b = torch.arange(-(-cols // COLS), dtype=torch.int64)
    last = (torch.clamp((b + 1) * COLS, max=cols) - 1) // group
    seen = (ctx - n + 1 + last).clamp(0, keys) if causal else torch.full_like(b, keys)
    tiles = ((seen + KEYS - 1) // KEYS).clamp_min(1) + ITEM_COST
    return [0, *tiles.cumsum(0).tolist()]


def check(starts, kv, group, causal, ctx, new, max_pages):
    heads = [units_before(group, causal, c, n, max_pages) for c, n in zip(ctx, new)]
    first = [0]
    for h in heads:
        first.append(first[-1] + kv * h[-1])
    total = first[-1]
    run = max(MIN_RUN, -(-total // CTAS))
    where, at, header = starts(kv, group, causal, ctx, new, max_pages)
    assert header == [run, total]
    for i in range(CTAS):
        begin = run * i
        assert at[i] == [begin, max(0, min(run, total - begin))], i
        if begin >= total:
            continue
        r = bisect.bisect_right(first, begin) - 1
        head, offset = divmod(begin - first[r], heads[r][-1])
        block = bisect.bisect_right(heads[r], offset) - 1
        assert where[i] == [r, head, block, offset - heads[r][block]], (i, where[i])
    return max(h[-1] for h in heads)


@pytest.mark.parametrize("kv,group,causal,ctx,new,max_pages", [
    (2, 4, True, [700, 40, 9, 300], [300, 40, 20, 100], 11),
    (3, 7, False, [2000, 5], [77, 1], 40),
    (2, 8, True, [10 + i % 300 for i in range(1200)], [i % 60 for i in range(1200)], 5),
])
def test_runs_begin_where_the_numbering_says(starts, kv, group, causal, ctx, new, max_pages):
    check(starts, kv, group, causal, ctx, new, max_pages)


@pytest.mark.parametrize("kv,group,causal,ctx,new,max_pages", [
    (1, 64, True, [2 ** 21], [2 ** 21], 2 ** 15),                                  # 2^32 key tiles and more in a head
    (2, 16, False, [300, 2 ** 26, 5000], [77, 2 ** 21 + 5, 400], 2 ** 20),
    (1, 32, True, [64] * 700 + [2 ** 22 + 3] + [100] * 9, [2] * 700 + [2 ** 22] + [70] * 9, 2 ** 16 + 1),
])
def test_runs_of_heads_with_more_tiles_than_31_bits_hold(starts, kv, group, causal, ctx, new, max_pages):
    assert check(starts, kv, group, causal, ctx, new, max_pages) > 2 ** 31


@pytest.mark.parametrize("kv,group,ctx,new", [
    (1, 1, [64], [2 ** 31 - 1]), (1, 1, [300, 64], [70, 2 ** 31 - 71]), (1, 8, [1, 64], [1, 2 ** 28 - 2]), (1, 3, [64], [(2 ** 31 - 1) // 3]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_runs_of_calls_with_columns_up_to_31_bits(starts, kv, group, ctx, new, causal):
    check(starts, kv, group, causal, ctx, new, 5)
