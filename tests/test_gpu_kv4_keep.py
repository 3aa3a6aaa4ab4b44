"""Keeping the accepted drafted tokens of the 4-bit cache, against the definition:
values, pages, lengths and counts are exact."""
import pytest
import torch

import kv4_reference as R
from test_gpu_kv4 import batch, dcc, make_cache, starts  # noqa: F401  (dcc: the fixture)

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def setup(dcc, seed, n, lens, heads, dim, group, dtype, layers=1, max_pages=None):
    g = torch.Generator().manual_seed(seed)
    cache, pools, table = make_cache(dcc, g, n, lens, heads, dim, group, dtype, layers, max_pages=max_pages)
    refs = torch.zeros(cache.pages, dtype=torch.int32)
    for p in table[table >= 0].tolist():
        refs[p] += 1
    cache.refs.copy_(refs.cuda())
    return cache, pools, table, refs


def plain(table, refs, lens, news, paths, counts):
    """The definition: (table, refs, lens, info, moves as (sequence, from, to) positions)."""
    table, refs, lens = [r[:] for r in table.tolist()], refs.tolist(), list(lens)
    counted, left, moves = list(refs), 0, []
    for s, t in enumerate(news):
        first, c, path = lens[s] - t, counts[s], paths[s][:max(0, counts[s])]
        ok = 0 <= c <= t and first >= 0 and all(0 <= x < t for x in path) and all(a < b for a, b in zip(path, path[1:]))
        own = [(x, i) for i, x in enumerate(path) if x != i] if ok else []
        if any(counted[table[s][(first + i) // R.PAGE]] != 1 for _, i in own):
            ok = False
        if not ok:
            left += 1
            continue
        moves += [(s, first + x, first + i) for x, i in own]
        for j in range(-(-(first + c) // R.PAGE), -(-lens[s] // R.PAGE)):
            refs[table[s][j]] -= 1
            table[s][j] = -1
        lens[s] = first + c
    return table, refs, lens, [refs.count(0), left, len(moves)], moves


def run(dcc, cache, pools, table, refs, lens, news, paths, counts, info=True):
    want = plain(table, refs, lens, news, paths, counts)
    flat = [x for p, t in zip(paths, news) for x in (p + [-7] * t)[:t]]
    out = torch.full((4,), 9, dtype=torch.int32, device="cuda") if info else None
    cache.keep(batch(news), i32(flat) if flat else torch.empty(0, dtype=torch.int32, device="cuda"), i32(counts),
               workspace=cache.pages_workspace(), info=out)
    assert cache.table.cpu().tolist() == want[0] and cache.refs.cpu().tolist() == want[1]
    assert cache.lengths.cpu().tolist() == want[2]
    if info:
        assert out.cpu().tolist()[:3] == want[3]
    dim, group, dtype = cache.head_dim, cache.group, {torch.bfloat16: "bf16", torch.float16: "fp16"}[cache.torch_dtype]
    for r in range(cache.n):
        for before, after in zip(R.values(pools[r], dim, group, dtype), R.values(cache.pools[r].cpu(), dim, group, dtype)):
            for s, x, y in want[4]:
                before_row = before[:, table[s, x // R.PAGE], :, x % R.PAGE]
                row = after[:, table[s, y // R.PAGE], :, y % R.PAGE]
                assert torch.equal(row.nan_to_num(7e9), before_row.nan_to_num(7e9)), (r, s, x, y)
            touched = torch.zeros(before.shape[1], R.PAGE, dtype=torch.bool)  # rows that some move goes to
            for s, _, y in want[4]:
                touched[table[s, y // R.PAGE], y % R.PAGE] = True
            same = (before.nan_to_num(7e9) == after.nan_to_num(7e9)).all(-1).all(2).all(0)
            assert same[~touched].all()
    return want


@pytest.mark.parametrize("dtype,dim,group", [("bf16", 128, 64), ("fp16", 64, 32), ("bf16", 64, 64), ("fp16", 128, 32)])
@pytest.mark.parametrize("n,heads,layers,lens,news,paths", [
    (1, 1, 1, [1], [1], [[0]]), (1, 1, 1, [1], [1], [[]]), (2, 2, 3, [70], [8], [[1, 3, 7]]),
    (8, 1, 2, [300, 64, 5, 0, 129], [40, 32, 5, 0, 2], [[0, 1, 7, 39], [31], [0, 1, 2, 3, 4], [], [1]]),
    (1, 3, 1, [200], [130], [list(range(1, 130, 2))]),            # over three pages, each onto others' places
    (2, 1, 1, [128, 128], [128, 64], [[], list(range(64))]),      # all given up; all kept
    (1, 1, 2, [500], [400], [list(range(3, 400))]),
    (1, 2, 1, [65, 66, 67], [3, 3, 3], [[2], [0, 2], [1, 2]]),
    (1, 1, 1, [90] * 40, [6] * 40, [[0, 1 + s % 5] for s in range(40)])])
def test_keep(dcc, dtype, dim, group, n, heads, layers, lens, news, paths):  # noqa: F811
    cache, pools, table, refs = setup(dcc, dim + group + sum(lens), n, lens, heads, dim, group, dtype, layers)
    run(dcc, cache, pools, table, refs, lens, news, paths, [len(p) for p in paths])
    assert dcc.dcc_local_check() == dcc.DCC_OK


def test_sequences_left_as_they_are(dcc):  # noqa: F811
    lens, news = [70] * 9 + [3], [8] * 9 + [5]
    paths = [[1, 1], [2, 1], [0, 8], [-1, 3], [0, 1], [0, 1], [0, 2], [5], [0, 4], [0]]
    counts = [2, 2, 2, 2, -1, 9, 2, 1, 2, 1]
    cache, pools, table, refs = setup(dcc, 4, 2, lens, 1, 128, 64, "bf16")
    want = run(dcc, cache, pools, table, refs, lens, news, paths, counts)
    assert want[3][1:] == [7, 3]
    assert dcc.dcc_local_check() == dcc.DCC_OK


def test_shared_pages(dcc):  # noqa: F811
    """A page of two sequences takes no moved row, but may be given up by one, or kept where nothing moves."""
    cache, pools, table, refs = setup(dcc, 5, 1, [70, 70, 70, 70], 1, 64, 32, "fp16")
    for s in (1, 2, 3):   # all on sequence 0's second page
        refs[table[s, 1]] -= 1
        table[s, 1] = table[0, 1]
        refs[table[s, 1]] += 1
    cache.table.copy_(table.cuda())
    cache.refs.copy_(refs.cuda())
    want = run(dcc, cache, pools, table, refs, [70] * 4, [5, 6, 6, 70], [[1, 3], [], [0, 1, 2], [4]], [2, 0, 3, 1])
    assert want[3][1] == 1 and want[2] == [70, 64, 67, 1]


def test_pages_outside_the_pool(dcc):  # noqa: F811
    cache, _, table, refs = setup(dcc, 6, 1, [200, 200], 1, 64, 32, "fp16")
    table[0, 3] = 10 ** 6      # among those the path reads
    table[1, 3] = -5           # only given up
    cache.table.copy_(table.cuda())
    before = cache.pools[0].clone()
    info = torch.zeros(4, dtype=torch.int32, device="cuda")
    cache.keep(batch([100, 100]), i32([50, 99] + [0] * 98 + [0, 1] + [0] * 98), i32([2, 2]),
               workspace=cache.pages_workspace(), info=info)
    assert dcc.dcc_local_check() == dcc.DCC_ERR_BOUNDS
    assert cache.lengths.tolist() == [200, 102] and info.tolist()[1:3] == [1, 0]
    assert torch.equal(before, cache.pools[0]) and cache.table[1].tolist()[2:] == [-1, -1]


def test_batch_that_leaves_the_path(dcc):  # noqa: F811
    """start past the path's tokens counts what is there; without info."""
    cache, pools, table, refs = setup(dcc, 7, 1, [90, 80], 1, 128, 64, "fp16")
    cache.keep(i32([0, 4, 9]), i32([1, 3, 0, 0, 2, 0]), i32([2, 1]), workspace=cache.pages_workspace())
    # the second sequence has rows 4 and 5 only: path [2] lies past them
    assert cache.lengths.tolist() == [88, 80]


@pytest.mark.parametrize("pages", [300, 5000])
def test_large_pools_and_a_graph(dcc, pages):  # noqa: F811
    """Books by one CTA and by a cluster; captured, replayed on restored state."""
    lens, news = [130] * 20, [9] * 20
    paths = [[s % 9] for s in range(20)]
    g = torch.Generator().manual_seed(pages)
    cache, pools, table = make_cache(dcc, g, 1, lens, 1, 64, 64, "bf16", spare=pages - 60, max_pages=4)
    refs = torch.zeros(pages, dtype=torch.int32)
    refs[table[table >= 0].long()] = 1
    cache.refs.copy_(refs.cuda())
    want = plain(table, refs, lens, news, paths, [1] * 20)
    path = i32([x for s in range(20) for x in (paths[s] + [0] * 8)])
    start, count, ws = batch(news), i32([1] * 20), cache.pages_workspace()
    info = torch.zeros(4, dtype=torch.int32, device="cuda")
    state = [(t, t.clone()) for t in (cache.table, cache.refs, cache.lengths, cache.pools[0])]

    def restore():
        for t, was in state:
            t.copy_(was)
    cache.keep(start, path, count, ws, info)   # (loads the kernels)
    restore()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.keep(start, path, count, ws, info)
    for _ in range(2):
        restore()
        ws.fill_(0xab)  # any content
        graph.replay()
        torch.cuda.synchronize()
        assert cache.table.tolist() == want[0] and cache.refs.tolist() == want[1]
        assert cache.lengths.tolist() == want[2] and info.tolist()[:3] == want[3]


def test_many_sequences_without_drafts(dcc):  # noqa: F811
    lens = [65] * 300
    cache, pools, table, refs = setup(dcc, 9, 1, lens, 1, 64, 64, "fp16")
    news = [0 if s % 3 else 2 for s in range(300)]
    run(dcc, cache, pools, table, refs, lens, news, [[1] if t else [] for t in news], [1 if t else 0 for t in news])
