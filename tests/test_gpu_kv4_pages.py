"""The page calls of the 4-bit cache against one-request-at-a-time forms: all
whole numbers, so tables, counts, lists and the pool's bytes must be equal."""
import random

import pytest
import torch

import kv4_reference as R

pytestmark = pytest.mark.gpu
PAGE = R.PAGE


@pytest.fixture(scope="module")
def dcc():
    from driven_collective_communication_gb300 import build
    build.build()
    from driven_collective_communication_gb300 import dcc as mod
    torch.cuda.set_device(0)
    return mod


def make(dcc, seed, n, layers, heads, dim, group, seqs, pages, mp, lens):
    rng = random.Random(seed)
    order = list(range(pages))
    rng.shuffle(order)
    table = [[-1] * mp for _ in range(seqs)]
    refs = [0] * pages
    for s, m in enumerate(lens):
        for j in range(-(-m // PAGE)):
            table[s][j] = order.pop()
            refs[table[s][j]] = 1
    g = torch.Generator().manual_seed(seed)
    pools = [torch.randint(0, 256, (layers, pages, heads, R.block_bytes(dim, group)), generator=g, dtype=torch.uint8)
             for _ in range(n)]
    t32 = dict(dtype=torch.int32, device="cuda")
    cache = dcc.Kv4Cache([p.cuda() for p in pools], torch.tensor(table, **t32), torch.tensor(lens, **t32),
                         torch.tensor(refs, **t32), heads, dim, group, "bf16")
    return cache, pools, R.PageBook(table, lens, refs)


def same_state(cache, book):
    assert cache.table.tolist() == book.table
    assert cache.lengths.tolist() == book.lens
    assert cache.refs.tolist() == book.refs


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def info():
    return torch.full((4,), -5, dtype=torch.int32, device="cuda")


SHAPES = [(1, 1, 1, 64, 32), (2, 2, 1, 128, 64), (3, 1, 2, 128, 32)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("seed", range(4))
def test_a_life_of_the_cache(dcc, shape, seed):
    """Reserve, fork, free and compact in turn on one cache, sharing included,
    until the pool has run out more than once."""
    n, layers, heads, dim, group = shape
    rng = random.Random(seed * 7 + dim)
    seqs, pages, mp = rng.choice([3, 17, 40]), rng.choice([5, 60, 211]), rng.choice([4, 9])
    cache, pools, book = make(dcc, seed, n, layers, heads, dim, group, seqs, pages, mp, [0] * seqs)
    ws = cache.pages_workspace()
    out = info()
    for step in range(12):
        add = [rng.choice([0, 0, -3, 1, 63, 64, 65, 200, 1000]) for _ in range(seqs)]
        cache.reserve(ints(add), ws, out)
        assert out.tolist()[:3] == book.reserve(add)
        same_state(cache, book)
        k = rng.randrange(0, seqs)
        perm = rng.sample(range(seqs), seqs)
        dst, rest = perm[:k], perm[k:]
        src = [rng.choice(rest) for _ in dst]
        before = [p.clone() for p in cache.pools]
        book.copies = []
        cache.fork(ints(src), ints(dst), ws, out)
        assert out.tolist()[:3] == book.fork(src, dst)
        same_state(cache, book)
        for p, b in zip(cache.pools, before):
            for x, y in book.copies:
                b[:, y] = b[:, x]
            assert torch.equal(p, b)
        gone = rng.sample(range(seqs), rng.randrange(0, seqs))
        cache.free(ints(gone), ws, out)
        assert out.tolist()[:3] == book.free(gone)
        same_state(cache, book)
        nt, nr, rm = torch.empty_like(cache.table), torch.empty_like(cache.refs), torch.empty_like(cache.refs)
        before = [p.clone() for p in cache.pools]
        table, refs, remap, moves, said = book.compact()
        if step % 2:
            nt, nr = cache.table, cache.refs  # in place
        cache.compact(nt, nr, rm, ws, out)
        assert out.tolist()[:2] == said
        assert nt.tolist() == table and nr.tolist() == refs and rm.tolist() == remap
        for p, b in zip(cache.pools, before):
            for x, y in moves:
                b[:, y] = b[:, x]
            assert torch.equal(p, b)
        if step % 2:
            book.table, book.refs = table, refs
        else:  # the old table still holds: nothing was overwritten
            for s, row in enumerate(book.table):
                for j, x in enumerate(row):
                    if x >= 0:
                        assert torch.equal(cache.pools[0][:, x], before[0][:, x])
                        assert torch.equal(cache.pools[0][:, table[s][j]], before[0][:, x])
            for p, b in zip(cache.pools, before):
                pass
    assert dcc.dcc_local_check() == dcc.DCC_OK


def test_many_pages(dcc):
    """More pages and sequences than one CTA's threads, and long rows."""
    seqs, mp = 2500, 70
    rng = random.Random(8)
    lens = [rng.choice([0, 1, 64, 100, 700, 70 * 64]) for _ in range(seqs)]
    pages = sum(-(-m // PAGE) for m in lens) + 1111
    cache, _, book = make(dcc, 8, 1, 1, 1, 64, 64, seqs, pages, mp, lens)
    ws, out = cache.pages_workspace(), info()
    perm = rng.sample(range(seqs), seqs)
    dst, rest = perm[:1200], perm[1200:]
    src = [rng.choice(rest) for _ in dst]
    cache.fork(ints(src), ints(dst), ws, out)
    assert out.tolist()[:3] == book.fork(src, dst)
    same_state(cache, book)
    add = [rng.choice([0, 1, 300]) for _ in range(seqs)]
    cache.reserve(ints(add), ws, out)
    assert out.tolist()[:3] == book.reserve(add)
    same_state(cache, book)
    gone = rng.sample(range(seqs), 1700)
    cache.free(ints(gone), ws, out)
    assert out.tolist()[:3] == book.free(gone)
    same_state(cache, book)
    rm = torch.empty_like(cache.refs)
    table, refs, remap, _, said = book.compact()
    cache.compact(cache.table, cache.refs, rm, ws, out)
    assert out.tolist()[:2] == said
    assert cache.table.tolist() == table and cache.refs.tolist() == refs and rm.tolist() == remap
    assert dcc.dcc_local_check() == dcc.DCC_OK


def test_forks_that_fail(dcc):
    """Named twice, a source that is dropped itself, out of range, no page left."""
    lens = [70, 70, 70, 64, 10, 0]
    cache, _, book = make(dcc, 1, 1, 1, 1, 64, 32, 6, 10, 2, lens)
    ws, out = cache.pages_workspace(), info()
    src, dst = [0, 0, 3, 9, 0, 2], [1, 1, 4, 5, 77, 3]
    cache.fork(ints(src), ints(dst), ws, out)
    assert out.tolist()[:3] == book.fork(src, dst)
    same_state(cache, book)
    assert dcc.dcc_local_check() == dcc.DCC_ERR_BOUNDS  # 9 and 77 are no sequences
    lens = [70, 70, 0, 0, 0]  # 4 pages held, one left
    cache, _, book = make(dcc, 2, 1, 1, 1, 64, 32, 5, 5, 2, lens)
    ws = cache.pages_workspace()
    src, dst = [0, 1, 0], [2, 3, 4]
    cache.fork(ints(src), ints(dst), ws, out)
    assert out.tolist()[:3] == book.fork(src, dst) == [0, 2, 1]
    same_state(cache, book)
    gone = [3, 2, 2, -1, 5]
    cache.free(ints(gone), ws, out)
    assert out.tolist()[:3] == book.free(gone)
    same_state(cache, book)
    assert dcc.dcc_local_check() == dcc.DCC_ERR_BOUNDS


def test_reserve_stops_at_the_end_of_the_pool(dcc):
    cache, _, book = make(dcc, 3, 1, 1, 1, 64, 32, 6, 6, 100, [1, 64, 0, 0, 30, 0])
    ws, out = cache.pages_workspace(), info()
    add = [5, 1, 129, 64, 20, 2 ** 31 - 1]
    cache.reserve(ints(add), ws, out)
    assert out.tolist()[:3] == book.reserve(add)
    same_state(cache, book)
    assert dcc.dcc_local_check() == dcc.DCC_OK


@pytest.mark.parametrize("shape", SHAPES)
def test_copy_pages(dcc, shape):
    n, layers, heads, dim, group = shape
    cache, pools, _ = make(dcc, 5, n, layers, heads, dim, group, 2, 31, 4, [100, 64])
    src, dst = [4, 4, 30, 0], [1, 29, 7, 12]
    cache.copy_pages(ints(src), ints(dst))
    for p, b in zip(cache.pools, pools):
        for x, y in zip(src, dst):
            b[:, y] = b[:, x]
        assert torch.equal(p.cpu(), b)
    assert dcc.dcc_local_check() == dcc.DCC_OK
    cache.copy_pages(ints([31, 2, -1]), ints([3, 40, 5]))  # nowhere: skipped, said
    for p, b in zip(cache.pools, pools):
        assert torch.equal(p.cpu(), b)
    assert dcc.dcc_local_check() == dcc.DCC_ERR_BOUNDS


def test_without_info_and_empty_lists(dcc):
    cache, _, book = make(dcc, 6, 1, 1, 1, 64, 32, 3, 8, 4, [100, 64, 0])
    ws = cache.pages_workspace()
    none = ints([])
    cache.fork(none, none, ws)
    cache.free(none, ws)
    cache.copy_pages(none, none)
    same_state(cache, book)
    cache.fork(ints([0]), ints([2]), ws)
    book.fork([0], [2])
    same_state(cache, book)
