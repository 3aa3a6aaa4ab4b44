"""Sequences of the 4-bit cache that grow, fork, keep a part of their drafted
tokens and grow on: whatever pages they share meanwhile, each reads back what was
appended to it.  Values, pages, lengths and counts are exact."""
import random

import pytest
import torch

import kv4_reference as R
from test_gpu_kv4 import batch, dcc  # noqa: F401  (dcc: the fixture)

pytestmark = pytest.mark.gpu
PAGE = R.PAGE


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def reserve(table, refs, lens, add):
    """The definition: (table, refs, lens, info, copies as (from, to) pages)."""
    table, counts, refs, lens = [list(r) for r in table], list(refs), list(refs), list(lens)
    left = [p for p, r in enumerate(refs) if r == 0]
    room, wanted, fails, given, copies = len(left), 0, 0, 0, []
    for s, a in enumerate(add):
        if a <= 0:
            continue
        held, new = -(-lens[s] // PAGE), -(-(lens[s] + a) // PAGE)
        if new > len(table[s]):
            fails += 1
            continue
        # the rest of a last page that has other owners is not this sequence's to write
        own = int(lens[s] % PAGE > 0 and counts[table[s][held - 1]] > 1)
        wanted += new - held + own
        if new - held + own > 0 and wanted > room:
            fails += 1
            continue
        for j in range(held - own, new):
            if j < held:
                refs[table[s][j]] -= 1
                copies.append((table[s][j], left[0]))
            table[s][j] = left.pop(0)
            refs[table[s][j]] = 1
            given += 1
        lens[s] += a
    return table, refs, lens, [refs.count(0), fails, given], copies


class Life:
    """A cache and, beside it, the tokens that each sequence was given."""

    def __init__(self, dcc, seed, seqs, pages, max_pages, n=2, layers=2, heads=1, dim=64, group=32, dtype="bf16"):
        self.dcc, self.g = dcc, torch.Generator().manual_seed(seed)
        self.cache = dcc.Kv4Cache.create(n, layers, pages, seqs, max_pages, heads, dim, group, dtype)
        self.shape, self.dtype = (layers, n, 2, heads, dim), dtype
        self.ws, self.info = self.cache.pages_workspace(), torch.full((4,), -5, dtype=torch.int32, device="cuda")
        self.tokens = [[] for _ in range(seqs)]  # of every sequence: numbers of its tokens
        self.data = []                           # by number: [layers, n, 2 (k, v), heads, dim]

    def books(self):
        return self.cache.table.tolist(), self.cache.refs.tolist(), self.cache.lengths.tolist()

    def grow(self, add):
        """Room for add[s] more tokens, and those; returns the call's info."""
        c = self.cache
        table, refs, lens, said, _ = reserve(*self.books(), add)
        c.reserve(ints(add), self.ws, self.info)
        assert self.info.tolist()[:3] == said
        assert (c.table.tolist(), c.refs.tolist(), c.lengths.tolist()) == (table, refs, lens)
        news = [m - len(t) for m, t in zip(lens, self.tokens)]
        T, (layers, n, _, heads, dim) = sum(news), self.shape
        if T == 0:
            return said
        x = torch.randn(T, *self.shape, generator=self.g).to(R.TD[self.dtype])
        for s, t in enumerate(news):
            self.tokens[s] += range(len(self.data), len(self.data) + t)
            self.data += list(x[sum(news[:s]):][:t])
        start = batch(news)
        for layer in range(layers):
            k, v = ([x[:, layer, r, i].contiguous().cuda() for r in range(n)] for i in range(2))
            c.append(k, v, start, layer=layer)
        return said

    def fork(self, src, dst):
        self.cache.fork(ints(src), ints(dst), self.ws, self.info)
        said = self.info.tolist()[:3]
        for s, d in zip(src, dst):
            self.tokens[d] = list(self.tokens[s]) if self.cache.lengths[d] else []
        return said

    def free(self, seqs):
        self.cache.free(ints(seqs), self.ws, self.info)
        for s in seqs:
            self.tokens[s] = []

    def keep(self, news, paths):
        """Of the last news[s] tokens those of paths[s]; returns the call's info."""
        flat = [x for p, t in zip(paths, news) for x in (list(p) + [-1] * t)[:t]]
        table, refs, lens = self.books()
        self.cache.keep(batch(news), ints(flat), ints([len(p) for p in paths]), self.ws, self.info)
        left = 0
        for s, (t, p) in enumerate(zip(news, paths)):
            first = lens[s] - t
            if any(x != i and refs[table[s][(first + i) // PAGE]] != 1 for i, x in enumerate(p)):
                left += 1
                continue
            drafted = self.tokens[s][first:]
            self.tokens[s] = self.tokens[s][:first] + [drafted[x] for x in p]
        said = self.info.tolist()[:3]
        assert said[1] == left
        return said

    def check(self):
        c, (layers, n, _, heads, dim) = self.cache, self.shape
        assert self.dcc.dcc_local_check() == self.dcc.DCC_OK
        table, refs, lens = self.books()
        assert lens == [len(t) for t in self.tokens]
        held = [p for r, m in zip(table, lens) for p in r[:-(-m // PAGE)]]
        assert refs == [held.count(p) for p in range(c.pages)]
        T, start = sum(lens), batch(lens)
        if T == 0:
            return
        x = torch.stack([self.data[i] for t in self.tokens for i in t])
        for layer in range(layers):
            k, v = ([torch.empty(T, heads, dim, dtype=R.TD[self.dtype], device="cuda") for _ in range(n)] for _ in range(2))
            c.read(k, v, start, layer=layer)
            for r in range(n):
                for i, got in enumerate((k[r], v[r])):
                    want = R.quantise(x[:, layer, r, i], c.group, self.dtype).to(torch.float32).to(R.TD[self.dtype])
                    assert torch.equal(got.cpu(), want), (layer, r, i)


@pytest.mark.parametrize("dtype,dim,group", [("bf16", 128, 64), ("fp16", 64, 32), ("bf16", 64, 64), ("fp16", 128, 32)])
@pytest.mark.parametrize("context,drafted,kept", [
    (60, 32, (2, 4)),    # the first sequence goes on inside a page of both, the second at its end
    (123, 5, (2, 0)), (123, 5, (0, 0)), (123, 5, (5, 3)), (60, 100, (50, 3)), (1, 127, (0, 1)), (64, 64, (0, 63))])
def test_drafts_of_forked_sequences(dcc, dtype, dim, group, context, drafted, kept):  # noqa: F811
    life = Life(dcc, context + drafted, 3, 16, 4, dim=dim, group=group, dtype=dtype)
    life.grow([context, 7, 0])
    life.grow([drafted, 0, 0])
    life.fork([0], [2])
    life.check()
    said = life.keep([drafted, 0, drafted], [range(kept[0]), [], range(kept[1])])
    assert said[1:] == [0, 0]
    life.check()
    life.grow([3, 0, 0])      # one of the two: the other one's tokens stay
    life.check()
    life.grow([0, 1, 70])
    life.check()
    life.keep([3, 0, 70], [[1], [], [0, 5, 64]])  # (rows move in pages of their own)
    life.check()


@pytest.mark.parametrize("pages", [40, 5000])
def test_owners_that_grow_at_once(dcc, pages):  # noqa: F811
    """All owners of a page leave it in one call: it returns to the pool.  Books by one CTA and by a cluster."""
    life = Life(dcc, pages, 6, pages, 4, n=3, layers=2)
    life.grow([100, 0, 0, 0, 128, 0])
    life.grow([28, 0, 0, 0, 0, 0])
    life.fork([0, 0, 0, 4], [1, 2, 3, 5])
    life.keep([28] * 4 + [0, 0], [range(k) for k in (1, 2, 3, 27)] + [[], []])
    life.check()
    life.grow([5, 3, 40, 1, 1, 0])
    life.check()
    life.keep([1, 62, 3, 10, 60, 0], [[], [], [], [], range(2), []])
    life.check()
    life.grow([1, 1, 1, 1, 1, 1])
    life.check()
    life.free(list(range(6)))
    life.check()


def test_a_pool_without_a_page_for_the_copy(dcc):  # noqa: F811
    """A sequence that needs a page of its own and finds none keeps its length and its part of the page."""
    life = Life(dcc, 3, 3, 4, 3, n=1, layers=1)
    life.grow([128, 64, 0])
    life.fork([0], [2])
    life.keep([100, 0, 0], [range(90), [], []])
    life.check()
    life.grow([0, 1, 0])                # the last free page
    assert life.grow([1, 0, 0])[1] == 1
    assert life.grow([10 ** 6, 62, 0])[1] == 1
    life.check()
    life.free([1])
    assert life.grow([20, 0, 1]) == [0, 1, 2]  # the copy and a page; none is left for the other's next page
    life.check()


def test_captured(dcc):  # noqa: F811
    life = Life(dcc, 9, 4, 12, 3, n=2, layers=3, heads=2, dim=128, group=64)
    life.grow([64, 64, 0, 0])
    life.fork([0, 1], [2, 3])
    life.keep([9, 9, 0, 0], [range(4), range(5), [], []])
    c, add = life.cache, ints([2, 0, 3, 60])
    state = [(t, t.clone()) for t in (c.table, c.refs, c.lengths, *c.pools)]
    table, refs, lens, said, copies = reserve(*life.books(), add.tolist())
    assert len(copies) == 1
    want = [p.clone() for p in c.pools]
    for p in want:
        for x, y in copies:
            p[:, y] = p[:, x]
    c.reserve(add, life.ws, life.info)  # (loads the kernel)
    for t, was in state:
        t.copy_(was)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.reserve(add, life.ws, life.info)
    for _ in range(2):
        for t, was in state:
            t.copy_(was)
        life.ws.fill_(0xab)  # any content
        graph.replay()
        torch.cuda.synchronize()
        assert (c.table.tolist(), c.refs.tolist(), c.lengths.tolist()) == (table, refs, lens)
        assert life.info.tolist()[:3] == said
        assert all(torch.equal(p, w) for p, w in zip(c.pools, want))


@pytest.mark.parametrize("seed", range(6))
def test_any_life(dcc, seed):  # noqa: F811
    """Growing, forking, keeping and freeing in any order, in a pool that runs out."""
    rng = random.Random(seed)
    seqs, pages, mp = rng.choice([4, 9]), rng.choice([12, 30]), 5
    life = Life(dcc, seed, seqs, pages, mp, n=rng.choice([1, 2]), layers=rng.choice([1, 2]))
    for _ in range(14):
        life.grow([rng.choice([0, 0, 1, 5, 40, 64, 65]) for _ in range(seqs)])
        life.check()
        if rng.random() < 0.7:
            perm = rng.sample(range(seqs), seqs)
            dst = perm[:rng.randrange(0, seqs // 2 + 1)]
            life.fork([rng.choice(perm[len(dst):]) for _ in dst], dst)
            life.check()
        news = [rng.randrange(0, min(len(t), 70) + 1) for t in life.tokens]
        paths = []
        for t in news:
            k = rng.randrange(0, t + 1)
            paths.append(range(k) if rng.random() < 0.7 else sorted(rng.sample(range(t), k)))
        life.keep(news, paths)
        life.check()
        if rng.random() < 0.3:
            life.free(rng.sample(range(seqs), 1))
            life.check()
