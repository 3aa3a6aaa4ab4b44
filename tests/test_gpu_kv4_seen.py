"""Attention of trees of drafted tokens and with windows that keep first tokens,
over the 4-bit cache, against 64 bits.  Which kernel a call takes follows from its
rows; the bound is that of the kernel that rounds more (kv4_bounds.py), and of the
streaming kernel where few rows make the choice plain."""
import math

import pytest
import torch

import kv4_bounds as B
import kv4_reference as R
import seen_reference as S
from test_gpu_kv4 import batch, dcc, make_cache, starts  # noqa: F401  (dcc: the fixture)

pytestmark = pytest.mark.gpu
TD = R.TD
SHAPES = [("bf16", 128, 64), ("fp16", 64, 32), ("bf16", 64, 64), ("fp16", 128, 32)]


def attend(dcc, cache, g, n, heads, dim, dtype, lens, news, share, window, sinks, masks=None, words=None, max_new=None,
           rows_more=0, pad=0, scale=None, ws=None, q=None):
    """One call.  masks: a list of sets per sequence's drafted tokens, None: causal with sinks."""
    T, Hq = sum(news) + rows_more, heads * share
    if q is None:
        q = [torch.randn(T, Hq + pad, dim, generator=g).to(TD[dtype]) for _ in range(n)]
    qd = [x.cuda()[:, :Hq] for x in q]
    out = [torch.full((T, Hq, dim), 7.0, dtype=TD[dtype], device="cuda") for _ in range(n)]
    lse = [torch.full((T, Hq), 7.0, dtype=torch.float32, device="cuda") for _ in range(n)]
    ws = cache.attention_workspace(Hq) if ws is None else ws
    kw = dict(max_new=max_new or max(news + [1]), workspace=ws, lse=lse, window=window, sinks=sinks, scale=scale)
    if masks is None:
        cache.attention_sinks(qd, out, batch(news), **kw)
    else:
        words = words or -(-max(news + [1]) // 32)
        rows = [m for s in masks for m in s] + [set()] * rows_more
        cache.attention_tree(qd, out, batch(news), S.pack(rows, words).cuda(), **kw)
    assert dcc.dcc_local_check() == dcc.DCC_OK
    return [x[:, :Hq] for x in q], [x.cpu() for x in out], [x.cpu() for x in lse]


def check(cache, table, n, heads, dim, group, dtype, lens, news, share, window, sinks, masks, q, out, lse, kernel,
          max_new=None, scale=None, norm=True):
    scale = dim ** -0.5 if scale is None else scale
    T, first = q[0].shape[0], starts(news)
    written = torch.zeros(T, dtype=torch.bool)
    total = B.Totals(dtype)
    for r in range(n):
        K, V = B.parts(cache.pools[r].cpu()[0], dim, group, dtype)
        for s, (m, t) in enumerate(zip(lens, news)):
            rows = min(t, max_new or t)
            if rows == 0:
                continue
            a = first[s]
            written[a:a + rows] = True
            held = max(0, m)
            seen = S.seen_rows(m, t, rows, window, sinks, masks and masks[s])
            pages = table[s, :-(-held // R.PAGE)].long()
            for h in range(heads):
                k, v = B.rows_of(K, pages, h, held), B.rows_of(V, pages, h, held)
                for x in range(h * share, (h + 1) * share):
                    want, L, tol, tol_lse, rough = S.exact(k, v, q[r][a:a + rows, x].double(), seen, scale, dtype, kernel)
                    got, gl = out[r][a:a + rows, x].double(), lse[r][a:a + rows, x].double()
                    off = (got - want).abs()
                    assert (off <= tol).all(), (r, s, x, (off / tol).max().item())
                    none = ~seen.any(-1) if held else torch.ones(rows, dtype=torch.bool)
                    assert (got[none] == 0).all() and (gl[none] == -math.inf).all()
                    assert ((gl - L).abs()[~none] <= tol_lse[~none]).all()
                    total.add(got, want, tol, rough)
        for x in (out[r], lse[r]):
            assert (x[~written] == 7.0).all()
    if norm and total.ref:
        total.check()


@pytest.mark.parametrize("dtype,dim,group", SHAPES)
@pytest.mark.parametrize("n,heads,lens,news,share,window,sinks", [
    (1, 1, [1], [1], 1, 1, 1), (2, 2, [300, 5, 64, 0, 1000], [1, 1, 1, 1, 1], 4, 100, 4),
    (1, 1, [700], [1], 8, 64, 70), (3, 1, [129, 513], [1, 1], 2, 1, 1), (1, 2, [400, 200], [3, 5], 2, 130, 66),
    (8, 1, [2000, 77], [1, 1], 3, 256, 1), (1, 1, [640], [1], 1, 128, 64), (1, 1, [641], [1], 16, 127, 192),
    (1, 1, [500], [4], 1, 40, 10 ** 9), (2, 1, [300], [2], 1, 10 ** 9, 4), (1, 1, [300, 90], [2, 1], 1, 0, 4)])
def test_sinks_streaming(dcc, dtype, dim, group, n, heads, lens, news, share, window, sinks):  # noqa: F811
    g = torch.Generator().manual_seed(dim + group + sum(lens))
    cache, _, table = make_cache(dcc, g, n, lens, heads, dim, group, dtype)
    q, out, lse = attend(dcc, cache, g, n, heads, dim, dtype, lens, news, share, window, sinks, pad=2)
    check(cache, table, n, heads, dim, group, dtype, lens, news, share, window, sinks, None, q, out, lse, "streaming")


@pytest.mark.parametrize("dtype,dim,group", SHAPES)
@pytest.mark.parametrize("n,heads,lens,news,share,window,sinks,rows_more", [
    (2, 1, [700, 300], [130, 100], 4, 100, 4, 2), (1, 2, [900], [257], 3, 300, 130, 0), (8, 1, [600], [64], 8, 128, 1, 0),
    (1, 1, [500, 64, 0, 33], [200, 64, 0, 33], 8, 33, 64, 1), (1, 1, [4096], [40], 8, 2000, 300, 0),
    (1, 1, [5, 130], [9, 64], 8, 50, 5, 0)])  # four rows before position zero
def test_sinks_of_many_rows(dcc, dtype, dim, group, n, heads, lens, news, share, window, sinks, rows_more):  # noqa: F811
    g = torch.Generator().manual_seed(dim + group + sum(lens))
    cache, _, table = make_cache(dcc, g, n, lens, heads, dim, group, dtype)
    q, out, lse = attend(dcc, cache, g, n, heads, dim, dtype, lens, news, share, window, sinks, rows_more=rows_more)
    check(cache, table, n, heads, dim, group, dtype, lens, news, share, window, sinks, None, q, out, lse, "prompt")


@pytest.mark.parametrize("dtype,dim,group", SHAPES)
@pytest.mark.parametrize("n,heads,lens,news,share,window,sinks", [
    (1, 1, [1], [1], 1, 0, 0), (1, 1, [8], [8], 1, 0, 0), (2, 2, [300, 5, 64, 0, 1000], [7, 5, 1, 0, 8], 2, 0, 0),
    (1, 1, [130, 70], [4, 3], 4, 60, 3), (1, 1, [700], [5], 3, 64, 70), (8, 1, [200, 200], [2, 2], 8, 0, 0),
    (1, 3, [1000], [8], 2, 4, 1), (1, 1, [3], [5], 2, 0, 0)])  # two drafted tokens before position zero
def test_tree_streaming(dcc, dtype, dim, group, n, heads, lens, news, share, window, sinks):  # noqa: F811
    g = torch.Generator().manual_seed(dim + group + sum(lens))
    cache, _, table = make_cache(dcc, g, n, lens, heads, dim, group, dtype)
    masks = [S.tree(g, t) for t in news]
    q, out, lse = attend(dcc, cache, g, n, heads, dim, dtype, lens, news, share, window, sinks, masks, pad=1)
    check(cache, table, n, heads, dim, group, dtype, lens, news, share, window, sinks, masks, q, out, lse, "streaming")


@pytest.mark.parametrize("dtype,dim,group", SHAPES)
@pytest.mark.parametrize("n,heads,lens,news,share,window,sinks,words,rows_more", [
    (2, 1, [700, 300, 64], [63, 32, 33], 4, 0, 0, 2, 1), (1, 2, [900], [70], 8, 0, 0, 4, 0),
    (1, 1, [400, 31, 0, 129], [64, 31, 0, 65], 8, 100, 66, 3, 0), (8, 1, [2000], [32], 8, 0, 0, 1, 0),
    (1, 1, [300, 256], [256, 256], 2, 0, 0, 8, 0), (4, 1, [1300, 900, 500, 700], [16, 64, 40, 17], 8, 0, 0, 32, 3),
    (1, 1, [6000], [24], 16, 0, 0, 1, 0), (1, 1, [20, 190], [33, 64], 3, 7, 2, 2, 0)])
def test_tree_of_many_rows(dcc, dtype, dim, group, n, heads, lens, news, share, window, sinks, words, rows_more):  # noqa: F811
    g = torch.Generator().manual_seed(dim + group + sum(lens))
    cache, _, table = make_cache(dcc, g, n, lens, heads, dim, group, dtype)
    masks = [S.tree(g, t) for t in news]
    q, out, lse = attend(dcc, cache, g, n, heads, dim, dtype, lens, news, share, window, sinks, masks, words,
                         rows_more=rows_more)
    check(cache, table, n, heads, dim, group, dtype, lens, news, share, window, sinks, masks, q, out, lse, "prompt")


@pytest.mark.parametrize("share", [1, 8])
@pytest.mark.parametrize("dtype,dim,group", SHAPES[:2])
def test_masks_of_any_kind(dcc, dtype, dim, group, share):  # noqa: F811
    """Rows that see nothing, only others, all, later ones, and bits past the drafted tokens."""
    g = torch.Generator().manual_seed(7 + share)
    lens, news = [40, 0, 200, 33], [40, 0, 37, 33]
    cache, _, table = make_cache(dcc, g, 2, lens, 1, dim, group, dtype)
    masks = [[set(int(x) for x in torch.randint(0, 64, (5,), generator=g)) for _ in range(t)] for t in news]
    masks[0][0] = set()                # no context either: nothing
    masks[0][39] = {63, 45}            # past the drafted tokens: nothing
    masks[0][5] = set(range(64))
    masks[2][0], masks[2][36] = set(), {36, 37, 63}
    masks[3][32] = {0, 31, 32}
    q, out, lse = attend(dcc, cache, g, 2, 1, dim, dtype, lens, news, share, 0, 0, masks, 2)
    check(cache, table, 2, 1, dim, group, dtype, lens, news, share, 0, 0, masks, q, out, lse, "prompt", norm=False)


@pytest.mark.parametrize("share", [1, 8])
def test_a_chain_is_causal_attention(dcc, share):  # noqa: F811
    """A tree without branches: what the causal call gives, with and without a window."""
    g = torch.Generator().manual_seed(3)
    lens, news = [500, 77], [5, 3]
    cache, _, _ = make_cache(dcc, g, 2, lens, 2, 128, 64, "bf16")
    masks = [[set(range(i + 1)) for i in range(t)] for t in news]
    for window in (0, 100):
        q, out, lse = attend(dcc, cache, g, 2, 2, 128, "bf16", lens, news, share, window, 0, masks)
        want = [torch.empty_like(x).cuda() for x in out]
        logs = [torch.empty_like(x).cuda() for x in lse]
        cache.attention([x.cuda() for x in q], want, batch(news), max_new=5, workspace=cache.attention_workspace(2 * share),
                        lse=logs, window=window)
        for a, b in zip(out + lse, want + logs):
            assert torch.allclose(a.float(), b.cpu().float(), rtol=2.0 ** -7, atol=2.0 ** -8)


@pytest.mark.parametrize("news,share", [([6], 2), ([40], 8)])
@pytest.mark.parametrize("dtype,dim,group", SHAPES)
def test_hidden_keys_may_hold_anything(dcc, dtype, dim, group, news, share):  # noqa: F811
    """NaN and infinity in drafted tokens and in context that a window hides reach only the rows that see them."""
    g = torch.Generator().manual_seed(11)
    lens = [300]
    cache, pools, table = make_cache(dcc, g, 1, lens, 1, dim, group, dtype)
    ng, half = dim // group, R.PAGE * dim // 2
    first = lens[0] - news[0]
    masks = [[{0, i} if i % 2 else {i} for i in range(news[0])]]
    bad = [first + 3, first + 4, 50, 51]    # two drafted tokens; two that the window hides (of them 50 is no sink)
    for x in bad:
        blk = cache.pools[0][0, int(table[0, x // R.PAGE]), 0]
        for w in range(2):
            par = blk[2 * half + w * R.PAGE * ng * 4:2 * half + (w + 1) * R.PAGE * ng * 4].view(TD[dtype]).view(R.PAGE, ng, 2)
            par[x % R.PAGE, 0, w] = math.nan if x >= first else math.inf
    for window, sinks in ((100, 40), (100, 0)):
        q, out, lse = attend(dcc, cache, g, 1, 1, dim, dtype, lens, news, share, window, sinks, masks)
        sees = torch.tensor([i in (3, 4) for i in range(news[0])])
        assert torch.isnan(out[0][sees]).any(-1).all() and torch.isfinite(out[0][~sees]).all()
        clean = cache.pools[0].cpu().clone()
        keep = cache.pools[0]
        for x in bad:   # the bound's inputs: as if the hidden ones were zeros
            b = clean[0, int(table[0, x // R.PAGE]), 0]
            for w in range(2):
                b[2 * half + w * R.PAGE * ng * 4:2 * half + (w + 1) * R.PAGE * ng * 4].view(TD[dtype]).view(R.PAGE, ng, 2)[x % R.PAGE] = 0
        cache.pools[0] = clean
        good = [i for i in range(news[0]) if i not in (3, 4)]
        seen = S.seen_rows(lens[0], news[0], news[0], window, sinks, masks[0])[good]
        K, V = B.parts(clean[0], dim, group, dtype)
        pages = table[0].long()
        k, v = B.rows_of(K, pages, 0, lens[0]), B.rows_of(V, pages, 0, lens[0])
        for x in range(share):
            want, _, tol, _, _ = S.exact(k, v, q[0][good, x].double(), seen, dim ** -0.5, dtype, "prompt")
            assert ((out[0][good, x].double() - want).abs() <= tol).all()
        cache.pools[0] = keep


@pytest.mark.parametrize("share,news", [(1, [9, 4]), (8, [40, 33])])
def test_rows_past_max_new_stay(dcc, share, news):  # noqa: F811
    g = torch.Generator().manual_seed(5)
    lens = [400, 100]
    cache, _, table = make_cache(dcc, g, 1, lens, 1, 128, 64, "fp16")
    masks = [S.tree(g, t) for t in news]
    for m in (None, masks):
        window, sinks = (90, 5) if m is None else (0, 0)
        q, out, lse = attend(dcc, cache, g, 1, 1, 128, "fp16", lens, news, share, window, sinks, m, max_new=news[1] + 1,
                             words=2)
        check(cache, table, 1, 1, 128, 64, "fp16", lens, news, share, window, sinks, m, q, out, lse, "prompt",
              max_new=news[1] + 1)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
@pytest.mark.parametrize("news,share", [([6, 3], 2), ([40, 20], 8)])
def test_scales(dcc, scale, news, share):  # noqa: F811
    g = torch.Generator().manual_seed(6)
    lens = [300, 90]
    cache, _, table = make_cache(dcc, g, 1, lens, 1, 64, 32, "bf16")
    masks = [S.tree(g, t) for t in news]
    q, out, lse = attend(dcc, cache, g, 1, 1, 64, "bf16", lens, news, share, 80, 9, masks, scale=scale)
    check(cache, table, 1, 1, 64, 32, "bf16", lens, news, share, 80, 9, masks, q, out, lse, "prompt", scale=scale,
          norm=False)


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("news,share", [([6, 3], 2), ([48, 20], 8)])
def test_repeats_bit_for_bit_in_a_graph_and_on_another_stream(dcc, news, share, tree):  # noqa: F811
    g = torch.Generator().manual_seed(8)
    lens = [3000, 700]
    cache, _, _ = make_cache(dcc, g, 2, lens, 1, 128, 64, "bf16")
    q = [torch.randn(sum(news), share, 128, generator=g).bfloat16().cuda() for _ in range(2)]
    rows = [m for t in news for m in S.tree(g, t)]
    mask, start, ws = S.pack(rows, 2).cuda(), batch(news), cache.attention_workspace(share)

    def call(out, lse, stream=None):
        kw = dict(max_new=max(news), workspace=ws, lse=lse, window=500 if not tree else 0, sinks=4, stream=stream)
        if tree:
            cache.attention_tree(q, out, start, mask, **kw)
        else:
            cache.attention_sinks(q, out, start, **kw)

    def buffers():
        return ([torch.empty_like(x) for x in q],
                [torch.empty(sum(news), share, dtype=torch.float32, device="cuda") for _ in q])
    want = buffers()
    call(*want)
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), buffers()
    with torch.cuda.stream(side):
        call(*got)
    side.synchronize()
    replay = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*replay)
        call(*replay)
    for _ in range(3):
        for x in replay[0] + replay[1]:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(want[0] + want[1], got[0] + got[1], replay[0] + replay[1]):
            assert torch.equal(a, b) and torch.equal(a, c)
    assert dcc.dcc_local_check() == dcc.DCC_OK


@pytest.mark.parametrize("news,share", [([3], 2), ([40], 8)])
def test_missing_pages_are_reported(dcc, news, share):  # noqa: F811
    """A page number outside the pool: recorded, its keys not seen."""
    g = torch.Generator().manual_seed(9)
    cache, _, table = make_cache(dcc, g, 1, [300], 1, 128, 64, "fp16")
    q = torch.randn(sum(news), share, 128, generator=g).half().cuda()
    out = torch.zeros_like(q)
    ws = cache.attention_workspace(share)
    mask = S.pack(S.tree(g, news[0]), 2).cuda()
    cache.table[0, 1] = 10 ** 6
    cache.attention_tree([q], [out], batch(news), mask, max_new=news[0], workspace=ws)
    assert dcc.dcc_local_check() == dcc.DCC_ERR_BOUNDS
    assert torch.isfinite(out).all() and out.abs().max() > 0
    cache.table[0, 1] = table[0, 1].item()
    cache.attention_tree([q], [out], batch(news), mask, max_new=news[0], workspace=ws)
    assert dcc.dcc_local_check() == dcc.DCC_OK


@pytest.mark.parametrize("dtype,dim,group", SHAPES)
@pytest.mark.parametrize("new,window", [(3, 0), (4, 0), (4, 700)])
def test_two_passes_of_the_streaming_kernel(dcc, dtype, dim, group, new, window):  # noqa: F811
    """Rows that it takes in two goes, over a row of the table long enough for the rule."""
    g = torch.Generator().manual_seed(new + dim)
    lens, news = [1500, 70], [new, 2]
    share = 8 if dim == 128 else 10
    need = [-(-m // R.PAGE) for m in lens]
    cache, _, table = make_cache(dcc, g, 1, lens, 1, dim, group, dtype, max_pages=5000 if window == 0 else max(need))
    masks = [S.tree(g, t) for t in news]
    q, out, lse = attend(dcc, cache, g, 1, 1, dim, dtype, lens, news, share, window, 9 if window else 0, masks)
    check(cache, table, 1, 1, dim, group, dtype, lens, news, share, window, 9 if window else 0, masks, q, out, lse, "prompt")


@pytest.mark.parametrize("share", [1, 8])
@pytest.mark.parametrize("tree", [True, False])
def test_idle_slots(dcc, share, tree):  # noqa: F811
    """Two sequences with rows among a thousand slots without any."""
    g = torch.Generator().manual_seed(12)
    lens, news = [0] * 1000, [0] * 1000
    for s, (m, t) in {3: (300, 9), 977: (700, 5)}.items():
        lens[s], news[s] = m, t
    lens[500] = 200  # holds tokens, brings none
    cache, _, table = make_cache(dcc, g, 2, lens, 1, 128, 64, "bf16")
    masks = [S.tree(g, t) for t in news] if tree else None
    window, sinks = (0, 0) if tree else (100, 70)
    q, out, lse = attend(dcc, cache, g, 2, 1, 128, "bf16", lens, news, share, window, sinks, masks)
    check(cache, table, 2, 1, 128, 64, "bf16", lens, news, share, window, sinks, masks, q, out, lse, "prompt")


def test_two_calls_at_once(dcc):  # noqa: F811
    """On two streams, with a workspace each, over and over: as one after the other."""
    g = torch.Generator().manual_seed(13)
    lens, news = [3000, 700], [40, 9]
    cache, _, _ = make_cache(dcc, g, 2, lens, 1, 128, 64, "bf16")
    q = [torch.randn(sum(news), 8, 128, generator=g).bfloat16().cuda() for _ in range(2)]
    mask, start = S.pack([m for t in news for m in S.tree(g, t)], 2).cuda(), batch(news)
    streams, ws = [torch.cuda.Stream() for _ in range(2)], [cache.attention_workspace(8) for _ in range(2)]

    def call(i, out):
        with torch.cuda.stream(streams[i]):
            if i == 0:
                cache.attention_tree(q, out, start, mask, max_new=40, workspace=ws[0])
            else:
                cache.attention_sinks(q, out, start, max_new=40, workspace=ws[1], window=300, sinks=70)
    want = [[torch.empty_like(x) for x in q] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(2):
        call(i, want[i])
        torch.cuda.synchronize()
    got = [[[torch.empty_like(x) for x in q] for _ in range(2)] for _ in range(6)]
    torch.cuda.synchronize()
    for pair in got:
        for i in range(2):
            call(i, pair[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for pair in got for i in range(2) for a, b in zip(pair[i], want[i]))
    assert dcc.dcc_local_check() == dcc.DCC_OK


@pytest.mark.parametrize("news,share", [([5, 2], 2), ([40, 33], 8)])
def test_layers(dcc, news, share):  # noqa: F811
    """Each layer's own pages."""
    g = torch.Generator().manual_seed(14)
    lens = [300, 90]
    cache, _, table = make_cache(dcc, g, 2, lens, 2, 64, 32, "fp16", layers=3)
    start, mask = batch(news), S.pack([m for t in news for m in S.tree(g, t)], 2).cuda()
    q = [torch.randn(sum(news), 2 * share, 64, generator=g).half().cuda() for _ in range(2)]
    ws = cache.attention_workspace(2 * share)
    for layer in range(3):
        alone = dcc.Kv4Cache([p[layer:layer + 1] for p in cache.pools], cache.table, cache.lengths, None, 2, 64, 32, "fp16")
        for tree in (True, False):
            got, want = ([torch.empty_like(x) for x in q] for _ in range(2))
            for c, out, at in ((cache, got, layer), (alone, want, 0)):
                if tree:
                    c.attention_tree(q, out, start, mask, max_new=max(news), workspace=ws, layer=at)
                else:
                    c.attention_sinks(q, out, start, max_new=max(news), workspace=ws, window=60, sinks=5, layer=at)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert dcc.dcc_local_check() == dcc.DCC_OK
