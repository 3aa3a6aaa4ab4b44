"""The 4-bit cache on the GPU: append, read and attention against 64-bit forms.

Append and read are exact: codes, steps and minima are determined by the
definition (IEEE fp32 arithmetic on 16-bit inputs), and a value read back is
lo + step * code rounded once.

Attention, with u the type's unit roundoff and e = 2^-23 (an fp32 rounding, or
truncation, per operation): keys may enter the first product rounded to the
type (u per element), so a score is off by at most ds = (u + (D + 8) e) *
scale * sum|q K|; the probabilities are off by a factor within exp(+-2 ds) and
another rounding u, values by u, sums of n terms by n e relative to sum p|V|,
and the result is rounded once (by half the smallest subnormal, 2^-25 in fp16,
where it lies below the normal numbers):
  |out - exact| <= (2 u + expm1(2 ds) + 2 n e) * sum p|V| (1 + small) + u |exact| + tiny
  |lse - exact| <= ds + n e + 4 e |lse|
"""
import math

import pytest
import torch

import kv4_reference as R

pytestmark = pytest.mark.gpu
TD, U, PAGE = R.TD, R.U, R.PAGE
E = 2.0 ** -23
TINY = {"bf16": 1e-30, "fp16": 2.0 ** -25}


@pytest.fixture(scope="module")
def dcc():
    from driven_collective_communication_gb300 import build
    build.build()
    from driven_collective_communication_gb300 import dcc as mod
    torch.cuda.set_device(0)
    return mod


def make_cache(dcc, g, n, lens, heads, dim, group, dtype, layers=1, spare=2, max_pages=None, poison=True):
    need = [-(-m // PAGE) for m in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).tolist()
    mp = max_pages or max(need + [1])
    table = torch.full((len(lens), mp), -1, dtype=torch.int32)
    for s, c in enumerate(need):
        for j in range(c):
            table[s, j] = order.pop()
    pools = [R.random_pool(g, layers, pages, heads, dim, group, dtype) for _ in range(n)]
    if poison:
        for p in pools:
            R.poison(p, table, lens, dim, group)
    cache = dcc.Kv4Cache([p.cuda() for p in pools], table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                         torch.zeros(pages, dtype=torch.int32).cuda(), heads, dim, group, dtype)
    return cache, pools, table


def starts(news):
    out = [0]
    for t in news:
        out.append(out[-1] + t)
    return out


def batch(news):
    return torch.tensor(starts(news), dtype=torch.int32).cuda()


def test_reference_places_are_a_permutation():
    for dim in (64, 128):
        assert sorted(R.k_nibble(dim, d) for d in range(dim)) == list(range(dim))
        for t in range(PAGE):
            assert sorted(R.v_nibble(dim, d, t) for d in range(dim)) == list(range(dim))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64)])
@pytest.mark.parametrize("n,heads,lens,news,layer,layers", [
    (1, 1, [1], [1], 0, 1), (2, 3, [70, 64, 1, 200], [70, 1, 1, 65], 1, 2),
    (8, 1, [5, 0, 130], [2, 0, 130], 0, 1), (3, 2, [64] * 20, [1] * 20, 0, 1),
    (1, 2, [3, 40], [5, 1], 0, 1),            # two rows before position zero: skipped
    (1, 1, [1] * 300, [1] * 300, 2, 3)])
def test_append_then_read(dcc, dtype, dim, group, n, heads, lens, news, layer, layers):
    g = torch.Generator().manual_seed(dim + group + sum(lens))
    cache, pools, table = make_cache(dcc, g, n, lens, heads, dim, group, dtype, layers)
    T = sum(news)
    k = [(torch.randn(T, heads, dim, generator=g) * 1.7 + 0.3).to(TD[dtype]) for _ in range(n)]
    v = [torch.randn(T, heads, dim, generator=g).to(TD[dtype]) for _ in range(n)]
    k[0][0, 0, :group] = 1.25                  # a constant group
    v[0][T // 2, 0, :4] = torch.tensor([0.0, -0.0, 1e-7, -3.0]).to(TD[dtype])
    start = batch(news)
    cache.append([x.cuda() for x in k], [x.cuda() for x in v], start, layer=layer)
    fill = 7.0
    ko = [torch.full((T, heads, dim), fill, dtype=TD[dtype], device="cuda") for _ in range(n)]
    vo = [torch.full((T, heads, dim), fill, dtype=TD[dtype], device="cuda") for _ in range(n)]
    cache.read(ko, vo, start, layer=layer)
    assert dcc.dcc_local_check() == dcc.DCC_OK
    row_pos = []
    for s, (m, t) in enumerate(zip(lens, news)):
        row_pos += [(s, m - t + i) for i in range(t)]
    skipped = torch.tensor([p < 0 for _, p in row_pos])
    for r in range(n):
        for got, x in ((ko[r], k[r]), (vo[r], v[r])):
            want = R.quantise(x, group, dtype).to(torch.float32).to(TD[dtype])
            want[skipped] = fill
            assert torch.equal(got.cpu(), want)
        # only the batch's rows of this layer changed
        before_k, before_v = R.values(pools[r], dim, group, dtype)
        after_k, after_v = R.values(cache.pools[r].cpu(), dim, group, dtype)
        touched = torch.zeros(pools[r].shape[:2] + (PAGE,), dtype=torch.bool)
        for s, p in row_pos:
            if p >= 0:
                touched[layer, table[s, p // PAGE], p % PAGE] = True
        for a, b in ((after_k, before_k), (after_v, before_v)):
            same = ((a == b) | (a.isnan() & b.isnan())).all(-1).all(2)
            assert same[~touched].all()


@pytest.mark.parametrize("dtype,dim,group", [("bf16", 128, 64), ("fp16", 64, 32), ("bf16", 64, 64), ("fp16", 128, 32)])
def test_append_then_read_of_many_rows(dcc, dtype, dim, group):
    """Batches large enough that a group of lanes takes several rows: runs that
    cross sequences (some without rows) and pages, rows before position zero,
    rows of no sequence at the end, a row count that is no multiple."""
    n, heads = 8, 4
    lens = [700, 3, 0, 64, 129] + [1] * 30 + [5, 401]
    news = [650, 5, 0, 64, 2] + [1] * 30 + [0, 401]
    g = torch.Generator().manual_seed(12)
    cache, _, _ = make_cache(dcc, g, n, lens, heads, dim, group, dtype)
    T = sum(news) + 67
    k, v = ([torch.randn(T, heads, dim, generator=g).to(TD[dtype]) for _ in range(n)] for _ in range(2))
    start = batch(news)
    cache.append([x.cuda() for x in k], [x.cuda() for x in v], start)
    ko, vo = ([torch.full((T, heads, dim), 7.0, dtype=TD[dtype], device="cuda") for _ in range(n)] for _ in range(2))
    cache.read(ko, vo, start)
    assert dcc.dcc_local_check() == dcc.DCC_OK
    there = torch.tensor([m - t + i >= 0 for m, t in zip(lens, news) for i in range(t)] + [False] * 67)
    for got, x in zip(ko + vo, k + v):
        want = R.quantise(x, group, dtype).to(torch.float32).to(TD[dtype])
        want[~there] = 7.0
        assert torch.equal(got.cpu(), want)


def test_append_of_special_values(dcc):
    """NaN and infinities read back as NaN in their own group only; a range
    that overflows the type as well; the largest finite values survive."""
    g = torch.Generator().manual_seed(3)
    for dtype in ("bf16", "fp16"):
        big = torch.finfo(TD[dtype]).max
        cache, _, _ = make_cache(dcc, g, 1, [6], 1, 128, 32, dtype)
        x = torch.randn(6, 1, 128, generator=g).to(TD[dtype])
        x[0, 0, 3], x[1, 0, 40], x[2, 0, 127] = math.nan, math.inf, -math.inf
        x[3, 0, 64], x[3, 0, 65] = big, -big
        x[4, 0, :32] = -big
        x[5, 0, 0] = torch.finfo(TD[dtype]).tiny / 4  # subnormal
        out = [torch.empty_like(x).cuda() for _ in range(2)]
        cache.append([x.cuda()], [x.cuda()], batch([6]))
        cache.read([out[0]], [out[1]], batch([6]))
        want = R.quantise(x, 32, dtype).to(torch.float32).to(TD[dtype])
        if dtype == "bf16":
            assert want[3, 0, 64].isnan()  # 2 * max has no bf16 step
        for o in out:
            assert torch.equal(o.cpu().isnan(), want.isnan())
            assert torch.equal(o.cpu().nan_to_num(9.0), want.nan_to_num(9.0))


def test_append_strided_rows(dcc):
    """K and V as slices of one fused projection, in place."""
    g = torch.Generator().manual_seed(4)
    cache, _, _ = make_cache(dcc, g, 2, [33, 90], 2, 64, 32, "bf16")
    qkv = [torch.randn(34, 10, 64, generator=g).bfloat16().cuda() for _ in range(2)]
    k, v = [x[:, 6:8] for x in qkv], [x[:, 8:10] for x in qkv]
    cache.append(k, v, batch([33, 1]))
    ko, vo = [torch.empty(34, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)], \
             [torch.empty(34, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cache.read(ko, vo, batch([33, 1]))
    for r in range(2):
        assert torch.equal(ko[r].double(), R.quantise(k[r], 32, "bf16").float().bfloat16().double())
        assert torch.equal(vo[r].double(), R.quantise(v[r], 32, "bf16").float().bfloat16().double())


def check_attention(dcc, dtype, dim, group, n, heads, share, lens, news, window=0, scale=None, seed=0, q_scale=1.0,
                    with_lse=True, max_new=None, layers=1, layer=0, extra_rows=0, stream=None, strided=False, powers=None):
    g = torch.Generator().manual_seed(seed + 31 * dim + group + heads + share)
    cache, pools, table = make_cache(dcc, g, n, lens, heads, dim, group, dtype, layers)
    if powers:  # K and V of single tokens multiplied by powers of two: powers = (of K, of V), drawn from
        for pool in cache.pools:
            par = pool.view(TD[dtype]).view(*pool.shape[:-1], -1)[..., PAGE * dim // 2:]
            par = par.view(*pool.shape[:-1], 2, PAGE, -1)
            for side, of in enumerate(powers):
                e = torch.tensor(of)[torch.randint(len(of), (*par.shape[:-3], PAGE, 1), generator=g)]
                par[..., side, :, :] *= torch.exp2(e.double()).to(TD[dtype]).cuda()
    T, Hq = sum(news) + extra_rows, heads * share
    wide = Hq + (2 * heads if strided else 0)
    q = [(q_scale * torch.randn(T, wide, dim, generator=g)).to(TD[dtype]).cuda()[:, :Hq] for _ in range(n)]
    fill = 3.0
    out = [torch.full((T, Hq, dim), fill, dtype=TD[dtype], device="cuda") for _ in range(n)]
    lse = [torch.full((T, Hq), fill, device="cuda") for _ in range(n)] if with_lse else None
    ws = cache.attention_workspace(Hq)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    start = batch(news)
    for _ in range(2):  # twice: the workspace is left as it was found
        cache.attention(q, out, start, max_new=max_new or max(news), workspace=ws, lse=lse, scale=scale,
                        window=window, layer=layer, stream=stream)
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    assert dcc.dcc_local_check(stream) == dcc.DCC_OK
    sc = dim ** -0.5 if scale is None else scale
    u, st = U[dtype], starts(news)
    for r in range(n):
        K, V = R.values(cache.pools[r][layer], dim, group, dtype)  # [pages, heads, 64, dim]
        got_o, got_l = out[r].double(), lse[r].double() if with_lse else None
        for s, (m, t) in enumerate(zip(lens, news)):
            if t == 0:
                continue
            rows = slice(st[s], st[s + 1])
            pg = table[s, :-(-m // PAGE)].long().cuda()
            pos = torch.arange(m - t, m, device="cuda")
            for h in range(heads):
                Kh = K[pg, h].reshape(-1, dim)[:m]
                Vh = V[pg, h].reshape(-1, dim)[:m]
                for x in range(share):
                    qq = q[r][rows, h * share + x].double()
                    o, l, pv, mag = R.attention(Kh, Vh, qq, pos, window, sc)
                    o, l, pv, mag = o.cuda(), l.cuda(), pv.cuda(), mag.cuda()
                    ds = (u + (dim + 8) * E) * mag
                    tol = (2 * u + torch.expm1(2 * ds) + 2 * max(m, 1) * E)[:, None] * pv * 1.01 + u * o.abs() + TINY[dtype]
                    err = (got_o[rows, h * share + x] - o).abs()
                    assert (err <= tol).all(), (r, s, h, x, (err / tol).max())
                    if with_lse:
                        gl = got_l[rows, h * share + x]
                        empty = torch.isinf(l)
                        assert torch.equal(torch.isinf(gl), empty) and (gl[empty] < 0).all()
                        e2 = (gl - l)[~empty].abs()
                        assert (e2 <= (ds + max(m, 1) * E + 4 * E * l.abs())[~empty] + 1e-6).all(), (e2.max())
                        assert (got_o[rows, h * share + x][empty] == 0).all()
        if extra_rows:
            assert (out[r][T - extra_rows:] == fill).all()
    return cache, q, out, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64)])
@pytest.mark.parametrize("n,heads,share,lens", [
    (1, 1, 1, [1]), (1, 1, 8, [777]), (8, 1, 8, [64, 1, 65, 0, 300]), (2, 2, 4, [129, 4000]),
    (3, 1, 5, [63, 62, 2]), (1, 4, 16, [200, 64, 128]), (2, 1, 7, [1] * 70), (1, 1, 33, [100])])
def test_decode(dcc, dtype, dim, group, n, heads, share, lens):
    check_attention(dcc, dtype, dim, group, n, heads, share, lens, [1] * len(lens))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group", [(64, 32), (128, 64)])
@pytest.mark.parametrize("heads,share,lens,news,window", [
    (1, 4, [300, 5, 64], [5, 5, 1], 0), (2, 2, [1000], [3], 100), (1, 8, [70, 130], [2, 8], 64),
    (2, 1, [40, 41, 42], [2, 0, 7], 1), (1, 3, [2000, 10], [4, 10], 1), (1, 8, [90], [4], 65)])
def test_several_tokens(dcc, dtype, dim, group, heads, share, lens, news, window):
    check_attention(dcc, dtype, dim, group, 2, heads, share, lens, news, window)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64)])
@pytest.mark.parametrize("heads,share,lens,news,window", [
    (1, 8, [200], [200], 0), (2, 4, [513, 70], [100, 70], 0), (1, 1, [300], [300], 0), (1, 16, [1000], [33], 0),
    (2, 3, [400, 129, 1], [129, 129, 1], 50), (1, 5, [700], [311], 128)])
def test_prompt_chunks(dcc, dtype, dim, group, heads, share, lens, news, window):
    check_attention(dcc, dtype, dim, group, 2, heads, share, lens, news, window)


@pytest.mark.parametrize("news", [[3, 40, 1], [4, 1, 1]])
def test_rows_before_position_zero_and_idle_slots(dcc, news):
    """More new rows than the sequence holds: those before position zero see
    nothing; an idle slot sees nothing; rows of no sequence stay."""
    check_attention(dcc, "bf16", 128, 64, 2, 1, 8, [1, 20, 0], news, extra_rows=3)


def test_large_and_tiny_scores(dcc):
    """Scores of a few hundred (one key takes all) and of almost zero."""
    check_attention(dcc, "bf16", 128, 64, 1, 1, 8, [500, 64], [1, 1], scale=4.0)
    check_attention(dcc, "fp16", 64, 32, 1, 1, 8, [500, 64], [1, 1], scale=4.0)
    check_attention(dcc, "fp16", 128, 32, 1, 2, 2, [500, 64], [40, 2], scale=1e-6)
    check_attention(dcc, "bf16", 64, 32, 1, 2, 2, [500, 300], [100, 2], scale=-0.5)


@pytest.mark.parametrize("dtype,dim,group", [("bf16", 128, 64), ("fp16", 64, 32)])
def test_zero_scale_and_unusual_queries(dcc, dtype, dim, group):
    """Scale 0 (every key counts the same), queries far from 1, many tiny pages."""
    check_attention(dcc, dtype, dim, group, 1, 1, 8, [500, 64, 0], [1, 1, 1], scale=0.0)
    check_attention(dcc, dtype, dim, group, 1, 2, 3, [500, 70], [4, 1], scale=1e-4, q_scale=1000.0)
    check_attention(dcc, dtype, dim, group, 1, 1, 8, [300], [1], scale=1000.0, q_scale=1e-3)
    check_attention(dcc, "bf16", dim, group, 2, 1, 8, [300, 20], [1, 1], scale=1e-28, q_scale=1e27)
    check_attention(dcc, dtype, dim, group, 1, 1, 2, [33] * 700, [1] * 700)  # more sequences than a CTA's threads


def test_without_lse_layers_and_strided_queries(dcc):
    check_attention(dcc, "bf16", 128, 64, 2, 2, 4, [100, 300], [1, 1], with_lse=False, layers=3, layer=2, strided=True)
    check_attention(dcc, "fp16", 64, 32, 2, 2, 4, [100, 300], [90, 20], with_lse=False, layers=2, layer=1, strided=True)


def test_on_another_stream(dcc):
    check_attention(dcc, "bf16", 128, 64, 2, 1, 8, [3000, 10, 700], [1, 1, 1], stream=torch.cuda.Stream())
    check_attention(dcc, "bf16", 128, 64, 2, 1, 8, [300, 100], [200, 30], stream=torch.cuda.Stream())


def test_long_sequence(dcc):
    check_attention(dcc, "bf16", 128, 64, 1, 1, 2, [40001], [1])
    check_attention(dcc, "fp16", 64, 32, 1, 1, 1, [70003, 1], [1, 1])


@pytest.mark.parametrize("new", [1, 60])
def test_nan_reaches_only_the_rows_that_see_it(dcc, new):
    g = torch.Generator().manual_seed(9)
    m = 200
    for which in ("k", "v"):
        cache, _, _ = make_cache(dcc, g, 1, [m, m], 1, 128, 64, "bf16")
        x = torch.randn(2 * m, 1, 128, generator=g).bfloat16()
        y = x.clone()
        y[m - 30, 0, 5] = math.nan  # the first sequence's position m - 30
        k, v = (y, x) if which == "k" else (x, y)
        cache.append([k.cuda()], [v.cuda()], batch([m, m]))
        q = torch.randn(2 * new, 8, 128, generator=g).bfloat16().cuda()
        out = torch.empty_like(q)
        cache.attention([q], [out], batch([new, new]), max_new=new, workspace=cache.attention_workspace(8))
        sees = torch.arange(m - new, m) >= m - 30
        bad = out[:new].isnan().any(-1).any(-1).cpu()
        assert torch.equal(bad, sees) and not out[new:].isnan().any()


# The prompt kernel runs where (ranks x kv heads x sequences) x (rows / 16)
# passes 100 (few pages): these do.
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64)])
@pytest.mark.parametrize("heads,share,lens,news,window", [
    (4, 4, [90, 300, 64, 1], [30, 20, 25, 1], 0),        # a single, partial row tile
    (2, 8, [16, 200, 129], [16, 33, 129], 0),            # exactly one row tile; two
    (1, 3, [2000, 30, 500, 0], [90, 90, 85, 4], 70),     # window, more rows than tokens, an idle slot
    (4, 16, [65, 1000], [17, 40], 1), (4, 1, [128, 256, 383], [128, 100, 129], 0)])
def test_prompt_kernel(dcc, dtype, dim, group, heads, share, lens, news, window):
    check_attention(dcc, dtype, dim, group, 8, heads, share, lens, news, window, extra_rows=2)


def test_prompt_kernel_scores_scales_and_streams(dcc):
    check_attention(dcc, "bf16", 128, 64, 8, 2, 8, [500, 64], [60, 40], scale=4.0)
    check_attention(dcc, "fp16", 64, 32, 8, 2, 8, [500, 300], [60, 100], scale=-2.0)
    check_attention(dcc, "fp16", 128, 32, 8, 2, 8, [500, 64], [60, 40], scale=0.0)
    check_attention(dcc, "bf16", 128, 64, 8, 2, 8, [500, 64], [60, 40], with_lse=False, strided=True, layers=2, layer=1,
                    stream=torch.cuda.Stream(), max_new=60)


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("dtype,group", [("bf16", 64), ("fp16", 32)])
def test_nan_in_the_prompt_kernel(dcc, which, dtype, group):
    g = torch.Generator().manual_seed(10)
    n, m, new = 8, 200, 60
    cache, _, _ = make_cache(dcc, g, n, [m, m], 1, 128, group, dtype)
    x = torch.randn(2 * m, 1, 128, generator=g).to(TD[dtype])
    y = x.clone()
    y[m - 30, 0, 5], y[m - 10, 0, 120] = math.nan, math.inf
    k, v = (y, x) if which == "k" else (x, y)
    cache.append([k.cuda()] * n, [v.cuda()] * n, batch([m, m]))
    q = torch.randn(2 * new, 8, 128, generator=g).to(TD[dtype]).cuda()
    out = [torch.empty_like(q) for _ in range(n)]
    cache.attention([q] * n, out, batch([new, new]), max_new=new, workspace=cache.attention_workspace(8))
    sees = torch.arange(m - new, m) >= m - 30
    for o in out:
        assert torch.equal(o[:new].isnan().any(-1).any(-1).cpu(), sees) and not o[new:].isnan().any()


def test_bad_pages_in_the_prompt_kernel(dcc):
    """A missing page is skipped: its keys are seen by nobody."""
    g = torch.Generator().manual_seed(11)
    n, lens, new = 8, [300, 300], 100
    cache, _, table = make_cache(dcc, g, n, lens, 1, 128, 64, "bf16")
    q = [torch.randn(2 * new, 8, 128, generator=g).bfloat16().cuda() for _ in range(n)]
    out = [torch.empty_like(x) for x in q]
    cache.table[1, 2] = cache.pages + 3
    cache.attention(q, out, batch([new, new]), max_new=new, workspace=cache.attention_workspace(8))
    assert dcc.dcc_local_check() == dcc.DCC_ERR_BOUNDS
    K, V = R.values(cache.pools[3][0], 128, 64, "bf16")
    keep = torch.tensor([j for j in range(300) if not 128 <= j < 192])
    pg = table[1, :5].long().cuda()
    Kh, Vh = K[pg, 0].reshape(-1, 128)[:300].cpu(), V[pg, 0].reshape(-1, 128)[:300].cpu()
    for i in (0, 57, 99):
        pos = 200 + i
        seen = keep[keep <= pos]
        for h in (0, 7):
            o, _, pv, mag = R.attention(Kh[seen], Vh[seen], q[3][new + i, h].double().cpu()[None],
                                        torch.tensor([10 ** 6]), 0, 128 ** -0.5)
            ds = (U["bf16"] + 136 * E) * mag
            tol = (2 * U["bf16"] + torch.expm1(2 * ds) + 600 * E)[:, None] * pv * 1.01 + U["bf16"] * o.abs()
            assert ((out[3][new + i, h].cpu().double() - o).abs() <= tol).all()


def test_prompt_kernel_past_four_gigabytes(dcc):
    block = R.block_bytes(128, 64)
    pages = (1 << 32) // block + 300
    pool = torch.zeros(1, pages, 1, block, dtype=torch.uint8, device="cuda")
    row = [pages - 1, 3, pages - 200]
    one = dcc.Kv4Cache([pool], torch.tensor([row], dtype=torch.int32, device="cuda"),
                       torch.tensor([150], dtype=torch.int32, device="cuda"), None, 1, 128, 64, "bf16")
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(150, 1, 128, generator=g).bfloat16() for _ in range(2))
    one.append([k.cuda()], [v.cuda()], batch([150]))
    many = dcc.Kv4Cache([pool], torch.tensor([row] * 16, dtype=torch.int32, device="cuda"),
                        torch.full((16,), 150, dtype=torch.int32, device="cuda"), None, 1, 128, 64, "bf16")
    q = torch.randn(1600, 4, 128, generator=g).bfloat16()
    out = torch.empty(1600, 4, 128, dtype=torch.bfloat16, device="cuda")
    many.attention([q.cuda()], [out], batch([100] * 16), max_new=100, workspace=many.attention_workspace(4))
    K, V = R.quantise(k, 64, "bf16")[:, 0], R.quantise(v, 64, "bf16")[:, 0]
    for s in (0, 15):
        for h in (0, 3):
            rows = slice(100 * s, 100 * s + 100)
            o, _, pv, mag = R.attention(K, V, q[rows, h].double(), torch.arange(50, 150), 0, 128 ** -0.5)
            ds = (U["bf16"] + 136 * E) * mag
            tol = (2 * U["bf16"] + torch.expm1(2 * ds) + 300 * E)[:, None] * pv * 1.01 + U["bf16"] * o.abs()
            assert ((out[rows, h].cpu().double() - o).abs() <= tol).all()


def test_pages_past_four_gigabytes(dcc):
    """Page numbers whose byte offsets pass 32 bits."""
    block = R.block_bytes(128, 64)
    pages = (1 << 32) // block + 300
    pool = torch.zeros(1, pages, 1, block, dtype=torch.uint8, device="cuda")
    table = torch.tensor([[pages - 1, 3, pages - 200]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([150], dtype=torch.int32, device="cuda")
    cache = dcc.Kv4Cache([pool], table, lens, None, 1, 128, 64, "bf16")
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(150, 1, 128, generator=g).bfloat16() for _ in range(2))
    cache.append([k.cuda()], [v.cuda()], batch([150]))
    ko, vo = (torch.empty(150, 1, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache.read([ko], [vo], batch([150]))
    assert torch.equal(ko.cpu(), R.quantise(k, 64, "bf16").float().bfloat16())
    assert torch.equal(vo.cpu(), R.quantise(v, 64, "bf16").float().bfloat16())
    K, V = R.quantise(k, 64, "bf16")[:, 0], R.quantise(v, 64, "bf16")[:, 0]
    for new in (1, 100):
        q = torch.randn(new, 4, 128, generator=g).bfloat16()
        out = torch.empty(new, 4, 128, dtype=torch.bfloat16, device="cuda")
        cache.attention([q.cuda()], [out], batch([new]), max_new=new, workspace=cache.attention_workspace(4))
        for h in range(4):
            o, _, pv, mag = R.attention(K, V, q[:, h].double(), torch.arange(150 - new, 150), 0, 128 ** -0.5)
            ds = (U["bf16"] + 136 * E) * mag
            tol = (2 * U["bf16"] + torch.expm1(2 * ds) + 300 * E)[:, None] * pv * 1.01 + U["bf16"] * o.abs()
            assert ((out[:, h].cpu().double() - o).abs() <= tol).all()


def test_bad_page_numbers_are_reported_and_skipped(dcc):
    """A table entry that is no page: the call skips it and says so."""
    g = torch.Generator().manual_seed(6)
    cache, _, _ = make_cache(dcc, g, 1, [130], 1, 128, 64, "bf16")
    good = cache.table.clone()
    q = torch.randn(1, 8, 128, generator=g).bfloat16().cuda()
    x = torch.randn(130, 1, 128, generator=g).bfloat16().cuda()
    ws = cache.attention_workspace(8)
    for entry in (-1, cache.pages, 1 << 30):
        cache.table.copy_(good)
        cache.table[0, 1] = entry
        out = torch.empty_like(q)
        cache.attention([q], [out], batch([1]), max_new=1, workspace=ws)
        assert dcc.dcc_local_check() == dcc.DCC_ERR_BOUNDS
        assert dcc.dcc_local_check() == dcc.DCC_OK
        cache.append([x], [x], batch([130]))
        assert dcc.dcc_local_check() == dcc.DCC_ERR_BOUNDS
    cache.table.copy_(good)
    cache.lengths.fill_(64 * cache.max_pages + 5)  # longer than its row
    cache.attention([q], [torch.empty_like(q)], batch([1]), max_new=1, workspace=ws)
    assert dcc.dcc_local_check() == dcc.DCC_ERR_BOUNDS


@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64)])
@pytest.mark.parametrize("powers,q_scale,scale", [
    (([0, 0, -30, 5], [0]), 1.0, None), (([0, -3, 18], [0]), 1.0, 2.0 ** -21), (([0], [0, 0, -25, 9]), 1.0, None),
    (([100, 90], [-60, 60]), 1e-30, 0.05), (([-90, -100], [-20]), 1e27, -0.5),
    (([0] * 299 + [-30], [0] * 299 + [20]), 1.0, None)])  # some pages only
def test_prompt_wide_ranges(dcc, dim, group, powers, q_scale, scale):
    """bf16 tokens whose values leave the range of 16-bit floats, beside others that do not."""
    check_attention(dcc, "bf16", dim, group, 8, 2, 8, [500, 300], [60, 100], scale=scale, q_scale=q_scale, powers=powers)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_prompt_calls_back_to_back(dcc, dtype):
    """Calls on caches in turn, nothing waited for between them: pages come from memory in any order."""
    g = torch.Generator().manual_seed(5)
    sets = []
    for _ in range(3):
        cache, _, _ = make_cache(dcc, g, 8, [4096], 1, 128, 64, dtype)
        q = [torch.randn(512, 8, 128, generator=g).to(TD[dtype]).cuda() for _ in range(8)]
        sets.append((cache, q, [torch.empty_like(x) for x in q], cache.attention_workspace(8)))
    start = batch([512])

    def run(s):
        s[0].attention(s[1], s[2], start, max_new=512, workspace=s[3])

    want = []
    for s in sets:
        run(s)
        torch.cuda.synchronize()
        want.append([x.clone() for x in s[2]])
    for i in range(240):
        run(sets[i % 3])
    assert dcc.dcc_local_check() == dcc.DCC_OK
    for s, w in zip(sets, want):
        assert all(torch.equal(a, b) for a, b in zip(s[2], w))
