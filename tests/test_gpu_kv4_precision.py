"""How exact the attention over the 4-bit cache is, both kernels: every element
within kv4_bounds, every case's 2-norm within a limit that bf16 operands (3.0e-3)
or sums that lose bits (1.5e-3 in fp16) do not meet, and no case that a result
of zeros would pass."""
import pytest
import torch

import kv4_bounds as B
import kv4_reference as R
from test_attention_plan import plan  # noqa: F401  (a fixture)
from test_gpu_kv4 import batch, make_cache, starts

pytestmark = pytest.mark.gpu
TD = R.TD


@pytest.fixture(scope="module")
def dcc():
    from driven_collective_communication_gb300 import build
    build.build()
    from driven_collective_communication_gb300 import dcc as mod
    torch.cuda.set_device(0)
    return mod


def check(dcc, plan, kernel, dtype, dim, group, n, heads, share, lens, news, window=0, scale=None, q_scale=1.0,  # noqa: F811
          powers=None, seed=0):
    g = torch.Generator().manual_seed(1000 + seed + dim + group + share)
    cache, _, table = make_cache(dcc, g, n, lens, heads, dim, group, dtype)
    assert plan(heads=n * heads, seqs=len(lens), pages=table.shape[1], dim=dim, share=share, tokens=sum(news),
                max_new=max(news))["prompt"] == (kernel == "prompt")
    if powers:  # K and V of single tokens times powers of two drawn from powers = (of K, of V)
        for pool in cache.pools:
            par = pool.view(TD[dtype]).view(*pool.shape[:-1], -1)[..., R.PAGE * dim // 2:]
            par = par.view(*pool.shape[:-1], 2, R.PAGE, -1)
            for side, of in enumerate(powers):
                e = torch.tensor(of)[torch.randint(len(of), (*par.shape[:-3], R.PAGE, 1), generator=g)]
                par[..., side, :, :] *= torch.exp2(e.double()).to(TD[dtype]).cuda()
    T, Hq = sum(news), heads * share
    q = [(q_scale * torch.randn(T, Hq, dim, generator=g)).to(TD[dtype]).cuda() for _ in range(n)]
    out = [torch.full((T, Hq, dim), 3.0, dtype=TD[dtype], device="cuda") for _ in range(n)]
    lse = [torch.full((T, Hq), 3.0, device="cuda") for _ in range(n)]
    cache.attention(q, out, batch(news), max_new=max(news), workspace=cache.attention_workspace(Hq), lse=lse, scale=scale,
                    window=window)
    assert dcc.dcc_local_check() == dcc.DCC_OK
    sc, st = dim ** -0.5 if scale is None else scale, starts(news)
    totals = B.Totals(dtype, kernel == "prompt" and dtype == "bf16" and powers is not None and any(powers[1]))
    for r in {0, n - 1}:
        K, V = B.parts(cache.pools[r][0], dim, group, dtype)
        for s, (m, t) in enumerate(zip(lens, news)):
            rows, pg = slice(st[s], st[s + 1]), table[s, :-(-m // R.PAGE)].long().cuda()
            pos = torch.arange(m - t, m, device="cuda")
            for h in range(heads):
                Kh, Vh = B.rows_of(K, pg, h, m), B.rows_of(V, pg, h, m)
                for x in range(share):
                    o, l, tol, tol_l, rough = B.exact(Kh, Vh, q[r][rows, h * share + x].double(), pos, window, sc, dtype, kernel)
                    got, gl = out[r][rows, h * share + x].double(), lse[r][rows, h * share + x].double()
                    err = (got - o).abs()
                    assert (err <= tol).all(), (r, s, h, x, (err / tol).max())
                    none = torch.isinf(l)
                    assert torch.equal(torch.isinf(gl), none) and (got[none] == 0).all()
                    assert ((gl - l).abs() <= tol_l)[~none].all(), ((gl - l).abs() / tol_l)[~none].max()
                    totals.add(got, o, tol, rough)
    return totals.check()


SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group", SHAPES)
@pytest.mark.parametrize("n,heads,share,lens,news,window", [
    (1, 1, 8, [777], [1], 0), (8, 1, 8, [64, 1, 65, 0, 300], [1] * 5, 0), (2, 2, 4, [129, 4000], [1, 1], 0),
    (1, 1, 33, [100], [1], 0), (2, 1, 4, [300, 5, 64], [5, 5, 1], 0), (2, 2, 2, [1000], [3], 100),
    (1, 1, 8, [200, 200], [40, 40], 0)])
def test_streaming(dcc, plan, dtype, dim, group, n, heads, share, lens, news, window):  # noqa: F811
    check(dcc, plan, "streaming", dtype, dim, group, n, heads, share, lens, news, window)


def test_streaming_over_a_long_sequence(dcc, plan):  # noqa: F811
    check(dcc, plan, "streaming", "fp16", 128, 32, 1, 1, 4, [70003], [1])
    check(dcc, plan, "streaming", "bf16", 128, 64, 1, 1, 2, [70003], [1])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group", SHAPES)
@pytest.mark.parametrize("heads,share,lens,news,window", [
    (4, 4, [90, 300, 64, 1], [30, 20, 25, 1], 0), (2, 8, [16, 200, 129], [16, 33, 129], 0),
    (1, 3, [2000, 30, 500, 0], [90, 90, 85, 4], 70), (1, 8, [441], [300], 0)])
def test_prompt(dcc, plan, dtype, dim, group, heads, share, lens, news, window):  # noqa: F811
    check(dcc, plan, "prompt", dtype, dim, group, 8, heads, share, lens, news, window)


@pytest.mark.parametrize("kernel,n,news", [("streaming", 1, [1, 1]), ("streaming", 1, [9, 2]), ("prompt", 8, [60, 40])])
@pytest.mark.parametrize("dtype,dim,group", [("bf16", 128, 64), ("fp16", 64, 32), ("fp16", 128, 32)])
@pytest.mark.parametrize("scale,q_scale", [(4.0, 1.0), (-0.5, 1.0), (0.0, 1.0), (1000.0, 1e-3), (1e-4, 1000.0)])
def test_scales(dcc, plan, kernel, n, news, dtype, dim, group, scale, q_scale):  # noqa: F811
    check(dcc, plan, kernel, dtype, dim, group, n, 1, 8, [500, 64], news, scale=scale, q_scale=q_scale)


@pytest.mark.parametrize("dim,group", SHAPES)
@pytest.mark.parametrize("powers,q_scale,scale", [
    (([0, 0, -30, 5], [0]), 1.0, None), (([0, -3, 18], [0]), 1.0, 2.0 ** -21), (([0], [0, 0, -25, 9]), 1.0, None),
    (([100, 90], [-60, 60]), 1e-30, 0.05), (([-90, -100], [-20]), 1e27, -0.5),
    (([0] * 299 + [-30], [0] * 299 + [20]), 1.0, None)])
@pytest.mark.parametrize("kernel,n,news", [("streaming", 1, [1, 1]), ("prompt", 8, [60, 100])])
def test_wide_ranges(dcc, plan, kernel, n, news, dim, group, powers, q_scale, scale):  # noqa: F811
    check(dcc, plan, kernel, "bf16", dim, group, n, 1, 8, [500, 300], news, scale=scale, q_scale=q_scale, powers=powers)
