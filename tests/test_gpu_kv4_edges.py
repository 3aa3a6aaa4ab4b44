"""Attention over the 4-bit cache at the ends of its types' ranges, in both
kernels (few rows: streaming; many: prompt), against 64 bits, within the bounds
of kv4_bounds.  A value that the rounded-up step puts past the type's largest
number may count as the largest: 65,536 as 65,504 in fp16, off by 2^-11 of it,
which the prompt kernel's bound has for each element of K and V.
"""
import math

import pytest
import torch

import kv4_bounds as B
import kv4_reference as R
from test_gpu_kv4 import batch, make_cache

pytestmark = pytest.mark.gpu
TD = R.TD
# ranks, new tokens of each of two sequences, the kernel that runs
FORMS = {"one token": (1, 1, "streaming"), "streaming": (1, 40, "streaming"), "prompt": (8, 60, "prompt")}


@pytest.fixture(scope="module")
def dcc():
    from driven_collective_communication_gb300 import build
    build.build()
    from driven_collective_communication_gb300 import dcc as mod
    torch.cuda.set_device(0)
    return mod


def run(dcc, cache, table, q, lens, news, n, share, group, dtype, kernel, window=0, rows=None):
    """Attention on every rank; checks the first and the last against 64 bits."""
    D = q.shape[-1]
    q = q.cuda()
    out = [torch.full_like(q, 7.0) for _ in range(n)]
    cache.attention([q] * n, out, batch(news), max_new=max(news), workspace=cache.attention_workspace(share),
                    window=window)
    assert dcc.dcc_local_check() == dcc.DCC_OK
    at = [0]
    for t in news:
        at.append(at[-1] + t)
    for r in {0, n - 1}:
        K, V = B.parts(cache.pools[r][0], D, group, dtype)
        for s, (m, t) in enumerate(zip(lens, news)):
            pg = table[s, :-(-m // R.PAGE)].long().cuda()
            Kh, Vh = B.rows_of(K, pg, 0, m), B.rows_of(V, pg, 0, m)
            pos = torch.arange(m - t, m, device="cuda")
            take = torch.ones(t, dtype=torch.bool, device="cuda") if rows is None else rows(s, pos)
            for x in range(share):
                o, _, tol, _, _ = B.exact(Kh, Vh, q[at[s]:at[s + 1], x].double(), pos, window, D ** -0.5, dtype, kernel)
                err = (out[r][at[s]:at[s + 1], x].double() - o).abs()
                assert (err <= tol)[take].all(), (r, s, x, (err / tol)[take].max())
    return out


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dim,group", [(128, 64), (128, 32), (64, 64), (64, 32)])
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("lo,hi", [(0.0, 65504.0), (-65504.0, 65504.0), (-65504.0, 0.0), (-65504.0, -3e4), (65504.0, 65504.0)])
def test_fp16_groups_as_wide_as_the_type(dcc, form, dim, group, side, lo, hi):
    """One key in thirty whose group spans lo .. hi; rows before it and after it."""
    n, new, kernel = FORMS[form]
    g = torch.Generator().manual_seed(21)
    m = 200
    cache, _, table = make_cache(dcc, g, n, [m, m], 1, dim, group, "fp16")
    x = torch.randn(2 * m, 1, dim, generator=g).half()
    y = x.clone()
    for at in (m - 30, m - 61, m - 90, 3):
        y[at, 0, dim - group:] = (lo + (hi - lo) * torch.rand(group, generator=g)).clamp(-65504, 65504).half()
        y[at, 0, dim - group], y[at, 0, dim - group + 1] = lo, hi
    k, v = (y, x) if side == "k" else (x, y)
    cache.append([k.cuda()] * n, [v.cuda()] * n, batch([m, m]))
    q = torch.randn(2 * new, 8, dim, generator=g)
    q = (q * 2.0 ** -16 if side == "k" else q).half()  # scores of a few
    run(dcc, cache, table, q, [m, m], [new, new], n, 8, group, "fp16", kernel)


@pytest.mark.parametrize("form", FORMS)
def test_bf16_values_of_v_as_large_as_the_type(dcc, form):
    """A step rounded up past bf16's largest number: rows that do not see the
    key must not see an infinity either (those that do may overflow)."""
    n, new, kernel = FORMS[form]
    g = torch.Generator().manual_seed(22)
    m = 200
    cache, _, table = make_cache(dcc, g, n, [m, m], 1, 128, 64, "bf16")
    k = torch.randn(2 * m, 1, 128, generator=g).bfloat16()
    v = torch.randn(2 * m, 1, 128, generator=g).bfloat16()
    at = m - 20
    v[at, 0, 64], v[at, 0, 65] = -1.32e36, torch.finfo(torch.bfloat16).max
    cache.append([k.cuda()] * n, [v.cuda()] * n, batch([m, m]))
    assert (R.values(cache.pools[0][0].cpu(), 128, 64, "bf16")[1].abs() > torch.finfo(torch.bfloat16).max).any()
    q = torch.randn(2 * new, 8, 128, generator=g).bfloat16()
    out = run(dcc, cache, table, q, [m, m], [new, new], n, 8, 64, "bf16", kernel, rows=lambda s, pos: (pos < at) | (s == 1))
    assert not out[0].isnan().any()


@pytest.mark.parametrize("form", FORMS)
def test_nan_and_infinities_beside_large_groups(dcc, form):
    """A key with NaN in one group and a group as wide as the type in another:
    NaN for the rows that see it, nothing for the others."""
    n, new, kernel = FORMS[form]
    g = torch.Generator().manual_seed(23)
    m = 200
    for side in "kv":
        cache, _, _ = make_cache(dcc, g, n, [m, m], 1, 128, 32, "fp16")
        x = torch.randn(2 * m, 1, 128, generator=g).half()
        y = x.clone()
        y[m - 30, 0, 0], y[m - 30, 0, 1] = 65504.0, 0.0
        y[m - 30, 0, 40] = math.nan
        k, v = (y, x) if side == "k" else (x, y)
        cache.append([k.cuda()] * n, [v.cuda()] * n, batch([m, m]))
        q = torch.randn(2 * new, 8, 128, generator=g).half().cuda()
        out = torch.empty_like(q)
        cache.attention([q] * n, [out] + [torch.empty_like(q) for _ in range(n - 1)], batch([new, new]), max_new=new,
                        workspace=cache.attention_workspace(8))
        sees = torch.arange(m - new, m) >= m - 30
        assert torch.equal(out[:new].isnan().any(-1).any(-1).cpu(), sees) and torch.isfinite(out[new:]).all()
        assert torch.isfinite(out[:new][~sees]).all()


@pytest.mark.parametrize("window", [1 << 30, (1 << 31) - 1, (1 << 30) - 1])
@pytest.mark.parametrize("n,lens,news", [(1, [3, 70], [8, 1]), (1, [3, 70], [1, 1]), (8, [3, 70], [60, 60])])
def test_windows_longer_than_any_sequence(dcc, window, n, lens, news):
    """Nothing is hidden, also from a batch with rows before position zero."""
    g = torch.Generator().manual_seed(24)
    cache, _, _ = make_cache(dcc, g, n, lens, 1, 128, 64, "bf16")
    q = torch.randn(sum(news), 8, 128, generator=g).bfloat16().cuda()
    outs = []
    for w in (0, window):
        outs.append([torch.full_like(q, 7.0) for _ in range(n)])
        cache.attention([q] * n, outs[-1], batch(news), max_new=max(news), workspace=cache.attention_workspace(8), window=w)
    assert dcc.dcc_local_check() == dcc.DCC_OK
    assert outs[0][0].any() and all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,value", [("bf16", 1e20), ("bf16", -1e16), ("bf16", 3e30), ("bf16", 1e-30), ("fp16", 60000.0)])
@pytest.mark.parametrize("dim,group", [(128, 64), (64, 32)])
def test_constant_groups_of_v(dcc, form, dtype, value, dim, group):
    """Groups whose step is zero, the same in every key: V itself comes out; beside them ordinary ones."""
    n, new, kernel = FORMS[form]
    g = torch.Generator().manual_seed(25)
    m = 200
    for constant in (dim, dim - group):  # all groups, or all but one
        cache, _, table = make_cache(dcc, g, n, [m, m], 1, dim, group, dtype)
        k = torch.randn(2 * m, 1, dim, generator=g).to(TD[dtype])
        v = torch.randn(2 * m, 1, dim, generator=g).to(TD[dtype])
        v[..., :constant] = value
        cache.append([k.cuda()] * n, [v.cuda()] * n, batch([m, m]))
        q = torch.randn(2 * new, 8, dim, generator=g).to(TD[dtype])
        out = run(dcc, cache, table, q, [m, m], [new, new], n, 8, group, dtype, kernel)
        exact = torch.tensor(value).to(TD[dtype]).double().item()
        assert ((out[0][..., :constant].double() / exact - 1).abs() <= 2 * R.U[dtype]).all()


@pytest.mark.parametrize("form,news", [("one token", [1, 1]), ("streaming", [3, 5]), ("streaming", [40, 7]), ("prompt", [60, 61])])
@pytest.mark.parametrize("dtype,small,large", [("bf16", 1.0, 1e12), ("bf16", 1e-20, 1e8), ("fp16", 2.0 ** -18, 6e4)])
@pytest.mark.parametrize("dim,group", [(128, 64), (64, 32), (128, 32)])
@pytest.mark.parametrize("window", [0, 21])
def test_rows_do_not_lose_bits_to_keys_they_do_not_see(dcc, form, news, dtype, small, large, dim, group, window):
    """V of every fifth of the newest tokens is larger than the rest by more than
    a product's 16 bits can span: rows before such a token, or past its window,
    are as exact as without it."""
    n, _, kernel = FORMS[form]
    g = torch.Generator().manual_seed(26)
    m = 200
    cache, _, table = make_cache(dcc, g, n, [m, m], 1, dim, group, dtype)
    k = torch.randn(2 * m, 1, dim, generator=g).to(TD[dtype])
    v = torch.randn(2 * m, 1, dim, generator=g) * small
    huge = [(s, at) for s, t in enumerate(news) for at in range(m - t + 1, m, 5)]
    for s, at in huge:
        v[s * m + at] *= large / small / 4
    cache.append([k.cuda()] * n, [v.clamp(-6e4, 6e4).to(TD[dtype]).cuda() if dtype == "fp16" else v.to(TD[dtype]).cuda()] * n,
                 batch([m, m]))
    q = torch.randn(sum(news), 8, dim, generator=g).to(TD[dtype])

    def rows(s, pos):  # those that see none of them
        w = window or m
        return torch.stack([((at > pos) | (at <= pos - w)) for t, at in huge if t == s] +
                           [torch.ones_like(pos, dtype=torch.bool)]).all(0)
    run(dcc, cache, table, q, [m, m], news, n, 8, group, dtype, kernel, window=window, rows=rows)
