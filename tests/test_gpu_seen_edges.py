"""Trees and windows with sinks at the ends of the cache types' ranges, with few and
many rows, against 64 bits, within the bounds of seen_reference.exact (whose prompt
form holds for a value past the type's largest number, which may count as that)."""
import pytest
import torch

import kv4_bounds as B
import kv4_reference as R
import seen_reference as S
from test_gpu_kv4 import batch, dcc, make_cache, starts  # noqa: F401  (dcc: the fixture)

pytestmark = pytest.mark.gpu
TD = R.TD
FORMS = {"one token": (1, "streaming"), "few rows": (2, "streaming"), "many rows": (40, "prompt")}


def run(dcc, cache, table, q, lens, news, share, group, dtype, kernel, window, sinks, masks):
    D = q.shape[-1]
    n, q = len(cache.pools), q.cuda()
    out = [torch.full_like(q, 7.0) for _ in range(n)]
    kw = dict(max_new=max(news), workspace=cache.attention_workspace(share), window=window, sinks=sinks)
    if masks is None:
        cache.attention_sinks([q] * n, out, batch(news), **kw)
    else:
        mask = S.pack([m for s in masks for m in s], -(-max(news) // 32)).cuda()
        cache.attention_tree([q] * n, out, batch(news), mask, **kw)
    assert dcc.dcc_local_check() == dcc.DCC_OK
    at = starts(news)
    K, V = B.parts(cache.pools[n - 1][0].cpu(), D, group, dtype)
    for s, (m, t) in enumerate(zip(lens, news)):
        pg = table[s, :-(-m // R.PAGE)].long()
        k, v = B.rows_of(K, pg, 0, m), B.rows_of(V, pg, 0, m)
        seen = S.seen_rows(m, t, t, window, sinks, masks and masks[s])
        for x in range(share):
            want, _, tol, _, _ = S.exact(k, v, q[at[s]:at[s + 1], x].cpu().double(), seen, D ** -0.5, dtype, kernel)
            err = (out[n - 1][at[s]:at[s + 1], x].cpu().double() - want).abs()
            assert (err <= tol).all(), (s, x, (err / tol).max())


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dim,group", [(128, 64), (128, 32), (64, 64), (64, 32)])
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("lo,hi", [(0.0, 65504.0), (-65504.0, 65504.0), (-65504.0, -3e4), (65504.0, 65504.0), (-3e4, -1e3)])
def test_fp16_groups_as_wide_as_the_type(dcc, form, dim, group, side, lo, hi, tree):  # noqa: F811
    new, kernel = FORMS[form]
    g = torch.Generator().manual_seed(21)
    m = 200
    cache, _, table = make_cache(dcc, g, 2, [m, m], 1, dim, group, "fp16")
    x = torch.randn(2 * m, 1, dim, generator=g).half()
    y = x.clone()
    for at in (m - 1, m - 30, m - 61, m - 90, 3):
        y[at, 0, dim - group:] = (lo + (hi - lo) * torch.rand(group, generator=g)).clamp(-65504, 65504).half()
        y[at, 0, dim - group], y[at, 0, dim - group + 1] = lo, hi
    k, v = (y, x) if side == "k" else (x, y)
    cache.append([k.cuda()] * 2, [v.cuda()] * 2, batch([m, m]))
    q = torch.randn(2 * new, 8, dim, generator=g)
    q = (q * 2.0 ** -16 if side == "k" else q).half()  # scores of a few
    masks = [S.tree(g, new) for _ in range(2)] if tree else None
    run(dcc, cache, table, q, [m, m], [new, new], 8, group, "fp16", kernel, 70, 5, masks)


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dim,group", [(128, 64), (64, 32)])
@pytest.mark.parametrize("value", [1e-30, 1e-5, 3.0, 1e5, 1e20])
def test_bf16_values_of_all_sizes(dcc, form, dim, group, value, tree):  # noqa: F811
    """V of one size throughout, from far below fp16's range to far above."""
    new, kernel = FORMS[form]
    g = torch.Generator().manual_seed(22)
    m = 200
    cache, _, table = make_cache(dcc, g, 2, [m, m], 1, dim, group, "bf16")
    k = torch.randn(2 * m, 1, dim, generator=g).bfloat16()
    v = (value * torch.randn(2 * m, 1, dim, generator=g)).bfloat16()
    cache.append([k.cuda()] * 2, [v.cuda()] * 2, batch([m, m]))
    q = torch.randn(2 * new, 8, dim, generator=g).bfloat16()
    masks = [S.tree(g, new) for _ in range(2)] if tree else None
    run(dcc, cache, table, q, [m, m], [new, new], 8, group, "bf16", kernel, 70, 5, masks)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dim,group", [(128, 64), (64, 32)])
@pytest.mark.parametrize("value", [1e-20, 1e-3, 1e6, 1e25])
def test_bf16_keys_of_all_sizes(dcc, form, dim, group, value):  # noqa: F811
    new, kernel = FORMS[form]
    g = torch.Generator().manual_seed(23)
    m = 200
    cache, _, table = make_cache(dcc, g, 2, [m, m], 1, dim, group, "bf16")
    k = (value * torch.randn(2 * m, 1, dim, generator=g)).bfloat16()
    v = torch.randn(2 * m, 1, dim, generator=g).bfloat16()
    cache.append([k.cuda()] * 2, [v.cuda()] * 2, batch([m, m]))
    q = (torch.randn(2 * new, 8, dim, generator=g) / value).bfloat16()
    run(dcc, cache, table, q, [m, m], [new, new], 8, group, "bf16", kernel, 70, 5, [S.tree(g, new) for _ in range(2)])
