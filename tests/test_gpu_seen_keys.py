"""How exactly the keys of an fp16 cache of 64 channels enter the scores of trees and
of windows with sinks on the kernel of many rows: as two fp16 numbers.

Queries have one channel and every row sees one key, so a score is one product and
no sum rounds.  With m the group's largest magnitude and e = 2^-24 (an fp32
rounding; a tensor core may truncate, 2 e), the key's value k enters with an error of
at most
  2^-22 (|step code| + |k|) <= 2^-22 (2 m + m) < 2^-20 m      (lo + step code in fp16: the
      product's error is exact, the sum's error is exact, what is added of both is rounded
      to fp16, 2^-11 of at most 2^-11 (|step code| + |k|), a little more for the sum),
  or, for a large group, fp32's rounding e |k| and fp16's of what the first number left,
      2^-11 * 2^-11 |k|;
the parts below fp16's normal numbers are multiples of 2^-24 and exact in the first form,
off by 2^-25 in the second.  The products with q are exact in fp32 (22 bits), their sum is
off by 2 e |s|.  lse = ln 2 (ref - 6 + log2 l) with ref = c s, c = scale log2 e rounded
twice, l = 2^6: 3 e |s| for c and its product, 2 (|s| / ln 2 + 6) e ln 2 for the two sums, one
rounding of log2 l (6 * 2 e) and of the product with ln 2, itself rounded (2 e |s|).
Together, with 1.01 for products of errors:
  |lse - exact| <= 1.01 (|scale q| (2^-20 m + 2^-24) + 9 e |s| + 24 e)."""
import math

import pytest
import torch

import kv4_bounds as B
import kv4_reference as R
import seen_reference as S
from test_gpu_kv4 import batch, dcc, make_cache  # noqa: F401  (dcc: the fixture)

pytestmark = pytest.mark.gpu
DIM, E = 64, 2.0 ** -24


def put(pool, group, which, step, lo):
    """Parameters [layers, pages, heads, 64, groups] of K (0) or V (1)."""
    ng, half, par = DIM // group, R.PAGE * DIM // 2, R.PAGE * (DIM // group) * 4
    x = torch.stack([step, lo], -1).to(torch.float16).contiguous().view(torch.uint8)
    pool[..., 2 * half + which * par:2 * half + (which + 1) * par] = x.reshape(*pool.shape[:3], par)


@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("kind", ["ordinary", "far", "large V", "large K", "small"])
@pytest.mark.parametrize("tree", [True, False])
def test_keys_in_two_numbers(dcc, group, kind, tree):  # noqa: F811
    g = torch.Generator().manual_seed(group + len(kind))
    n, lens, news, share = 2, [200, 64], [100, 64], 2
    scale = {"large K": 2.0 ** -10, "small": 64.0}.get(kind, 1.0)
    cache, pools, table = make_cache(dcc, g, n, lens, 1, DIM, group, "fp16", poison=False)
    for r, pool in enumerate(pools):
        shape = (*pool.shape[:3], R.PAGE, DIM // group)
        rand = lambda: torch.rand(shape, generator=g)  # noqa: E731
        sign = torch.where(rand() < 0.5, -1.0, 1.0)
        if kind == "far":          # a step far below lo: the code is mostly lost in one number
            put(pool, group, 0, 0.01 + 0.1 * rand(), sign * (20 + 40 * rand()))
        elif kind == "large V":    # V out of the fast form's range, K ordinary
            put(pool, group, 0, 0.01 + 0.1 * rand(), sign * (20 + 40 * rand()))
            put(pool, group, 1, 1 + rand(), torch.where(rand() < 0.3, 40000.0, 3.0))
        elif kind == "large K":
            put(pool, group, 0, 1 + 30 * rand(), sign * (33000 + 20000 * rand()))
        elif kind == "small":      # among fp16's subnormal numbers
            put(pool, group, 0, 2.0 ** -18 * (1 + 15 * rand()), sign * 2.0 ** -12 * rand())
        cache.pools[r].copy_(pool.cuda())
    T = sum(news)
    q = [torch.zeros(T, share, DIM, dtype=torch.float16) for _ in range(n)]
    for x in q:
        at = torch.randint(0, DIM, (T, share, 1), generator=g)
        x.scatter_(2, at, (torch.rand(T, share, 1, generator=g) + 0.5).half())
    out = [torch.empty(T, share, DIM, dtype=torch.float16, device="cuda") for _ in range(n)]
    lse = [torch.empty(T, share, dtype=torch.float32, device="cuda") for _ in range(n)]
    qd, kw = [x.cuda() for x in q], dict(max_new=max(news), workspace=cache.attention_workspace(share), lse=lse, scale=scale)
    if tree:   # a window that the row itself fills: nothing of the context
        masks = [{t - 1 - j} for t in news for j in range(t)]
        cache.attention_tree(qd, out, batch(news), S.pack(masks, 4).cuda(), window=1, **kw)
        sees = [[m - 1 - j for j in range(t)] for m, t in zip(lens, news)]
    else:      # (the first sinks of a window of one: keys 0 and, for row x, x; the row counts one of them where they meet)
        cache.attention_sinks(qd, out, batch(news), window=1, sinks=1, **kw)
        sees = [[m - t + j for j in range(t)] for m, t in zip(lens, news)]
    assert dcc.dcc_local_check() == dcc.DCC_OK
    once = 0
    for r in range(n):
        K, _ = B.parts(pools[r][0], DIM, group, "fp16")
        for s, (m, t) in enumerate(zip(lens, news)):
            step, lo, code = B.rows_of(K, table[s, :-(-m // R.PAGE)].long(), 0, m)
            k, most = lo + step * code, torch.maximum(lo.abs(), (lo + 15 * step).abs())
            rows = slice(sum(news[:s]), sum(news[:s]) + t)
            for h in range(share):
                qq, got = q[r][rows, h].double(), lse[r][rows, h].cpu().double()
                at = torch.tensor(sees[s])
                keys = [at] if tree else [at, torch.zeros_like(at)]
                scores = [scale * (qq * k[i]).sum(-1) for i in keys]
                rounded = [scale * (qq * k[i].half().double()).sum(-1) for i in keys]
                tols = [(scale * qq.abs() * (2.0 ** -20 * most[i] + E)).sum(-1) + 9 * E * x.abs() + 24 * E
                        for i, x in zip(keys, scores)]
                if not tree:   # ln(e^a + e^b) moves by at most the larger of the two errors
                    two = at != 0
                    scores, rounded = ([torch.where(two, torch.logaddexp(*x), x[0])] for x in (scores, rounded))
                    big = torch.maximum(*tols)
                    tols = [big + 60 * E]   # sums and logarithm of two terms
                tol = 1.01 * tols[0]
                off = (got - scores[0]).abs()
                assert (off <= tol).all(), (off / tol).max().item()
                once += ((rounded[0] - scores[0]).abs() > tol).sum().item()
    # a key rounded to one number would be seen, in rows enough
    assert kind == "small" or once > n * T * share // 4
