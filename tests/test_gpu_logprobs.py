"""Log probabilities, entropy and top alternatives against 64 bits.

With e = 2^-24 and s_j = scale (x_j - m): a difference of two numbers of up to 24
bits is rounded once, its product with scale log2 e (itself rounded) once, and the
exponential is off by 2^-22 of itself; so a term of Z is off by at most
(3 e |s_j| + 2^-22) of itself, and sums of up to 2^18 terms, a few dozen to a thread, by 100 e.
ln Z inherits the terms' mean; log p adds the rounding of s, of ln Z and of their
difference; so does the entropy, whose terms carry s_j again.  The ids are exact."""
import math

import pytest
import torch

from test_gpu_kv4 import dcc  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
TD = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E = 2.0 ** -24


def call(dcc, xs, target, top=0, vocab=None, scale=1.0, ws=None, entropy=True, stream=None):
    T = xs[0].shape[0]
    f = dict(dtype=torch.float32, device="cuda")
    lp = torch.full((T,), 7.0, **f) if target is not None else None
    en = torch.full((T,), 7.0, **f) if entropy else None
    ids = torch.full((T, top), 7, dtype=torch.int32, device="cuda") if top else None
    tl = torch.full((T, top), 7.0, **f) if top else None
    ws = dcc.token_logprobs_workspace(len(xs), T, xs[0].shape[1], top) if ws is None else ws
    dcc.dcc_token_logprobs(xs, target, lp, ws, entropy=en, top_ids=ids, top_logprobs=tl, vocab=vocab, scale=scale,
                           stream=stream)
    return lp, en, ids, tl


def plain(xs, target, top, vocab, scale):
    x = torch.cat([t.double() for t in xs], 1)[:, :vocab]
    y = x * scale
    m = y.amax(-1, keepdim=True)
    log = y - m - torch.log(torch.exp(y - m).sum(-1, keepdim=True))
    p = torch.exp(log)
    spread = torch.where(p > 0, (y - m).abs(), torch.zeros_like(y))
    entropy = -torch.where(p > 0, p * log, torch.zeros_like(p)).sum(-1)
    mean = (p * spread).sum(-1)          # of |s| over the distribution
    square = (p * spread * spread).sum(-1)
    lp = torch.where(target >= 0, log.gather(1, target.long().clamp(min=0)[:, None])[:, 0], torch.zeros_like(mean)) \
        if target is not None else None
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
    base = 3 * E * mean + 2.0 ** -22 + 100 * E      # of ln Z
    far = torch.where(torch.isfinite(log), (y - m).abs(), torch.zeros_like(y))
    tol = (base + 4 * E * (math.log(x.shape[1]) + 1))[:, None] + 4 * E * far
    tol_entropy = 2 * base + 4 * E * (entropy.abs() + mean) + 3 * E * square + (2.0 ** -22 + 100 * E) * (mean + 1)
    return lp, entropy, order, log, tol, tol_entropy


def check(dcc, xs, target, top, vocab=None, scale=1.0, ws=None):
    V = vocab or len(xs) * xs[0].shape[1]
    lp, en, ids, tl = call(dcc, xs, target, top, vocab, scale, ws)
    want, entropy, order, log, tol, tol_entropy = plain(xs, target, top, V, scale)

    def near(a, b, t):
        same = (a.double() == b) | ((a.double() - b).abs() <= t)  # (infinities are equal)
        assert same.all(), ((a.double() - b).abs() / t).nan_to_num(0).max().item()
    if target is not None:
        near(lp, want, tol.gather(1, target.long().clamp(min=0)[:, None])[:, 0])
    near(en, entropy, tol_entropy)
    if top:
        assert torch.equal(ids.long(), order)
        near(tl, log.gather(1, order), tol.gather(1, order))
    return lp, en, ids, tl


def logits(g, n, T, C, dtype, loud=3.0, stride=None):
    out = []
    for _ in range(n):
        x = torch.empty(T, stride or C, dtype=TD[dtype], device="cuda")[:, :C]
        x.copy_((torch.randn(T, C, generator=g) * loud).to(TD[dtype]))
        out.append(x)
    return out


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,T,C,vocab,top", [
    (1, 1, 1, None, 1), (1, 3, 2, None, 2), (2, 1, 7, 9, 5), (8, 2, 33, 257, 64), (1, 5, 1000, 999, 20),
    (8, 1, 4001, 32001, 5), (8, 1, 16031, None, 20), (3, 7, 12345, 30000, 1), (16, 2, 8192, None, 50),
    (8, 64, 4096, 32000, 20), (2, 300, 2049, 4097, 3), (1, 1300, 777, None, 7), (4, 1217, 500, 1501, 64), (1, 2, 152064, None, 20)])
def test_rows_of_all_sizes(dcc, dtype, n, T, C, vocab, top):  # noqa: F811
    g = torch.Generator().manual_seed(n + T + C)
    xs = logits(g, n, T, C, dtype)
    V = vocab or n * C
    target = torch.randint(0, V, (T,), generator=g).to(torch.int32).cuda()
    target[::5] = -1
    check(dcc, xs, target, top, vocab)
    assert dcc.dcc_local_check() == dcc.DCC_OK


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("stride,shift", [(1001, 0), (1004, 0), (1003, 1), (1008, 3), (2000, 5)])
def test_rows_that_begin_anywhere(dcc, dtype, stride, shift):  # noqa: F811
    g = torch.Generator().manual_seed(stride)
    xs = []
    for _ in range(3):
        buf = torch.full((9 * stride + 16,), math.nan, dtype=TD[dtype], device="cuda")  # around the rows: NaN
        x = buf[shift:shift + 9 * stride].view(9, stride)[:, :1000]
        x.copy_(torch.randn(9, 1000, generator=g) * 4)
        xs.append(x)
    check(dcc, xs, torch.arange(0, 2700, 300, dtype=torch.int32, device="cuda"), 10, vocab=2950)


@pytest.mark.parametrize("T", [3, 700])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "few values", "hidden", "lowest", "zeros", "peaks"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_orders_and_masks(dcc, dtype, kind, T):  # noqa: F811
    """Ties go to the lowest id, whatever the order of the values; masked tokens do not count."""
    g = torch.Generator().manual_seed(5)
    n, C = 4, 9001
    lowest = torch.finfo(TD[dtype]).min
    x = torch.randn(T, n * C, generator=g)
    if kind == "equal":
        x = torch.full_like(x, 1.5)
    elif kind == "rising":
        x = torch.arange(n * C).float().expand(T, -1) / 5000
    elif kind == "falling":
        x = -torch.arange(n * C).float().expand(T, -1) / 5000
    elif kind == "few values":
        x = torch.randint(0, 3, x.shape, generator=g).float()
    elif kind == "hidden":      # all but a handful, in the last rank
        x[:, :-7] = -math.inf
    elif kind == "lowest":      # all of a row's the lowest number of the type, or all but one
        x = torch.full_like(x, lowest)
        x[1::2, 20000] = 3.0
    elif kind == "zeros":       # both zeros are one value
        x = torch.where(torch.rand(x.shape, generator=g) < 0.5, torch.zeros_like(x), -torch.zeros_like(x))
    else:
        x[:, 12345] = 60.0
    x = x.to(TD[dtype]).cuda()
    xs = [t.contiguous() for t in x.split(C, 1)]
    target = torch.randint(0, n * C, (T,), generator=g).to(torch.int32).cuda()
    check(dcc, xs, target, 20)


@pytest.mark.parametrize("scale", [1e-3, 0.5, 1.0, 7.5, 300.0])
def test_temperatures(dcc, scale):  # noqa: F811
    g = torch.Generator().manual_seed(2)
    xs = logits(g, 2, 40, 5000, "bf16")
    check(dcc, xs, torch.randint(0, 10000, (40,), generator=g).to(torch.int32).cuda(), 4, scale=scale)


def test_far_values(dcc):  # noqa: F811
    """Logits whose difference passes 32 bits."""
    x = torch.full((4, 3000), -3e38, device="cuda")
    x[:, 17] = 3e38
    x[1, 18] = 3e38
    x[2, 2999] = math.nan
    x[3, 5] = -math.inf
    lp, en, ids, tl = call(dcc, [x], torch.tensor([17, 17, 17, 5], dtype=torch.int32, device="cuda"), 2)
    assert lp.tolist()[0] == 0.0 and abs(lp[1].item() + math.log(2)) < 1e-6 and math.isnan(lp[2]) and lp[3] == -math.inf
    assert en[0] == 0.0 and abs(en[1].item() - math.log(2)) < 1e-6 and math.isnan(en[2]) and en[3] == 0.0
    assert ids.tolist() == [[17, 0], [17, 18], [-1, -1], [17, 0]] and tl[0, 1] == -math.inf


@pytest.mark.parametrize("T", [4, 1300])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_rows_without_a_distribution(dcc, dtype, T):  # noqa: F811
    g = torch.Generator().manual_seed(3)
    xs = logits(g, 2, T, 3001, dtype)
    xs[1][0, 3000] = math.nan
    xs[0][1, 0] = math.inf
    for x in xs:
        x[2] = -math.inf
    xs[0][3, :] = math.nan
    target = torch.full((T,), 5, dtype=torch.int32, device="cuda")
    lp, en, ids, tl = call(dcc, xs, target, 3)
    for t in (lp, en, tl):
        assert torch.isnan(t[:4]).all() and torch.isfinite(t[4:]).all()
    assert (ids[:4] == -1).all() and (ids[4:] >= 0).all()


def test_targets(dcc):  # noqa: F811
    g = torch.Generator().manual_seed(4)
    xs = logits(g, 2, 4, 100, "fp16")
    xs[0][0, 7] = -math.inf
    target = torch.tensor([7, -1, -2 ** 31, 199], dtype=torch.int32, device="cuda")
    lp = check(dcc, xs, target, 0)[0]
    assert lp[0] == -math.inf and lp[1:3].tolist() == [0.0, 0.0]
    assert dcc.dcc_local_check() == dcc.DCC_OK
    target[1] = 198
    lp = call(dcc, xs, target, vocab=198)[0]
    assert dcc.dcc_local_check() == dcc.DCC_ERR_BOUNDS
    assert torch.isnan(lp[1]) and torch.isnan(lp[3]) and lp[2] == 0.0


def test_outputs_may_be_left_out(dcc):  # noqa: F811
    g = torch.Generator().manual_seed(6)
    xs = logits(g, 2, 5, 3000, "bf16")
    target = torch.arange(5, dtype=torch.int32, device="cuda")
    lp, en, ids, tl = call(dcc, xs, target, 6)
    assert torch.equal(call(dcc, xs, target, 0, entropy=False)[0], lp)
    assert torch.equal(call(dcc, xs, None, 0)[1], en)
    _, _, i, t = call(dcc, xs, None, 6, entropy=False)
    assert torch.equal(i, ids) and torch.equal(t, tl)


def test_one_workspace_for_calls_of_all_sizes_and_a_graph(dcc):  # noqa: F811
    """Calls of other sizes in between, other streams, replays: the same bits."""
    g = torch.Generator().manual_seed(7)
    ws = dcc.token_logprobs_workspace(8, 1, 1, dcc.DCC_TOP_MAX)
    cases = []
    for n, T, C, top, dtype in ((8, 1, 16000, 20, "bf16"), (2, 9, 700, 64, "fp32"), (8, 40, 4000, 0, "fp16"), (1, 2, 50000, 5, "fp32")):
        xs = logits(g, n, T, C, dtype)
        target = torch.randint(0, n * C, (T,), generator=g).to(torch.int32).cuda()
        cases.append((xs, target, top, check(dcc, xs, target, top, ws=ws)))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for xs, target, top, want in cases + cases[::-1]:
        with torch.cuda.stream(side):
            got = call(dcc, xs, target, top, ws=ws)
        side.synchronize()
        assert all(a is None or torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [call(dcc, xs, target, top, ws=ws) for xs, target, top, _ in cases]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for got, (_, _, _, want) in zip(outs, cases):
            assert all(a is None or torch.equal(a, b) for a, b in zip(got, want))


def test_after_the_column_parallel_layer(dcc):  # noqa: F811
    """Logits as dcc_linear leaves them."""
    g = torch.Generator().manual_seed(8)
    n, T, R, K = 4, 12, 1000, 512
    w = [(torch.randn(R, K, generator=g) * K ** -0.5 * 3).bfloat16().cuda() for _ in range(n)]
    x = torch.randn(T, K, generator=g).bfloat16().cuda()
    y = [torch.empty(T, R, dtype=torch.bfloat16, device="cuda") for _ in range(n)]
    dcc.dcc_linear(w, [x] * n, y)
    check(dcc, y, torch.randint(0, 3990, (T,), generator=g).to(torch.int32).cuda(), 8, vocab=3990)


def test_rows_past_four_gigabytes(dcc):  # noqa: F811
    x = torch.empty(2, 17000, 65600, dtype=torch.float16, device="cuda")  # 2.2 GB a rank, and rows 131,200 apart below
    for r in range(2):
        for a in range(0, 17000, 1000):
            x[r, a:a + 1000] = torch.randn(1000, 65600, device="cuda")
    wide = x.view(17000, 131200)
    rows = torch.cat([torch.arange(3), torch.arange(8400, 8403), torch.arange(16990, 17000)]).cuda()
    target = torch.arange(17000, dtype=torch.int32, device="cuda")
    for xs in ([x[0], x[1]], [wide]):
        lp, en, ids, tl = call(dcc, xs, target, 3)
        want, entropy, order, log, tol, tol_entropy = plain([t[rows] for t in xs], target[rows], 3, None, 1.0)
        assert torch.equal(ids[rows].long(), order)
        assert ((lp[rows].double() - want).abs() <= tol.gather(1, target[rows].long()[:, None])[:, 0]).all()
        assert ((en[rows].double() - entropy).abs() <= tol_entropy).all()
