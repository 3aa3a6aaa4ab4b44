"""The column-parallel linear layer against a 64-bit form.

With u the type's unit roundoff and e = 2^-23: a sum of k exact products plus
the bias in fp32, in any order and with truncating adds, is off by at most
g = (k + 2) e sum|w x| + e |bias|; every activation's slope is at most 1.13 and
its evaluation adds at most 32 e (|z| + 1); the residual adds e; one rounding:
  |y - exact| <= 1.13 g + 32 e (|z| + 1) + e |y| + u |y|  (+ the smallest subnormal)
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
TD = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
E = 2.0 ** -23


@pytest.fixture(scope="module")
def dcc():
    from driven_collective_communication_gb300 import build
    build.build()
    from driven_collective_communication_gb300 import dcc as mod
    torch.cuda.set_device(0)
    return mod


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def check(dcc, n, tokens, rows, k, dtype, act="none", bias=True, residual=False, in_place=False, shared_x=False,
          stream=None, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + tokens + 3 * rows + 7 * k)
    t = TD[dtype]

    def rand(*shape, scale=1.0):
        return (scale * torch.randn(*shape, device="cuda", generator=g)).to(t)
    w = [rand(rows, k, scale=k ** -0.5) for _ in range(n)]
    x = [rand(tokens, k)] * n if shared_x else [rand(tokens, k) for _ in range(n)]
    b = [rand(rows) for _ in range(n)] if bias else None
    res = [rand(tokens, rows) for _ in range(n)] if residual else None
    kept = [r.clone() for r in res] if residual else None
    y = res if in_place else [torch.full((tokens, rows), math.nan, dtype=t, device="cuda") for _ in range(n)]
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    dcc.dcc_linear(w, x, y, bias=b, residual=res, act=act, stream=stream)
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    assert dcc.dcc_local_check(stream) == dcc.DCC_OK
    for r in range(n):
        wd, xd = w[r].double(), x[r].double()
        z = xd @ wd.T
        g_err = (k + 2) * E * (xd.abs() @ wd.abs().T)
        if bias:
            z = z + b[r].double()
            g_err = g_err + E * b[r].double().abs()
        want = act64(z, act)
        if residual:
            want = want + kept[r].double()
        tol = 1.13 * g_err + 32 * E * (z.abs() + 1) + (E + U[dtype]) * want.abs() + 2.0 ** -25
        err = (y[r].double() - want).abs()
        assert (err <= tol).all(), (r, (err / tol).max())


ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,tokens,rows,k", [
    (1, 1, 8, 8), (1, 1, 1024, 4096), (8, 1, 136, 1000), (2, 2, 264, 72), (3, 7, 24, 520), (1, 8, 512, 64),
    (4, 9, 104, 2048), (2, 16, 8, 1024), (1, 17, 1000, 136), (8, 33, 64, 264), (1, 64, 136, 8), (2, 100, 520, 328),
    (1, 128, 128, 128), (1, 129, 264, 192), (2, 200, 1032, 64), (1, 255, 256, 1016), (1, 257, 512, 512),
    (2, 300, 72, 2056), (1, 513, 776, 96)])
def test_shapes(dcc, dtype, n, tokens, rows, k):
    i = tokens + rows // 8 + k // 8
    check(dcc, n, tokens, rows, k, dtype, act=ACTS[i % 5], bias=i % 3 != 0, residual=i % 2 == 0, in_place=i % 4 == 0)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("tokens", [1, 5, 40, 300])
def test_activations_with_every_epilogue(dcc, act, tokens):
    for bias in (False, True):
        for residual in (False, True):
            check(dcc, 2, tokens, 264, 200, "bf16", act, bias, residual)
            check(dcc, 2, tokens, 264, 200, "fp16", act, bias, residual, in_place=residual)


@pytest.mark.parametrize("tokens", [1, 3, 16, 64, 256, 700])
def test_one_x_for_all_ranks(dcc, tokens):
    check(dcc, 8, tokens, 128, 512, "bf16", "silu", shared_x=True)


@pytest.mark.parametrize("tokens", [1, 12, 150])
def test_integers_are_exact(dcc, tokens):
    g = torch.Generator().manual_seed(tokens)
    w = torch.randint(-3, 4, (264, 1016), generator=g).bfloat16().cuda()
    x = torch.randint(-2, 3, (tokens, 1016), generator=g).bfloat16().cuda()
    y = torch.empty(tokens, 264, dtype=torch.bfloat16, device="cuda")
    dcc.dcc_linear([w], [x], [y])
    assert torch.equal(y, (x.double() @ w.double().T).to(torch.float32).bfloat16())


@pytest.mark.parametrize("tokens", [2, 80, 400])
def test_non_finite_inputs_stay_in_their_row_and_column(dcc, tokens):
    """An infinity or NaN in x reaches its token only, one in a weight row its
    output column only; the padding of a tile adds nothing."""
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(136, 72, device="cuda", generator=g).bfloat16()
    x = torch.randn(tokens, 72, device="cuda", generator=g).bfloat16()
    x[1, 71] = math.inf
    w[7, 0] = math.nan
    y = torch.empty(tokens, 136, dtype=torch.bfloat16, device="cuda")
    dcc.dcc_linear([w], [x], [y])
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[1] = True
    want[:, 7] = True
    assert torch.equal(bad, want)


def test_on_another_stream(dcc):
    for tokens in (1, 30, 200):
        check(dcc, 2, tokens, 264, 328, "bf16", "gelu", stream=torch.cuda.Stream())


def test_extreme_activation_arguments(dcc):
    """exp overflows inside SILU, tanh and erf saturate: no NaN."""
    z = torch.tensor([-300.0, -90.0, -20.0, -1e-3, 0.0, 1e-3, 20.0, 90.0, 300.0, 1e4, -1e4, 3e4, 5.0, -5.0, 1.0, -1.0])
    w = torch.zeros(16, 8, dtype=torch.bfloat16, device="cuda")
    b = z.bfloat16().cuda()
    for tokens in (1, 64, 300):
        x = torch.zeros(tokens, 8, dtype=torch.bfloat16, device="cuda")
        y = torch.empty(tokens, 16, dtype=torch.bfloat16, device="cuda")
        for act in ACTS:
            dcc.dcc_linear([w], [x], [y], bias=[b], act=act)
            want = act64(b.double(), act).expand(tokens, 16)
            tol = 32 * E * (b.double().abs() + 1) + U["bf16"] * want.abs()
            assert ((y.double() - want).abs() <= tol).all(), (act, tokens)
