"""The decoder's calls launched after one another with no host wait between
them: each kernel may start while the one before it ends, so results must be
those of the same calls with a wait after each."""
import pytest
import torch

import kv4_reference as R
from test_gpu_kv4 import batch, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dcc():
    from driven_collective_communication_gb300 import build
    build.build()
    from driven_collective_communication_gb300 import dcc as mod
    torch.cuda.set_device(0)
    return mod


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group", [(64, 32), (128, 64)])
@pytest.mark.parametrize("tokens", [16, 64, 300])
def test_prompt_attention_and_linear_layers_in_turn(dcc, dtype, dim, group, tokens):
    """Kernels that share the tensor memory of an SM, small ones beside large
    ones: attention of a prompt, a layer of few tokens, one of many."""
    g = torch.Generator().manual_seed(7)
    n, lens, news = 8, [700, 300], [130, 100]
    cache, _, _ = make_cache(dcc, g, n, lens, 1, dim, group, dtype)
    t = R.TD[dtype]
    q = [torch.randn(230, 4, dim, generator=g).to(t).cuda() for _ in range(n)]
    attn = [torch.empty_like(x) for x in q]
    w = [(torch.randn(256, 4 * dim, generator=g) * 0.05).to(t).cuda() for _ in range(n)]
    ws = cache.attention_workspace(4)
    few = [x.view(230, -1)[:tokens] if tokens <= 230 else torch.randn(tokens, 4 * dim, generator=g).to(t).cuda() for x in attn]
    y = [torch.empty(tokens, 256, dtype=t, device="cuda") for _ in range(n)]
    z = [torch.empty(230, 256, dtype=t, device="cuda") for _ in range(n)]
    rows = [x.view(230, -1) for x in attn]
    start = batch(news)

    def step(wait):
        cache.attention(q, attn, start, max_new=130, workspace=ws)
        wait()
        dcc.dcc_linear(w, few, y, act="gelu")
        wait()
        dcc.dcc_linear(w, rows, z, act="silu")
        wait()

    step(torch.cuda.synchronize)
    want = [x.clone() for x in attn + y + z]
    for x in attn + y + z:
        x.zero_()
    for _ in range(50):
        step(lambda: None)
    assert dcc.dcc_local_check() == dcc.DCC_OK
    assert all(torch.equal(a, b) for a, b in zip(attn + y + z, want))
