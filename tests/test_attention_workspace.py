"""The attention calls' workspace: one size serves them all, and plain causal
attention asks only for what its own kernels use."""
import ctypes

import pytest
import torch

from test_gpu_kv4 import batch, make_cache
from test_ops_arguments import attend, dcc, desc  # noqa: F401  (dcc: the fixture)
from test_seen_arguments import sinks, tree

# a counter per CTA; per CTA two partials and one a warp (160 CTAs of 12 warps), each 16 rows of
# 128 channels with a maximum, a sum and 4 of padding, fp32
PLAIN = 1024 + 160 * (2 + 12) * 16 * (128 + 6) * 4


def test_each_call_asks_for_what_it_uses(dcc):  # noqa: F811
    ok, bad = dcc.DCC_OK, dcc.DCC_ERR_INVALID_ARG
    assert dcc.DCC_KV4_ATTENTION_BYTES == PLAIN
    for dim in (64, 128):
        d, n = desc(dcc, head_dim=dim), ctypes.c_size_t()
        assert dcc.raw_call("dcc_kv4_attention_workspace", ctypes.byref(d), 8, ctypes.byref(n)) == ok
        for call in (attend, sinks, tree):
            assert call(dcc, d, tokens=0, ws_bytes=n.value) == ok
        assert attend(dcc, d, tokens=0, ws_bytes=PLAIN) == ok
        assert attend(dcc, d, tokens=0, ws_bytes=PLAIN - 1) == bad
        # causal rows without sinks are plain attention
        for args in (dict(sinks=0), dict(window=0), dict(window=1 << 30)):
            assert sinks(dcc, d, tokens=0, ws_bytes=PLAIN, **args) == ok
        assert n.value > PLAIN
        for call in (sinks, tree):
            assert call(dcc, d, tokens=0, ws_bytes=n.value - 1) == bad


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,dim,group", [("bf16", 128, 64), ("fp16", 64, 32)])
@pytest.mark.parametrize("lens,news,share,window", [
    ([900, 70], [1, 1], 8, 0), ([20000, 3000, 5], [2, 1, 5], 4, 0), ([700, 4000], [1, 3], 8, 100), ([1500, 300], [700, 300], 2, 0)])
def test_plain_attention_in_its_own_size(dcc, dtype, dim, group, lens, news, share, window):  # noqa: F811
    """The same bits, and nothing behind it is touched."""
    g = torch.Generator().manual_seed(sum(lens))
    cache, _, _ = make_cache(dcc, g, 2, lens, 1, dim, group, dtype)
    q = [torch.randn(sum(news), share, dim, generator=g).to(cache.torch_dtype).cuda() for _ in range(2)]
    large = cache.attention_workspace(share)
    buf = torch.zeros(PLAIN + 4096, dtype=torch.uint8, device="cuda")
    buf[PLAIN:] = 77
    got = []
    for ws in (large, buf[:PLAIN]):
        out = [torch.empty_like(x) for x in q]
        cache.attention(q, out, batch(news), max(news), ws, window=window)
        got.append(out)
    assert dcc.dcc_local_check() == dcc.DCC_OK
    assert all(torch.equal(a, b) for a, b in zip(*got)) and (buf[PLAIN:] == 77).all()
