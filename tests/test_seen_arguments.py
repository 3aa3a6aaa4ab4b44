"""Refusals of the calls for drafted tokens, windows with sinks and log
probabilities: every one returns before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from test_ops_arguments import dcc, desc, ptrs  # noqa: F401  (dcc: the fixture)
from test_ops_binding import OnDevice, bf16, dev  # noqa: F401
from test_ops_overlaps import apart

WS, BIG = 1 << 20, 1 << 40


def tree(dcc, d, layer=0, q=None, out=None, lse=None, q_heads=8, tokens=4, q_stride=1024, start=1024, max_new=2,
         mask=2048, words=1, scale=0.1, window=0, sinks=0, ws=WS, ws_bytes=BIG):
    q = ptrs(3 << 30, 4 << 30) if q is None else q
    out = ptrs(5 << 30, 6 << 30) if out is None else out
    return dcc.raw_call("dcc_kv4_attention_tree", ctypes.byref(d) if d is not None else None, layer, q, out, lse, q_heads,
                        tokens, q_stride, start, max_new, mask, words, scale, window, sinks, ws, ws_bytes, None)


def sinks(dcc, d, layer=0, q=None, out=None, lse=None, q_heads=8, tokens=4, q_stride=1024, start=1024, max_new=2,
          scale=0.1, window=100, sinks=4, ws=WS, ws_bytes=BIG):
    q = ptrs(3 << 30, 4 << 30) if q is None else q
    out = ptrs(5 << 30, 6 << 30) if out is None else out
    return dcc.raw_call("dcc_kv4_attention_sinks", ctypes.byref(d) if d is not None else None, layer, q, out, lse, q_heads,
                        tokens, q_stride, start, max_new, scale, window, sinks, ws, ws_bytes, None)


@pytest.mark.parametrize("change,code", [
    (dict(n_ranks=0), "INVALID_ARG"), (dict(head_dim=96), "UNSUPPORTED"), (dict(group=16), "UNSUPPORTED"),
    (dict(dtype=1), "UNSUPPORTED"), (dict(table=None), "INVALID_ARG"), (dict(len=129), "MISALIGNED"),
    (dict(pool=ptrs(1 << 30, (2 << 30) + 8)), "MISALIGNED")])
def test_cache_descriptors(dcc, change, code):  # noqa: F811
    want, d = getattr(dcc, "DCC_ERR_" + code), desc(dcc, **change)
    assert tree(dcc, d) == want and sinks(dcc, d) == want
    assert dcc.raw_call("dcc_kv4_keep", ctypes.byref(d), 64, 64, 4, 64, None, WS, BIG, None) == want


def test_null_descriptor(dcc):  # noqa: F811
    bad = dcc.DCC_ERR_INVALID_ARG
    assert tree(dcc, None) == bad and sinks(dcc, None) == bad
    assert dcc.raw_call("dcc_kv4_keep", None, 64, 64, 4, 64, None, WS, BIG, None) == bad


@pytest.mark.parametrize("args,code", [
    (dict(layer=2), "INVALID_ARG"), (dict(q_heads=7), "INVALID_ARG"), (dict(q_heads=258), "INVALID_ARG"),
    (dict(max_new=0), "INVALID_ARG"), (dict(window=-1), "INVALID_ARG"), (dict(sinks=-1), "INVALID_ARG"),
    (dict(scale=float("nan")), "INVALID_ARG"), (dict(ws=None), "INVALID_ARG"), (dict(ws=WS + 4), "MISALIGNED"),
    (dict(ws_bytes=1 << 20), "INVALID_ARG"), (dict(start=None), "INVALID_ARG"), (dict(start=3), "MISALIGNED"),
    (dict(q_stride=1023), "MISALIGNED"), (dict(q_stride=512), "INVALID_ARG"), (dict(out=ptrs(5 << 30, None)), "INVALID_ARG"),
    (dict(out=ptrs(3 << 30, 6 << 30)), "INVALID_ARG"), (dict(out=ptrs(1 << 30, 6 << 30)), "INVALID_ARG"),
    (dict(lse=ptrs(7 << 30, 7 << 30)), "INVALID_ARG"), (dict(tokens=1 << 31), "INVALID_ARG")])
def test_attention(dcc, args, code):  # noqa: F811
    want = getattr(dcc, "DCC_ERR_" + code)
    assert tree(dcc, desc(dcc), **args) == want and sinks(dcc, desc(dcc), **args) == want


@pytest.mark.parametrize("args,code", [
    (dict(mask=None), "INVALID_ARG"), (dict(mask=2050), "MISALIGNED"), (dict(words=0), "INVALID_ARG"),
    (dict(words=33), "INVALID_ARG"), (dict(words=-1), "INVALID_ARG"), (dict(tokens=40, max_new=33), "INVALID_ARG"),
    (dict(tokens=33, max_new=1000), "INVALID_ARG"), (dict(tokens=2000, max_new=2000, words=32), "INVALID_ARG")])
def test_masks(dcc, args, code):  # noqa: F811
    assert tree(dcc, desc(dcc), **args) == getattr(dcc, "DCC_ERR_" + code)


def test_no_tokens_are_a_no_op(dcc):  # noqa: F811
    assert tree(dcc, desc(dcc), tokens=0) == dcc.DCC_OK and sinks(dcc, desc(dcc), tokens=0) == dcc.DCC_OK


@pytest.mark.parametrize("args", [dict(ws=5 << 30), dict(ws=1 << 30), dict(ws=3 << 30), dict(start=(5 << 30) + 64),
                                  dict(out=ptrs(5 << 30, 4096)), dict(lse=ptrs(7 << 30, WS + 64))])
def test_attention_overlaps(dcc, args):  # noqa: F811
    d = apart(dcc)
    assert tree(dcc, d, **args) == dcc.DCC_ERR_INVALID_ARG and sinks(dcc, d, **args) == dcc.DCC_ERR_INVALID_ARG
    assert tree(dcc, d, mask=(5 << 30) + 16) == dcc.DCC_ERR_INVALID_ARG      # the mask in an output
    assert tree(dcc, d, mask=WS + 4096) == dcc.DCC_ERR_INVALID_ARG           # and in the workspace


def test_keep(dcc):  # noqa: F811
    bad, mis, call = dcc.DCC_ERR_INVALID_ARG, dcc.DCC_ERR_MISALIGNED, dcc.raw_call
    d, n = ctypes.byref(apart(dcc)), ctypes.c_size_t()
    assert call("dcc_kv4_pages_workspace", d, ctypes.byref(n)) == dcc.DCC_OK
    start, path, count, info = 1 << 16, 1 << 17, 1 << 18, 1 << 19
    for i in range(3):
        a = [start, path, count]
        a[i] = None
        assert call("dcc_kv4_keep", d, a[0], a[1], 4, a[2], info, WS, n.value, None) == bad
        a[i] = [start, path, count][i] + 2
        assert call("dcc_kv4_keep", d, a[0], a[1], 4, a[2], info, WS, n.value, None) == mis
        for on in (4096, 8192, 12288, 1 << 30, (2 << 30) + 4096, WS + 16, info):  # table, lengths, counts, pools, workspace, info
            a[i] = on
            assert call("dcc_kv4_keep", d, a[0], a[1], 4, a[2], info, WS, BIG, None) == bad
    assert call("dcc_kv4_keep", d, start, path, 4, count, info + 2, WS, BIG, None) == mis
    assert call("dcc_kv4_keep", d, start, path, 4, count, info, WS, n.value - 4, None) == bad
    assert call("dcc_kv4_keep", d, start, path, 4, count, info, None, BIG, None) == bad
    assert call("dcc_kv4_keep", d, start, path, 4, count, info, WS + 4, BIG, None) == mis
    assert call("dcc_kv4_keep", d, start, path, 1 << 27, count, info, WS, BIG, None) == bad
    assert call("dcc_kv4_keep", d, start, path, 4, count, 8192, WS, BIG, None) == bad
    assert call("dcc_kv4_keep", ctypes.byref(desc(dcc, refs=None)), start, path, 4, count, info, WS, BIG, None) == bad


def lp(dcc, n=2, x=None, tokens=4, columns=100, stride=100, vocab=200, target=1 << 16, scale=1.0, top=2, logprob=1 << 17,
       entropy=1 << 18, ids=1 << 19, tops=3 << 18, ws=WS, ws_bytes=BIG, t=1):
    x = ptrs(1 << 30, 2 << 30) if x is None else x
    return dcc.raw_call("dcc_token_logprobs", n, x, tokens, columns, stride, vocab, target, scale, top, logprob, entropy, ids,
                        tops, ws, ws_bytes, t, None)


@pytest.mark.parametrize("args,code", [
    (dict(n=0), "INVALID_ARG"), (dict(n=17), "INVALID_ARG"), (dict(columns=0), "INVALID_ARG"), (dict(top=-1), "INVALID_ARG"),
    (dict(top=65), "INVALID_ARG"), (dict(t=0), "UNSUPPORTED"), (dict(t=9), "UNSUPPORTED"), (dict(scale=0.0), "INVALID_ARG"),
    (dict(scale=-1.0), "INVALID_ARG"), (dict(scale=float("nan")), "INVALID_ARG"), (dict(scale=float("inf")), "INVALID_ARG"),
    (dict(vocab=0), "INVALID_ARG"), (dict(vocab=201), "INVALID_ARG"), (dict(vocab=1), "INVALID_ARG"),  # fewer than top
    (dict(stride=99), "INVALID_ARG"), (dict(tokens=1 << 25), "INVALID_ARG"), (dict(columns=1 << 30, stride=1 << 30), "INVALID_ARG"),
    (dict(target=None), "INVALID_ARG"), (dict(logprob=None), "INVALID_ARG"), (dict(ids=None), "INVALID_ARG"),
    (dict(tops=None), "INVALID_ARG"), (dict(top=0), "INVALID_ARG"),
    (dict(top=0, ids=None, tops=None, target=None, logprob=None, entropy=None), "INVALID_ARG"),
    (dict(x=ptrs(1 << 30, None)), "INVALID_ARG"), (dict(x=ptrs(1 << 30, (2 << 30) + 2)), "MISALIGNED"),
    (dict(x=ptrs(1 << 30, (2 << 30) + 1), t=3), "MISALIGNED"), (dict(target=(1 << 16) + 2), "MISALIGNED"),
    (dict(entropy=(1 << 18) + 1), "MISALIGNED"), (dict(ws=WS + 8), "MISALIGNED"), (dict(ws=None), "INVALID_ARG"),
    (dict(ws_bytes=100), "INVALID_ARG"), (dict(entropy=1 << 17), "INVALID_ARG"), (dict(tops=(1 << 19) + 4), "INVALID_ARG"),
    (dict(ids=(1 << 30) + 64), "INVALID_ARG"), (dict(logprob=(2 << 30) + 1596), "INVALID_ARG"), (dict(ws=1 << 30), "INVALID_ARG"),
    (dict(target=1 << 17), "INVALID_ARG"), (dict(entropy=WS + 128), "INVALID_ARG")])
def test_logprobs(dcc, args, code):  # noqa: F811
    assert lp(dcc, **args) == getattr(dcc, "DCC_ERR_" + code)


def test_logprobs_of_nothing(dcc):  # noqa: F811
    assert lp(dcc, tokens=0) == dcc.DCC_OK
    n = ctypes.c_size_t()
    for args in ((0, 1, 1, 1), (17, 1, 1, 1), (1, 1, 0, 1), (1, 1, 1, 65), (1, 1, 1, -1)):
        assert dcc.raw_call("dcc_token_logprobs_workspace", *args, ctypes.byref(n)) == dcc.DCC_ERR_INVALID_ARG
    assert dcc.raw_call("dcc_token_logprobs_workspace", 1, 1, 1, 1, None) == dcc.DCC_ERR_INVALID_ARG


def test_binding(dcc):  # noqa: F811
    """Shapes and types that the binding refuses by itself."""
    x = [bf16(4, 8)] * 2
    i, f = dev(torch.zeros(4, dtype=torch.int32)), dev(torch.zeros(4))
    ws = dev(torch.zeros(1 << 20, dtype=torch.uint8))
    for bad in (dict(target=f), dict(target=i[:3]), dict(logprob=i), dict(entropy=dev(torch.zeros(8))[::2]),
                dict(top_ids=i), dict(top_ids=dev(torch.zeros(4, 2, dtype=torch.int32)), top_logprobs=f),
                dict(logits=[bf16(4, 8, 2)] * 2)):
        a = dict(logits=x, target=i, logprob=f, workspace=ws)
        a.update(bad)
        with pytest.raises(ValueError):
            dcc.dcc_token_logprobs(**a)
