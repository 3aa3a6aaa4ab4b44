"""Refusals of the calls around the cache and of the linear layer: every one
returns before anything is launched (no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def dcc():
    from driven_collective_communication_gb300 import build
    build.build()
    from driven_collective_communication_gb300 import dcc as mod
    return mod


VP = ctypes.c_void_p


def ptrs(*xs):
    return (VP * len(xs))(*xs)


def desc(dcc, **change):
    f = dict(n_ranks=2, layers=2, pages=8, seqs=3, max_pages=4, kv_heads=2, head_dim=128, group=64, dtype=dcc.DCC_BF16)
    pool, table, length, refs = change.pop("pool", ptrs(1 << 30, 2 << 30)), change.pop("table", 64), \
        change.pop("len", 128), change.pop("refs", 256)
    f.update(change)
    return dcc.dcc_kv4_t(pool, table, length, refs, *[f[k] for k in (
        "n_ranks", "layers", "pages", "seqs", "max_pages", "kv_heads", "head_dim", "group", "dtype")])


def append(dcc, d, layer=0, k=None, v=None, tokens=4, stride=256, start=1024, name="dcc_kv4_append"):
    k = ptrs(3 << 30, 4 << 30) if k is None else k
    v = ptrs(5 << 30, 6 << 30) if v is None else v
    return dcc.raw_call(name, ctypes.byref(d) if d is not None else None, layer, k, v, tokens, stride, start, None)


@pytest.mark.parametrize("change,code", [
    (dict(n_ranks=0), "INVALID_ARG"), (dict(n_ranks=17), "INVALID_ARG"), (dict(layers=0), "INVALID_ARG"),
    (dict(pages=0), "INVALID_ARG"), (dict(seqs=0), "INVALID_ARG"), (dict(max_pages=0), "INVALID_ARG"),
    (dict(max_pages=1 << 25), "INVALID_ARG"), (dict(pages=(1 << 28) + 1), "INVALID_ARG"),
    (dict(kv_heads=0), "INVALID_ARG"), (dict(head_dim=96), "UNSUPPORTED"), (dict(head_dim=256), "UNSUPPORTED"),
    (dict(group=16), "UNSUPPORTED"), (dict(group=128), "UNSUPPORTED"), (dict(dtype=1), "UNSUPPORTED"),
    (dict(dtype=0), "UNSUPPORTED"), (dict(dtype=9), "UNSUPPORTED"), (dict(table=None), "INVALID_ARG"),
    (dict(len=None), "INVALID_ARG"), (dict(table=66), "MISALIGNED"), (dict(len=129), "MISALIGNED"),
    (dict(pool=ptrs(1 << 30, None)), "INVALID_ARG"), (dict(pool=ptrs(1 << 30, (2 << 30) + 8)), "MISALIGNED"),
    (dict(pool=ptrs(1 << 30, (1 << 30) + 9216)), "INVALID_ARG")])
def test_cache_descriptors(dcc, change, code):
    want = getattr(dcc, "DCC_ERR_" + code)
    d = desc(dcc, **change)
    assert append(dcc, d) == want
    assert append(dcc, d, name="dcc_kv4_read") == want
    assert attend(dcc, d) == want
    ws = (VP(1 << 20), 1 << 30)
    if change.get("seqs") != 0:
        assert dcc.raw_call("dcc_kv4_free", ctypes.byref(d), 64, 1, None, *ws, None) == want
        assert dcc.raw_call("dcc_kv4_fork", ctypes.byref(d), 64, 64, 1, None, *ws, None) == want
        assert dcc.raw_call("dcc_kv4_reserve", ctypes.byref(d), 64, None, *ws, None) == want
        assert dcc.raw_call("dcc_kv4_compact", ctypes.byref(d), 64, 64, 64, None, *ws, None) == want
        assert dcc.raw_call("dcc_kv4_copy", ctypes.byref(d), 64, 64, 1, None) == want


def test_null_descriptor(dcc):
    bad = dcc.DCC_ERR_INVALID_ARG
    assert append(dcc, None) == bad and attend(dcc, None) == bad
    n = ctypes.c_size_t()
    for name, args in (("dcc_kv4_free", (None, 64, 1, None, 64, 64, None)), ("dcc_kv4_copy", (None, 64, 64, 1, None)),
                       ("dcc_kv4_fork", (None, 64, 64, 1, None, 64, 64, None)),
                       ("dcc_kv4_reserve", (None, 64, None, 64, 64, None)),
                       ("dcc_kv4_compact", (None, 64, 64, 64, None, 64, 64, None)),
                       ("dcc_kv4_pages_workspace", (None, ctypes.byref(n))),
                       ("dcc_kv4_attention_workspace", (None, 8, ctypes.byref(n))),
                       ("dcc_kv4_block_bytes", (128, 64, None))):
        assert dcc.raw_call(name, *args) == bad, name


def test_block_bytes(dcc):
    assert dcc.dcc_kv4_block_bytes(128, 64) == 9216
    assert dcc.dcc_kv4_block_bytes(64, 32) == 5120
    with pytest.raises(dcc.DccError):
        dcc.dcc_kv4_block_bytes(80, 32)


@pytest.mark.parametrize("args,code", [
    (dict(layer=-1), "INVALID_ARG"), (dict(layer=2), "INVALID_ARG"), (dict(start=None), "INVALID_ARG"),
    (dict(start=1026), "MISALIGNED"), (dict(stride=255), "INVALID_ARG"), (dict(stride=260), "MISALIGNED"),
    (dict(stride=128), "INVALID_ARG"), (dict(tokens=1 << 31), "INVALID_ARG"),
    (dict(k=ptrs(3 << 30, None)), "INVALID_ARG"), (dict(v=ptrs((5 << 30) + 8, 6 << 30)), "MISALIGNED"),
    (dict(k=ptrs((1 << 30) + 64, 4 << 30)), "INVALID_ARG")])
def test_rows(dcc, args, code):
    want = getattr(dcc, "DCC_ERR_" + code)
    assert append(dcc, desc(dcc), **args) == want
    assert append(dcc, desc(dcc), name="dcc_kv4_read", **args) == want


def attend(dcc, d, layer=0, q=None, out=None, lse=None, q_heads=8, tokens=4, q_stride=1024, start=1024, max_new=1,
           scale=0.1, window=0, ws=1 << 20, ws_bytes=1 << 40):
    q = ptrs(3 << 30, 4 << 30) if q is None else q
    out = ptrs(5 << 30, 6 << 30) if out is None else out
    return dcc.raw_call("dcc_kv4_attention", ctypes.byref(d) if d is not None else None, layer, q, out, lse, q_heads,
                        tokens, q_stride, start, max_new, scale, window, ws, ws_bytes, None)


@pytest.mark.parametrize("args,code", [
    (dict(layer=2), "INVALID_ARG"), (dict(q_heads=7), "INVALID_ARG"), (dict(q_heads=0), "INVALID_ARG"),
    (dict(q_heads=258), "INVALID_ARG"), (dict(max_new=0), "INVALID_ARG"), (dict(window=-1), "INVALID_ARG"),
    (dict(scale=float("nan")), "INVALID_ARG"), (dict(scale=float("inf")), "INVALID_ARG"),
    (dict(ws=None), "INVALID_ARG"), (dict(ws=(1 << 20) + 4), "MISALIGNED"), (dict(ws_bytes=8), "INVALID_ARG"),
    (dict(start=None), "INVALID_ARG"), (dict(start=3), "MISALIGNED"), (dict(q_stride=1023), "MISALIGNED"),
    (dict(q_stride=512), "INVALID_ARG"), (dict(out=ptrs(5 << 30, None)), "INVALID_ARG"),
    (dict(out=ptrs((5 << 30) + 2, 6 << 30)), "MISALIGNED"), (dict(out=ptrs(3 << 30, 6 << 30)), "INVALID_ARG"),
    (dict(out=ptrs(5 << 30, 5 << 30)), "INVALID_ARG"), (dict(out=ptrs(1 << 30, 6 << 30)), "INVALID_ARG"),
    (dict(lse=ptrs(7 << 30, None)), "INVALID_ARG"), (dict(lse=ptrs((7 << 30) + 2, 8 << 30)), "MISALIGNED"),
    (dict(lse=ptrs(7 << 30, 5 << 30)), "INVALID_ARG"), (dict(lse=ptrs(7 << 30, 7 << 30)), "INVALID_ARG")])
def test_attention(dcc, args, code):
    assert attend(dcc, desc(dcc), **args) == getattr(dcc, "DCC_ERR_" + code)


def test_page_calls(dcc):
    bad, mis = dcc.DCC_ERR_INVALID_ARG, dcc.DCC_ERR_MISALIGNED
    d = ctypes.byref(desc(dcc))
    n = ctypes.c_size_t()
    assert dcc.raw_call("dcc_kv4_pages_workspace", d, ctypes.byref(n)) == dcc.DCC_OK
    ok, ws = n.value, 1 << 20
    call = dcc.raw_call
    assert call("dcc_kv4_free", d, 64, 4, None, ws, ok, None) == bad        # more than there are sequences
    assert call("dcc_kv4_free", d, None, 1, None, ws, ok, None) == bad
    assert call("dcc_kv4_free", d, 64, 1, None, ws, ok - 4, None) == bad
    assert call("dcc_kv4_free", d, 64, 1, None, None, ok, None) == bad
    assert call("dcc_kv4_free", d, 64, 1, None, ws + 4, ok, None) == mis
    assert call("dcc_kv4_free", d, 65, 1, None, ws, ok, None) == mis
    assert call("dcc_kv4_free", d, 64, 1, 66, ws, ok, None) == mis
    assert call("dcc_kv4_fork", d, None, 64, 1, None, ws, ok, None) == bad
    assert call("dcc_kv4_fork", d, 64, None, 1, None, ws, ok, None) == bad
    assert call("dcc_kv4_reserve", d, None, None, ws, ok, None) == bad
    assert call("dcc_kv4_copy", d, 64, None, 1, None) == bad
    assert call("dcc_kv4_copy", d, 64, 64, 9, None) == bad
    assert call("dcc_kv4_copy", d, 62, 64, 1, None) == mis
    for i in range(3):
        out = [64, 64, 64]
        out[i] = None
        assert call("dcc_kv4_compact", d, *out, None, ws, ok, None) == bad
    no_refs = ctypes.byref(desc(dcc, refs=None))
    assert call("dcc_kv4_free", no_refs, 64, 1, None, ws, ok, None) == bad
    assert call("dcc_kv4_compact", no_refs, 64, 64, 64, None, ws, ok, None) == bad


def linear(dcc, n=2, w=None, x=None, b=None, res=None, y=None, tokens=4, rows=64, k=128, act=0, t=3):
    w = ptrs(1 << 30, 2 << 30) if w is None else w
    x = ptrs(3 << 30, 3 << 30) if x is None else x
    y = ptrs(5 << 30, 6 << 30) if y is None else y
    return dcc.raw_call("dcc_linear", n, w, x, b, res, y, tokens, rows, k, act, t, None)


@pytest.mark.parametrize("args,code", [
    (dict(n=0), "INVALID_ARG"), (dict(n=17), "INVALID_ARG"), (dict(act=-1), "INVALID_ARG"), (dict(act=5), "INVALID_ARG"),
    (dict(t=1), "UNSUPPORTED"), (dict(t=0), "UNSUPPORTED"), (dict(rows=60), "UNSUPPORTED"), (dict(k=100), "UNSUPPORTED"),
    (dict(k=0), "INVALID_ARG"), (dict(tokens=1 << 27), "INVALID_ARG"), (dict(rows=1 << 27), "INVALID_ARG"),
    (dict(w=ptrs(1 << 30, None)), "INVALID_ARG"), (dict(x=ptrs((3 << 30) + 8, 3 << 30)), "MISALIGNED"),
    (dict(b=ptrs(7 << 30, (8 << 30) + 2)), "MISALIGNED"), (dict(b=ptrs(7 << 30, None)), "INVALID_ARG"),
    (dict(res=ptrs(7 << 30, None)), "INVALID_ARG"), (dict(y=ptrs(5 << 30, 5 << 30)), "INVALID_ARG"),
    (dict(y=ptrs(1 << 30, 6 << 30)), "INVALID_ARG"), (dict(y=ptrs(5 << 30, 3 << 30)), "INVALID_ARG"),
    (dict(b=ptrs(5 << 30, 8 << 30)), "INVALID_ARG"), (dict(res=ptrs(6 << 30, 5 << 30)), "INVALID_ARG"),
    (dict(res=ptrs((5 << 30) + 16, 6 << 30)), "INVALID_ARG")])
def test_linear(dcc, args, code):
    assert linear(dcc, **args) == getattr(dcc, "DCC_ERR_" + code)


def test_linear_of_nothing_is_a_no_op(dcc):
    assert linear(dcc, tokens=0) == dcc.DCC_OK
    assert linear(dcc, rows=0) == dcc.DCC_OK
