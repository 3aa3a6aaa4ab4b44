"""Buffers of one call that overlap where it writes: refused before anything is
launched (no GPU needed).  Slices of one buffer that only interleave are not."""
import ctypes

import pytest

from test_ops_arguments import append, attend, dcc, desc, ptrs  # noqa: F401  (dcc: the fixture)

WS, BIG = 1 << 20, 1 << 40


def apart(dcc, **change):
    """A descriptor whose table, lengths and counts lie apart."""
    return desc(dcc, **{"table": 4096, "len": 8192, "refs": 12288, **change})


def read(dcc, **kw):
    return append(dcc, apart(dcc), name="dcc_kv4_read", **kw)


def test_read_into_overlapping_rows(dcc):  # noqa: F811
    bad = dcc.DCC_ERR_INVALID_ARG
    k, v = 3 << 30, 5 << 30
    row = 2 * 128 * 2  # bytes
    for kk, vv in ((ptrs(k, k), ptrs(v, 6 << 30)), (ptrs(k, 4 << 30), ptrs(v, v)),      # two ranks
                   (ptrs(k, 4 << 30), ptrs(k, 6 << 30)), (ptrs(k, 4 << 30), ptrs(v, k)),  # K on V
                   (ptrs(k, 4 << 30), ptrs(k + 3 * row, 6 << 30)),   # the last row of one, the first of the other
                   (ptrs(k + 16, 4 << 30), ptrs(k, 6 << 30))):
        assert read(dcc, k=kk, v=vv) == bad
    for shift in (16, row - 16, 3 * row + 16, 3 * 4 * row + 16, -(4 * row) + 16, -16):  # rows 4 wide apart, interleaved
        assert read(dcc, k=ptrs(k, 4 << 30), v=ptrs(k + shift, 6 << 30), stride=4 * row // 2) == bad, shift


def test_append_may_read_the_same_rows_for_all_ranks(dcc):  # noqa: F811
    # (passes the checks and stops at the device, which is not there)
    from conftest import gpu_available
    if gpu_available():
        pytest.skip("would launch")
    k = ptrs(3 << 30, 3 << 30)
    assert append(dcc, apart(dcc), k=k, v=k) == dcc.DCC_ERR_CUDA
    row = 512
    interleaved = dict(k=ptrs(3 << 30, 4 << 30), stride=4 * row // 2)
    for shift in (row, 2 * row + 16, 3 * row, -row, 16 * row):
        v = ptrs((3 << 30) + shift, (4 << 30) + shift)
        assert read(dcc, v=v, **interleaved) == dcc.DCC_ERR_CUDA, shift


@pytest.mark.parametrize("args", [dict(ws=5 << 30), dict(ws=(6 << 30) + 1024), dict(ws=1 << 30), dict(ws=3 << 30),
                                  dict(ws=4096), dict(ws=8192), dict(start=(5 << 30) + 64),
                                  dict(out=ptrs(5 << 30, 4096)), dict(out=ptrs(8192, 5 << 30)),
                                  dict(lse=ptrs(7 << 30, WS + 64))])
def test_attention(dcc, args):  # noqa: F811
    assert attend(dcc, apart(dcc), **args) == dcc.DCC_ERR_INVALID_ARG


def test_page_calls(dcc):  # noqa: F811
    bad = dcc.DCC_ERR_INVALID_ARG
    d = ctypes.byref(apart(dcc))
    n = ctypes.c_size_t()
    assert dcc.raw_call("dcc_kv4_pages_workspace", d, ctypes.byref(n)) == dcc.DCC_OK
    list_, info = 1 << 16, 1 << 17
    for on in (4096, 8192, 12288, 1 << 30, (2 << 30) + 4096):  # table, lengths, counts, pools
        assert dcc.raw_call("dcc_kv4_free", d, list_, 1, info, on, BIG, None) == bad
        assert dcc.raw_call("dcc_kv4_free", d, list_, 1, on, WS, BIG, None) == bad
        assert dcc.raw_call("dcc_kv4_free", d, on, 1, info, WS, BIG, None) == bad
        assert dcc.raw_call("dcc_kv4_fork", d, list_, on, 1, info, WS, BIG, None) == bad
        assert dcc.raw_call("dcc_kv4_fork", d, on, list_, 1, info, WS, BIG, None) == bad
        assert dcc.raw_call("dcc_kv4_reserve", d, on, info, WS, BIG, None) == bad
        assert dcc.raw_call("dcc_kv4_compact", d, 1 << 14, 1 << 15, on, info, WS, BIG, None) == bad
    assert dcc.raw_call("dcc_kv4_free", d, WS, 1, info, WS, BIG, None) == bad
    assert dcc.raw_call("dcc_kv4_free", d, list_, 1, WS + 16, WS, BIG, None) == bad


@pytest.mark.parametrize("new_table,new_refs,remap,info", [
    (8192, 1 << 15, 1 << 16, 1 << 17), (12288, 1 << 15, 1 << 16, 1 << 17), (4096 + 4, 1 << 15, 1 << 16, 1 << 17),
    (1 << 14, 4096, 1 << 16, 1 << 17), (1 << 14, 12288 + 4, 1 << 16, 1 << 17), (1 << 14, (1 << 14) + 8, 1 << 16, 1 << 17),
    (1 << 14, 1 << 15, (1 << 14) + 4, 1 << 17), (1 << 14, 1 << 15, (1 << 15) + 4, 1 << 17), (1 << 14, 1 << 15, WS, 1 << 17),
    (WS, 1 << 15, 1 << 16, 1 << 17), (1 << 14, 1 << 15, 1 << 16, (1 << 16) + 4), (1 << 14, 1 << 30, 1 << 16, 1 << 17)])
def test_compact(dcc, new_table, new_refs, remap, info):  # noqa: F811
    d = ctypes.byref(apart(dcc))
    assert dcc.raw_call("dcc_kv4_compact", d, new_table, new_refs, remap, info, WS, BIG, None) == dcc.DCC_ERR_INVALID_ARG


def test_compact_in_place_is_allowed(dcc):  # noqa: F811
    from conftest import gpu_available
    if gpu_available():
        pytest.skip("would launch")
    d = ctypes.byref(apart(dcc))
    assert dcc.raw_call("dcc_kv4_compact", d, 4096, 12288, 1 << 16, 1 << 17, WS, BIG, None) == dcc.DCC_ERR_CUDA
