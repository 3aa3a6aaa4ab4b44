"""The device record of the calls without a communicator.  The record is
written from the host here (no wait is made to run out): a failure that another
call left in it changes nothing for the calls after, and is reported once."""
import ctypes
import threading

import pytest
import torch

import kv4_reference as R
from test_gpu_kv4 import batch, make_cache

pytestmark = pytest.mark.gpu
TIMEOUT_OF_RANK_3 = 1 | 3 << 8 | 3 << 16


@pytest.fixture(scope="module")
def dcc():
    from driven_collective_communication_gb300 import build
    build.build()
    from driven_collective_communication_gb300 import dcc as mod
    torch.cuda.set_device(0)
    return mod


def write_record(dcc, *words):
    """words: out of range, gave up, tag of the call that gave up last."""
    torch.cuda.synchronize()
    f = getattr(ctypes.CDLL(dcc.LIB_PATH), "_ZN8dcc_host12local_statusEv")
    f.restype = ctypes.c_void_p
    host = (ctypes.c_uint64 * len(words))(*words)
    copy = ctypes.CDLL("libcudart.so.13").cudaMemcpy
    copy.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
    assert copy(f(), host, ctypes.sizeof(host), 1) == 0


@pytest.mark.parametrize("tokens", [1, 64, 256, 700])
def test_a_layer_beside_another_calls_failure(dcc, tokens):
    g = torch.Generator().manual_seed(tokens)
    w = [torch.randn(1032, 2056, generator=g).bfloat16().cuda() for _ in range(8)]
    x = [torch.randn(tokens, 2056, generator=g).bfloat16().cuda() for _ in range(8)]
    y = [torch.empty(tokens, 1032, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    dcc.dcc_linear(w, x, y)
    assert dcc.dcc_local_check() == dcc.DCC_OK
    want = [t.clone() for t in y]
    for t in y:
        t.zero_()
    write_record(dcc, 0, TIMEOUT_OF_RANK_3, 1 << 62)
    dcc.dcc_linear(w, x, y)
    assert dcc.dcc_local_check() == dcc.DCC_ERR_TIMEOUT
    assert dcc.dcc_local_check() == dcc.DCC_OK
    assert all(torch.equal(a, b) for a, b in zip(y, want))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new", [1, 300])
def test_attention_beside_another_calls_failure(dcc, dtype, new):
    g = torch.Generator().manual_seed(new)
    cache, _, _ = make_cache(dcc, g, 8, [3000, 700], 1, 128, 64, dtype)
    q = torch.randn(2 * new, 8, 128, generator=g).to(R.TD[dtype]).cuda()
    out = [torch.empty_like(q) for _ in range(8)]
    ws = cache.attention_workspace(8)

    def run():
        cache.attention([q] * 8, out, batch([new, new]), max_new=new, workspace=ws)
    run()
    assert dcc.dcc_local_check() == dcc.DCC_OK
    want = [t.clone() for t in out]
    for t in out:
        t.zero_()
    write_record(dcc, 0, TIMEOUT_OF_RANK_3, 1 << 62)
    run()
    assert dcc.dcc_local_check() == dcc.DCC_ERR_TIMEOUT
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_the_record_is_reported_once(dcc):
    for words, code in (((2, 0, 0), dcc.DCC_ERR_BOUNDS), ((2, TIMEOUT_OF_RANK_3, 5), dcc.DCC_ERR_TIMEOUT),
                        ((0, TIMEOUT_OF_RANK_3, 5), dcc.DCC_ERR_TIMEOUT)):
        write_record(dcc, *words)
        assert dcc.dcc_local_check() == code
        assert dcc.dcc_local_check() == dcc.DCC_OK


def test_failures_of_two_streams_are_all_reported(dcc):
    """Two threads, a stream each: calls that fail, and a check after each.  No
    failure may go unreported: one thread's check finds its own unless the other
    thread's has reported something since the call."""
    cache, _, _ = make_cache(dcc, torch.Generator().manual_seed(3), 1, [70], 1, 128, 64, "bf16")
    cache.table[0, 1] = -1
    x = torch.randn(70, 1, 128).bfloat16().cuda()
    start = batch([70])
    torch.cuda.synchronize()
    reports, lost, turns = [0, 0], [], 300

    def work(me):
        stream = torch.cuda.Stream()
        for i in range(turns):
            before = reports[1 - me]
            cache.append([x], [x], start, stream=stream)
            code = dcc.dcc_local_check(stream)
            if code == dcc.DCC_ERR_BOUNDS:
                reports[me] += 1
            elif reports[1 - me] == before and done[1 - me]:
                lost.append((me, i, code))  # nobody else is left who could have taken it
        done[me] = True

    done = [False, False]
    threads = [threading.Thread(target=work, args=(t,)) for t in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not lost and sum(reports) > 0
    assert dcc.dcc_local_check() == dcc.DCC_OK
