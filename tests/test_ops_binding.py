"""Refusals of the binding's own checks (shapes, strides, types, devices) of the
calls around the cache and of the linear layer: each raises before the library
is called, so host tensors that claim to be on a device stand in (no GPU
needed)."""
import pytest
import torch


@pytest.fixture(scope="module")
def dcc():
    from driven_collective_communication_gb300 import build
    build.build()
    from driven_collective_communication_gb300 import dcc as mod
    return mod


class OnDevice(torch.Tensor):
    """A host tensor that says it is on a CUDA device."""
    is_cuda = True


def dev(t):
    return t.as_subclass(OnDevice)


def bf16(*shape):
    return dev(torch.zeros(*shape, dtype=torch.bfloat16))


@pytest.mark.parametrize("step", [2, 3, 8])
def test_a_strided_vector_is_no_dense_row(dcc, step):
    whole = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="not dense"):
        dcc.Ranks([dev(whole[::step])])
    with pytest.raises(ValueError, match="not dense"):
        dcc.Ranks([dev(torch.zeros(16, step, dtype=torch.bfloat16)[:, 1])] * 2)
    dcc.Ranks([dev(whole[::step][:1])])  # one element has no stride
    assert dcc.Ranks([dev(whole[step:])]).dense


def test_a_broadcast_vector_is_no_dense_row(dcc):
    with pytest.raises(ValueError, match="not dense"):
        dcc.Ranks([dev(torch.zeros(1, dtype=torch.bfloat16).expand(16))])


def test_ranks(dcc):
    with pytest.raises(ValueError, match="CUDA"):
        dcc.Ranks([torch.zeros(4, 8)])
    for other in (bf16(4, 16), dev(torch.zeros(4, 8)), dev(torch.zeros(4, 16, dtype=torch.bfloat16)[:, :8])):
        with pytest.raises(ValueError, match="differ"):
            dcc.Ranks([bf16(4, 8), other])
    with pytest.raises(ValueError, match="not dense"):
        dcc.Ranks([dev(torch.zeros(8, 4, dtype=torch.bfloat16).T)])
    r = dcc.Ranks([dev(torch.zeros(4, 32, dtype=torch.bfloat16)[:, 8:16])])
    assert r.stride == 32 and not r.dense and r.shape == (4, 8)


def test_linear(dcc):
    w, x, y, b = [bf16(16, 8)], [bf16(4, 8)], [bf16(4, 16)], [bf16(16)]
    strided = dev(torch.zeros(32, dtype=torch.bfloat16)[::2])
    wide = dev(torch.zeros(4, 32, dtype=torch.bfloat16)[:, :16])
    for args, kw in (((w, x, y), dict(bias=[strided])), ((w, [bf16(4, 16)], y), {}), ((w, x, [bf16(5, 16)]), {}),
                     ((w, x, y), dict(bias=[bf16(8)])), ((w, x, y), dict(residual=[bf16(4, 8)])),
                     ((w, x, [wide]), {}), ((w, x, y), dict(residual=[wide])), ((w * 2, x, y), {}),
                     ((w, [dev(torch.zeros(4, 8))], y), {})):
        with pytest.raises(ValueError):
            dcc.dcc_linear(*args, **{"bias": b, **kw})
    with pytest.raises((ValueError, KeyError)):
        dcc.dcc_linear(w, x, y, bias=b, act="swish")


class Cache:
    """What the calls read of a cache before they marshal it."""
    kv_heads, head_dim, seqs, pages, max_pages, n, torch_dtype, ref = 1, 64, 2, 4, 2, 1, torch.bfloat16, None


def test_workspaces_are_dense_and_on_the_device(dcc):
    i32 = dev(torch.zeros(8, dtype=torch.int32))
    q, out = [bf16(2, 4, 64)], [bf16(2, 4, 64)]
    for ws in (torch.zeros(64, dtype=torch.uint8), dev(torch.zeros(64, 2, dtype=torch.uint8)[:, 0])):
        for call in (lambda: dcc.dcc_kv4_attention(Cache, 0, q, out, i32, 1, ws), lambda: dcc.dcc_kv4_reserve(Cache, i32, ws),
                     lambda: dcc.dcc_kv4_free(Cache, i32[:1], ws), lambda: dcc.dcc_kv4_fork(Cache, i32[:1], i32[1:2], ws),
                     lambda: dcc.dcc_kv4_compact(Cache, i32, i32, i32, ws)):
            with pytest.raises(ValueError, match="workspace"):
                call()


def test_index_tensors(dcc):
    ws = dev(torch.zeros(64, dtype=torch.uint8))
    for bad in (torch.zeros(8, dtype=torch.int32), dev(torch.zeros(8, dtype=torch.int64)),
                dev(torch.zeros(16, dtype=torch.int32)[::2]), dev(torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(ValueError, match="int32"):
            dcc.dcc_kv4_reserve(Cache, bad, ws)
