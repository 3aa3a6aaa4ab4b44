"""Calls for drafted tokens and log probabilities whose buffers are empty, half
given or out of range: what returns before anything is launched (no GPU needed)."""
import pytest
import torch

from test_ops_arguments import dcc, desc  # noqa: F401  (dcc: the fixture)
from test_ops_binding import bf16, dev  # noqa: F401
from test_seen_arguments import lp, tree


def f32(*shape):
    return dev(torch.zeros(*shape))


def i32(*shape):
    return dev(torch.zeros(*shape, dtype=torch.int32))


def test_half_of_the_alternatives(dcc):  # noqa: F811
    """Token numbers without their log probabilities, or these without those."""
    a = dict(logits=[bf16(4, 8)] * 2, target=i32(4), logprob=f32(4), workspace=dev(torch.zeros(1 << 20, dtype=torch.uint8)))
    for half in (dict(top_logprobs=f32(4, 2)), dict(top_ids=i32(4, 2)), dict(top_ids=i32(4, 0), top_logprobs=f32(4, 2)),
                 dict(top_ids=i32(4, 2), top_logprobs=f32(4, 0))):
        with pytest.raises(ValueError):
            dcc.dcc_token_logprobs(**a, **half)


def test_trees_of_no_tokens(dcc):  # noqa: F811
    """An empty batch has an empty mask, which has no address."""
    assert tree(dcc, desc(dcc), tokens=0, mask=None) == dcc.DCC_OK
    assert tree(dcc, desc(dcc), tokens=0, mask=None, words=0) == dcc.DCC_ERR_INVALID_ARG
    assert tree(dcc, desc(dcc), tokens=1, max_new=1, mask=None) == dcc.DCC_ERR_INVALID_ARG


def test_log_probabilities_of_no_tokens(dcc):  # noqa: F811
    none = dict(target=None, logprob=None, entropy=None, ids=None, tops=None)
    assert lp(dcc, tokens=0, **none) == dcc.DCC_OK
    assert lp(dcc, tokens=0, top=0, **none) == dcc.DCC_OK
    assert lp(dcc, tokens=0, top=65, **none) == dcc.DCC_ERR_INVALID_ARG
    assert lp(dcc, tokens=0, ws=None, **none) == dcc.DCC_ERR_INVALID_ARG
    ws = torch.zeros((1 << 20) + 16, dtype=torch.uint8)
    ws = dev(ws[-ws.data_ptr() % 16:])  # (as the GPU's allocations are)
    dcc.dcc_token_logprobs([bf16(0, 8)] * 2, i32(0), f32(0), ws, stream=0)
    dcc.dcc_token_logprobs([bf16(0, 8)] * 2, i32(0), f32(0), ws, entropy=f32(0), top_ids=i32(0, 3), top_logprobs=f32(0, 3),
                           stream=0)


@pytest.mark.parametrize("scale", [2.4e38, 3e38, 3.4028234e38])
def test_scales_whose_product_with_log2_e_is_infinite(dcc, scale):  # noqa: F811
    assert lp(dcc, scale=scale) == dcc.DCC_ERR_INVALID_ARG
