"""Calls for drafted tokens and log probabilities whose buffers are empty or half
given: what returns before anything is launched (no GPU needed)."""
import pytest
import torch

from test_ops_arguments import dcc  # noqa: F401  (dcc: the fixture)
from test_ops_binding import bf16, dev  # noqa: F401


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
