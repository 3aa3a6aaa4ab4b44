"""One row's log probabilities, scored alone and among others: a row is cut over more
or fewer CTAs by what the call brings, so the fp32 sums may differ in their last bits,
within the bounds that each call keeps; the ids may not."""
import pytest
import torch

from test_gpu_kv4 import dcc  # noqa: F401  (the fixture)
from test_gpu_logprobs import check, logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,C,top", [(8, 4001, 20), (2, 70001, 64), (1, 129, 3)])
def test_a_row_alone_and_among_others(dcc, dtype, n, C, top):  # noqa: F811
    g = torch.Generator().manual_seed(C)
    xs = logits(g, n, 1100, C, dtype)
    target = torch.randint(0, n * C, (1100,), generator=g).to(torch.int32).cuda()
    ids = None
    for T in (1100, 532, 64, 3, 1):  # one run a row, two, several, one batch a run
        got = check(dcc, [x[:T] for x in xs], target[:T], top)
        ids = got[2] if ids is None else ids
        assert torch.equal(got[2], ids[:T])
    assert dcc.dcc_local_check() == dcc.DCC_OK
