"""The example decoder block: the cache, its attention and pages, the
column-parallel layer and the row-parallel layer fused with the AllReduce run
together, prompts and single tokens and a beam step, against plain torch
operations on the cache's own values.

Both sides round the same intermediate results to bf16 (Q, the attention's
output, the hidden state twice, the activation); where a rounding falls the
other way the difference is one bf16 ulp of that value, 2^-8 of it, and the few
roundings after each other stay below 16 of them on the largest values (4
sigma): 16 * 4 * 2^-8 = 0.25 of the rms.
"""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [dict(), dict(n=2, q_heads=4, kv_heads=2, dim=64, hidden=512, ff=1024),
                                   dict(n=8, q_heads=2, kv_heads=1, dim=128, hidden=256, ff=2048)])
def test_decode_block(shape):
    from driven_collective_communication_gb300 import build
    build.build()
    from driven_collective_communication_gb300.examples import decode_block
    for off in decode_block.run(decode_block.Block(**shape), verbose=False):
        assert off < 0.25
