"""The example of drafted trees: reserve, cache, the tree's attention, the output
layer, log probabilities and the accepted branch kept, run together for several
steps, with and without a window, against plain torch operations on the cache's
own values.

The block's bound is that of test_gpu_decode_block.py (16 bf16 roundings of the
largest values: 0.25 of the rms).  Log probabilities are compared on the same
logits: both sides are fp32, log p = x - lse of values up to about 30, so a few
roundings of 2^-24 * 30 = 1.8e-6 each, 16 of them 3e-5."""
import pytest

pytestmark = pytest.mark.gpu

WIDE = [-1] + [(j - 1) // 2 for j in range(1, 39)]  # 39 drafted tokens: two words of a mask


@pytest.mark.parametrize("shape", [dict(), dict(n=2, q_heads=4, kv_heads=2, dim=64, hidden=512, ff=1024, window=100, sinks=4),
                                   dict(n=8, q_heads=2, kv_heads=1, dim=128, hidden=256, ff=2048, vocab=777, top=1),
                                   dict(n=2, q_heads=8, kv_heads=1, hidden=512, ff=1024, parents=WIDE, window=64, sinks=70)])
def test_speculate(shape):
    from driven_collective_communication_gb300 import build
    build.build()
    from driven_collective_communication_gb300.examples import speculate
    steps = speculate.run(speculate.Speculator(**shape), verbose=False)
    assert [len(k) for _, _, k in steps] == [3] * 7
    for off, lp, kept in steps:
        assert off < 0.25 and lp < 3e-5
    assert all(k == [0, 0, 0] for _, _, k in (steps[2], steps[5])) and all(min(steps[i][2]) >= 1 for i in (1, 3, 4, 6))
