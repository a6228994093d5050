"""The example that runs the projections, the cache, its attention and the log probabilities together."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode_q8_cache  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", [dict(), dict(hidden=256, q_heads=4, kv_heads=1, head_dim=128, mlp=512, vocab=1000)])
def test_scores_of_one_pass_are_those_of_the_steps(sizes):
    # The two differ by the cache's rounding alone: a block's scale grows as tokens arrive one by one, and its
    # codes are rounded again, half a step (1/254 of the block's largest value) each time.  A few of these, of
    # values around a third of the largest, are a percent or two of an attention output, which is one of the
    # sums that make up a logit of unit deviation; 0.25 is far above that, and far below what a token in
    # a wrong place, a wrong page or a missing key does to 60 x 4 log probabilities.
    tokens, logps, apart, ms, entropy = decode_q8_cache.run(layers=2, steps=60, prompt_lens=(1, 130, 37, 16), **sizes)
    assert tokens.shape == (60, 4) and tokens.min() >= 0 and ms > 0
    assert torch.all(torch.isfinite(logps)) and torch.all(logps < 0)
    assert apart.abs().max().item() < 0.25
    assert 0 < entropy < torch.log(torch.tensor(float(sizes.get("vocab", 49152)))).item()
