"""Host side of the benchmark."""

import pytest

import bench


@pytest.mark.parametrize("steps", [1, 2, 5, 20, 31, 32, 33, 1000])
@pytest.mark.parametrize("copies", [1, 2, 4, 7])
def test_every_leg_has_its_tokens(steps, copies):
    """A short run generates enough tokens for the multi-layer leg as well
    (a slice past the last token is empty, which the step refuses)."""
    n = bench.tokens_after_prefill(steps, copies, 8)
    per_copy = max(len(range(i, steps, copies)) for i in range(copies))
    assert n >= 2 * per_copy and n >= bench.LAYER_STEPS
    # the default run's data stay what they were
    assert bench.tokens_after_prefill(20000, copies, 8) == \
        2 * -(-20000 // copies) + 1
    assert bench.tokens_after_prefill(steps, copies, 0) == \
        2 * -(-steps // copies) + 1
