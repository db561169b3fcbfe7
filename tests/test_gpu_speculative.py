"""The speculative decoding example end to end: prompts, runs without commit, verification, commit."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.gpu
def test_speculative_example_keeps_the_states_of_what_it_emitted():
    import speculative_ssm
    texts, share, apart = speculative_ssm.run()
    assert 0.05 < share < 1
    lens = [5 + 37 * b for b in range(4)]
    assert all(len(t) >= n + 12 for t, n in zip(texts, lens))  # one token a step at least
    # the projections are the same matrix products on other batch shapes: a bf16 rounding of an input
    # may differ (2^-8 of it), the operators' own differences are far smaller
    assert apart <= 2 ** -6
