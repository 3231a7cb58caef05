"""rope_inv_freq where its formulas meet their ends: pairs that never turn, and arguments that are no numbers."""

import numpy as np
import pytest

import fp8_quantized_skinny_amd as sk


@pytest.mark.parametrize("rot", [2, 16, 64, 128])
@pytest.mark.parametrize("original", [1, 4, 6, 7, 50, 4096, 10 ** 9])
def test_pairs_of_few_and_of_many_turns(rot, original):
    """Fewer than `slow` turns over the original positions: divided by the whole factor; more than `fast`: as they are."""
    plain = sk.rope_inv_freq(rot, 10000.0).astype(np.float64)
    scaled = sk.rope_inv_freq(rot, 10000.0, factor=8.0, original=original, fast=32.0, slow=1.0)
    turns = plain * original / (2.0 * np.pi)
    share = plain / scaled
    assert (np.abs(share[turns < 1.0] - 8.0) <= 8.0 * 2.0 ** -22).all() and (np.abs(share[turns > 32.0] - 1.0) <= 2.0 ** -22).all()
    assert (share >= 1.0 - 2.0 ** -22).all() and (share <= 8.0 + 2.0 ** -19).all()


@pytest.mark.parametrize("name", ["base", "factor", "original", "fast", "slow"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_what_is_no_number_is_refused(name, value):
    with pytest.raises(ValueError):
        sk.rope_inv_freq(64, **{"factor": 2.0, "original": 4096, name: value})
