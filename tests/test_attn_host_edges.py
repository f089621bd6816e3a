"""Edges of the attention oracle and host checks, without a GPU."""
import math

import numpy as np
import pytest

from oracle import attn_oracle as A


@pytest.mark.parametrize("base,original,scaled", [(4.0, 131072.0, False), (1e4, 4.0, True)])
def test_yarn_whose_ramp_lies_on_one_side_of_the_pairs(base, original, scaled):
    f, _ = A.frequencies(64, base)
    turns = original * f / (2 * math.pi)
    assert (turns < 1).all() if scaled else (turns > 32).all()
    y, _ = A.frequencies(64, base, kind="yarn", factor=8, original=original)
    np.testing.assert_allclose(y, f / 8 if scaled else f, rtol=1e-15)
