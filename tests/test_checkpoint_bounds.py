"""How far a checkpoint's values may be from what was saved: the bounds that its entry states, by the 64-bit definition."""
import numpy as np
import pytest

import oracle.recurrence as ref

LARGEST = float(np.finfo(np.float32).max)


# just above 63.5 steps, which rounds by half a step; the type's largest value, 64 steps less 2^-18, whose code is cut to 63
@pytest.mark.parametrize("largest, bound", [(63.5 + 2.0 ** -14, 127), (LARGEST, 64)])
def test_the_bounds_are_met(largest, bound):
    x = np.zeros((1, 32))
    x[0, 0] = largest
    off = abs(ref.checkpoint(x, LARGEST)[2][0, 0] - largest) / largest
    assert 0.999 / bound <= off <= 1 / bound and off > 2.0 ** -7


def test_the_bounds_hold():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 32)) * 2.0 ** rng.uniform(-140, 120, (200, 1))
    off = np.abs(ref.checkpoint(x)[2] - x).max(1)
    assert (off <= np.maximum(np.abs(x).max(1) / 127, 2.0 ** -128)).all()
    assert (off > np.abs(x).max(1) / 127).any()            # below the least scale
