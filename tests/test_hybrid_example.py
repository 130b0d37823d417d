"""The hybrid mixer example: the operators together with a long convolution."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_hybrid_mixer():
    """The loss falls; tokens decoded one by one agree with the prompt run as a
    whole to the rounding of the outputs (both within 1.25 u of the same values,
    u = 2^-8)."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import hybrid_mixer
    finally:
        sys.path.pop(0)
    r = hybrid_mixer.run(batch=2, tokens=1024, steps=4, hidden=512, decode=5)
    assert r["shape"] == (2, 1024, 512)
    assert r["losses"][-1] < r["losses"][0]
    assert r["decode_difference"] < 2.5 * 2.0 ** -8
