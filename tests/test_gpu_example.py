"""The 8-bit example runs and its results are what 8-bit operands allow."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu


def test_fp8_moe_example():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import fp8_moe
    errors = fp8_moe.main(["--tokens", "200", "--hidden", "512", "--inter", "384", "--experts", "6", "--topk", "2", "--batch", "5"])
    # A value in e4m3 is off by 2^-4 of itself at most, in e5m2 by 2^-3; their squares average a third of that (an error
    # spread evenly up to the bound) or less.  A product's norm carries both operands' shares; the expert layer has two
    # products of quantised weights after each other, the first under a product of two factors.
    e4, e5 = 2.0 ** -4 / 3 ** 0.5, 2.0 ** -3 / 3 ** 0.5
    both = lambda a, b: (a * a + b * b) ** 0.5
    assert errors["y"] < both(e4, e4) and errors["dx"] < both(e5, e4) and errors["dW"] < both(e5, e4)
    assert errors["experts"] < both(both(e4, 2 * e4), 2.0 ** -8)
