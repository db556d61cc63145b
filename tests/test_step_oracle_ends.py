"""The references of oracle/steps.py at the ends of their ranges (no GPU)."""
import numpy as np

from oracle import steps as os_


def test_largest_weights_by_hand():
    """6 2^125 is the largest value of a weight: the codes of 4 and 6 times 2^126 are past bfloat16."""
    row = np.array([3e38, -3e38, 1.5 * 2.0 ** 127, 2.0 ** 125] + [0.0] * 28)
    got, byte = os_.encode_weights(row)
    assert byte == 252 and np.array_equal(got[:4], [6 * 2.0 ** 125, -6 * 2.0 ** 125, 6 * 2.0 ** 125, 2.0 ** 125])
    assert os_.encode_weights(np.full(32, 1.5 * 2.0 ** 126))[1] == 251
