"""The code check itself: mistakes that a tolerance of one neighbour lets pass."""
import numpy as np
import pytest

import blockref as ref
from fp8checks import assert_full_range


def rows():
    rng = np.random.default_rng(0)
    return ref.quant_rows(rng.standard_normal((32, 4096)))


def test_right_codes_pass():
    q, s = rows()
    assert_full_range(q, s)
    z = np.zeros((3, 256), np.uint8)
    assert_full_range(z, np.zeros((2, 3), np.float32))


@pytest.mark.parametrize("wrong,match", [(0x7F, "NaN"), (0xFF, "NaN"), (0x7D, "not 448"), (0xFD, "not 448")])
def test_a_wrong_code_in_place_of_448_is_found(wrong, match):
    q, s = rows()
    bad = q.copy()
    at = np.argwhere(bad == (wrong & 0x80 | 0x7E))
    m, k = next((m, k) for m, k in at if (bad[m, k // 128 * 128:k // 128 * 128 + 128] & 0x7F == 0x7E).sum() == 1)
    bad[m, k] = wrong
    ref.assert_codes8(bad, s, q, s)  # (one neighbour in 0.1 % of the codes passes there)
    with pytest.raises(AssertionError, match=match):
        assert_full_range(bad, s)
