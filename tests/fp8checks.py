"""A check of FP8 activation codes that needs no reference: finite tokens have no NaN code, and the largest value of
every group is +-448."""
import numpy as np


def assert_full_range(q, s, what=""):
    """q uint8 [M][K], s float32 [K / 128][M], of finite tokens.

    s is max|h| / 448 rounded to float32, off by at most 2^-24 of itself where it is a normal
    number, so the quotient of the largest value lies within 448 (1 +- 2^-23): between 432 and
    464, which is 448 in e4m3 (its next neighbours would be 416 and 480).  Groups whose
    scale is not normal are left out of that part."""
    M, K = q.shape
    nan = (q & 0x7F) == 0x7F
    assert not nan.any(), f"{what}: {np.count_nonzero(nan)} codes are NaN"
    top = (q & 0x7F).reshape(M, K // 128, 128).max(-1).T
    normal = s >= 2.0 ** -126
    assert np.all(np.isfinite(s)) and np.all(top[normal] == 0x7E), f"{what}: a group's largest code is not 448"
    assert np.all(top[s == 0] == 0), f"{what}: a group without a scale has codes"
