"""What the 16-bit levels of the 8-bit product cost, as the header states it
per width for the built-in codebooks: the root mean square of the levels'
error over N(0,1), relative to the levels' own."""

from math import erf, sqrt

import numpy as np
import pytest

import rotated_codebook_bit_amd as cq

try:
    cq.lib()
except ImportError:
    pytest.skip("libcq.so is not built", allow_module_level=True)


@pytest.mark.parametrize("bits,stated", [(cq.TERNARY, 4e-8), (2, 4e-8), (3, 1e-6), (4, 7e-6)])
def test_stated_error(bits, stated):
    t, lv = cq.q8_levels(bits), cq.codebook(bits).astype(np.float64)
    m = 256.0 * np.array(t.hi[:len(lv)]) + np.array(t.lo[:len(lv)])
    cdf = [0.0] + [0.5 + 0.5 * erf(e / sqrt(2)) for e in (lv[1:] + lv[:-1]) / 2] + [1.0]
    share = np.diff(cdf)
    error = sqrt((share * (lv - t.scale * m) ** 2).sum() / (share * lv ** 2).sum())
    assert stated / 8 < error <= stated  # the statement is neither broken nor far from the truth
