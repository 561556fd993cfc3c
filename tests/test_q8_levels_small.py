"""Codebooks so small that the 8-bit product's scale would leave float32's
normal range: refused, where the scale had lost its bits (or was 0, the product
then all zeros); whatever is accepted meets its levels to within 2.1e-5 of the
largest, and so does its scale divided by sqrt(G) as the product uses it."""

import numpy as np
import pytest

import rotated_codebook_bit_amd as cq

try:
    cq.lib()
except ImportError:
    pytest.skip("libcq.so is not built", allow_module_level=True)

TINY = float(np.finfo(np.float32).tiny)


@pytest.mark.parametrize("bits", [cq.TERNARY, 2, 3, 4])
def test_small_codebooks(bits):
    base = cq.codebook(bits).astype(np.float64)
    accepted = 0
    for e in range(-149, 1):
        lv = (base * 2.0 ** e).astype(np.float32)
        if np.any(np.diff(lv) <= 0):
            continue  # not strictly ascending any more: refused as any such table
        top = np.abs(lv.astype(np.float64)).max()
        try:
            t = cq.q8_levels(bits, lv)
        except cq.CQError as err:
            assert err.status == -2 and top / 24576 < 32 * TINY, (e, err)
            continue
        accepted += 1
        m = 256.0 * np.array(t.hi[:len(lv)]) + np.array(t.lo[:len(lv)])
        for scale in (float(t.scale), float(np.float32(np.float32(t.scale) / np.float32(16.0))) * 16):
            # 2.1e-5, and the levels' own rounding to float32
            assert np.abs(lv.astype(np.float64) - scale * m).max() <= (2.1e-5 + 2.0 ** -22) * top, (e, scale)
    assert accepted >= 100  # ordinary ones are not refused
