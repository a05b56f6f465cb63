"""The parts in 8 bits that probabilities are split into (csrc/fa_serve8.cu), over every fp16 number that they may be."""

import numpy as np
import pytest


def e5m2(h):
    """The nearest e5m2 as the kernel takes it: half a step up in the magnitude's bits, the low byte off."""
    return ((h.view(np.uint16).astype(np.uint32) + 0x80) & 0xFF00).astype(np.uint16).view(np.float16)


@pytest.mark.parametrize("parts,most,below", [(3, 2.0 ** -21, 2.0 ** -10), (4, 2.0 ** -23, 2.0 ** -12)])
def test_how_far_the_parts_are_off(parts, most, below):
    x = np.arange(0, 0x7801, dtype=np.uint16).view(np.float16)
    assert x[-1] == 2.0 ** 15
    left, held = x.copy(), np.zeros(x.shape)
    for z in range(parts):
        p = e5m2(left)
        assert np.isfinite(p).all()
        held += p.astype(np.float64) * (1.0 if z < 2 else 1.0 / 64)
        assert ((left.astype(np.float64) - p.astype(np.float64)) == (left - p).astype(np.float64)).all()  # no rounding
        left = left - p
        if z == 1:
            assert (left.astype(np.float64) * 64 == (left * np.float16(64)).astype(np.float64)).all()
            left = left * np.float16(64)
    off = np.abs(held - x.astype(np.float64))
    assert off.max() == most and not off[x >= below].any()
