"""The host forms of the 4-bit append's bytes against each other."""
import numpy as np
import pytest

import layer_ref as ref
from append_codes_ref import TABLE, bytes_of, exact_bytes, nearest_scale, values


def test_scales_and_ties():
    assert np.array_equal(nearest_scale(TABLE), np.arange(127))
    middle = (TABLE[1:] + TABLE[:-1]) / 2
    assert np.array_equal(nearest_scale(middle), np.arange(126) + np.arange(126) % 2)
    assert nearest_scale(1e9) == 126 and nearest_scale(2.0 ** -10) == 0 and nearest_scale(2.0 ** -10 * 1.001) == 1
    x = np.zeros((1, 16))
    x[0, :8] = [7, 0.5, 1.5, -2.5, 3.5, -6.5, 0.75, 0.25]
    for f in (bytes_of, exact_bytes):
        codes, scale = f(x, 1.0)
        assert codes[0, :8].tolist() == [7, 0, 2, -2, 4, -6, 1, 0] and scale.tolist() == [[0x38]]


@pytest.mark.parametrize("ftype", ["f16", "bf16"])
def test_the_two_forms(ftype):
    """Equal where a factor is a power of two; elsewhere a border may lie between fp32's quotient and the exact one."""
    for f in (1.0, 0.5, 4.0, 2.0 ** -20):
        x = ref.f64(values(300, 2, 128, ftype, f, 6))
        for a, b in zip(bytes_of(x, f), exact_bytes(x, f)):
            assert np.array_equal(a, b)
    for f in (1 / 3, 0.7, 0.1):
        x = ref.f64(values(300, 2, 128, ftype, f, 7))
        (a, sa), (b, sb) = bytes_of(x, f), exact_bytes(x, f)
        same = np.repeat(sa == sb, 16, -1)
        assert (np.abs(sa - sb) <= 1).all() and (np.abs(a - b)[same] <= 1).all()
