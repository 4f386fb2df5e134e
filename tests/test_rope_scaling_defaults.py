"""What a scaling of the rotary frequencies means where only its name, factor
and original length are given."""
import numpy as np
import pytest

from oracle import decode_step as od

gbb = pytest.importorskip("gemm_block_bit_amd")


@pytest.mark.parametrize("scaling,high", [("bands", 4.0), ("yarn", 32.0)])
def test_published_bounds_are_the_defaults(scaling, high):
    given = dict(scaling=scaling, factor=8.0, original_len=4096.0)
    got = gbb.rope_table(128, 300, 500000.0, **given)
    assert np.array_equal(got, gbb.rope_table(128, 300, 500000.0, low=1.0, high=high, **given))
    other = gbb.rope_table(128, 300, 500000.0, low=1.0, high=36.0 - high, **given)
    assert not np.array_equal(got, other)
    # the 64-bit formulas: one rounding to fp32, an angle below 2^9 rounded in 64 bits
    ref = od.rope_table(128, 300, 500000.0, low=1.0, high=high, **given)
    assert np.all(np.abs(got - ref) <= 0.5 * np.spacing(np.abs(got)) + 2.0 ** -42)


def test_one_bound_given():
    given = dict(scaling="yarn", factor=8.0, original_len=4096.0)
    assert np.array_equal(gbb.rope_table(64, 40, low=2.0, **given), gbb.rope_table(64, 40, low=2.0, high=32.0, **given))
    assert np.array_equal(gbb.rope_table(64, 40, high=4.0, **given), gbb.rope_table(64, 40, low=1.0, high=4.0, **given))
