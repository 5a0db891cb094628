"""What the 8-bit format's reading (c + 1/2) s adds to rows, in the mean: by the format's definition, no GPU."""
import numpy as np
import pytest

import q8_ref as ref


def read_back(x, s):
    return (ref.codes(x, s).astype(np.float64) - 128 + 0.5) * s


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("E", [-40, 0, 5])
def test_bf16_numbers_are_read_back_half_a_step_of_theirs_high(E, sign):
    """All 128 bf16 numbers of a binade of one sign, from the block's largest binade to that of the scale: the mean of
    (value - x) is half their distance, whatever the sign."""
    s = 2.0 ** (E - 6)
    assert ref.scale_of(1.5 * 2.0 ** E) == s
    for e in range(E - 6, E + 1):
        x = sign * (1 + np.arange(128) / 128) * 2.0 ** e
        step = 2.0 ** (e - 7)
        error = read_back(x, s) - x
        assert np.abs(error).max() <= s / 2
        assert error.mean() == step / 2    # the binade is 2^(e - E + 6) whole steps of the codes, of s / step numbers each
    assert read_back(0.0, s) == s / 2
    small = np.arange(1, 64) / 64 * s  # below s: the two signs' errors cancel
    assert (read_back(small, s) - small + read_back(-small, s) + small).sum() == 0


def test_numbers_anywhere_between_the_codes_keep_their_mean():
    """fp32 numbers (rotated keys): the mean error of n of them, each within s / 2 and evenly spread there, is below five
    standard deviations s / sqrt(12 n), and their step's half, 2^-17 s at most."""
    rng = np.random.default_rng(1)
    n, s = 1 << 18, 2.0 ** -6
    x = rng.uniform(-1.9, 1.9, n).astype(np.float32).astype(np.float64)
    error = read_back(x, s) - x
    assert abs(error.mean()) <= 5 * s / np.sqrt(12 * n) + 2.0 ** -17 * s


@pytest.mark.parametrize("e", [-149, -133, -127, -126, -121, -120, -119, 0, 127])
def test_largest_error_of_a_block(e):
    """s / 2 for a block whose largest magnitude a has the exponent e: a / 128 at most, but 2^-127 where a is below 2^-120."""
    s = np.float64(ref.scale_of(2.0 ** e))
    x = np.append(np.random.default_rng(2).uniform(-2.0 ** e, 2.0 ** e, 1000), [2.0 ** e, -2.0 ** e, 0.0])
    assert np.abs(read_back(x, s) - x).max() <= s / 2
    assert s / 2 <= max(2.0 ** e / 128, 2.0 ** -127) and (s / 2 <= 2.0 ** e / 128) == (e >= -120)
