"""The bound that the page-scale attention's notes state for q as the sum of two E4M3 terms, over every
bf16 value: a row is scaled by a power of two so that its largest element lies in [2^7, 2^8); hi is
the nearest E4M3 value, lo that of what is left. The sum is exact for elements of at least 2^-9 of
the largest and off by at most 2^-17 of it below. No GPU is used."""

import numpy as np

import oracle


def e4m3(x):
    return oracle.e4m3_decode(oracle.e4m3_encode(x))


def test_two_terms_over_every_magnitude():
    # the non-negative bf16 values below 2^8, down to 0
    bits = np.arange(0, 0x4380, dtype=np.uint32) << 16
    x = bits.view(np.float32).astype(np.float64)
    assert x.max() < 256.0
    hi = e4m3(x)
    err = np.abs(x - hi - e4m3(x - hi))
    assert (err[x >= 2.0 ** -2] == 0).all()       # 2^-9 of a largest element of 2^7
    assert err.max() <= 2.0 ** -10                # 2^-17 of it
    # neither can be stated tighter: elements just below 2^-9 of 2^7 are not exact, and some are off
    # by more than 2^-18 of it
    assert (err[(x < 2.0 ** -2) & (x >= 2.0 ** -3)] > 0).any() and err.max() > 2.0 ** -11
