"""The scale bytes that an INT4 page may hold (CPU): the unpacking's fp16 products
are finite and exact up to 0xE7, and not from the next one on."""
import numpy as np

import kv4_ref as ref


def _exact(x):
    with np.errstate(over="ignore"):
        return np.array_equal(x, x.astype(np.float16).astype(np.float64))


def test_the_largest_scale_byte():
    assert ref.SCALES[0xE7] == 15360 and ref.SCALES[0xE8] == 16384
    s = ref.SCALES[:0xE8]
    for f in (1, 264, 24):                                     # s / 64 and the two biases times it
        assert _exact(s / 64 * f)
    assert not _exact(ref.SCALES[0xE8:0xE9] / 64 * 264)
    # a code's value under an exponent, taken off again by one multiply-add: exact
    for base, bias in ((256, 264), (16, 24)):
        for u in range(16):
            v = (base + u) * (s / 64) - bias * (s / 64)
            assert np.array_equal(v, (u - 8) * s / 64) and _exact(v)


def test_appends_stay_below_it():
    x = np.full(128, 65504, np.float16)
    assert ref.SCALES[ref.quantise_row(x)[1]].max() == 10240
