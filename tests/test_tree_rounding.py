"""How the tree attention holds an INT4 key, replayed in host arithmetic for every scale and code: half
the key in fp16, and what that rounding dropped as the upper byte of its fp16 form (E5M2)."""

import numpy as np


def test_a_key_keeps_its_bits_down_to_scales_of_2_to_the_minus_5():
    scales = np.arange(1, 0x7000, dtype=np.uint16).view(np.float16)
    s = scales[scales <= np.float16(9360)].astype(np.float64)   # the largest scale: 65504 / 7
    assert s[0] == 2.0 ** -24 and s[-1] > 8000
    for code in range(1, 8):   # signs only mirror it
        half = code / 2 * s
        h = half.astype(np.float16).astype(np.float64)
        rest = (half - h).astype(np.float16)
        low = (rest.view(np.uint16) & 0xff00).view(np.float16).astype(np.float64)
        off = 2 * np.abs(half - h - low)
        assert (off[s >= 2.0 ** -5] == 0).all()
        key = code * s
        assert (off <= np.minimum(2.0 ** -11 * key, 2.0 ** -15) + 2.0 ** -24).all()
        # the remainder itself, which meets the rounded query: half an ulp of the halved key, doubled
        assert (2 * np.abs(half - h) <= 2.0 ** -11 * key + 2.0 ** -24).all()


def test_a_value_is_off_by_half_an_ulp_or_the_smallest_step():
    scales = np.arange(1, 0x7bff, dtype=np.uint16).view(np.float16)
    s = scales.astype(np.float64)
    for code in range(1, 8):
        v = code * s
        v = v[v <= 65504]
        off = np.abs(v - 2 * (v / 2).astype(np.float16).astype(np.float64))
        assert (off <= np.maximum(2.0 ** -11 * v, 2.0 ** -24)).all()
