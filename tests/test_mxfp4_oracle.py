"""The MXFP4 oracle against the format's tables."""
import numpy as np

from host_offloaded_weight_gb300 import lstream as L
from oracle import mxfp4 as mx


def test_pitches_match_the_library():
    for K in (1, 31, 32, 127, 128, 129, 512, 513, 1000, 13824):
        assert (L.lsk_mxfp4_code_pitch(K), L.lsk_mxfp4_scale_pitch(K)) == (mx.code_pitch(K), mx.scale_pitch(K))
    assert L.lsk_mxfp4_code_pitch(0) == 0 and L.lsk_mxfp4_scale_pitch(-5) == 0


def test_elements_round_to_nearest_ties_to_even():
    v = np.zeros((1, 32))
    v[0, :16] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.9, 0.26, 0.74, -0.25, -3.5, -7.9, 0.0, 5.1]
    c, s = mx.encode(v)
    assert s[0, 0] == 127                                # max 7.9: floor(log2) = 2, scale 2^0
    assert mx.decode(c, s, 32)[0, :16].tolist() == [4, 0, 1, 1, 2, 2, 4, 4, 6, 0.5, 0.5, 0, -4, -6, 0, 6]


def test_every_value_of_the_format_keeps_itself():
    mags = np.concatenate((mx.MAGNITUDES, -mx.MAGNITUDES, mx.MAGNITUDES, -mx.MAGNITUDES))
    for e in (-125, -3, 0, 60, 125):
        v = np.ldexp(mags, e)[None]
        c, s = mx.encode(v)
        assert s[0, 0] == e + 127 and np.array_equal(mx.decode(c, s, 32), v)


def test_relative_error_of_normal_values():
    """Within a block an element is off by at most half a step: 1/4 of the scale below 2, 1 at the top, 2 when saturated."""
    v = np.random.default_rng(0).standard_normal((50, 320))
    c, s = mx.encode(v)
    step = np.ldexp(1.0, s[:, np.arange(320) // 32].astype(int) - 127)
    assert np.all(np.abs(mx.decode(c, s, 320) - v) <= 2.0 * step)
    assert np.all(c[:, 160:] == 0) and np.all(s[:, 10:] == 0)


def test_non_finite_blocks_read_as_nan():
    v = np.ones((1, 96))
    v[0, 40] = np.inf
    v[0, 70] = np.nan
    c, s = mx.encode(v)
    assert s[0, :3].tolist() == [125, 255, 255]
    d = mx.decode(c, s, 96)
    assert np.array_equal(np.isnan(d[0]), np.arange(96) >= 32)


def test_error_bound_of_each_range_of_magnitudes():
    """Half a step: 1/4 of the scale below 2, 1/2 below 4, 1 up to 6; what saturates is off by its distance from 6."""
    v = np.random.default_rng(1).standard_normal((200, 320)) * np.exp2(np.random.default_rng(2).integers(-8, 8, (200, 1)))
    c, s = mx.encode(v)
    step = np.ldexp(1.0, s[:, np.arange(320) // 32].astype(int) - 127)
    a, err = np.abs(v) / step, np.abs(mx.decode(c, s, 320) - v) / step
    bound = np.select([a < 2, a < 4, a <= 6], [0.25, 0.5, 1.0], a - 6)
    assert np.all(err <= bound * (1 + 1e-12)) and a.max() < 8
    for lo, hi in ((0, 2), (2, 4), (4, 6), (6, 8)):
        assert ((a >= lo) & (a < hi)).sum() > 100
