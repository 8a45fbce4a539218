"""Pins of the 8-bit oracle: hand-worked codes, rounding by definition, scales at their borders."""
import numpy as np

from oracle import fp8 as F


def test_codes_by_hand():
    # 1 = 2^0: exponent 7 -> 0x38; 1.125 -> 0x39; 448 = 1.75 2^8 -> 0x7E; 2^-9 -> 0x01; 2^-6 -> 0x08
    want = {0.0: 0x00, 1.0: 0x38, 1.125: 0x39, 448.0: 0x7E, 2.0 ** -9: 0x01, 2.0 ** -6: 0x08, -1.5: 0xBC, 240.0: 0x77}
    for v, c in want.items():
        assert F.e4m3_bytes(np.array([v]))[0] == c
        assert F.e4m3_values(np.array([c]))[0] == v
    assert np.isnan(F.e4m3_values(np.array([0x7F, 0xFF]))).all()


def test_ties_go_to_even_and_steps_are_halves():
    got = F.e4m3_round(np.array([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, -17.0]))   # between 16, 18, 20; 0, 2^-9, 2^-8
    np.testing.assert_array_equal(got, [16.0, 20.0, 0.0, 2.0 ** -8, -16.0])
    x = np.random.default_rng(3).uniform(2.0 ** -6, 448, 20000)
    assert np.max(np.abs(F.e4m3_round(x) - x) / x) <= 2.0 ** -4
    grid = F.e4m3_values(np.arange(127))
    np.testing.assert_array_equal(F.e4m3_bytes(grid), np.arange(127))


def test_scales_at_their_borders():
    b = F.scale_bytes(np.array([448.0, np.nextafter(448.0, 449), 1.75, 1.7500001, 0.0, 2.0 ** -140, np.inf, np.nan,
                                3.4028234663852886e38]))
    np.testing.assert_array_equal(b, [127, 128, 119, 120, 27, 27, 255, 255, 247])


def test_tiles_and_rows():
    x = np.random.default_rng(5).standard_normal((130, 200)) * np.logspace(-3, 3, 200)
    codes, b = F.fp8_quantize(x)
    assert codes.shape == (130, 256) and b.shape == (130, 2) and not codes[:, 200:].any()
    v = F.fp8_values(codes, b)[:, :200]
    top = np.stack([np.abs(x[:, :128]).max(1), np.abs(x[:, 128:]).max(1)], 1)
    # half a step of four significant bits, or of the smallest code: top > 224 2^(b - 127)
    assert np.all(np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, np.repeat(top, 128, 1)[:, :200] / 224 * 2.0 ** -10))
    tc, tb = F.fp8_quantize(x, tiles=True)
    assert tb.shape == (2, 2)
    back, backb = F.fp8_quantize(x.T, tiles=True)
    np.testing.assert_array_equal(tb.T, backb)
    np.testing.assert_array_equal(tc[:, :200].T, back[:, :130])
    np.testing.assert_array_equal(F.fp8_values(tc, tb, tiles=True)[:, :200].T, F.fp8_values(back, backb, tiles=True)[:, :130])
