"""Pins of the 4-bit cache oracle (oracle/fp4.py): the code grid, ties, round trips, the selection rule."""
import numpy as np

from oracle import fp4 as F


def test_codes_ties_and_saturation():
    x = np.array([0.0, 0.25, 0.2500001, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.0001, 6.0, 100.0, -0.75, -2.5, -7.0])
    want = [0, 0, 0.5, 1, 1, 2, 2, 4, 4, 6, 6, 6, -1, -2, -6]
    assert F.e2m1_values(F.e2m1_codes(x)).tolist() == want


def test_every_code_is_a_fixed_point():
    codes = np.arange(16, dtype=np.uint8)
    assert np.array_equal(F.e2m1_codes(F.e2m1_values(codes)) & 7, codes & 7)
    assert np.array_equal(F.e2m1_values(F.e2m1_codes(F.e2m1_values(codes))), F.e2m1_values(codes))


def test_rows_round_trip_and_error_bound():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 512)).astype(np.float32).astype(np.float64)
    x[3, 64:96] = 0
    codes, scales = F.quantize(x)
    rows = F.pack(codes, scales, np.zeros((50, 128), np.uint8))
    c2, s2 = F.unpack(rows)
    assert np.array_equal(c2, codes) and np.array_equal(s2, scales)
    back = F.dequantize_rows(rows)[:, :512].reshape(50, 16, 32)
    s = scales.astype(np.float64)[..., None]
    a = np.abs(x.reshape(50, 16, 32))
    # half the widest spacing at that height, or the cut at 6 s (amax <= 6 s (1 + 2^-11))
    spacing = np.where(a < 2 * s, 0.5, np.where(a < 4 * s, 1.0, 2.0)) * s
    assert np.all(np.abs(back - x.reshape(50, 16, 32)) <= np.maximum(spacing / 2, 6 * s * 2.0 ** -11) + 1e-12)
    exact = F.e2m1_values(rng.integers(0, 8, (4, 512)).astype(np.uint8)) * 0.25
    exact[:, ::32] = 1.5                                           # every group reaches 6 x 0.25
    codes, scales = F.quantize(exact)
    assert np.array_equal(F.dequantize_rows(F.pack(codes, scales, np.zeros((4, 128), np.uint8)))[:, :512], exact)


def test_code8_half_way_goes_to_even():
    codes, scale = F.code8(np.array([[2.0, 1.0, -1.0, 0.0]]))
    assert codes.tolist() == [[127, 64, -64, 0]] and scale[0] == np.float32(2.0 / 127)
    codes, scale = F.code8(np.zeros((1, 4)))
    assert codes.tolist() == [[0, 0, 0, 0]] and scale[0] == 0


def test_select_keeps_the_ends_and_breaks_ties_low():
    q = np.zeros((2, 576))
    q[0, 0], q[1, 1] = 1.0, -1.0
    codes = np.zeros((10, 576))
    codes[:, 0] = [0, 5, 9, 9, 9, 1, 0, 0, 0, 0]
    codes[6, 1] = -12                                    # the second head's best page
    assert F.select(q, codes, np.ones(10, np.float32), 600, 5, 1, 1) == [0, 2, 3, 6, 9]
    assert F.select(q, codes, np.ones(10, np.float32), 320, 5, 1, 1) == [0, 1, 2, 3, 4]


def test_build_tables_by_hand():
    table = [[7, -1, -1], [3, 4, -1], [-1, -1, -1]]
    t, lens, cu, slots, pos, head, bad = F.build_tables([63, 100, 0], [2, 1, 1], table, [9, 8, 5], 1, 6)
    assert t == [[7, 8, -1], [3, 4, -1], [5, -1, -1]] and lens == [65, 101, 1] and cu == [0, 2, 3, 4]
    assert slots == [7 * 64 + 63, 8 * 64, 4 * 64 + 36, 5 * 64, -1, -1] and pos == [63, 64, 100, 0, -1, -1]
    assert head == 3 and not bad
