"""Pins for the oracle of the four-bit operators: the format by hand, nearest
codes against a dense search, and the cache against plain arrays."""
import numpy as np
import pytest

from oracle import fp4, tokens as ot

rng = np.random.default_rng(8)


def test_values_by_hand():
    codes = np.zeros((1, 16), np.uint8)
    codes[0, :4] = [0x10, 0x32, 0x54, 0x76]
    codes[0, 4:8] = [0x98, 0xba, 0xdc, 0xfe]
    v = fp4.values(codes, np.array([[128]], np.uint8))[0]
    np.testing.assert_array_equal(v[:8], [0, 1, 2, 3, 4, 6, 8, 12])
    np.testing.assert_array_equal(v[8:16], [0, -1, -2, -3, -4, -6, -8, -12])
    assert np.signbit(v[8]) and not v[16:].any()
    assert np.isnan(fp4.values(codes, np.array([[255]], np.uint8))).all()
    assert fp4.values(codes, np.array([[0]], np.uint8))[0, 1] == 2.0 ** -128


def test_every_code_comes_back():
    for e in (-125, -3, 0, 17, 125):
        v = np.concatenate([fp4.SIZES, -fp4.SIZES, fp4.SIZES, -fp4.SIZES]) * 2.0 ** e
        codes, scales = fp4.quantise(v)
        assert scales[0] == e + 127
        np.testing.assert_array_equal(fp4.values(codes, scales), v)


@pytest.mark.parametrize("a,e", [(6.0, 0), (6.999, 0), (7.0, 1), (4.0, 0), (3.5, 0), (3.499, -1), (1.75, -1), (0.0, -125),
                                 (7 * 2.0 ** -126, -125), (3e38, 125)])
def test_the_largest_value_decides_the_scale(a, e):
    x = np.zeros(32)
    x[5] = -a
    _, scales = fp4.quantise(x)
    assert scales[0] == e + 127


def test_ties_go_to_the_even_code_and_six_is_the_last():
    x = np.zeros(32)
    x[:9] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, -2.5]
    np.testing.assert_array_equal(fp4.values(*fp4.quantise(x))[:9], [0, 1, 1, 2, 2, 4, 4, 6, -2])
    x = np.full(32, 7.9 * 2.0 ** 125)
    np.testing.assert_array_equal(fp4.values(*fp4.quantise(x)), np.full(32, 6 * 2.0 ** 125))


def test_no_value_is_off_by_more_than_half_its_step():
    x = rng.standard_normal((200, 64)) * np.exp(rng.standard_normal((200, 1)) * 5)
    codes, scales = fp4.quantise(x)
    y = fp4.values(codes, scales)
    unit = np.repeat(2.0 ** (scales.astype(float) - 127), 32, -1)
    r = np.abs(x) / unit
    step = np.where(r < 2, 0.5, np.where(r < 4, 1.0, 2.0))
    assert np.all(np.abs(x - y) <= unit * step / 2)


def test_values_that_are_not_finite_take_their_group_along():
    x = np.ones((2, 64))
    x[0, 3], x[1, 40] = np.inf, np.nan
    y = fp4.values(*fp4.quantise(x))
    assert np.isnan(y[0, :32]).all() and np.isnan(y[1, 32:]).all()
    assert (y[0, 32:] == 1).all() and (y[1, :32] == 1).all()


def test_cache_keeps_tokens_by_their_places():
    k, v = rng.standard_normal((2, 2, 40, 3, 64))
    codes, scales = np.zeros((5, 2, 3, 32, 32), np.uint8), np.full((5, 2, 3, 32, 2), 255, np.uint8)
    table = np.array([[4, 1, 9], [2, -1, 0]], np.int32)
    start, count = np.array([20, 50]), np.array([40, 30])
    c, s = fp4.append(k, v, codes, scales, table, start, count)
    ko, vo = fp4.read(c, s, table, 40, start, count)
    want = fp4.values(*fp4.quantise(k)), fp4.values(*fp4.quantise(v))
    for got, w in zip((ko, vo), want):
        np.testing.assert_array_equal(got[0], w[0])          # places 20 .. 59: pages 4 and 1
        assert not got[1, :14].any() and not got[1, 30:].any()  # 50 .. 63 have no page; past count
        np.testing.assert_array_equal(got[1, 14:30], w[1, 14:30])
    assert (s[3] == 255).all() and (s[0, :, :, 16:] == 255).all()


@pytest.mark.parametrize("causal", [False, True])
def test_attention_equals_that_of_plain_keys(causal):
    B, Tq, Hq, Hk, D, page = 2, 3, 4, 2, 64, 32
    codes = rng.integers(0, 256, (6, 2, Hk, page, D // 2), dtype=np.uint8)
    scales = rng.integers(124, 128, (6, 2, Hk, page, D // 32), dtype=np.uint8)
    table = np.array([[3, 0, 5], [1, 4, 2]], np.int32)
    length, q_len = np.array([70, 96]), np.array([3, 2])
    q = rng.standard_normal((B, Tq, Hq, D))
    got, mean_abs, _ = fp4.attention(q, codes, scales, table, length, q_len, causal)
    k, v = fp4.read(codes, scales, table, 96)
    empty = np.zeros((0, Hk, D))
    want, want_abs, _ = ot.prefix_attention(q, empty, empty, k, v, length, q_len, None, causal)
    np.testing.assert_allclose(got, want, atol=1e-13)
    np.testing.assert_allclose(mean_abs, want_abs, atol=1e-13)
    # a column without a page: its tokens do not count
    table[0, 1] = 6
    mask = np.ones((B, 96), bool)
    mask[0, 32:64] = False
    got, _, _ = fp4.attention(q, codes, scales, table, length, q_len, causal)
    want, _, _ = ot.prefix_attention(q, empty, empty, k, v, length, q_len, mask, causal)
    np.testing.assert_allclose(got, want, atol=1e-13)
