"""Pins of the attention side's oracle (oracle/attention.py), and the layout
queries that need no GPU."""

import numpy as np
import pytest

from moe_layer_05_amd import binding
from oracle import attention as oa
from oracle import rope as orope


@pytest.mark.parametrize("D", [64, 128, 192, 256])
def test_tile_places_are_a_permutation(D):
    """Every half byte and scale byte of a tile has exactly one owner."""
    nibbles = [2 * b + s // 4 for f in (oa.k_place, oa.v_place) for t in range(16) for d in range(D)
               for b, s in [f(D, t, d)]]
    scales = [f(D, t, g) for f in (oa.k_scale_place, oa.v_scale_place) for t in range(16)
              for g in range(D // 32)]
    used = sorted(nibbles + [2 * s + i for s in scales for i in (0, 1)])
    assert used == list(range(2 * 17 * D))


def test_v_places_by_hand():
    # D = 192: one chunk of 128 features, a last one of 64
    base = 8 * 192 + 96
    assert oa.v_place(192, 0, 0) == (base, 0)
    assert oa.v_place(192, 5, 9) == (base + ((1 * 16 + 1) * 4 + 1) * 4, 4)
    assert oa.v_place(192, 15, 191) == (base + 1024 + ((3 * 16 + 15) * 4 + 3) * 2 + 1, 4)


def test_quantise_by_hand():
    x = np.zeros(64)
    x[:5] = [7.0, -5.0, 2.5, 0.25, -0.75]     # 7 -> 6; 5 ties to 4; 2.5 to 2; .25 to 0; .75 to 1
    x[32:34] = [7.0001, 1.0]                  # above 7: the next power of two
    c, s = oa.quantise(x)
    assert list(s) == [127, 128]
    assert list(oa.values(c, s)[:5]) == [6.0, -4.0, 2.0, 0.0, -1.0]
    assert list(oa.values(c, s)[32:34]) == [8.0, 1.0]


def test_quantise_bounds():
    """No value is off by more than half a step of its interval, the largest
    by at most half the top one; groups scale by powers of two."""
    r = np.random.default_rng(0)
    x = r.standard_normal((200, 64)) * np.exp2(r.integers(-40, 40, (200, 1)))
    c, s = oa.quantise(x)
    y = oa.values(c, s)
    unit = np.repeat(2.0 ** (s.astype(float) - 127), 32, -1)
    a = np.abs(x) / unit
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    assert (np.abs(x - y) / unit <= step / 2).all()
    c2, s2 = oa.quantise(x * 8)
    assert np.array_equal(c, c2) and np.array_equal(s + 3, s2)


def test_quantise_extremes():
    big, tiny = np.float64(3.3895313892515355e38), 2.0 ** -133
    for v, byte in ((big, 252), (tiny, 2), (0.0, 2), (np.inf, 255), (np.nan, 255)):
        c, s = oa.quantise(np.full(32, v))
        assert s[0] == byte
        if byte == 255:
            assert np.isnan(oa.values(c, s)).all()
    assert np.isfinite(np.float32(oa.values(*oa.quantise(np.full(32, big))))).all()


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_is_the_inverse_of_the_inverse(inter):
    r = np.random.default_rng(1)
    T, NH, D, R = 7, 2, 64, 32
    x = r.standard_normal((T, NH, D))
    pos = r.integers(0, 50, T)
    ang = np.arange(50)[:, None] * 10000.0 ** (-np.arange(R // 2) * 2 / R)
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    y, _ = oa.norm_rope(x, None, 0.0, pos, table, R, inter)
    back = orope.inv_rope(y.astype(np.float32), pos, table, R, inter)
    assert np.abs(back - x).max() < 1e-5
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))


def test_norm_by_hand():
    x = np.zeros((1, 1, 16))
    x[..., 0], x[..., 8] = 3.0, 4.0
    table = np.zeros((1, 16), np.float32)
    table[:, 8] = 1.0                                  # a quarter turn of the first pair
    y, _ = oa.norm_rope(x, np.full(16, 2.0), 0.0, [0], table, 16, False)
    r = 2.0 / np.sqrt(25.0 / 16)
    assert y[0, 0, 0] == pytest.approx(-4 * r) and y[0, 0, 8] == pytest.approx(3 * r)


def test_attend_by_hand():
    k = np.array([[0.0], [np.log(3.0)]])
    v = np.array([[1.0], [5.0]])
    out, lse, spread, _ = oa.attend([[1.0], [1.0], [1.0]], k, v, 1.0, sees=[2, 1, 0])
    assert out[:, 0] == pytest.approx([4.0, 1.0, 0.0])
    assert lse[0] == pytest.approx(np.log(4.0)) and lse[1] == 0 and lse[2] == -np.inf
    assert spread[0, 0] == pytest.approx(4.0)


def test_put_get_round_trip():
    r = np.random.default_rng(2)
    for D in (64, 128, 192, 256):
        pages = r.integers(0, 256, (2, 2, 2, 17 * D)).astype(np.uint8)
        before = pages.copy()
        k, v = r.standard_normal((2, D))
        oa.put(pages, 1, 0, 21, k, v)
        a, b = oa.get(pages, 1, 0, 21)
        assert np.array_equal(a, oa.values(*oa.quantise(k)))
        assert np.array_equal(b, oa.values(*oa.quantise(v)))
        assert (before != pages).sum() <= 17 * D // 16      # no other token's bytes
        for t in (20, 22):
            assert np.array_equal(oa.get(pages, 1, 0, t), oa.get(before, 1, 0, t), equal_nan=True)


def test_page_bytes():
    L = binding.lib()
    assert L.moe_cache4_page_bytes(64, 3, 128) == 3 * 4 * 17 * 128
    for bad in ((8, 1, 128), (0, 1, 128), (4112, 1, 128), (16, 0, 128), (16, 1, 96), (-16, 1, 64)):
        assert L.moe_cache4_page_bytes(*bad) == 0, bad
