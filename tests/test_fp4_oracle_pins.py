"""The oracle of the 4-bit experts and of the input norm against hand-worked values,
exhaustive rounding and finite differences (CPU)."""
import numpy as np
import pytest

from oracle import fp4_oracle as Q


def test_codes_by_hand():
    y = [0, 0.24, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 4.99, 5.0, 5.01, 6.0]
    want = [0, 0, 0, 1, 2, 2, 4, 4, 6, 6, 6, 7, 7]
    assert Q.e2m1_codes(np.array(y)).tolist() == want
    assert Q.e2m1_codes(-np.array(y)).tolist() == [c + 8 for c in want]
    assert Q.of_codes(np.arange(16)).tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6,
                                                  0, -.5, -1, -1.5, -2, -3, -4, -6]


def test_rounding_is_to_nearest_with_even_codes_on_ties():
    y = np.arange(0, 6 * 256 + 1) / 256
    v = Q.of_codes(Q.e2m1_codes(y))
    for yi, vi, c in zip(y, v, Q.e2m1_codes(y)):
        best = min(abs(yi - g) for g in Q.GRID)
        assert abs(yi - vi) == best
        if sum(abs(yi - g) == best for g in Q.GRID) == 2:
            assert c % 2 == 0


@pytest.mark.parametrize("amax,b", [(0.0, 0), (6.0, 127), (6.0001, 128), (3.0, 126), (3.01, 127),
                                    (12.0, 128), (2.0 ** -126, 0), (np.inf, 255), (np.nan, 255),
                                    (3.3895313892515355e38, 253)])
def test_scale_byte(amax, b):
    assert Q.scale_byte(amax) == b


def test_nothing_is_clamped_and_scales_are_smallest():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 64)) * np.exp(3 * rng.standard_normal((50, 1)))
    c, b = Q.quantize(x)
    m = np.abs(x.reshape(50, 2, 32)).max(-1)
    assert (m <= 6 * Q.scale(b)).all() and (m > 6 * Q.scale(b - 1)).all()
    step = np.repeat(Q.scale(b), 32, 1) * np.array([.5, .5, .5, .5, 1, 1, 2, 2])[c & 7]
    assert (np.abs(Q.values(c, b) - x) <= step / 2 + 1e-300).all()
    assert (Q.roundtrip(Q.roundtrip(x)) == Q.roundtrip(x)).all()


def test_layouts():
    c = np.arange(64).reshape(2, 32) % 16
    assert (Q.unpack(Q.pack(c)) == c).all()
    assert Q.pack(np.array([[3, 10]])).tolist() == [[3 | 10 << 4]]
    b = np.arange(30).reshape(3, 10)
    s = Q.groups(b, rows=4)
    assert s.shape == (2, 4, 8) and s[1, 2, 1] == b[2, 9] and s[1, 2, 2] == 0 and s[0, 3].max() == 0
    assert (Q.ungroup(s, 3, 10) == b).all()


def test_a_block_that_is_not_finite_takes_its_own_rows_alone():
    x = np.ones((3, 64))
    x[1, 40] = np.nan
    v = Q.roundtrip(x)
    assert np.isnan(v[1, 32:]).all() and np.isfinite(v[1, :32]).all() and np.isfinite(v[[0, 2]]).all()


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(1)
    r, w, dy = rng.standard_normal((4, 12)), rng.standard_normal(12), rng.standard_normal((4, 12))
    eps = 0.05
    f = lambda r, w: (Q.rms_norm(r, w, eps)[0] * dy).sum()  # noqa: E731
    dx, dw = Q.rms_norm_bwd(dy, r, w, Q.rms_norm(r, w, eps)[1])
    d = 1e-6
    for i in np.ndindex(4, 12):
        e = np.zeros((4, 12))
        e[i] = d
        assert abs((f(r + e, w) - f(r - e, w)) / (2 * d) - dx[i]) < 1e-7
    for j in range(12):
        e = np.zeros(12)
        e[j] = d
        assert abs((f(r, w + e) - f(r, w - e)) / (2 * d) - dw[j]) < 1e-7


def test_norm_by_hand():
    y, rstd = Q.rms_norm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.0)
    assert np.allclose(rstd, 1 / np.sqrt(12.5)) and np.allclose(y, [[3 / 12.5 ** .5, 8 / 12.5 ** .5]])


def test_forward_by_hand():
    x = np.zeros((2, 32))
    x[0, 0], x[1, 1] = 2.0, 1.0
    w1 = np.zeros((1, 64, 32))
    w1[0, 0, 0], w1[0, 32, 0] = 1.0, 3.0  # gate 2, up 6 in column 0 of row 0
    w2 = np.zeros((1, 32, 32))
    w2[0, 5, 0] = 0.5
    s = Q.ffn_forward(x, [0, 2], w1, w2)
    h = 2 / (1 + np.exp(-2.0)) * 6  # 10.57: scale 2, 5.28 -> 6 (past the tie at 5)
    assert abs(s["h"][0, 0] - h) < 1e-12 and s["o"][0, 5] == 6.0 and s["o"][1].max() == 0
