"""The oracle of the 8-bit experts against brute force: every e4m3 value, the
rounding at and beside ties, the scale rule at its borders, and the gradient
stages against central differences."""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as O


def e4m3_values():
    """All finite e4m3 values from the format's definition."""
    out = set()
    for e in range(16):
        for m in range(8):
            if e == 15 and m == 7:
                continue  # NaN
            v = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
            out |= {v, -v}
    return np.array(sorted(out))


def test_e4m3_is_the_nearest_value_ties_to_even():
    v = e4m3_values()
    assert v.max() == 448 and np.abs(v[v != 0]).min() == 2.0 ** -9
    assert np.array_equal(O.e4m3(v), v)
    mid = (v[1:] + v[:-1]) / 2
    even = {float(x): i for i, x in enumerate(v[v >= 0])}
    for lo, hi, m in zip(v[:-1], v[1:], mid):
        want = lo if even[abs(lo)] % 2 == 0 else hi
        assert O.e4m3(m) == want, m
        assert O.e4m3(np.nextafter(m, lo)) == lo and O.e4m3(np.nextafter(m, hi)) == hi


def test_bf16_agrees_with_torch():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(4000) * 10.0 ** rng.uniform(-42, 38, 4000),
                        [0, -0.0, 3.4e38, -3.4e38, 2.0 ** -134, 1.5 * 2.0 ** -133, np.inf]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    assert np.array_equal(O.bf16(x), want)


@pytest.mark.parametrize("exp", [-140, -119, -118, -20, 0, 1, 100, 119])
def test_scale_is_the_smallest_that_does_not_clamp(exp):
    top = np.ldexp(448.0, exp)
    for amax, want in ((top, exp + 127), (np.nextafter(top, np.inf), exp + 128),
                       (np.nextafter(top, 0), exp + 127)):
        assert O.scale_byte(amax) == max(want, 0)
    assert O.scale_byte(0.0) == 0
    assert O.scale_byte(np.inf) == 255 and O.scale_byte(np.nan) == 255


def test_rows_blocks_and_words():
    rng = np.random.default_rng(2)
    x = O.bf16(rng.standard_normal((5, 320)) * 2.0 ** rng.integers(-20, 20, (5, 1)))
    x[1, 130] = np.inf
    x[2, :128] = 0
    q, b = O.quantize_rows(x)
    assert b.shape == (5, 3) and b[1, 1] == 255 and b[2, 0] == 0
    assert np.isnan(q[1, 128:256]).all() and np.isfinite(np.delete(q, 1, 0)).all()
    v = O.values_rows(q, b)
    fin = np.isfinite(v)
    # half a step of a 4-bit significand, or of the smallest step under the block's scale
    tol = np.maximum(2.0 ** -4 * np.abs(x), np.repeat(np.ldexp(1.0, b - 137), 128, 1)[:, :320])
    assert (np.abs(v - x)[fin] <= tol[fin]).all()
    words = np.zeros((1, 5, 4), np.int64)
    words[0, :, :3] = b
    assert np.array_equal(O.unpack_words(words, 3), b)


def test_weights_share_a_scale_in_each_block():
    rng = np.random.default_rng(3)
    w = O.bf16(rng.standard_normal((2, 192, 320)))
    w[0, :128, :128] *= 64
    q, b = O.quantize_weights(w)
    assert b.shape == (2, 2, 3)
    for m in range(2):
        for i in range(2):
            for j in range(3):
                blk = w[m, 128 * i:128 * i + 128, 128 * j:128 * j + 128]
                assert b[m, i, j] == O.scale_byte(np.abs(blk).max())
    qt, bt = O.quantize_weights(np.swapaxes(w, 1, 2))  # one quantisation serves both directions
    assert np.array_equal(np.swapaxes(qt, 1, 2), q) and np.array_equal(np.swapaxes(bt, 1, 2), b)


def test_gradient_stages_against_differences():
    """sum(d_o * o) moved by each x and by each a, central differences in float64."""
    rng = np.random.default_rng(4)
    E, H, F = 3, 6, 4
    off = np.array([0, 2, 2, 5])
    x, d_o = rng.standard_normal((5, H)), rng.standard_normal((5, H))
    w1, w2 = rng.standard_normal((E, 2 * F, H)), rng.standard_normal((E, H, F))
    f = O.ffn_forward(x, off, w1, w2, round16=O.identity)
    g = O.ffn_dgrad(d_o, f["a"], off, w1, w2, round16=O.identity)
    eps = 1e-6

    def loss_x(x):
        return (O.ffn_forward(x, off, w1, w2, round16=O.identity)["o"] * d_o).sum()

    def loss_a(a):
        return (O.grouped(O.swiglu(a), off, w2) * d_o).sum()

    for fn, at, grad in ((loss_x, x, g["dx_perm"]), (loss_a, f["a"], g["da"])):
        for i in np.ndindex(at.shape):
            up, dn = at.copy(), at.copy()
            up[i] += eps
            dn[i] -= eps
            assert abs((fn(up) - fn(dn)) / (2 * eps) - grad[i]) < 1e-7 * (1 + abs(grad[i]))
