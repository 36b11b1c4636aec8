"""The fp64 reference of the 4-bit microscaled layers, pinned against brute force and closed forms."""
import numpy as np
import pytest

from oracle import mx_ref as M


def test_values():
    assert M.E2M1[:8].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6] and (M.E2M1[8:] == -M.E2M1[:8]).all()


def test_rounding_against_all_values():
    v = np.concatenate([np.linspace(-9, 9, 1441), [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 1e300, -1e300]])
    codes = M.round_e2m1(v)
    for x, c in zip(v, codes):
        d = np.abs(M.E2M1 - np.clip(x, -6, 6))
        assert d[c] == d.min()
        near = [k for k in range(16) if d[k] == d.min() and (k >= 8) == bool(np.signbit(x))]
        assert len(near) == 1 or c % 2 == 0     # a tie goes to the even code


@pytest.mark.parametrize("scaling", ["floor", "ceil"])
def test_scales_are_the_powers_of_two_they_should_be(scaling):
    rng = np.random.default_rng(1)
    tops = np.concatenate([np.exp(20 * rng.standard_normal(200)), 2.0 ** np.arange(-30, 30), 6 * 2.0 ** np.arange(-30, 30),
                           np.nextafter(6 * 2.0 ** np.arange(-30.0, 30), np.inf)])
    for top, c in zip(tops, M.scale_codes(tops, scaling)):
        s = 2.0 ** (int(c) - 127)
        if scaling == "floor":
            assert 4 * s <= top < 8 * s
        else:
            assert top <= 6 * s and top > 3 * s
    assert M.scale_codes([0.0, 2.0 ** -140, 1e-45, np.inf, np.nan], scaling).tolist() == [1, 1, 1, 255, 255]


@pytest.mark.parametrize("scaling", ["floor", "ceil"])
def test_quantize_error_and_codes(scaling):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 96)) * np.exp(2 * rng.standard_normal((5, 1)))
    codes, s = M.ref_quantize(x, scaling)
    y = M.dequantize(codes, s)
    step = np.repeat(M.scale_values(s), 32, axis=1)
    over = np.abs(x) > 6 * step
    assert (np.abs(y) <= 6 * step).all() and (scaling == "floor" or not over.any())
    assert (np.abs(x - y)[~over] <= np.maximum(0.25 * step, np.abs(x) / 4)[~over] + 1e-12).all()
    assert (M.unpack(M.pack(codes)) == codes).all()
    x[2, 40] = np.inf
    codes, s = M.ref_quantize(x, scaling)
    assert s[2, 1] == 255 and (codes[2, 32:64] == 0).all() and np.isnan(M.dequantize(codes, s)[2, 32:64]).all()
    assert np.isfinite(M.dequantize(codes, s)[2, :32]).all()


def test_grouped_and_layer_against_loops():
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal((7, 64)), rng.standard_normal((3, 5, 64))
    y, b, written = M.ref_grouped(x, w, [1, 3, 3, 6], np.array([0, 6, 2, -1, 7, 1, 1]))
    assert written.tolist() == [False, True, True, True, True, True, False]
    assert np.allclose(y[1], w[0] @ x[6]) and np.allclose(y[5], w[2] @ x[1]) and (y[3:5] == 0).all()
    w1, w2 = rng.standard_normal((3, 64, 64)), rng.standard_normal((3, 64, 32))
    ids, p = np.array([[0, 2], [-1, 1], [3, 5], [1, 1]]), rng.random((4, 2))
    for kind in ("silu", "gelu_tanh"):
        out, size, spread = M.ref_mlp(x[:4], ids, p, w1, w2, kind, 1e-6)
        assert (out[2] == 0).all() and (size >= np.abs(out) - 1e-12).all() and (spread[[0, 1, 3]] > 0).all()
        y = w1[1] @ x[3]
        g = y[:32]
        a = g / (1 + np.exp(-g)) if kind == "silu" else 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))
        assert np.allclose(out[3], (p[3, 0] + p[3, 1]) * (w2[1] @ (a * y[32:])))


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_activation_slope_bound(kind):
    g = np.linspace(-30, 30, 600001)
    a, _ = M.activation(g, kind)
    assert np.abs(np.diff(a) / np.diff(g)).max() < 1.13
