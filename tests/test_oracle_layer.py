"""Pins of the fp64 oracle of the operators around the attention: closed forms, invariants, and every
gradient against central differences."""

import math

import numpy as np
import pytest

import block_sparse_masked_segment_b200 as opr
from oracle import layer_oracle as lo
from oracle import opr_oracle as orc


def central(f, x, dy, h=1e-6):
    """Gradient of sum(f(x) dy) by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, dn = x.copy(), x.copy()
        up[i] += h
        dn[i] -= h
        g[i] = ((f(up) - f(dn)) * dy).sum() / (2 * h)
    return g


def test_rotation_is_the_known_one_for_whole_heads_in_the_half_layout():
    rng = np.random.default_rng(0)
    x, pos = rng.standard_normal((5, 3, 16)), np.array([0, 1, 7, 100000, 3])
    freq, scale = lo.frequencies(16, 1e4)
    assert scale == 1.0
    np.testing.assert_allclose(lo.rotate(x, pos, freq), orc.rope(x, pos, 1e4), atol=1e-9)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_invariants(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 2, 12))
    freq, _ = lo.frequencies(8, 100.0)
    pos = np.array([0, 3, -5, 11])
    y = lo.rotate(x, pos, freq, interleaved)
    np.testing.assert_array_equal(y[..., 8:], x[..., 8:])  # passed through
    np.testing.assert_allclose(y[0], x[0])                 # position 0
    np.testing.assert_allclose((y * y).sum(-1), (x * x).sum(-1))
    np.testing.assert_allclose(lo.rotate(y, pos, freq, interleaved, inverse=True), x)
    # a product of two rotated heads depends on the difference of their positions only
    q, k = rng.standard_normal((2, 1, 1, 8))
    dot = [(lo.rotate(q, [m + 3], freq, interleaved) * lo.rotate(k, [m], freq, interleaved)).sum() for m in (0, 9)]
    assert dot[0] == pytest.approx(dot[1], abs=1e-12)


def test_interleaved_is_the_half_layout_permuted():
    rng = np.random.default_rng(2)
    x, pos = rng.standard_normal((3, 2, 8)), np.array([1, 2, 3])
    freq, _ = lo.frequencies(8, 50.0)
    perm = np.array([0, 2, 4, 6, 1, 3, 5, 7])  # entry j of the half layout is entry perm[j] of the interleaved
    np.testing.assert_allclose(lo.rotate(x, pos, freq, True)[..., perm], lo.rotate(x[..., perm], pos, freq, False))


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients_of_norm_and_rotation_against_differences(interleaved):
    rng = np.random.default_rng(3)
    x, dy = rng.standard_normal((2, 3, 2, 6))
    w, pos = rng.standard_normal(6), np.array([0, 4, 9])
    freq, _ = lo.frequencies(4, 30.0)
    f = lambda x, w: lo.norm_rotate(x, w, pos, freq, 1e-2, interleaved, 1.3)  # noqa: E731
    dx, dw = lo.norm_rotate_bwd(dy, x, w, pos, freq, 1e-2, interleaved, 1.3)
    np.testing.assert_allclose(dx, central(lambda v: f(v, w), x, dy), atol=1e-7)
    np.testing.assert_allclose(dw, central(lambda v: f(x, v), w, dy), atol=1e-7)


@pytest.mark.parametrize("activation", [None, "silu", "gelu", "gelu_tanh"])
def test_gradients_of_the_product_against_differences(activation):
    rng = np.random.default_rng(4)
    x, w, b, r = (rng.standard_normal(s) for s in ((3, 4), (5, 4), 5, (3, 5)))
    dy, add = rng.standard_normal((3, 5)), rng.standard_normal((3, 4))
    y, z = lo.linear(x, w, b, activation, r)
    np.testing.assert_allclose(y - r, lo.act(x @ w.T + b, activation))
    dx, dw, db, _ = lo.linear_bwd(dy, x, w, z, activation, add)
    f = lambda x, w, b: lo.linear(x, w, b, activation, r)[0]  # noqa: E731
    np.testing.assert_allclose(dx - add, central(lambda v: f(v, w, b), x, dy), atol=1e-7)
    np.testing.assert_allclose(dw, central(lambda v: f(x, v, b), w, dy), atol=1e-7)
    np.testing.assert_allclose(db, central(lambda v: f(x, w, v), b, dy), atol=1e-7)


def test_frequencies_closed_forms():
    plain, _ = lo.frequencies(8, 1e4)
    np.testing.assert_allclose(plain, [1.0, 0.1, 0.01, 0.001])
    np.testing.assert_allclose(lo.frequencies(8, 1e4, "linear", 4.0)[0], plain / 4)
    # ntk: the highest frequency stays, the lowest is divided by the factor
    ntk, _ = lo.frequencies(8, 1e4, "ntk", 4.0)
    assert ntk[0] == 1.0 and ntk[-1] == pytest.approx(plain[-1] / 4)
    for rule in ("yarn", "wavelength"):
        f, scale = lo.frequencies(64, 1e4, rule, 4.0, 8192, 1.0, 32.0)
        p, _ = lo.frequencies(64, 1e4)
        assert f[0] == p[0] and f[-1] == pytest.approx(p[-1] / 4) and (np.diff(f) < 0).all()
        assert scale == (pytest.approx(0.1 * math.log(4) + 1) if rule == "yarn" else 1.0)


@pytest.mark.parametrize("rot_dim", [2, 20, 64, 128, 256])
@pytest.mark.parametrize("rule", ["plain", "linear", "ntk", "yarn", "wavelength"])
def test_library_frequencies_match_the_oracle(rule, rot_dim):
    """opr_rotary_frequencies is host code.  Both sides round a pow, a log (for yarn inside a floor and
    a ceiling, away from whole numbers here) and a few products: 1e-13 relative."""
    if rule == "ntk" and rot_dim == 2:
        with pytest.raises(opr.OprError):
            opr.opr_rotary_frequencies(rot_dim, 1e4, rule, 4.0, 8192.0, device="cpu")
        return
    for base, factor, length, low, high in ((1e4, 4.0, 8192.0, 1.0, 32.0), (1e6, 2.5, 4097.0, 1.0, 4.0)):
        f, s = opr.opr_rotary_frequencies(rot_dim, base, rule, factor, length, low, high, device="cpu")
        rf, rs = lo.frequencies(rot_dim, base, rule, factor, length, low, high)
        np.testing.assert_allclose(f.numpy(), rf, rtol=1e-13)
        assert s == pytest.approx(rs, rel=1e-14)
