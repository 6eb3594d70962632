"""fp64 CPU oracle of the operators around the attention: rotary positions, the norm of each head of
q and k with the rotation, and the matrix product with its epilogue.  TEST INFRASTRUCTURE ONLY (see
opr_oracle).  Every function evaluates the definition with numpy in float64; the gradients are
written out by hand and pinned against differences by the tests.
"""

from __future__ import annotations

import math

import numpy as np


def frequencies(rot_dim, base, rule="plain", factor=1.0, length=0.0, low_turns=1.0, high_turns=32.0):
    """(frequency of each pair in radians per position, factor on the rotated values)."""
    out, scale = [], 1.0
    for j in range(rot_dim // 2):
        f = base ** (-2.0 * j / rot_dim)
        if rule == "linear":
            f = f / factor
        elif rule == "ntk":
            f = (base * factor ** (rot_dim / (rot_dim - 2.0))) ** (-2.0 * j / rot_dim)
        elif rule == "yarn":
            def where(turns):  # the (real) pair index that makes `turns` turns over the original length
                return rot_dim * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo = max(math.floor(where(high_turns)), 0)
            hi = min(math.ceil(where(low_turns)), rot_dim - 1)
            ramp = min(max((j - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            f = f * (1 - ramp) + f / factor * ramp
            scale = 0.1 * math.log(factor) + 1.0
        elif rule == "wavelength":
            wavelength = 2 * math.pi / f
            if wavelength > length / low_turns:
                f = f / factor
            elif wavelength >= length / high_turns:
                t = (length / wavelength - low_turns) / (high_turns - low_turns)
                f = (1 - t) * f / factor + t * f
        out.append(f)
    return np.array(out), scale


def pair_indices(rot_dim, interleaved):
    j = np.arange(rot_dim // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rot_dim // 2)


def rotate(x, pos, freq, interleaved=False, scale=1.0, inverse=False):
    """x [tokens, heads, d] with its first 2 len(freq) entries rotated by pos * freq."""
    ia, ib = pair_indices(2 * len(freq), interleaved)
    angle = np.asarray(pos, dtype=np.float64)[:, None, None] * freq
    c, s = scale * np.cos(angle), scale * np.sin(angle)
    if inverse:
        s = -s
    y = np.array(x, dtype=np.float64)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia] = a * c - b * s
    y[..., ib] = a * s + b * c
    return y


def norm(x, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def norm_rotate(x, w, pos, freq, eps, interleaved=False, scale=1.0):
    return rotate(norm(x, eps) * w, pos, freq, interleaved, scale)


def norm_rotate_bwd(dy, x, w, pos, freq, eps, interleaved=False, scale=1.0):
    """(dx, dw): with g the gradient before the rotation, xh the normed head and u = g w,
    dw = sum g xh and dx = (u - xh mean(u xh)) / sqrt(mean(x^2) + eps)."""
    g = rotate(dy, pos, freq, interleaved, scale, inverse=True)
    xh = norm(x, eps)
    u = g * w
    dx = (u - xh * (u * xh).mean(-1, keepdims=True)) / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return dx, (g * xh).sum((0, 1))


def _phi(z):
    """Distribution function of the normal law."""
    return 0.5 * (1.0 + np.vectorize(math.erf)(z / math.sqrt(2.0))) if z.size else z.copy()


_C = math.sqrt(2.0 / math.pi)


def act(z, name):
    if name == "silu":
        return z / (1.0 + np.exp(-z))
    if name == "gelu":
        return z * _phi(z)
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(_C * (z + 0.044715 * z ** 3)))
    return z


def act_slope(z, name):
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s + z * s * (1.0 - s)
    if name == "gelu":
        return _phi(z) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        t = np.tanh(_C * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _C * (1.0 + 3 * 0.044715 * z * z)
    return np.ones_like(z)


def linear(x, w, bias=None, activation=None, residual=None):
    """(y, z): z = x w^T + bias, y = act(z) + residual."""
    z = x @ w.T
    if bias is not None:
        z = z + bias
    y = act(z, activation)
    return (y if residual is None else y + residual), z


def linear_bwd(dy, x, w, z=None, activation=None, dx_residual=None):
    """(dx, dw, db, dz)."""
    dz = dy if activation is None else dy * act_slope(z, activation)
    dx = dz @ w
    return (dx if dx_residual is None else dx + dx_residual), dz.T @ x, dz.sum(0), dz
