"""CPU model of qk_norm_rope and its gradient: float64, one row at a time as the formulas say.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  A head's row x is normed, y = x w / sqrt(mean(x^2) + eps), and
its pair i turned by pos * f_i: the pair read as a complex number is multiplied by exp(i pos f_i).  The gradient of the
norm is written with its Jacobian, dx_c = sum_e dy_e w_e (delta_ec / s - x_e x_c / (D s^3)), s = sqrt(mean(x^2) + eps).
"""
from __future__ import annotations

import numpy as np


def pairs(rot, interleaved):
    """Channel numbers [rot / 2, 2] of the pairs."""
    n = rot // 2
    i = np.arange(n)
    return np.stack([2 * i, 2 * i + 1], -1) if interleaved else np.stack([i, i + n], -1)


def turn(x, angle, rot, interleaved):
    """Rows x [..., D] with pair i turned by angle [..., rot / 2]."""
    p = pairs(rot, interleaved)
    out = np.array(x, dtype=np.float64)
    z = (out[..., p[:, 0]] + 1j * out[..., p[:, 1]]) * np.exp(1j * angle)
    out[..., p[:, 0]], out[..., p[:, 1]] = z.real, z.imag
    return out


def angles(pos, inv_freq, axis):
    """[B, T, rot / 2] from positions [axes, B, T]."""
    pos = np.asarray(pos, dtype=np.float64)
    if not len(inv_freq):
        return np.zeros(pos.shape[1:] + (0,))
    return np.stack([pos[a] * f for a, f in zip(axis, inv_freq)], -1)


def forward(x, w, eps, angle, interleaved):
    """x [B, T, H, D] -> [B, H, T, D]; w [D] or None."""
    x = np.asarray(x, dtype=np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)
    return turn(x, angle[:, :, None], 2 * angle.shape[-1], interleaved).transpose(0, 2, 1, 3)


def backward(d, x, w, eps, angle, interleaved):
    """d [B, H, T, D], x [B, T, H, D] -> gradient of x, gradient of w (or None)."""
    d = turn(np.asarray(d, dtype=np.float64).transpose(0, 2, 1, 3), -angle[:, :, None], 2 * angle.shape[-1], interleaved)
    if w is None:
        return d, None
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    D = x.shape[-1]
    s = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dw = (d * x / s).sum((0, 1, 2))
    dy = d * w
    jac = np.eye(D) / s[..., None] - x[..., :, None] * x[..., None, :] / (D * s[..., None] ** 3)
    return np.einsum("...e,...ec->...c", dy, jac), dw
