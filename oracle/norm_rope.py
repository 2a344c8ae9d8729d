"""CPU oracle of the per-head RMS norm with the position rotation and its backward:
float64 numpy, in the definition's own terms."""
from __future__ import annotations

import numpy as np


def _pairs(rot: int, interleaved: bool):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(y, cos, sin, interleaved: bool):
    """z_a = y_a c - y_b s, z_b = y_b c + y_a s on the first 2 len(cos) elements of the
    last axis; cos and sin broadcast against the pairs."""
    a, b = _pairs(2 * cos.shape[-1], interleaved)
    z = np.array(y, dtype=np.float64)
    z[..., a] = y[..., a] * cos - y[..., b] * sin
    z[..., b] = y[..., b] * cos + y[..., a] * sin
    return z


def _angles(cos_sin, positions):
    half = cos_sin.shape[1] // 2
    rows = np.asarray(cos_sin, dtype=np.float64)[positions]
    return rows[:, None, :half], rows[:, None, half:]


def norm_rope_fwd(x, w, cos_sin, positions, eps, interleaved, out):
    """Rows of x [rows, heads, d] into a copy of ``out``; rows whose position is negative
    or past the table keep out's. ``w`` None: ones."""
    x = np.asarray(x, dtype=np.float64)
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, dtype=np.float64)
    out = np.array(out, dtype=np.float64)
    live = (positions >= 0) & (positions < cos_sin.shape[0])
    xl = x[live]
    y = xl / np.sqrt(np.mean(xl * xl, axis=-1, keepdims=True) + eps) * w
    out[live] = rotate(y, *_angles(cos_sin, positions[live]), interleaved)
    return out


def norm_rope_bwd(x, dz, w, cos_sin, positions, eps, interleaved, dx_out):
    """(dx, dw) of :func:`norm_rope_fwd` for the upstream gradient dz."""
    x, dz = np.asarray(x, dtype=np.float64), np.asarray(dz, dtype=np.float64)
    d = x.shape[-1]
    w = np.ones(d) if w is None else np.asarray(w, dtype=np.float64)
    dx = np.array(dx_out, dtype=np.float64)
    live = (positions >= 0) & (positions < cos_sin.shape[0])
    xl = x[live]
    cos, sin = _angles(cos_sin, positions[live])
    g = rotate(dz[live], cos, -sin, interleaved)   # the transpose of a rotation turns back
    r = 1.0 / np.sqrt(np.mean(xl * xl, axis=-1, keepdims=True) + eps)
    # d/dx_e of x_f r w_f: r w_f (e == f) - x_f w_f r^3 x_e / d
    dx[live] = g * w * r - xl * r ** 3 / d * np.sum(g * w * xl, axis=-1, keepdims=True)
    return dx, np.sum(g * xl * r, axis=(0, 1))
