"""fp64 oracle of the query/key norm with rotation and of its gradients.

For a head row x at position t with weight w:
    r = 1 / sqrt(mean(x^2) + eps),  u = r x w,  y = R(a_t) u
with R the rotation of the pairs (i, i + D/2); the angle's cosine and sine come
from a given [rows, D/2, 2] table (a value the caller holds), or from
oracle.rope_ref's angles.
"""
import numpy as np


def rotate(u, table, inverse=False):
    """u [..., tokens, heads, D] by table [tokens, D/2, 2]."""
    c, s = table[:, None, :, 0], table[:, None, :, 1]
    s = -s if inverse else s
    a, b = np.split(u, 2, axis=-1)
    return np.concatenate((a * c - b * s, a * s + b * c), axis=-1)


def norm(x, w, eps):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return r * x * w


def norm_rope(x, w, table, eps):
    """w None: rotation only."""
    return rotate(x if w is None else norm(x, w, eps), table)


def norm_rope_bwd(x, w, table, dy, eps):
    """(dx, dw) and the magnitudes the fp32 kernel's error bound is stated in:
    the sums of absolute terms of dx and of dw."""
    D = x.shape[-1]
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    du = rotate(dy, table, inverse=True)
    g = du * w
    axes = tuple(range(x.ndim - 1))
    dw = (du * r * x).sum(axes)
    dx = r * (g - r * r * x * (g * x).sum(-1, keepdims=True) / D)
    a, b = np.split(np.abs(dy), 2, axis=-1)
    du_abs = np.concatenate((a + b, a + b), axis=-1)
    g_abs = du_abs * np.abs(w)
    dx_abs = r * (g_abs + r * r * np.abs(x) * (g_abs * np.abs(x)).sum(-1, keepdims=True) / D)
    dw_abs = (du_abs * np.abs(r * x)).sum(axes)
    return dx, dw, dx_abs, dw_abs
