"""fp64 CPU oracle for the norms with positions: rows normalised, pairs of their
columns rotated, and the gradients by the formulas.

TEST INFRASTRUCTURE ONLY.  Imported by ``tests/``; the product library never
imports or calls it and shares no code with it.  Plain numpy in float64; the
angles of far positions are reduced in numpy's longest type first.
"""
from __future__ import annotations

import numpy as np

_TWO_PI = 2 * np.longdouble("3.14159265358979323846264338327950288")


def angles(pos, freq):
    """theta [..., n] of coordinates [axes, ...] and frequencies [axes, n]."""
    pos, freq = np.asarray(pos, dtype=np.longdouble), np.asarray(freq, dtype=np.longdouble)
    return np.fmod(np.tensordot(pos, freq, (0, 0)), _TWO_PI).astype(np.float64)


def columns(n, first, halves):
    """Columns (u, v) of the n pairs."""
    p = np.arange(n)
    return (first + p, first + n + p) if halves else (first + 2 * p, first + 2 * p + 1)


def rotate(y, theta, first, halves):
    """y [..., D] with its pairs turned by theta [..., n]."""
    u, v = columns(theta.shape[-1], first, halves)
    o = np.array(y, dtype=np.float64)
    c, s = np.cos(theta), np.sin(theta)
    o[..., u] = y[..., u] * c - y[..., v] * s
    o[..., v] = y[..., u] * s + y[..., v] * c
    return o


def norm(x, w, eps):
    x = np.asarray(x, dtype=np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return y if w is None else y * np.asarray(w, dtype=np.float64)


def forward(x, w, eps, theta, first, halves):
    return rotate(norm(x, w, eps), theta, first, halves)


def backward(x, w, eps, theta, first, halves, g):
    """(dx, dw) for the cotangent g; dw summed over all rows."""
    x = np.asarray(x, dtype=np.float64)
    g = rotate(np.asarray(g, dtype=np.float64), -theta, first, halves)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h = g if w is None else g * np.asarray(w, dtype=np.float64)
    dx = r * (h - x * r * r * (h * x).mean(-1, keepdims=True))
    return dx, (g * x * r).reshape(-1, x.shape[-1]).sum(0)


# ---------------------------------------------------------------------------
# bounds of the fp32 arithmetic, elementwise.  A unit is 2^-24, the rounding of an
# fp32 operation.  cos and sin, 3 units:
#   the phase, in turns: a frequency is cut off below 2^-64, so each of up to four axes
#   is off by 2^-33, and what is left of a quarter turn is cut off below 2^-34: together
#   0.06 units of radians;
#   the rest in radians, pi/4 at most: rounded to fp32, times 2 pi 2^-34 as an fp32 number
#   (off by 0.47 units) and rounded: 2.47 pi/4 = 1.94 units, 2 with the phase's.  Of that
#   sin(pi/4) reaches cos, 1.42 units, and 2.47 x cos x + 0.06 sin, 1.43;
#   the series end at x^8 and x^9: x^10/10! = 0.41 units, x^11/11! = 0.03;
#   their evaluation: the last addition 0.5 (results from 0.5 to 1), and before it x^2,
#   the inner sum and for sin x^3, 0.48 units for cos and 0.26 for sin:
#   cos 2.81, sin 2.22.
# r: the sum of D squares D units at most, halved by the root, and 3 for the root
# itself.  A result u cos - v sin: r's and two roundings of u and v, 3 of cos and
# sin and 2 of the sum: D/2 + 10 units of |u| + |v|.
# ---------------------------------------------------------------------------
UNIT = 2.0 ** -24


def rotated_magnitude(y, theta, first, halves):
    """|u| + |v| at the columns of pairs, |y| elsewhere."""
    u, v = columns(theta.shape[-1], first, halves)
    a = np.abs(y)
    m = a.copy()
    m[..., u] = a[..., u] + a[..., v]
    m[..., v] = a[..., u] + a[..., v]
    return m


def forward_bound(x, w, eps, theta, first, halves):
    """Of |out - forward| before the rounding to the type."""
    return (x.shape[-1] / 2 + 10) * UNIT * rotated_magnitude(norm(x, w, eps), theta, first, halves)


def rotate_bound(x, theta, first, halves):
    return 6 * UNIT * rotated_magnitude(np.asarray(x, dtype=np.float64), theta, first, halves)


def backward_bound(x, w, eps, theta, first, halves, g):
    """Of |dx - backward| and |dw - backward| before the rounding to the type.
    g' is off by 6 units of |u| + |v| of its pair, h by 7; the mean of h x by D + 8
    units of the mean of |h x|; x r^2 times it by 2 (D/2 + 3) + 3 more; the last
    difference and product by 3 with r's D/2 + 3.  dw: a term by 6 + D/2 + 5, and
    the sum over n rows by n units of the sum of magnitudes."""
    x = np.asarray(x, dtype=np.float64)
    D = x.shape[-1]
    gm = rotated_magnitude(np.asarray(g, dtype=np.float64), theta, first, halves)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    hm = gm if w is None else gm * np.abs(np.asarray(w, dtype=np.float64))
    dx = r * (hm * (D / 2 + 13) + np.abs(x) * r * r * (hm * np.abs(x)).mean(-1, keepdims=True) * (2.5 * D + 23)) * UNIT
    terms = (gm * np.abs(x) * r).reshape(-1, D)
    return dx, terms.sum(0) * (D / 2 + 11 + len(terms)) * UNIT
