"""Rotary positions in double precision, from the definition.

TEST INFRASTRUCTURE ONLY (see the package docstring): the library never
imports this module.

Pins: tests/test_rope.py (complex numbers, the inverse, distances that alone
matter to a product of rotated vectors).
"""
import numpy as np


def rotate(x, freqs, axis, positions, interleaved=False, inverse=False):
    """x [..., T, d] with pair i of its columns turned by freqs[i] * positions[axis[i], t] (positions [axes, T], or
    [axes, B, T] for x [B, H, T, d]); the columns behind the pairs as they are."""
    x = np.asarray(x, np.float64)
    positions = np.asarray(positions)
    y = x.copy()
    n = len(freqs)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        # whole turns off in extended precision: positions reach 2^31
        turns = np.longdouble(freqs[i]) / (2 * np.longdouble(np.pi) + np.longdouble(2.4492935982947064e-16)) * positions[axis[i]]
        angle = ((turns - np.round(turns)) * (2 * np.longdouble(np.pi))).astype(np.float64)
        if angle.ndim == 2:
            angle = angle[:, None]                       # over the heads
        c, s = np.cos(angle), np.sin(angle) * (-1.0 if inverse else 1.0)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y
