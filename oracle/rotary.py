"""Norm and rotary positions of heads by definition, in fp64."""
from __future__ import annotations

import numpy as np


def turn(x, position, inv_freq, neighbours=False, factor=1.0, eps=None, gain=None):
    """x [D] of one head at position (one number for each frequency) -> y [D]."""
    x = np.asarray(x, np.float64)
    if eps is not None:
        x = x / np.sqrt((x * x).mean() + eps) * (1.0 if gain is None else np.asarray(gain, np.float64))
    y, half = x.copy(), len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if neighbours else (i, i + half)
        # whole turns drop out in extended precision where the platform has it; the positions of the tests need no more than fp64
        angle = float(position[i]) * float(inv_freq[i])
        c, s = factor * np.cos(angle), factor * np.sin(angle)
        y[a], y[b] = x[a] * c - x[b] * s, x[b] * c + x[a] * s
    return y
