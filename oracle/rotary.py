"""Plain CPU oracle of rotary positions (float64 numpy).

TEST INFRASTRUCTURE ONLY: the CUDA library never uses it.

x [N, H, D], positions [N], inv_freq [rot/2] (its values as they are): pairs of
the first rot values as complex numbers times scale exp(+-i position inv_freq).
The product position * inv_freq is reduced modulo 2 pi in extended precision
where numpy has one, else in 64 bits.
"""
from __future__ import annotations

import numpy as np


def turn(x, positions, inv_freq, interleaved=False, scale=1.0, inverse=False):
    x = np.asarray(x, np.float64)
    f = np.asarray(inv_freq, np.float64)
    rot = 2 * f.size
    ang = np.asarray(positions, np.longdouble)[:, None] * f.astype(np.longdouble)[None]
    w = scale * np.exp((-1j if inverse else 1j) * np.asarray(ang % (2 * np.longdouble(np.pi)), np.float64))[:, None]
    y = x.copy()
    if interleaved:
        z = (x[..., 0:rot:2] + 1j * x[..., 1:rot:2]) * w
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = (x[..., :rot // 2] + 1j * x[..., rot // 2:rot]) * w
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y
