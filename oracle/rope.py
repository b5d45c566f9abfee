"""Rotary positions in fp64 on the CPU, from the definition.

Pair j of a row at position t is the complex number a + i b; it is multiplied by mscale * exp(i t f_j) (its conjugate for
gradients).  The angle is reduced to one turn in exact rational arithmetic, so that far positions lose nothing.
"""

from fractions import Fraction

import numpy as np

# 1 / (2 pi) to 60 digits.
_TURN = Fraction("0.159154943091895335768883763372514362034459645740456448747667")


def angles(positions, freq):
    """[..., len(freq)] angles in radians within half a turn, for whole positions."""
    t = np.asarray(positions)
    out = np.empty(t.shape + (len(freq),))
    per = [Fraction(float(f)) * _TURN for f in freq]
    for at in np.ndindex(t.shape):
        for j, f in enumerate(per):
            x = int(t[at]) * f
            x -= round(x)
            out[at + (j,)] = float(x) * 2.0 * np.pi
    return out


def rotate(x, theta, rot, interleaved=False, mscale=1.0, inverse=False):
    """x [..., d] fp64 turned by theta [..., rot / 2] (broadcast over the axes ahead)."""
    y = np.array(x, dtype=np.float64, copy=True)
    lo, hi = (np.s_[..., 0:rot:2], np.s_[..., 1:rot:2]) if interleaved else (np.s_[..., :rot // 2], np.s_[..., rot // 2:rot])
    z = (x[lo] + 1j * x[hi]) * (mscale * np.exp((-1j if inverse else 1j) * theta))
    y[lo], y[hi] = z.real, z.imag
    return y
