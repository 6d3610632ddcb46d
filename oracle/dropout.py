"""Counter-based dropout (oracle side).

TEST INFRASTRUCTURE: see oracle/__init__.py for who may use this module.

Element e (row-major) of the tensor takes its 16 random bits u from Philox
call e >> 3 with third counter word 2 (philox.sr_bits' layout, whose
orientations 0 and 1 are the stochastic rounding's); with t = p * 65536 rounded
to the nearest integer, ties to even, it is kept iff u >= t and scaled by
fp32(65536 / (65536 - t)).
"""

import numpy as np

from . import philox

STREAM = 2


def threshold(p):
    return int(np.rint(65536.0 * p))


def keep(shape, p, seed, offset, rows=None):
    """The mask of a (rows, cols) tensor (or of its sampled rows)."""
    return philox.sr_bits(seed, offset, STREAM, *shape, rows=rows) >= threshold(p)


def dropout(x, mask, p, residual=None):
    """fp32 result before the rounding to the output's type (x, residual fp32)."""
    t = threshold(p)
    scale = np.float32(0.0) if t == 65536 else np.float32(65536.0 / (65536 - t))
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.where(mask, (x * scale).astype(np.float32), np.float32(0.0))
        return y if residual is None else (residual + y).astype(np.float32)
