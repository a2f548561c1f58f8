"""Float64 (numpy) root-mean-square norm, 8-bit values with a scale for each block of 128, their product, and clipping,
with the magnitudes that rounding errors scale with. Independent of the CUDA library.

e4m3: sign, 4 bits of exponent (bias 7), 3 of significand; subnormals of step 2^-9; largest 448; no infinities, NaN at the
exponent's and significand's highest values.
"""
import numpy as np

BLOCK = 128
TOP = 448.0


def rms_norm_fwd(x, r, w, eps):
    """(y, rstd) of x + r (r already rounded into x, or None)."""
    h = x if r is None else x + r
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    y = h * rstd[:, None]
    return (y if w is None else y * w), rstd


def rms_norm_bwd(dy, h, w, dh, eps):
    """(dx, dweight)."""
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    hhat = h * rstd[:, None]
    g = dy if w is None else dy * w
    dx = rstd[:, None] * (g - hhat * (g * hhat).mean(1, keepdims=True))
    return (dx if dh is None else dx + dh), (dy * hhat).sum(0)


def step(v):
    """The distance of neighbouring e4m3 values around |v| (up to 448)."""
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    return 2.0 ** (np.minimum(e, 8) - 3)


def round_e4m3(v):
    """The nearest e4m3 value, ties to the even significand, saturated."""
    s = step(v)
    return np.clip(np.rint(v / s) * s, -TOP, TOP)


def block_max(x, block_rows):
    """[rows / block_rows, cols / 128]: the largest magnitude of each block."""
    rows, cols = x.shape
    up, across = -(-rows // block_rows), -(-cols // BLOCK)
    wide = np.zeros((up * block_rows, across * BLOCK))
    wide[:rows, :cols] = np.abs(x)
    return wide.reshape(up, block_rows, across, BLOCK).max((1, 3), initial=0.0)


def scales(x, block_rows):
    s = block_max(x, block_rows) / TOP
    return np.where(s < 2.0 ** -126, 1.0, s)


def spread(scale, shape):
    """A scale for each element."""
    rows, cols = shape
    block_rows = 1 if scale.shape[0] == rows else BLOCK
    return np.repeat(np.repeat(scale, block_rows, 0)[:rows], BLOCK, 1)[:, :cols]


def quantize(x, block_rows):
    s = scales(x, block_rows)
    return round_e4m3(x / spread(s, x.shape)), s


def matmul(qa, sa, qb, sb):
    """(a b^T, sum of the magnitudes of its terms)."""
    a, b = qa * spread(sa, qa.shape), qb * spread(sb, qb.shape)
    return a @ b.T, np.abs(a) @ np.abs(b).T


def clip(grads, max_norm, eps):
    norm = np.sqrt(sum((g * g).sum() for g in grads))
    return norm, [g * min(1.0, max_norm / (norm + eps)) for g in grads]
