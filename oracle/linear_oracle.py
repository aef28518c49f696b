"""Float64 oracle of the 8-bit operators of linear layers (include/muon_linear.h)."""

from __future__ import annotations

import numpy as np

BLOCK = 128


def _poisoned(x):
    return ~np.isfinite(x).all(axis=-1)


def nearest(x):
    """The nearest integers, ties to the even one."""
    return np.rint(x)


def row_codes(x):
    """(codes, scales) of the rows of x: scale = max|row| / 127, code = nearest(127 x / max|row|)."""
    x = np.asarray(x, np.float64)
    bad = _poisoned(x)
    x = np.where(bad[:, None], 0.0, x)
    top = np.abs(x).max(axis=1, initial=0.0)
    codes = nearest(127.0 * x / np.where(top > 0, top, 1.0)[:, None])
    return codes, np.where(bad, np.nan, top / 127.0)


def block_codes(x):
    """(codes, scales) of the blocks of 128 columns: the smallest power of two 2^e, -126 <= e <= 121,
    with max|block| <= 127 2^e where there is one."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    groups = -(-cols // BLOCK)
    padded = np.zeros((rows, groups * BLOCK))
    padded[:, :cols] = x
    blocks = padded.reshape(rows, groups, BLOCK)
    bad = _poisoned(blocks)
    blocks = np.where(bad[..., None], 0.0, blocks)
    top = np.abs(blocks).max(axis=2, initial=0.0)
    powers = 2.0 ** np.arange(-126, 122)
    scale = powers[np.minimum((top[..., None] > 127.0 * powers).sum(axis=-1), len(powers) - 1)]
    codes = np.clip(nearest(blocks / scale[..., None]), -127, 127)
    return codes.reshape(rows, groups * BLOCK)[:, :cols], np.where(bad, np.nan, scale)


def decode(codes, scale, block):
    """The values that codes stand for."""
    codes, scale = np.asarray(codes, np.float64), np.asarray(scale, np.float64)
    if not block:
        return codes * scale.reshape(-1, 1)
    return codes * np.repeat(scale, BLOCK, axis=1)[:, :codes.shape[1]]


def product(a, b):
    """out = a b^T of (codes, scales) by row."""
    (qa, sa), (qb, sb) = a, b
    return (qa @ qb.T) * sa[:, None] * sb[None, :]


def weight_grad(dy, codes, scale):
    """(dy^T x, the sum of the terms' magnitudes) of a checkpoint's codes and scales."""
    x = decode(codes, scale, True)
    dy = np.asarray(dy, np.float64)
    return dy.T @ x, np.abs(dy).T @ np.abs(x)
