"""Float64 oracle of the global gradient norm and of clipping by it."""

from __future__ import annotations

import math

import numpy as np

CLIP_EPS = 1e-6


def grad_norm(grads, kind: str = "l2") -> float:
    """Norm over all elements of a list of arrays: sqrt of the sum of squares, or the largest
    magnitude.  Values are scaled by the largest power of two first, so that no square leaves
    the range of a float64."""
    arrays = [np.asarray(g, dtype=np.float64).reshape(-1) for g in grads]
    flat = np.concatenate(arrays) if arrays else np.zeros(0)
    if np.isnan(flat).any():
        return math.nan
    top = float(np.max(np.abs(flat))) if flat.size else 0.0
    if kind == "inf" or top == 0.0 or math.isinf(top):
        return top
    scale = 2.0 ** math.frexp(top)[1]
    return scale * math.sqrt(float(np.sum(np.square(flat / scale))))


def clip_coef(norm: float, max_norm: float) -> float:
    """min(1, max_norm / (norm + 1e-6)); NaN for a NaN norm."""
    if math.isnan(norm):
        return math.nan
    return min(1.0, max_norm / (norm + CLIP_EPS))


def clip_grads(grads, norm: float, max_norm: float):
    c = clip_coef(norm, max_norm)
    with np.errstate(invalid="ignore"):
        return [np.asarray(g, dtype=np.float64) * c for g in grads]
