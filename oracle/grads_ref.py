"""Float64 oracle of the norm of many gradients and of clipping (test infrastructure; numpy on
the CPU, written from the definitions in ``include/nsmuon.h``)."""

from __future__ import annotations

import numpy as np


def _norm(x):
    """The 2-norm, scaled by the largest element: squares leave no range."""
    x = np.asarray(x, dtype=np.float64).reshape(-1)
    if x.size == 0:
        return 0.0
    if np.isnan(x).any():
        return float("nan")
    most = np.max(np.abs(x))
    if most == 0 or most == np.inf:
        return float(most)
    return float(most * np.sqrt(np.sum((x / most) ** 2)))


def grad_norm(grads):
    """(norm of all, norm of each)"""
    norms = np.array([_norm(g) for g in grads])
    return _norm(norms), norms


def clip_grads(grads, max_norm):
    norm, norms = grad_norm(grads)
    factor = max_norm / norm if np.isfinite(norm) and norm > max_norm else 1.0
    return [np.asarray(g, dtype=np.float64) * factor for g in grads], norm, norms
