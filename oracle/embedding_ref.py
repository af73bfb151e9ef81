"""Float64 oracle of the embedding lookup and its gradient (test infrastructure; numpy on the
CPU, written from the definitions in ``include/nsmuon.h``)."""

from __future__ import annotations

import numpy as np


def embedding(weight, tokens, scale=1.0):
    weight = np.asarray(weight, dtype=np.float64)
    out = np.zeros((len(tokens), weight.shape[1]))
    for r, t in enumerate(tokens):
        if 0 <= t < len(weight):
            out[r] = scale * weight[t]
    return out


def embedding_backward(d_out, tokens, vocab, scale=1.0, old=None):
    """(gradient, the sum of the sizes of what was added, rows that were added to each)"""
    d_out = np.asarray(d_out, dtype=np.float64)
    grad, size, count = np.zeros((vocab, d_out.shape[1])), np.zeros((vocab, d_out.shape[1])), np.zeros(vocab, dtype=np.int64)
    for r, t in enumerate(tokens):
        if 0 <= t < vocab:
            grad[t] += scale * d_out[r]
            size[t] += abs(scale) * np.abs(d_out[r])
            count[t] += 1
    if old is not None:
        grad, size = grad + old, size + np.abs(old)
    return grad, size, count
