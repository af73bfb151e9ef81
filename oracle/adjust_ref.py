"""Float64 oracle of the penalties, biases and grammar masks on logits (test infrastructure;
numpy on the CPU, one row at a time, written from the definitions in ``include/nsmuon.h``)."""

from __future__ import annotations

import numpy as np


def _counts(vocab, history, row, length, history_row):
    """How often each token occurs in the row's history."""
    counts = np.zeros(vocab, dtype=np.int64)
    if history is None:
        return counts
    line = row if history_row is None else int(history_row[row])
    if not 0 <= line < len(history):
        return counts
    n = history.shape[1] if length is None else min(max(int(length[row]), 0), history.shape[1])
    for token in history[line, :n]:
        if 0 <= token < vocab:
            counts[token] += 1
    return counts


def _allowed(vocab, mask, row, mask_row):
    if mask is None:
        return np.ones(vocab, dtype=bool)
    line = row if mask_row is None else int(mask_row[row])
    if not 0 <= line < len(mask):
        return np.ones(vocab, dtype=bool)
    v = np.arange(vocab)
    return (mask[line][v // 32].astype(np.int64) >> (v % 32)) & 1 == 1


def _at(values, row, default):
    return default if values is None else float(values[row])


def adjust(x, history=None, length=None, history_row=None, repetition=None, frequency=None, presence=None,
           bias_index=None, bias=None, mask=None, mask_row=None):
    """(the adjusted logits, the sum of what was added to each: the size its rounding errors have)."""
    x = np.asarray(x, dtype=np.float64)
    rows, vocab = x.shape
    out, size = x.copy(), np.abs(x)
    with np.errstate(invalid="ignore", over="ignore"):
        for r in range(rows):
            counts = _counts(vocab, history, r, length, history_row)
            theta, f, p = _at(repetition, r, 1.0), _at(frequency, r, 0.0), _at(presence, r, 0.0)
            for v in np.nonzero(counts)[0]:
                a = x[r, v] / theta if x[r, v] > 0 else x[r, v] * theta
                out[r, v] = a - (f * counts[v] + p)
                size[r, v] = abs(a) + abs(f) * counts[v] + abs(p)
            if bias is not None:
                for v, b in zip(bias_index[r], bias[r]):
                    if 0 <= v < vocab:
                        out[r, v] += b
                        size[r, v] += abs(b)
            out[r, ~_allowed(vocab, mask, r, mask_row)] = -np.inf
    return out, size


def adjust_backward(x, d_out, history=None, length=None, history_row=None, repetition=None, mask=None, mask_row=None):
    grad = np.asarray(d_out, dtype=np.float64).copy()
    rows, vocab = grad.shape
    for r in range(rows):
        if repetition is not None:
            theta = float(repetition[r])
            for v in np.nonzero(_counts(vocab, history, r, length, history_row))[0]:
                grad[r, v] *= 1 / theta if x[r, v] > 0 else theta
        grad[r, ~_allowed(vocab, mask, r, mask_row)] = 0.0
    return grad
