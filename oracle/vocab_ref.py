"""Float64 oracle of the losses over a vocabulary: log probabilities of given tokens, with
entropy and top alternatives, and distillation from a teacher's top logits (test
infrastructure; numpy on the CPU, one row at a time, written from the definitions in
``include/nsmuon.h``)."""

from __future__ import annotations

from typing import Dict, Optional

import numpy as np


def _softmax_row(y: np.ndarray, lse: Optional[float] = None):
    """(lse, q, log q) of one row; with ``lse`` given, relative to that one.  log q is taken
    from the differences to the largest y, which stay exact where y is huge."""
    top = np.max(y)
    if lse == -np.inf or (lse is None and top == -np.inf):
        return -np.inf, np.zeros_like(y), np.full_like(y, -np.inf)
    if lse is None:
        total = np.log(np.sum(np.exp(y - top)))
        lse, log_q = top + total, (y - top) - total
    else:
        log_q = y - lse
    return lse, np.exp(log_q), log_q


def _log_sum(log_q: np.ndarray) -> float:
    """log sum exp(log_q), -inf of nothing; no term underflows beside the largest."""
    top = np.max(log_q) if len(log_q) else -np.inf
    return float(top) if top == -np.inf else float(top + np.log(np.sum(np.exp(log_q - top))))


def _entropy(q: np.ndarray, log_q: np.ndarray) -> float:
    some = q > 0
    return float(-np.sum(q[some] * log_q[some]))


def logprobs(x: np.ndarray, tokens, temperature: float = 1.0, k: int = 0) -> Dict[str, np.ndarray]:
    x = np.asarray(x, dtype=np.float64)
    rows, vocab = x.shape
    out = {"logprob": np.zeros(rows), "entropy": np.zeros(rows), "lse": np.zeros(rows),
           "top_logprob": np.full((rows, k), -np.inf), "top_index": np.full((rows, k), -1, dtype=np.int32)}
    with np.errstate(invalid="ignore", divide="ignore"):
        for r in range(rows):
            y = x[r] / temperature
            if np.isnan(y).any() or np.max(y) == np.inf:
                for name in ("logprob", "entropy", "lse"):
                    out[name][r] = np.nan
                out["top_logprob"][r] = np.nan
                if tokens is None or not 0 <= tokens[r] < vocab:
                    out["logprob"][r] = 0.0
                continue
            lse, q, log_q = _softmax_row(y)
            out["lse"][r] = lse
            out["entropy"][r] = _entropy(q, log_q)
            if tokens is not None and 0 <= tokens[r] < vocab:
                out["logprob"][r] = log_q[tokens[r]]
            order = np.argsort(-x[r], kind="stable")[:k]
            order = order[x[r][order] > -np.inf]
            out["top_index"][r, :len(order)] = order
            out["top_logprob"][r, :len(order)] = log_q[order]
    return out


def logprobs_grad(x: np.ndarray, tokens, d_logprob, d_entropy, temperature: float = 1.0, lse=None,
                  entropy=None) -> np.ndarray:
    """Gradient of sum(d_logprob logprob + d_entropy entropy); from given lse and entropy the
    backward pass alone."""
    x = np.asarray(x, dtype=np.float64)
    rows, vocab = x.shape
    grad = np.zeros_like(x)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        for r in range(rows):
            has = tokens is not None and 0 <= tokens[r] < vocab
            w = float(d_logprob[r]) if d_logprob is not None and has else 0.0
            h = float(d_entropy[r]) if d_entropy is not None else 0.0
            if w == 0.0 and h == 0.0:
                continue
            y = x[r] / temperature
            if lse is None and (np.isnan(y).any() or np.max(y) == np.inf):
                grad[r] = np.nan
                continue
            given, q, log_q = _softmax_row(y, None if lse is None else float(lse[r]))
            if given == -np.inf:
                continue
            big_h = float(entropy[r]) if entropy is not None else _entropy(q, log_q)
            some = q > 0
            g = -w * q
            g[some] -= h * q[some] * (log_q[some] + big_h)
            if has and x[r, tokens[r]] != -np.inf:
                g[tokens[r]] += w
            grad[r] = g / temperature
    return grad


def _teacher(x_row, teacher_row, index_row, temperature, tail):
    """Token -> (p, log p) of the row's entries that count, and p_rest before the student's say."""
    vocab = len(x_row)
    kept = {}
    for z, v in zip(teacher_row, index_row):
        if 0 <= v < vocab and int(v) not in kept:
            kept[int(v)] = float(z)
    tokens = np.array(list(kept), dtype=np.int64)
    z = np.array([kept[int(v)] for v in tokens])
    if tail:
        p = np.exp(z)
        return tokens, p, z, max(0.0, 1.0 - float(np.sum(p))), len(tokens) > 0
    if len(tokens) == 0 or np.max(z) == -np.inf:
        return tokens, np.zeros(len(z)), np.full(len(z), -np.inf), 0.0, False
    y = z / temperature
    log_p = y - np.max(y)
    log_p = log_p - np.log(np.sum(np.exp(log_p)))
    return tokens, np.exp(log_p), log_p, 0.0, True


def distill(x, teacher, index, temperature: float = 1.0, tail: bool = False) -> Dict[str, np.ndarray]:
    x = np.asarray(x, dtype=np.float64)
    rows = x.shape[0]
    out = {"loss": np.zeros(rows), "lse": np.zeros(rows), "rest": np.zeros(rows)}
    with np.errstate(invalid="ignore", divide="ignore"):
        for r in range(rows):
            y = x[r] / temperature
            if np.isnan(y).any() or np.max(y) == np.inf:
                for name in out:
                    out[name][r] = np.nan
                tokens, p, log_p, p_rest, any_entry = _teacher(x[r], teacher[r], index[r], temperature, tail)
                if not any_entry:
                    out["loss"][r] = 0.0
                continue
            lse, q, log_q = _softmax_row(y)
            tokens, p, log_p, p_rest, any_entry = _teacher(x[r], teacher[r], index[r], temperature, tail)
            outside = np.ones(len(y), dtype=bool)
            outside[tokens] = False
            rest = _log_sum(log_q[outside])
            out["lse"][r] = lse
            out["rest"][r] = rest
            if not any_entry:
                continue
            loss = 0.0
            for v, pv, lp in zip(tokens, p, log_p):
                if pv > 0:
                    loss += pv * (lp - log_q[v])
            if p_rest > 0 and rest > -np.inf:
                loss += p_rest * (np.log(p_rest) - rest)
            out["loss"][r] = loss
    return out


def distill_grad(x, teacher, index, d_loss, temperature: float = 1.0, tail: bool = False, lse=None,
                 rest=None) -> np.ndarray:
    x = np.asarray(x, dtype=np.float64)
    rows = x.shape[0]
    grad = np.zeros_like(x)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        for r in range(rows):
            w = 1.0 if d_loss is None else float(d_loss[r])
            tokens, p, log_p, p_rest, any_entry = _teacher(x[r], teacher[r], index[r], temperature, tail)
            if w == 0.0 or not any_entry:
                continue
            y = x[r] / temperature
            if lse is None and (np.isnan(y).any() or np.max(y) == np.inf):
                grad[r] = np.nan
                continue
            given, q, log_q = _softmax_row(y, None if lse is None else float(lse[r]))
            if given == -np.inf:
                continue
            outside = np.ones(len(y), dtype=bool)
            outside[tokens] = False
            if rest is not None:
                log_rest = float(rest[r])
            else:
                log_rest = _log_sum(log_q[outside])
            if log_rest == -np.inf:
                p_rest = 0.0
            g = q * (float(np.sum(p)) + p_rest)
            g[tokens] -= p
            if tail and p_rest > 0:
                g[outside] -= p_rest * np.exp(log_q[outside] - log_rest)
            g[x[r] == -np.inf] = 0.0
            grad[r] = w * g / temperature
    return grad
