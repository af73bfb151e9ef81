"""Distillation's gradient at entries whose teacher and student are far apart: a score of
almost no mass (its probability a subnormal number or nothing in fp32) on a token that the
student holds likely, and the other way round, against the float64 oracle.

Tolerances as in test_gpu_vocab_loss.py: a probability q or p has a relative error of 2 E(V)
plus 4 u times the size of the logs that it comes from, a subnormal one an error of the
smallest step beside, and the gradient w / t (q - p) is rounded once: w / t (q + p) times that
error.  A score further than 104 below the largest has no mass in fp32, so the sizes of the
teacher's logs stop at 130 (what the largest may be above 0 is below 26 here)."""

import numpy as np
import pytest
import torch

from oracle import vocab_ref as ref
from test_gpu_vocab_loss import SMALLEST, STEP, U, close, e_of, finite, on_gpu, outputs, softmax

pytestmark = pytest.mark.gpu

# A warp per row, a block per row, a cluster per row, rows that fit no cluster's shared memory.
ROWS = [(300, "bf16", 6), (300, "fp32", 6), (1999, "fp16", 6), (8001, "bf16", 700), (8001, "fp32", 6), (50257, "bf16", 6),
        (131072, "fp32", 6), (500003, "fp32", 2)]


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_orthogonalized_gb300 as m
    m.lib()
    return m


def check(nsm, x, dtype, z, index, temperature, tail):
    rows, vocab = x.shape
    logits, seen = on_gpu(x, dtype, pad=3, offset=1)
    teacher, ix = torch.from_numpy(z).float().cuda(), torch.from_numpy(index).cuda()
    w = np.linspace(0.5, 1.5, rows).astype(np.float32)
    d_loss = torch.from_numpy(w).cuda()
    o = outputs(rows)
    g = torch.full_like(logits, float("nan"))
    back = torch.full_like(logits, float("nan"))
    nsm.distill_grad(logits, teacher, ix, d_loss, g, o["loss"], o["lse"], o["rest"], temperature=temperature, tail=tail)
    nsm.distill_backward(logits, teacher, ix, o["lse"], o["rest"] if tail else None, d_loss, back,
                         temperature=temperature, tail=tail)
    few = [0, rows // 2, rows - 1]
    seen, w = seen[few], w[few]
    z, index = teacher.double().cpu().numpy()[few], index[few]
    fwd = ref.distill(seen, z, index, temperature, tail)
    want = ref.distill_grad(seen, z, index, w, temperature, tail)
    assert np.isfinite(want).all()
    q, log_q = softmax(seen, temperature)
    p = np.zeros_like(q)
    for r in range(len(few)):
        tok, pr, _, p_rest, _ = ref._teacher(seen[r], z[r], index[r], temperature, tail)
        p[r, tok] = pr
        if tail:
            out = np.ones(vocab, dtype=bool)
            out[tok] = False
            p[r, out] += p_rest * np.exp(log_q[r, out] - fwd["rest"][r])
    logs = finite(fwd["lse"]) + finite(seen).max(axis=1) / temperature + 130
    rel = 2 * e_of(vocab) + 4 * U * (finite(log_q) + logs[:, None])
    tol = (w / temperature)[:, None] * (q + p) * rel + 1.01 * STEP[dtype] * finite(want) + SMALLEST[dtype]
    close(g[few], want, tol, "gradient in one call")
    close(back[few], want, 2 * tol, "backward alone")  # the stored lse and rest carry their own errors


def rows_with_entries(vocab, rows, scores, spread):
    """Rows of a bell, and entries at random tokens, one of them far ahead in the student."""
    rng = np.random.default_rng(vocab + rows)
    x = rng.normal(size=(rows, vocab)) * spread
    index = np.stack([rng.permutation(vocab)[:len(scores)] for _ in range(rows)])
    for r in range(rows):
        x[r, index[r, 1 + r % (len(scores) - 1)]] += 6 * spread  # a token of almost no mass, not the first
    return x, np.tile(np.asarray(scores, dtype=np.float64), (rows, 1)), index


@pytest.mark.parametrize("vocab,dtype,rows", ROWS)
def test_entries_of_almost_no_mass_with_the_tail(nsm, vocab, dtype, rows):
    scores = [-0.25, -80.0, -90.0, -95.0, -100.0, -103.0, -110.0, -1e30, -np.inf]
    check(nsm, *_ordered(rows_with_entries(vocab, rows, scores, 1.0), dtype), 1.0, True)


@pytest.mark.parametrize("vocab,dtype,rows", ROWS)
@pytest.mark.parametrize("temperature", [0.05, 0.1])
def test_scores_far_apart_at_a_low_temperature(nsm, vocab, dtype, rows, temperature):
    scores = [1.0, 0.9, -3.0, -3.75, -4.5, -8.0, -8.5, -9.0, -9.5, -10.0, -11.0, -60.0]
    check(nsm, *_ordered(rows_with_entries(vocab, rows, scores, 2 * temperature), dtype), temperature, False)


@pytest.mark.parametrize("vocab,dtype,rows", ROWS)
def test_a_student_far_from_likely_scores(nsm, vocab, dtype, rows):
    # the teacher's mass where the student has none: the gradient is -p there
    scores = [-0.7, -1.2, -3.0, -6.0]
    x, z, index = rows_with_entries(vocab, rows, scores, 1.0)
    for r in range(rows):
        x[r, index[r, :2]] = (-90.0, -120.0)
    check(nsm, *_ordered((x, z, index), dtype), 1.0, True)


def _ordered(case, dtype):
    x, z, index = case
    return x, dtype, z, index
