"""Rows of the vocabulary losses in batches of every size: the values of other rows never
change a row's bits, their number only the order of its sums.

The tolerances are those of test_gpu_vocab_loss.py; two results of the same row differ by at
most both their errors."""

import numpy as np
import pytest
import torch

from test_gpu_vocab_loss import SMALLEST, STEP, U, close, e_of, finite, outputs, softmax

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_orthogonalized_gb300 as m
    m.lib()
    return m


def every_call(nsm, x, tokens, teacher, index, w):
    """The results of every call on these rows."""
    rows = x.shape[0]
    o = outputs(rows, 9)
    nsm.logprobs(x, tokens, o["logprob"], o["entropy"], o["lse"], o["top_logprob"], o["top_index"])
    plain = torch.empty(rows, device="cuda")
    nsm.logprobs(x, tokens, plain)
    r = {n: o[n] for n in ("logprob", "entropy", "lse", "top_logprob", "top_index")}
    r["without alternatives"] = plain
    loss = outputs(rows)
    nsm.distill(x, teacher, index, loss["loss"], loss["lse"], loss["rest"], tail=True)
    r["loss"], r["rest"] = loss["loss"], loss["rest"]
    for name, call in (("logprobs_grad", lambda g: nsm.logprobs_grad(x, tokens, w, None, g)),
                       ("logprobs_backward", lambda g: nsm.logprobs_backward(x, tokens, o["lse"], None, w, None, g)),
                       ("distill_grad", lambda g: nsm.distill_grad(x, teacher, index, w, g, tail=True)),
                       ("distill_backward", lambda g: nsm.distill_backward(x, teacher, index, loss["lse"], loss["rest"], w, g,
                                                                           tail=True))):
        r[name] = torch.empty_like(x)
        call(r[name])
    return r


def batch(rows, vocab):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * 3).bfloat16()
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    teacher = torch.randn(rows, 12, generator=g, device="cuda").log_softmax(1) - 0.1
    index = torch.arange(12, device="cuda") + torch.randint(0, vocab - 12, (rows, 1), generator=g, device="cuda")
    w = torch.rand(rows, generator=g, device="cuda") + 0.5
    return x, tokens, teacher, index, w


@pytest.mark.parametrize("vocab", [515, 8001, 50257, 131072])
def test_the_number_of_rows_changes_last_bits_at_most(nsm, vocab):
    # batches on both sides of where blocks a row, pieces a row and threads change
    most = 2049
    whole = batch(most, vocab)
    want = every_call(nsm, *whole)
    e = e_of(vocab)
    for rows in (1, 18, 19, 37, 38, 75, 76, 151, 152, 303, 304, 607, 608, 2047, 2048):
        got = every_call(nsm, *(t[:rows] for t in whole))
        few = sorted({0, rows // 2, rows - 1})
        q, log_q = softmax(whole[0][few].double().cpu().numpy(), 1.0)
        p = np.zeros_like(q)  # where a gradient is a difference
        for j, r in enumerate(few):
            p[j, whole[3][r].cpu().numpy()] = 1.0
            p[j, int(whole[1][r])] = 1.0
        weight = whole[4][few].double().cpu().numpy()[:, None]
        for name, t in got.items():
            a, b = t[few], want[name][few].double().cpu().numpy()
            if name == "top_index":
                assert np.array_equal(a.cpu().numpy(), b)
            elif t.dim() == 2 and t.shape[1] == vocab:
                tol = 2 * weight * (q + p) * (4 * e + 4 * U * (finite(log_q) + 60)) + 2.1 * STEP["bf16"] * finite(b) + 2 * SMALLEST["bf16"]
                close(a, b, 2 * tol if name.endswith("backward") else tol, f"{name} of {rows} rows")
            else:
                close(a, b, 2 * (4 * e + 8 * U * (finite(b) + 60)), f"{name} of {rows} rows")


@pytest.mark.parametrize("rows,vocab", [(40, 515), (700, 8001), (300, 50257), (2100, 50257), (5, 131072), (2, 1 << 20)])
def test_the_values_of_other_rows_change_nothing(nsm, rows, vocab):
    x, tokens, teacher, index, w = batch(rows, vocab)
    first = every_call(nsm, x, tokens, teacher, index, w)
    keep = rows // 2
    others = torch.arange(rows, device="cuda") != keep
    x[others] = torch.randn(1, vocab, device="cuda").bfloat16() * 9
    x[(keep + 1) % rows, ::3] = float("nan")
    tokens[others] = -1
    teacher[others] = float("nan")
    w[others] = 0.0
    again = every_call(nsm, x, tokens, teacher, index, w)
    for name, t in first.items():
        assert torch.equal(t[keep:keep + 1].contiguous().view(torch.uint8),
                           again[name][keep:keep + 1].contiguous().view(torch.uint8)), name
