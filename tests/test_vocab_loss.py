"""Losses over a vocabulary, without a GPU: the float64 oracle against central differences
and against plain identities, and every refusal of the C ABI and of the binding (all of
them are returned before a CUDA call)."""

import ctypes

import numpy as np
import pytest

from oracle import vocab_ref as ref


def _row(seed, vocab=37, spread=2.0):
    return np.random.default_rng(seed).normal(size=(1, vocab)) * spread


@pytest.mark.parametrize("temperature", [1.0, 0.7, 2.5])
@pytest.mark.parametrize("weights", [(1.3, 0.0), (0.0, -0.7), (-0.4, 0.9)])
def test_oracle_logprob_gradient_against_differences(temperature, weights):
    x = _row(1)
    x[0, 5] = -np.inf
    w, h = weights
    tokens = [11]

    def value(z):
        o = ref.logprobs(z, tokens, temperature)
        return w * o["logprob"][0] + h * o["entropy"][0]

    g = ref.logprobs_grad(x, tokens, [w], [h], temperature)
    step = 1e-5
    for v in range(x.shape[1]):
        if x[0, v] == -np.inf:
            assert g[0, v] == 0.0
            continue
        up, down = x.copy(), x.copy()
        up[0, v] += step
        down[0, v] -= step
        # third derivatives are of order 1 / t^3: the difference is good to about step^2
        assert abs((value(up) - value(down)) / (2 * step) - g[0, v]) < 1e-8


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("temperature", [1.0, 2.0])
def test_oracle_distill_gradient_against_differences(tail, temperature):
    x = _row(2)
    index = np.array([[3, 30, -1, 17, 3, 99]])
    z = np.array([[1.0, 0.3, 5.0, -0.5, 9.0, 7.0]])
    if tail:
        z = z - 2.0
    g = ref.distill_grad(x, z, index, [0.8], temperature, tail)
    step = 1e-5
    for v in range(x.shape[1]):
        up, down = x.copy(), x.copy()
        up[0, v] += step
        down[0, v] -= step
        d = 0.8 * (ref.distill(up, z, index, temperature, tail)["loss"][0]
                   - ref.distill(down, z, index, temperature, tail)["loss"][0]) / (2 * step)
        assert abs(d - g[0, v]) < 1e-8


def test_oracle_distill_of_the_whole_row_is_the_divergence():
    # entries over every token, scores the teacher's logits: the plain KL of two softmaxes
    x, y = _row(3, 19), _row(4, 19)
    index = np.arange(19)[None]
    q = np.exp(x[0]) / np.exp(x[0]).sum()
    p = np.exp(y[0]) / np.exp(y[0]).sum()
    want = np.sum(p * np.log(p / q))
    assert abs(ref.distill(x, y, index)["loss"][0] - want) < 1e-12
    log_p = np.log(p)[None]
    assert abs(ref.distill(x, log_p, index, tail=True)["loss"][0] - want) < 1e-12
    # the student equal to the teacher: no loss and no gradient, with any subset of entries
    log_q = np.log(q)[None]
    part = index[:, :7]
    assert abs(ref.distill(x, log_q[:, :7], part, tail=True)["loss"][0]) < 1e-12
    assert np.abs(ref.distill_grad(x, log_q[:, :7], part, None, tail=True)).max() < 1e-12


@pytest.fixture(scope="module")
def nsm():
    import os

    import newton_schulz_orthogonalized_gb300 as m
    if not os.path.exists(m.LIB_PATH):
        from newton_schulz_orthogonalized_gb300 import _build
        _build.build()
    m.lib()
    return m


X, G, TOK, F = 0x10000000, 0x20000000, 0x30000000, 0x40000000


def _logprobs(nsm, x=X, dtype=0, rows=4, vocab=100, ld=100, tokens=TOK, wide=1, t=1.0, k=0, logprob=F,
              entropy=0, lse=0, top=0, top_index=0):
    return nsm.lib().nsm_logprobs(x, dtype, rows, vocab, ld, tokens, wide, t, k, logprob, entropy, lse, top,
                                  top_index, None)


def test_logprobs_refusals(nsm):
    E = nsm
    assert _logprobs(nsm, x=0) == E.NSM_ERR_NULL
    assert _logprobs(nsm, dtype=3) == E.NSM_ERR_ARG
    assert _logprobs(nsm, dtype=-1) == E.NSM_ERR_ARG
    assert _logprobs(nsm, rows=-1) == E.NSM_ERR_SHAPE
    assert _logprobs(nsm, rows=1 << 31) == E.NSM_ERR_SHAPE
    assert _logprobs(nsm, vocab=0) == E.NSM_ERR_SHAPE
    assert _logprobs(nsm, vocab=(1 << 20) + 1, ld=1 << 21) == E.NSM_ERR_SHAPE
    assert _logprobs(nsm, ld=99) == E.NSM_ERR_SHAPE
    assert _logprobs(nsm, ld=1 << 62) == E.NSM_ERR_SHAPE
    assert _logprobs(nsm, x=X + 1) == E.NSM_ERR_ALIGN
    assert _logprobs(nsm, x=X + 2, dtype=2) == E.NSM_ERR_ALIGN
    assert _logprobs(nsm, tokens=TOK + 4) == E.NSM_ERR_ALIGN
    assert _logprobs(nsm, logprob=F + 2) == E.NSM_ERR_ALIGN
    for t in (0.0, -1.0, float("nan"), float("inf"), 1e-7, 1e7):
        assert _logprobs(nsm, t=t) == E.NSM_ERR_ARG
    assert _logprobs(nsm, k=129, top=F + 0x1000, top_index=F + 0x2000) == E.NSM_ERR_ARG
    assert _logprobs(nsm, k=-1) == E.NSM_ERR_ARG
    assert _logprobs(nsm, k=5) == E.NSM_ERR_NULL
    assert _logprobs(nsm, tokens=0) == E.NSM_ERR_NULL
    assert _logprobs(nsm, logprob=0) == E.NSM_ERR_NULL  # nothing is asked for
    assert _logprobs(nsm, lse=F + 8) == E.NSM_ERR_ARG  # overlaps logprob
    assert _logprobs(nsm, logprob=X + 16) == E.NSM_ERR_ARG  # overlaps the logits
    assert "overlap" in nsm.last_error()
    assert _logprobs(nsm, rows=0, x=0, tokens=0) == E.NSM_OK
    assert nsm.last_launch_count() == 0


def _logprobs_grad(nsm, x=X, rows=4, ld=100, tokens=TOK, dl=F, dh=0, g=G, ldd=100, logprob=0):
    return nsm.lib().nsm_logprobs_grad(x, 0, rows, 100, ld, tokens, 1, 1.0, dl, dh, g, ldd, logprob, 0, 0, None)


def test_logprobs_grad_refusals(nsm):
    E = nsm
    assert _logprobs_grad(nsm, g=0) == E.NSM_ERR_NULL
    assert _logprobs_grad(nsm, dl=0) == E.NSM_ERR_NULL
    assert _logprobs_grad(nsm, tokens=0) == E.NSM_ERR_NULL
    assert _logprobs_grad(nsm, ldd=99) == E.NSM_ERR_SHAPE
    assert _logprobs_grad(nsm, g=G + 1) == E.NSM_ERR_ALIGN
    assert _logprobs_grad(nsm, g=X + 200) == E.NSM_ERR_ARG  # shifted over the logits
    assert _logprobs_grad(nsm, g=X, ldd=104) == E.NSM_ERR_ARG  # in place at another stride
    assert _logprobs_grad(nsm, logprob=F) == E.NSM_ERR_ARG  # the output over the weights
    assert _logprobs_grad(nsm, rows=0, x=0) == E.NSM_OK


def test_logprobs_backward_refusals(nsm):
    L, E = nsm.lib(), nsm

    def call(lse=F, entropy=0, dl=F + 0x1000, dh=0, g=G, tokens=TOK):
        return L.nsm_logprobs_backward(X, 0, 4, 100, 100, tokens, 1, 1.0, lse, entropy, dl, dh, g, 100, None)

    assert call(lse=0) == E.NSM_ERR_NULL
    assert call(g=0) == E.NSM_ERR_NULL
    assert call(dl=0) == E.NSM_ERR_NULL
    assert call(tokens=0) == E.NSM_ERR_NULL
    assert call(dh=F + 0x2000) == E.NSM_ERR_NULL  # without the entropy
    assert call(g=F) == E.NSM_ERR_ARG


def _distill(nsm, teacher=TOK, td=0, ldt=8, index=TOK + 0x1000, wide=1, ldi=8, k=8, t=1.0, loss=F, rows=4, lse=0):
    return nsm.lib().nsm_distill(X, 0, rows, 100, 100, teacher, td, ldt, index, wide, ldi, k, t, 0, loss, lse, 0, None)


def test_distill_refusals(nsm):
    L, E = nsm.lib(), nsm
    assert _distill(nsm, teacher=0) == E.NSM_ERR_NULL
    assert _distill(nsm, index=0) == E.NSM_ERR_NULL
    assert _distill(nsm, loss=0) == E.NSM_ERR_NULL
    assert _distill(nsm, td=7) == E.NSM_ERR_ARG
    assert _distill(nsm, k=0) == E.NSM_ERR_ARG
    assert _distill(nsm, k=129, ldt=200, ldi=200) == E.NSM_ERR_ARG
    assert _distill(nsm, ldt=7) == E.NSM_ERR_SHAPE
    assert _distill(nsm, ldi=7) == E.NSM_ERR_SHAPE
    assert _distill(nsm, teacher=TOK + 1) == E.NSM_ERR_ALIGN
    assert _distill(nsm, index=TOK + 0x1004) == E.NSM_ERR_ALIGN
    assert _distill(nsm, loss=TOK) == E.NSM_ERR_ARG
    assert _distill(nsm, lse=F) == E.NSM_ERR_ARG
    assert _distill(nsm, t=0.0) == E.NSM_ERR_ARG
    assert _distill(nsm, rows=0) == E.NSM_OK
    entries = (TOK, 0, 8, TOK + 0x1000, 1, 8, 8, 1.0)
    assert L.nsm_distill_grad(X, 0, 4, 100, 100, *entries, 0, 0, 0, 100, F, 0, 0, None) == E.NSM_ERR_NULL
    assert L.nsm_distill_grad(X, 0, 4, 100, 100, *entries, 0, 0, X + 64, 100, F, 0, 0, None) == E.NSM_ERR_ARG
    back = L.nsm_distill_backward
    assert back(X, 0, 4, 100, 100, *entries, 0, 0, 0, 0, G, 100, None) == E.NSM_ERR_NULL  # lse
    assert back(X, 0, 4, 100, 100, *entries, 1, F, 0, 0, G, 100, None) == E.NSM_ERR_NULL  # rest, with the tail
    assert back(X, 0, 4, 100, 100, *entries, 0, F, 0, 0, 0, 100, None) == E.NSM_ERR_NULL  # d_logits


def test_binding_refuses_host_tensors(nsm):
    import torch
    x = torch.zeros(3, 10)
    with pytest.raises(ValueError):
        nsm.logprobs(x, torch.zeros(3, dtype=torch.int64), torch.zeros(3))
    with pytest.raises(ValueError):
        nsm.distill(x, torch.zeros(3, 2), torch.zeros(3, 2, dtype=torch.int64), torch.zeros(3))


def test_timing_kinds_cover_the_losses(nsm):
    ms = ctypes.c_double(-1)
    for kind in (nsm.KIND_LOGPROBS, nsm.KIND_DISTILL):
        assert nsm.lib().nsm_timing_read_kind(kind, ctypes.byref(ms), None, None) == nsm.NSM_OK
        assert ms.value == 0.0
    assert nsm.lib().nsm_timing_read_kind(10, ctypes.byref(ms), None, None) == nsm.NSM_ERR_ARG
