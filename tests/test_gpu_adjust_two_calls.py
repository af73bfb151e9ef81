"""Penalties over two histories in two calls: repetition over the prompt and the answer to fp32, then
frequency, presence, biases and a mask in place, over the answer alone."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

from oracle import adjust_ref as ref  # noqa: E402


@pytest.mark.parametrize("kind", ["bfloat16", "float16", "float32"])
def test_repetition_over_more_than_the_others(kind):
    import torch

    import newton_schulz_orthogonalized_gb300 as nsm
    rows, vocab, prompt, answer, k = 5, 9001, 200, 60, 4
    g = torch.Generator(device="cuda").manual_seed(7)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * 3).to(getattr(torch, kind))
    tokens = torch.randint(0, vocab, (rows, prompt + answer), generator=g, device="cuda")
    tokens[:, ::4] = tokens[:, 1:2].clone()
    theta, frequency, presence = (0.5 + torch.rand(rows, generator=g, device="cuda") for _ in range(3))
    later = dict(history=tokens[:, prompt:], frequency=frequency, presence=presence,
                 bias_index=torch.randint(0, vocab, (rows, k), generator=g, device="cuda"), bias=torch.randn(rows, k, generator=g, device="cuda"),
                 mask=torch.randint(-2 ** 31, 2 ** 31, (rows, (vocab + 31) // 32), generator=g, device="cuda").int())
    out = torch.empty(rows, vocab, device="cuda")
    nsm.adjust_logits(x, out, history=tokens, repetition=theta)
    nsm.adjust_logits(out, out, **later)
    host = {n: t.cpu().numpy() for n, t in later.items()}
    first, _ = ref.adjust(x.double().cpu().numpy(), history=tokens.cpu().numpy(), repetition=theta.cpu().numpy())
    want, size = ref.adjust(first, **host)
    got = out.double().cpu().numpy()
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    fine = np.isfinite(want)
    # fp32: quotient or product, penalty, difference, a sum per bias, and either call's rounding; half the least subnormal
    tol = (5 + k) * 2.0 ** -24 * size + 2.0 ** -150
    assert np.all(np.abs(got[fine] - want[fine]) <= tol[fine] * 1.0001)
    # the gradient: repetition's and the mask's in one call
    d_out = torch.randn(rows, vocab, generator=g, device="cuda")
    d = torch.empty_like(x)
    nsm.adjust_logits_backward(x, d_out, d, history=tokens, repetition=theta, mask=later["mask"])
    exact = ref.adjust_backward(x.double().cpu().numpy(), d_out.double().cpu().numpy(), history=tokens.cpu().numpy(),
                                repetition=theta.cpu().numpy(), mask=host["mask"])
    half, least = torch.finfo(x.dtype).eps / 2, {"bfloat16": 2.0 ** -134, "float16": 2.0 ** -25, "float32": 2.0 ** -150}[kind]
    assert np.all(np.abs(d.double().cpu().numpy() - exact) <= ((2.0 ** -24 + half) * np.abs(exact) + least) * 1.0001)
