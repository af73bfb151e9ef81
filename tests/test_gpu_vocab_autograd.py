"""The vocabulary losses write through raw pointers: torch has to know what was written, so
that a tensor saved for a backward pass and overwritten raises there, as torch's own in-place
operations do."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_orthogonalized_gb300 as m
    m.lib()
    return m


def _case(rows=4, vocab=300):
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, vocab, generator=gen, device="cuda")
    tokens = torch.arange(rows, device="cuda")
    index = torch.arange(3, device="cuda").repeat(rows, 1)
    return x, tokens, torch.zeros(rows, 3, device="cuda"), index, torch.ones(rows, device="cuda")


def _calls(nsm, place, o):
    """Each call with what it writes (place: its gradient goes over the logits)."""
    x, tokens, teacher, index, w = _case()
    g = x if place else torch.empty_like(x)
    return {
        "logprobs": (lambda: nsm.logprobs(x, tokens, o["logprob"], o["entropy"], o["lse"], o["top"], o["top_index"]),
                     [o["logprob"], o["entropy"], o["lse"], o["top"], o["top_index"]], x),
        "logprobs_grad": (lambda: nsm.logprobs_grad(x, tokens, w, w, g, o["logprob"], o["entropy"], o["lse"]),
                          [g, o["logprob"], o["entropy"], o["lse"]], x),
        "logprobs_backward": (lambda: nsm.logprobs_backward(x, tokens, w, w, w, w, g), [g], x),
        "distill": (lambda: nsm.distill(x, teacher, index, o["loss"], o["lse"], o["rest"], tail=True),
                    [o["loss"], o["lse"], o["rest"]], x),
        "distill_grad": (lambda: nsm.distill_grad(x, teacher, index, w, g, o["loss"], o["lse"], o["rest"], tail=True),
                         [g, o["loss"], o["lse"], o["rest"]], x),
        "distill_backward": (lambda: nsm.distill_backward(x, teacher, index, w, w, w, g, tail=True), [g], x),
    }


CALLS = ["logprobs", "logprobs_grad", "logprobs_backward", "distill", "distill_grad", "distill_backward"]


@pytest.mark.parametrize("place", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_every_written_tensor_has_a_new_version(nsm, name, place):
    o = {n: torch.empty(4, device="cuda") for n in ("logprob", "entropy", "lse", "loss", "rest")}
    o["top"], o["top_index"] = torch.empty(4, 2, device="cuda"), torch.empty(4, 2, dtype=torch.int32, device="cuda")
    call, written, logits = _calls(nsm, place, o)[name]
    before, read = [t._version for t in written], logits._version
    call()
    assert all(t._version > v for t, v in zip(written, before))
    if not any(t is logits for t in written):
        assert logits._version == read


def test_a_saved_tensor_overwritten_in_place_raises(nsm):
    # a soft cap's tanh saves its output: its gradient from what was written there would be wrong
    h, tokens, teacher, index, w = _case()
    for call in (lambda z: nsm.logprobs_grad(z, tokens, w, None, z), lambda z: nsm.distill_grad(z, teacher, index, w, z)):
        leaf = h.clone().requires_grad_()
        logits = torch.tanh(leaf)
        call(logits.detach())
        with pytest.raises(RuntimeError):
            logits.backward(logits.detach().clone())


def test_in_place_where_nothing_was_saved(nsm):
    x, tokens, _, _, w = _case()
    hidden = torch.randn(4, 16, device="cuda")
    weight = torch.randn(16, x.shape[1], device="cuda")
    grads = []
    for place in (False, True):
        leaf = weight.clone().requires_grad_()
        logits = hidden @ leaf
        d_logits = logits.detach() if place else torch.empty_like(logits)
        nsm.logprobs_grad(logits.detach(), tokens, w, None, d_logits)
        logits.backward(d_logits)
        grads.append(leaf.grad)
    assert torch.equal(grads[0], grads[1])


def test_inference_mode(nsm):
    with torch.inference_mode():
        x, tokens, _, _, w = _case()
        logprob = torch.empty(4, device="cuda")
        nsm.logprobs(x, tokens, logprob)
        want = torch.log_softmax(x.double(), 1).gather(1, tokens[:, None])[:, 0]
        assert torch.allclose(logprob.double(), want, atol=1e-5)
