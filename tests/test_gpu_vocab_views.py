"""Logits and gradient as views of one buffer that share no element: side by side in every
row, which is no overlap, and overlapping, which is refused."""

import pytest
import torch

from test_gpu_vocab_loss import e_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_orthogonalized_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("vocab", [77, 1003, 8200])
@pytest.mark.parametrize("swap", [False, True])
def test_side_by_side(nsm, vocab, swap):
    rows = 6
    buf = torch.full((rows, 2 * vocab + 40), 3.0, device="cuda")
    x, g = buf[:, :vocab], buf[:, vocab:2 * vocab]
    if swap:
        x, g = g, x
    teacher = buf[:, 2 * vocab:2 * vocab + 5]  # read there too
    gen = torch.Generator(device="cuda").manual_seed(vocab)
    x.copy_(torch.randn(rows, vocab, generator=gen, device="cuda"))
    teacher.copy_(torch.randn(rows, 5, generator=gen, device="cuda"))
    tokens = torch.arange(rows, device="cuda")
    index = torch.arange(5, device="cuda").repeat(rows, 1)
    w = torch.ones(rows, device="cuda")
    alone, teacher_alone, want = x.clone(), teacher.clone(), torch.empty(rows, vocab, device="cuda")
    lse = torch.empty(rows, device="cuda")
    for write, read in ((lambda a, t, d: nsm.logprobs_grad(a, tokens, w, None, d), alone),
                        (lambda a, t, d: nsm.logprobs_backward(a, tokens, lse, None, w, None, d), alone),
                        (lambda a, t, d: nsm.distill_grad(a, t, index, w, d), alone),
                        (lambda a, t, d: nsm.distill_backward(a, t, index, lse, None, w, d), alone)):
        nsm.logprobs(alone, tokens, lse=lse)
        write(alone, teacher_alone, want)
        write(x, teacher, g)
        # the sums may be grouped by another alignment of the row: each probability within twice
        # the error of a sum of exponentials, the first columns' 1 - q and q - p absolutely
        e = 4 * e_of(vocab)
        assert torch.allclose(g[:, 6:], want[:, 6:], rtol=e, atol=0.0)
        assert torch.allclose(g[:, :6], want[:, :6], rtol=0.0, atol=e)
        assert torch.equal(x, read) and torch.equal(teacher, teacher_alone)
        assert bool((buf[:, 2 * vocab + 5:] == 3.0).all())


def test_overlapping_views_are_refused(nsm):
    rows, vocab = 6, 1003
    buf = torch.zeros(rows, 2 * vocab + 40, device="cuda")
    x = buf[:, :vocab]
    tokens, w = torch.arange(rows, device="cuda"), torch.ones(rows, device="cuda")
    index = torch.arange(5, device="cuda").repeat(rows, 1)
    for first in (1, vocab - 1):
        with pytest.raises(nsm.NsmError):
            nsm.logprobs_grad(x, tokens, w, None, buf[:, first:first + vocab])
    # a gradient that ends in the next row's logits, and one over the teacher
    flat = buf.view(-1)
    wraps = flat[vocab + 41:vocab + 41 + (rows - 1) * buf.shape[1]].view(rows - 1, buf.shape[1])[:, :vocab]
    with pytest.raises(nsm.NsmError):
        nsm.logprobs_grad(x[:rows - 1], tokens[:rows - 1], w[:rows - 1], None, wraps)
    with pytest.raises(nsm.NsmError):
        nsm.distill_grad(x, buf[:, 2 * vocab - 1:2 * vocab + 4], index, w, buf[:, vocab:2 * vocab])
    assert nsm.device_status() == nsm.NSM_OK
