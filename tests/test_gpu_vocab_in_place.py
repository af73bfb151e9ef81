"""Every gradient of the vocabulary losses over its own logits: the bits that it has in a
buffer of its own, with rows in one warp, in a block, in a cluster and in pieces, and entries
everywhere in the row (what one thread reads of it another overwrites)."""

import pytest
import torch

pytestmark = pytest.mark.gpu

SHAPES = [(40, 259, 0, torch.bfloat16), (1000, 515, 1, torch.float16), (300, 1021, 3, torch.float32), (500, 2041, 5, torch.bfloat16),
          (60, 8001, 7, torch.bfloat16), (3, 50257, 1, torch.bfloat16), (700, 20001, 0, torch.float32), (5, 131073, 3, torch.float16),
          (2, 500003, 1, torch.float32)]


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_orthogonalized_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("rows,vocab,lead,dtype", SHAPES)
@pytest.mark.parametrize("call", ["logprobs_grad", "logprobs_backward", "distill_grad", "distill_backward"])
def test_the_same_bits_in_place(nsm, rows, vocab, lead, dtype, call):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    whole = (torch.randn(rows, vocab, generator=g, device="cuda") * 3).to(dtype)
    x = torch.empty(rows * vocab + 8, dtype=dtype, device="cuda")[lead:lead + rows * vocab].view(rows, vocab)
    k = min(128, vocab)
    index = torch.rand(rows, vocab, generator=g, device="cuda").topk(k, dim=1).indices
    teacher = torch.randn(rows, k, generator=g, device="cuda").log_softmax(1) - 0.1
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    w, h = torch.randn(rows, generator=g, device="cuda"), torch.randn(rows, generator=g, device="cuda")
    lse, entropy, rest, loss = (torch.empty(rows, device="cuda") for _ in range(4))
    x.copy_(whole)
    nsm.logprobs(x, tokens, lse=lse, entropy=entropy)
    nsm.distill(x, teacher, index, loss, rest=rest, tail=True)
    calls = {"logprobs_grad": lambda out: nsm.logprobs_grad(x, tokens, w, h, out),
             "logprobs_backward": lambda out: nsm.logprobs_backward(x, tokens, lse, entropy, w, h, out),
             "distill_grad": lambda out: nsm.distill_grad(x, teacher, index, w, out, tail=True),
             "distill_backward": lambda out: nsm.distill_backward(x, teacher, index, lse, rest, w, out, tail=True)}
    # another buffer at the same alignment, so that the vectors are the same
    want = torch.empty(rows * vocab + 8, dtype=dtype, device="cuda")[lead:lead + rows * vocab].view(rows, vocab)
    calls[call](want)
    for _ in range(20):
        x.copy_(whole)
        calls[call](x)
        assert torch.equal(x, want)
