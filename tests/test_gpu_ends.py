"""A training step's use of the vocabulary's two ends and the gradients' norm together, against the float64
oracles: tokens in by the embedding, logits adjusted and scored, the loss's gradient back through the
adjustment and into the tied weight, which the head's gradient reached first, all clipped, and the
optimizer's step."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

from oracle import adjust_ref, embedding_ref, grads_ref, vocab_ref  # noqa: E402


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_orthogonalized_gb300 as m
    m.lib()
    return m


def _host(t):
    return t.detach().double().cpu().numpy()


def _setup(nsm, torch):
    """A tied embedding and head, sequences of tokens, sampling penalties and a grammar."""
    sequences, length, vocab, width = 3, 40, 1003, 64
    rows = sequences * length
    g = torch.Generator(device="cuda").manual_seed(11)
    opt = nsm.MuonAdamW([("model.embed_tokens.weight", (vocab, width)), ("layers.0.proj.weight", (width, width))], adam_lr=1e-2)
    for n in ("model.embed_tokens.weight", "layers.0.proj.weight"):
        opt.param(n).copy_(torch.randn(opt.param(n).shape, generator=g, device="cuda") * 0.3)
    tokens = (vocab * torch.rand(sequences, length, generator=g, device="cuda") ** 3).long()
    at = torch.arange(rows, device="cuda")
    kw = {"history": tokens, "history_row": (at // length).int(), "length": (at % length).int(),
          "repetition": torch.full((rows,), 1.3, device="cuda"),
          "mask": torch.randint(-2 ** 31, 2 ** 31, (4, (vocab + 31) // 32), generator=g, device="cuda").int(),
          "mask_row": (at % 5 - 1).int()}
    extra = {"frequency": torch.full((rows,), 0.2, device="cuda"), "presence": torch.full((rows,), 0.1, device="cuda")}
    sampled = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    # sampled under the grammar
    word = kw["mask"][kw["mask_row"].clamp(min=0).long(), sampled // 32]
    banned = (((word >> (sampled % 32).int()) & 1) == 0) & (kw["mask_row"] >= 0)
    return opt, tokens, kw, extra, torch.where(banned, -100, sampled), torch.randn(rows, generator=g, device="cuda") / rows


def _step(nsm, torch, s, ws, clip_ws):
    """One step on preallocated tensors `s`; nothing is allocated but by the products."""
    opt, w = s["opt"], s["opt"].param("model.embed_tokens.weight")
    proj = s["opt"].param("layers.0.proj.weight")
    nsm.embedding(w, s["tokens"].view(-1), s["x"], scale=2.0)
    h = s["x"].float() @ proj
    s["h"].copy_(h)
    s["logits"].copy_(h @ w.T)
    nsm.adjust_logits(s["logits"], s["adjusted"], **s["kw"], **s["extra"])
    nsm.logprobs_grad(s["adjusted"], s["sampled"], s["weight"], None, s["d_adjusted"], s["logprob"])
    nsm.adjust_logits_backward(s["logits"], s["d_adjusted"], s["d_logits"], **s["kw"])
    s["d_w"].copy_(s["d_logits"].T @ s["h"])        # the head's part
    d_h = s["d_logits"] @ w
    s["d_proj"].copy_(s["x"].float().T @ d_h)
    s["d_x"].copy_(d_h @ proj.T)
    nsm.embedding_backward(s["d_x"], s["tokens"].view(-1), s["d_w"], ws, scale=2.0, accumulate=True)
    nsm.clip_grads(s["table"], 0.02, s["norm"], s["norms"], workspace=clip_ws)


def _tensors(nsm, torch):
    opt, tokens, kw, extra, sampled, weight = _setup(nsm, torch)
    rows, (vocab, width) = tokens.numel(), opt.param("model.embed_tokens.weight").shape

    def f(*shape):
        return torch.empty(*shape, device="cuda")

    s = {"opt": opt, "tokens": tokens, "kw": kw, "extra": extra, "sampled": sampled, "weight": weight, "x": f(rows, width),
         "h": f(rows, width), "logits": f(rows, vocab), "adjusted": f(rows, vocab), "d_adjusted": f(rows, vocab), "logprob": f(rows),
         "d_logits": f(rows, vocab), "d_w": f(vocab, width), "d_proj": f(width, width), "d_x": f(rows, width), "norm": f(1), "norms": f(2)}
    s["table"] = nsm.GradTable([s["d_proj"], s["d_w"]], [opt.grad("layers.0.proj.weight"), opt.grad("model.embed_tokens.weight")])
    ws = torch.empty(nsm.embedding_workspace_bytes(rows, vocab, width), dtype=torch.uint8, device="cuda")
    return s, ws, torch.empty(s["table"].workspace_bytes, dtype=torch.uint8, device="cuda")


def test_a_training_step(nsm):
    import torch
    s, ws, clip_ws = _tensors(nsm, torch)
    torch.backends.cuda.matmul.allow_tf32 = False
    _step(nsm, torch, s, ws, clip_ws)
    # each piece against its oracle, on the tensors that it got
    kw, extra = {n: t.cpu().numpy() for n, t in s["kw"].items()}, {n: t.cpu().numpy() for n, t in s["extra"].items()}
    w, tok = _host(s["opt"].param("model.embed_tokens.weight")), s["tokens"].view(-1).cpu().numpy()
    eps = 2.0 ** -24
    want = embedding_ref.embedding(w, tok, 2.0)
    assert np.array_equal(_host(s["x"]), want)  # a product with 2 is exact
    x = _host(s["logits"])
    want, size = adjust_ref.adjust(x, **kw, **extra)
    got, fine = _host(s["adjusted"]), np.isfinite(want)
    assert np.array_equal(np.isneginf(got), ~fine) and np.all(np.abs(got[fine] - want[fine]) <= 4 * eps * size[fine])
    sampled, weight = s["sampled"].cpu().numpy(), _host(s["weight"])
    ref = vocab_ref.logprobs(got, sampled)
    # of a sum of exponentials over 1003 logits, as for the losses alone, and of the values' size
    tol = 2 * (108 + 1003 / 256) * eps + 8 * eps * np.abs(ref["logprob"])
    assert np.all(np.abs(_host(s["logprob"]) - ref["logprob"]) <= tol)
    d_adj = vocab_ref.logprobs_grad(got, sampled, weight, None)
    assert np.linalg.norm(_host(s["d_adjusted"]) - d_adj) <= 1e-5 * np.linalg.norm(d_adj)
    d = adjust_ref.adjust_backward(x, _host(s["d_adjusted"]), **kw)
    assert np.all(np.abs(_host(s["d_logits"]) - d) <= 2 * eps * np.abs(d))
    # the whole gradient by the formulas in 64 bits; fp32 products of 1003 and of 120 terms
    proj, dl, h = _host(s["opt"].param("layers.0.proj.weight")), _host(s["d_logits"]), _host(s["h"])
    d_x = dl @ w @ proj.T
    d_w, _, _ = embedding_ref.embedding_backward(d_x, tok, 1003, 2.0, old=dl.T @ h)
    assert np.linalg.norm(_host(s["d_w"]) - d_w) <= 1e-5 * np.linalg.norm(d_w)
    clipped, norm, norms = grads_ref.clip_grads([_host(s["d_proj"]), _host(s["d_w"])], 0.02)
    assert norm > 0.02 and abs(s["norm"].item() - norm) <= 40 * eps * norm
    assert np.all(np.abs(_host(s["norms"]) - norms) <= 40 * eps * norms)
    for name, c in zip(("layers.0.proj.weight", "model.embed_tokens.weight"), clipped):
        assert np.all(np.abs(_host(s["opt"].grad(name)) - c) <= (2.0 ** -8 + 50 * eps) * np.abs(c) + 2.0 ** -134)
    before = {n: s["opt"].param(n).clone() for n in ("layers.0.proj.weight", "model.embed_tokens.weight")}
    s["opt"].step()
    assert all(not torch.equal(before[n], s["opt"].param(n)) for n in before)
    assert nsm.device_status() == nsm.NSM_OK


def test_the_step_captured_and_replayed(nsm):
    """The calls in one graph, with new tokens each time, give the bits of the same calls made one by one."""
    import torch
    torch.backends.cuda.matmul.allow_tf32 = False
    s, ws, clip_ws = _tensors(nsm, torch)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        _step(nsm, torch, s, ws, clip_ws)
        _step(nsm, torch, s, ws, clip_ws)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(nsm, torch, s, ws, clip_ws)
    names = ("x", "adjusted", "logprob", "d_logits", "d_w", "norm", "norms")
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        s["tokens"].copy_(torch.randint(-1, 1003, s["tokens"].shape, generator=g, device="cuda"))
        s["weight"].copy_(torch.randn(s["weight"].shape, generator=g, device="cuda") / 100)
        graph.replay()
        first = {n: s[n].clone() for n in names}
        slots = [t.clone() for t in s["table"].out]
        _step(nsm, torch, s, ws, clip_ws)
        for n in names:
            assert torch.equal(first[n].view(torch.int32), s[n].view(torch.int32)), n
        for a, b in zip(slots, s["table"].out):
            assert torch.equal(a, b)
