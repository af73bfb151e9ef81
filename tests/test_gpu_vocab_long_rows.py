"""Loss and gradient of log probabilities in one call where a row fits no cluster's shared
memory and is read twice, against the float64 oracle (tolerances: test_gpu_vocab_loss.py)."""

import numpy as np
import pytest
import torch

from oracle import vocab_ref as ref
from test_gpu_vocab_loss import U, close, e_of, finite, gradient_tolerance, make_rows, make_tokens, on_gpu, outputs, softmax

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_orthogonalized_gb300 as m
    m.lib()
    return m


# 16-byte vectors past eight blocks' shared memory
@pytest.mark.parametrize("dtype,vocab", [("fp32", 500003), ("bf16", 1 << 20), ("fp16", 1000001)])
@pytest.mark.parametrize("weights", ["token", "entropy", "both"])
def test_gradients_of_rows_that_fit_no_cluster(nsm, dtype, vocab, weights):
    rows, t = 8, 0.9
    x = make_rows(vocab, rows, vocab)
    tokens = make_tokens(vocab, rows, vocab)
    logits, seen = on_gpu(x, dtype, pad=3, offset=1)
    rng = np.random.default_rng(vocab)
    w = rng.normal(size=rows).astype(np.float32)
    w[rows - 1] = 0.0
    h = (rng.normal(size=rows) * 0.3).astype(np.float32)
    d_l = torch.from_numpy(w).cuda() if weights != "entropy" else None
    d_h = torch.from_numpy(h).cuda() if weights != "token" else None
    tk = torch.from_numpy(tokens).cuda()
    o = outputs(rows)
    g = torch.full_like(logits, float("nan"))
    nsm.logprobs_grad(logits, tk, d_l, d_h, g, o["logprob"], o["entropy"], o["lse"], temperature=t)
    fwd = ref.logprobs(seen, tokens, t)
    e = e_of(vocab)
    close(o["logprob"], fwd["logprob"], 2 * e + 4 * U * finite(fwd["logprob"]), "logprob")
    close(o["entropy"], fwd["entropy"], 2 * e * (1 + finite(fwd["entropy"])), "entropy")
    want = ref.logprobs_grad(seen, tokens, None if d_l is None else w, None if d_h is None else h, t)
    q, log_q = softmax(seen, t)
    scale = ((np.abs(w) if d_l is not None else 0) + (np.abs(h) * (1 + finite(fwd["entropy"])) if d_h is not None else 0)) / t
    scale = np.broadcast_to(scale, (rows,))
    close(g, want, gradient_tolerance(dtype, vocab, want, scale, q, log_q, tokens), "gradient")
    nsm.logprobs_grad(logits, tk, d_l, d_h, logits, temperature=t)  # in place: the same bits
    assert torch.equal(logits, g)
