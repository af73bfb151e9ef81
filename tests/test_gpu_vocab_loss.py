"""Losses over a vocabulary on the GPU against the float64 oracle: log probabilities of given
tokens with entropy and top alternatives, distillation from top logits, forward, backward
and in one call.

Tolerances, from the arithmetic.  u = 2^-24 is fp32's unit.  An exponential has a relative
error of at most 2^-22 from ex2 plus what its argument's rounding gives: (x - ref) and its
product with log2(e)/t are each good to u, and terms further than about 30 below the largest
do not matter, so 60 u; one more factor of ex2 when partial sums meet.  A sum of V terms
passes through at most V/256 additions in one thread and some 40 across threads, each u of
the sum.  So a sum of exponentials is relatively good to

    E(V) = (4 + 60 + 4 + 40 + V/256) u

and its logarithm absolutely to that, plus 2 u of the results' own sizes.  Differences of
two such numbers (a log probability, an entropy, a loss term) get twice E.  A gradient is a
probability (relative error E plus 4 u times its own |log q|, and |lse| u where a stored
lse is read back) times weights, rounded once to its type; fp16 and subnormal steps add half
of the type's smallest step.
"""

import numpy as np
import pytest
import torch

from oracle import vocab_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": U}  # half a unit in the last place: 8, 11, 24 bits
SMALLEST = {"bf16": 2.0 ** -126, "fp16": 2.0 ** -25, "fp32": 2.0 ** -126}


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_orthogonalized_gb300 as m
    m.lib()
    return m


def e_of(vocab):
    return (108 + vocab / 256) * U


def on_gpu(x, dtype, pad=0, offset=0):
    """x as a view of a wider buffer: row stride vocab + pad, first element `offset` in.  What
    surrounds the rows is NaN, so that reading it would show."""
    rows, vocab = x.shape
    buf = torch.full((rows * (vocab + pad) + offset + 8,), float("nan"), dtype=TYPES[dtype], device="cuda")
    view = buf[offset:offset + rows * (vocab + pad)].view(rows, vocab + pad)[:, :vocab]
    view.copy_(torch.from_numpy(x).to(TYPES[dtype]))
    return view, view.double().cpu().numpy()


def make_rows(seed, rows, vocab, spread=3.0):
    """Rows of several kinds: a bell, one token far ahead, masked tokens, nothing left, all
    equal, the lowest values, a rising row, large values of both signs."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, vocab)) * spread
    for r in range(rows):
        kind = r % 8
        if kind == 1:
            x[r, rng.integers(vocab)] += 25
        elif kind == 2:
            x[r, rng.random(vocab) < 0.6] = -np.inf
        elif kind == 3:
            x[r] = -np.inf
        elif kind == 4:
            x[r] = 0.5
        elif kind == 5:
            x[r] = -65504.0
        elif kind == 6:
            x[r] = np.sort(x[r])
        elif kind == 7:
            x[r] = np.round(x[r]) * 500
    return x


def make_tokens(seed, rows, vocab):
    rng = np.random.default_rng(seed + 1)
    t = rng.integers(0, vocab, rows)
    t[rng.random(rows) < 0.2] = -100
    if rows > 2:
        t[1], t[2] = vocab, vocab - 1
    return t


def close(got, want, tol, what):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        bad = ~same & ~(np.abs(got - want) <= tol)
    if bad.any():
        at = tuple(int(v) for v in np.argwhere(bad)[0])
        limit = np.broadcast_to(tol, want.shape)[at]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {at}: {got[at]!r} for "
                             f"{want[at]!r}, allowed {limit!r}")


def finite(a):
    return np.where(np.isfinite(a), np.abs(a), 0.0)


def outputs(rows, k=0):
    o = {n: torch.full((rows,), 7.0, device="cuda") for n in ("logprob", "entropy", "lse", "loss", "rest")}
    o["top_logprob"] = torch.full((rows, k), 7.0, device="cuda")
    o["top_index"] = torch.full((rows, k), 7, dtype=torch.int32, device="cuda")
    return o


VOCABS = [1, 2, 7, 8, 9, 63, 259, 1000, 2048, 4099, 16384, 50257, 131072, 262147]


def check_logprobs(nsm, x, dtype, tokens, temperature, k, pad=0, offset=0, wide=True):
    logits, seen = on_gpu(x, dtype, pad, offset)
    rows, vocab = x.shape
    o = outputs(rows, k)
    t = torch.from_numpy(tokens).to(torch.int64 if wide else torch.int32).cuda()
    top = {"top_logprob": o["top_logprob"], "top_index": o["top_index"]} if k else {}
    nsm.logprobs(logits, t, o["logprob"], o["entropy"], o["lse"], temperature=temperature, **top)
    want = ref.logprobs(seen, tokens, temperature, k)
    e = e_of(vocab)
    span = finite(seen).max(axis=1) / temperature
    close(o["lse"], want["lse"], e + 4 * U * (finite(want["lse"]) + span), "lse")
    close(o["logprob"], want["logprob"], 2 * e + 4 * U * finite(want["logprob"]), "logprob")
    close(o["entropy"], want["entropy"], 2 * e * (1 + finite(want["entropy"])), "entropy")
    if k:
        assert np.array_equal(o["top_index"].cpu().numpy(), want["top_index"])
        close(o["top_logprob"], want["top_logprob"], 2 * e + 4 * U * finite(want["top_logprob"]), "top_logprob")
    return logits, seen, t, o


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", VOCABS)
def test_logprobs(nsm, dtype, vocab):
    rows = 9 if vocab < 100000 else 8
    x = make_rows(vocab, rows, vocab)
    check_logprobs(nsm, x, dtype, make_tokens(vocab, rows, vocab), 1.0, min(20, vocab))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 5), (8, 8), (16, 2)])
def test_logprobs_strides(nsm, dtype, pad, offset):
    for vocab in (5, 1001, 8200):
        x = make_rows(pad + offset, 9, vocab)
        check_logprobs(nsm, x, dtype, make_tokens(3, 9, vocab), 0.8, min(7, vocab), pad, offset, wide=False)


@pytest.mark.parametrize("temperature", [0.05, 0.7, 3.0, 100.0])
def test_logprobs_temperatures(nsm, temperature):
    x = make_rows(5, 8, 3001)
    check_logprobs(nsm, x, "bf16", make_tokens(5, 8, 3001), temperature, 5)


@pytest.mark.parametrize("k", [1, 2, 31, 64, 127, 128])
@pytest.mark.parametrize("vocab", [100, 128, 1500, 2600, 33001])
def test_top_alternatives(nsm, k, vocab):
    # also where fewer than k logits are left, and where bf16 values repeat a lot
    for dtype in ("bf16", "fp32"):
        x = make_rows(k, 8, vocab, spread=1.0)
        check_logprobs(nsm, x, dtype, make_tokens(k, 8, vocab), 1.0, k)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_top_alternatives_in_few_places(nsm, dtype):
    # the largest logits all at one distance from one another, so that few threads hold
    # them, and rows of two values only, with zeros of both signs
    vocab, rows = 70000, 6
    rng = np.random.default_rng(8)
    x = rng.normal(size=(rows, vocab))
    for r, stride in enumerate((1024, 2048, 4096, 8192)):
        at = np.arange(r, vocab, stride)
        x[r, at] = 40 + rng.normal(size=len(at))
        for j in range(1, 8):  # and whole vectors there
            x[r, np.minimum(at + j, vocab - 1)] = 40 + rng.normal(size=len(at))
    x[4] = np.where(rng.random(vocab) < 0.5, 0.0, -0.0)
    x[5] = np.where(rng.random(vocab) < 0.001, 1.0, -1.0)
    for k in (1, 20, 128):
        check_logprobs(nsm, x, dtype, make_tokens(1, rows, vocab), 1.0, k)


def test_top_alternatives_many_in_few_vectors(nsm):
    # fewer threads than k have any logit left, and they have more than a thousand of them
    vocab = 200000
    x = np.full((2, vocab), -np.inf)
    rng = np.random.default_rng(9)
    for block in range(0, vocab, 2048):
        x[0, block:block + 512] = rng.normal(size=512)[: max(0, min(512, vocab - block))]
        x[1, block:block + 24] = 1.0
    check_logprobs(nsm, x, "bf16", np.array([0, 1]), 1.0, 128)
    check_logprobs(nsm, x, "fp32", np.array([0, 1]), 1.0, 128)


def test_lowest_values_and_huge_values(nsm):
    # the types' lowest finite value is a logit like any other, also beside larger ones
    low = float(torch.finfo(torch.bfloat16).min)
    x = np.full((4, 3000), low)
    x[1, 17] = 0.0
    x[2, :] = 1e38
    x[3, ::2] = 3e38
    for dtype in ("bf16", "fp32"):
        logits, seen = on_gpu(x, dtype)
        o = outputs(4)
        tokens = np.array([5, 17, 9, 2])
        nsm.logprobs(logits, torch.from_numpy(tokens).cuda(), o["logprob"], o["entropy"], o["lse"])
        want = ref.logprobs(seen, tokens)
        close(o["logprob"], want["logprob"], 2 * e_of(3000), "logprob")
        close(o["entropy"], want["entropy"], 2 * e_of(3000) * 10, "entropy")
        close(o["lse"], want["lse"], 4 * U * finite(want["lse"]) + e_of(3000), "lse")
        g = torch.empty_like(logits)
        ones = torch.ones(4, device="cuda")
        nsm.logprobs_grad(logits, torch.from_numpy(tokens).cuda(), ones, None, g)
        close(g, ref.logprobs_grad(seen, tokens, np.ones(4), None), STEP[dtype] * 1.01 + e_of(3000), "gradient")


def test_not_a_number_stays_in_its_row(nsm):
    x = make_rows(3, 9, 5003)
    x[0, 77] = np.nan
    x[4, 4000] = np.inf
    x[3, 5] = np.nan  # an otherwise empty row
    logits, seen, t, o = check_logprobs(nsm, x, "fp32", make_tokens(3, 9, 5003), 1.0, 11)
    w = torch.ones(9, device="cuda")
    w[0] = 0.0  # no weight: zeros whatever the row holds
    g = torch.empty_like(logits)
    tokens = t.cpu().numpy()
    nsm.logprobs_grad(logits, t, w, None, g)
    want = ref.logprobs_grad(seen, tokens, w.cpu().numpy(), None)
    assert np.array_equal(np.isnan(g.cpu().numpy()), np.isnan(want))
    assert not g[0].any()


def gradient_tolerance(dtype, vocab, want, scale, q, log_q, tokens, lse=None):
    """Per element: the probability's error times the weights (at the token 1 - q takes the
    place of q: three products and its own rounding), and the one rounding to the type."""
    e = 2 * e_of(vocab) + 4 * U * finite(log_q) + (0 if lse is None else 4 * U * finite(lse)[:, None])
    token = np.zeros_like(q)
    for r, v in enumerate(tokens):
        if 0 <= v < vocab:
            token[r, v] = 5 * U * scale[r]
    return token + scale[:, None] * q * e * (1 + finite(log_q)) + 1.01 * STEP[dtype] * finite(want) + SMALLEST[dtype]


def softmax(seen, temperature):
    y = seen / temperature
    top = np.max(y, axis=1, keepdims=True)
    top = np.where(np.isfinite(top), top, 0.0)
    s = np.exp(y - top)
    total = s.sum(axis=1, keepdims=True)
    total = np.where(total == 0, 1.0, total)
    return s / total, (y - top) - np.log(total)


GRAD_VOCABS = [1, 3, 8, 17, 259, 1000, 4099, 20001, 50257, 131073, 300007]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", GRAD_VOCABS)
@pytest.mark.parametrize("weights", ["token", "entropy", "both"])
def test_logprobs_gradients(nsm, dtype, vocab, weights):
    rows, t = 8, 0.9
    x = make_rows(vocab + 1, rows, vocab)
    tokens = make_tokens(vocab, rows, vocab)
    logits, seen = on_gpu(x, dtype, pad=vocab % 5, offset=vocab % 3)
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
    close(g, want, gradient_tolerance(dtype, vocab, want, scale, q, log_q, tokens), "gradient in one call")
    # the backward pass alone, from the library's own statistics
    back = torch.full_like(logits, float("nan"))
    nsm.logprobs_backward(logits, tk, o["lse"], o["entropy"], d_l, d_h, back, temperature=t)
    lse, ent = o["lse"].double().cpu().numpy(), o["entropy"].double().cpu().numpy()
    want = ref.logprobs_grad(seen, tokens, None if d_l is None else w, None if d_h is None else h, t, lse, ent)
    close(back, want, gradient_tolerance(dtype, vocab, want, scale, q, log_q, tokens, lse), "backward alone")
    # in place gives the same bits
    place = logits.clone() if logits.is_contiguous() else logits
    nsm.logprobs_grad(place, tk, d_l, d_h, place, temperature=t)
    if place.data_ptr() % 16 == logits.data_ptr() % 16 and place.stride() == logits.stride():
        assert torch.equal(place, g)


def make_entries(seed, x, k, temperature, tail):
    """Entries around the student's largest logits, some missing, some given twice."""
    rng = np.random.default_rng(seed)
    rows, vocab = x.shape
    index = np.full((rows, k), -1, dtype=np.int64)
    z = rng.normal(size=(rows, k))
    for r in range(rows):
        noisy = np.where(np.isfinite(x[r]), x[r], -1e3) / 300 + rng.normal(size=vocab) * 2
        n = min(k, vocab)
        order = np.argsort(-noisy, kind="stable")[:n]
        index[r, :n] = order
        if tail:
            y = noisy - noisy.max()
            z[r, :n] = (y - np.log(np.exp(y).sum()))[order]
        else:
            z[r, :n] = noisy[order]
    if k > 3 and rows > 5:
        index[1, 2] = index[1, 0]   # given twice
        index[1, 3] = vocab + 7     # outside
        index[2, :] = -1            # no entries
        z[4, 1] = -np.inf           # an entry without mass
    return z, index


def check_distill(nsm, x, dtype, k, temperature, tail, teacher_dtype="fp32", pad=0, offset=0, wide=True, seed=0):
    rows, vocab = x.shape
    logits, seen = on_gpu(x, dtype, pad, offset)
    z, index = make_entries(seed + k, x, k, temperature, tail)
    teacher = torch.from_numpy(z).to(TYPES[teacher_dtype]).cuda()
    z = teacher.double().cpu().numpy()
    ix = torch.from_numpy(index).to(torch.int64 if wide else torch.int32).cuda()
    want = ref.distill(seen, z, index, temperature, tail)
    e = e_of(vocab)
    # a term is p times a difference of logs: sum p is at most about 1
    logs = finite(want["lse"]) + finite(seen).max(axis=1) / temperature + 40
    loss_tol = 4 * e + 8 * U * logs * (1 if tail else 2)
    o = outputs(rows)
    nsm.distill(logits, teacher, ix, o["loss"], o["lse"], o["rest"], temperature=temperature, tail=tail)
    span = finite(seen).max(axis=1) / temperature
    close(o["lse"], want["lse"], e + 4 * U * (finite(want["lse"]) + span), "lse")
    close(o["rest"], want["rest"], 2 * e + 4 * U * (finite(want["rest"]) + span), "rest")
    close(o["loss"], want["loss"], loss_tol + 4 * U * finite(want["loss"]), "loss")
    rng = np.random.default_rng(3)
    w = rng.normal(size=rows).astype(np.float32)
    w[rows - 1] = 0.0
    d_loss = torch.from_numpy(w).cuda()
    g = torch.full_like(logits, float("nan"))
    o2 = outputs(rows)
    nsm.distill_grad(logits, teacher, ix, d_loss, g, o2["loss"], o2["lse"], o2["rest"], temperature=temperature,
                     tail=tail)
    close(o2["loss"], want["loss"], loss_tol + 4 * U * finite(want["loss"]), "loss in one call")
    wg = ref.distill_grad(seen, z, index, w, temperature, tail)
    q, log_q = softmax(seen, temperature)
    p = np.zeros_like(q)
    for r in range(rows):
        tok, pr, _, p_rest, some = ref._teacher(seen[r], z[r], index[r], temperature, tail)
        if some:
            p[r, tok] = pr
            if tail and np.isfinite(want["rest"][r]):
                out = np.ones(vocab, dtype=bool)
                out[tok] = False
                p[r, out] += p_rest * np.exp(log_q[r, out] - want["rest"][r])
    # q and p (the teacher's logs are as large as `logs`) each with the error of a probability
    scale = np.abs(w) / temperature
    rel = 2 * e + 4 * U * (finite(log_q) + logs[:, None])
    tol = scale[:, None] * (q + p) * rel + 1.01 * STEP[dtype] * finite(wg) + SMALLEST[dtype]
    close(g, wg, tol, "gradient in one call")
    back = torch.full_like(logits, float("nan"))
    nsm.distill_backward(logits, teacher, ix, o["lse"], o["rest"] if tail else None, d_loss, back,
                         temperature=temperature, tail=tail)
    close(back, wg, 2 * tol, "backward alone")  # the stored lse and rest carry their own errors
    place = logits.clone() if logits.is_contiguous() else logits
    nsm.distill_grad(place, teacher, ix, d_loss, place, temperature=temperature, tail=tail)
    if place.data_ptr() % 16 == logits.data_ptr() % 16 and place.stride() == logits.stride():
        assert torch.equal(place, g)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", GRAD_VOCABS)
@pytest.mark.parametrize("tail", [False, True])
def test_distill(nsm, dtype, vocab, tail):
    x = make_rows(vocab, 8, vocab)
    check_distill(nsm, x, dtype, 16, 1.0, tail, seed=vocab)


@pytest.mark.parametrize("k", [1, 2, 5, 33, 127, 128])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_entries(nsm, k, tail):
    x = make_rows(k, 8, 2003)
    check_distill(nsm, x, "bf16", k, 1.5, tail, "bf16" if not tail else "fp32", pad=3, offset=1, wide=False, seed=k)
    check_distill(nsm, x[:, :100], "fp32", k, 1.0, tail, "fp16" if not tail else "fp32", seed=k)


RING = [("bf16", 50257, 640, 0), ("fp16", 100003, 320, 1), ("fp32", 33001, 640, 3), ("fp32", 70001, 320, 0),
        ("bf16", 131072, 330, 0), ("bf16", 262147, 100, 5), ("bf16", 40000, 700, 8)]


@pytest.mark.parametrize("dtype,vocab,rows,pad", RING)
@pytest.mark.parametrize("op", ["logprobs", "entropy", "distill", "tail"])
def test_gradients_of_many_long_rows(nsm, dtype, vocab, rows, pad, op):
    # rows enough to go round the GPU, each too long for several to a block's shared memory:
    # against the oracle for some of every kind of row, and every row's numbers
    base = make_rows(vocab, 16, vocab)
    order = np.arange(rows) % 16
    buf = torch.full((rows * (vocab + pad) + 8,), float("nan"), dtype=TYPES[dtype], device="cuda")
    logits = buf[3:3 + rows * (vocab + pad)].view(rows, vocab + pad)[:, :vocab]
    logits.copy_(torch.from_numpy(base).to(TYPES[dtype]).cuda()[torch.from_numpy(order).cuda()])
    # rows differ by one logit each
    spot = torch.arange(rows, device="cuda") * 131 % vocab
    alive = ~torch.isinf(logits[torch.arange(rows, device="cuda"), spot])
    logits[torch.arange(rows, device="cuda")[alive], spot[alive]] += 1.0
    rng = np.random.default_rng(vocab)
    w = rng.normal(size=rows).astype(np.float32)
    w[::11] = 0.0
    weight = torch.from_numpy(w).cuda()
    t = 1.1
    sample = sorted({0, rows - 1, *range(rows // 2, rows // 2 + 8), *rng.integers(0, rows, 6).tolist()})
    seen = logits[sample].double().cpu().numpy()
    o = outputs(rows)
    g = torch.full_like(logits, float("nan"))
    e = e_of(vocab)
    q, log_q = softmax(seen, t)
    if op in ("logprobs", "entropy"):
        tokens = make_tokens(vocab, rows, vocab)
        h = (rng.normal(size=rows) * 0.2).astype(np.float32) if op == "entropy" else None
        d_h = torch.from_numpy(h).cuda() if h is not None else None
        tk = torch.from_numpy(tokens).cuda()
        nsm.logprobs_grad(logits, tk, weight, d_h, g, o["logprob"], o["entropy"], o["lse"], temperature=t)
        fwd = ref.logprobs(seen, tokens[sample], t)
        close(o["logprob"][sample], fwd["logprob"], 2 * e + 4 * U * finite(fwd["logprob"]), "logprob")
        close(o["entropy"][sample], fwd["entropy"], 2 * e * (1 + finite(fwd["entropy"])), "entropy")
        want = ref.logprobs_grad(seen, tokens[sample], w[sample], None if h is None else h[sample], t)
        scale = (np.abs(w[sample]) + (0 if h is None else np.abs(h[sample]) * (1 + finite(fwd["entropy"])))) / t
        close(g[sample], want, gradient_tolerance(dtype, vocab, want, scale, q, log_q, tokens[sample]), "gradient")
        alone = torch.empty(rows, device="cuda")
        nsm.logprobs(logits, tk, alone, temperature=t)
        close(o["logprob"], alone.double().cpu().numpy(), 4 * e + 8 * U * finite(alone.double().cpu().numpy()), "logprob")
        back = torch.full_like(logits, float("nan"))
        nsm.logprobs_backward(logits, tk, o["lse"], o["entropy"], weight, d_h, back, temperature=t)
        again = torch.full_like(logits, float("nan"))
        nsm.logprobs_grad(logits, tk, weight, d_h, again, temperature=t)
        nsm.logprobs_grad(logits, tk, weight, d_h, logits, temperature=t)
    else:
        tail = op == "tail"
        z16, index16 = make_entries(7, base, 40, t, tail)
        z, index = z16[order], index16[order]
        teacher, ix = torch.from_numpy(z).float().cuda(), torch.from_numpy(index).cuda()
        z = teacher.double().cpu().numpy()
        nsm.distill_grad(logits, teacher, ix, weight, g, o["loss"], o["lse"], o["rest"], temperature=t, tail=tail)
        fwd = ref.distill(seen, z[sample], index[sample], t, tail)
        logs = finite(fwd["lse"]) + finite(seen).max(axis=1) / t + 40
        tol = 4 * e + 8 * U * logs * (1 if tail else 2) + 4 * U * finite(fwd["loss"])
        close(o["loss"][sample], fwd["loss"], tol, "loss")
        want = ref.distill_grad(seen, z[sample], index[sample], w[sample], t, tail)
        p = np.zeros_like(q)
        for j, r in enumerate(sample):
            tok, pr, _, p_rest, some = ref._teacher(seen[j], z[r], index[r], t, tail)
            if some:
                p[j, tok] = pr
                if tail and np.isfinite(fwd["rest"][j]):
                    out = np.ones(vocab, dtype=bool)
                    out[tok] = False
                    p[j, out] += p_rest * np.exp(log_q[j, out] - fwd["rest"][j])
        rel = 2 * e + 4 * U * (finite(log_q) + logs[:, None])
        tol = (np.abs(w[sample]) / t)[:, None] * (q + p) * rel + 1.01 * STEP[dtype] * finite(want) + SMALLEST[dtype]
        close(g[sample], want, tol, "gradient")
        alone = torch.empty(rows, device="cuda")
        nsm.distill(logits, teacher, ix, alone, temperature=t, tail=tail)
        ref_loss = alone.double().cpu().numpy()
        span = 40 + float(logits.float()[torch.isfinite(logits)].abs().max()) / t
        close(o["loss"], ref_loss, 8 * e + 32 * U * span * 2 + 8 * U * finite(ref_loss), "loss")
        back = torch.full_like(logits, float("nan"))
        nsm.distill_backward(logits, teacher, ix, o["lse"], o["rest"] if tail else None, weight, back, temperature=t, tail=tail)
        again = torch.full_like(logits, float("nan"))
        nsm.distill_grad(logits, teacher, ix, weight, again, temperature=t, tail=tail)
        nsm.distill_grad(logits, teacher, ix, weight, logits, temperature=t, tail=tail)
    assert torch.equal(again, g)  # the same bits again
    assert torch.equal(logits, g)  # and in place
    # every row against the backward pass alone, whose statistics carry their own rounding: a
    # step of the type and the statistics' error on values of at most the row's weight
    far = (back.float() - g.float()).abs()
    lse_size = 8 * e + 16 * U * (float(o["lse"][torch.isfinite(o["lse"])].abs().max()) + 40)
    allowed = 2.1 * STEP[dtype] * g.float().abs() + lse_size * (2 * weight.abs() / t + 1)[:, None] * 2 + 2 * SMALLEST[dtype]
    assert bool((far <= allowed).all())


def test_distill_without_weights_is_weight_one(nsm):
    x = make_rows(11, 8, 700)
    logits, seen = on_gpu(x, "fp32")
    z, index = make_entries(4, x, 9, 1.0, False)
    teacher, ix = torch.from_numpy(z).float().cuda(), torch.from_numpy(index).cuda()
    a, b = torch.empty_like(logits), torch.empty_like(logits)
    nsm.distill_grad(logits, teacher, ix, None, a)
    nsm.distill_grad(logits, teacher, ix, torch.ones(8, device="cuda"), b)
    assert torch.equal(a, b)


def test_distill_not_a_number(nsm):
    x = make_rows(3, 8, 1500)
    x[0, 7] = np.nan
    logits, seen = on_gpu(x, "fp32")
    z, index = make_entries(4, x, 9, 1.0, False)
    z[4, 3] = np.nan
    z[6, 0] = np.inf
    teacher, ix = torch.from_numpy(z).float().cuda(), torch.from_numpy(index).cuda()
    o = outputs(8)
    w = torch.ones(8, device="cuda")
    w[6] = 0.0
    g = torch.empty_like(logits)
    nsm.distill_grad(logits, teacher, ix, w, g, o["loss"])
    loss = o["loss"].cpu().numpy()
    assert np.isnan(loss[[0, 4, 6]]).all() and not np.isnan(loss[[1, 2, 5, 7]]).any()
    assert torch.isnan(g[0]).any() and torch.isnan(g[4]).any() and not g[6].any()
    assert not torch.isnan(g[[1, 2, 3, 5, 7]]).any()


def test_the_teachers_top_is_the_students_target(nsm):
    # logprobs' alternatives go into distill with the tail as they are; the teacher itself as
    # the student has no loss and no gradient
    x = np.random.default_rng(5).normal(size=(6, 9000)) * 3
    logits, _ = on_gpu(x, "fp32")
    o = outputs(6, 50)
    nsm.logprobs(logits, None, lse=o["lse"], top_logprob=o["top_logprob"], top_index=o["top_index"])
    g = torch.empty_like(logits)
    nsm.distill_grad(logits, o["top_logprob"], o["top_index"], None, g, o["loss"], tail=True)
    tol = 4 * e_of(9000) + 80 * U
    assert float(o["loss"].abs().max()) <= tol
    assert float(g.abs().max()) <= tol


@pytest.mark.parametrize("op", ["logprobs", "distill"])
def test_gradient_against_differences(nsm, op):
    # the kernels' own losses along one direction: f(x + s d) - f(x - s d) over 2 s.  Each
    # loss is off by at most 4 E, so the quotient by 4 E / s, and the third derivative along
    # d (entries +-1, at most 8 in size) adds 8 s^2 / 6.
    vocab, rows, s = 6000, 4, 2.0 ** -6
    rng = np.random.default_rng(12)
    x = rng.normal(size=(rows, vocab)) * 2
    d = np.sign(rng.normal(size=(rows, vocab)))
    tokens = torch.from_numpy(rng.integers(0, vocab, rows)).cuda()
    z, index = make_entries(2, x * 300, 12, 1.0, True)
    teacher, ix = torch.from_numpy(z).float().cuda(), torch.from_numpy(index).cuda()
    base = torch.from_numpy(x).float().cuda()
    # steps that are exact in fp32
    base = torch.round(base * 256) / 256
    step = torch.from_numpy(d).float().cuda() * s
    one = torch.ones(rows, device="cuda")

    def value(y):
        o = outputs(rows)
        if op == "logprobs":
            nsm.logprobs(y, tokens, o["logprob"], o["entropy"])
            return (o["logprob"].double() + 0.5 * o["entropy"].double())
        nsm.distill(y, teacher, ix, o["loss"], tail=True)
        return o["loss"].double()

    g = torch.empty_like(base)
    if op == "logprobs":
        nsm.logprobs_grad(base, tokens, one, 0.5 * one, g)
    else:
        nsm.distill_grad(base, teacher, ix, None, g, tail=True)
    along = (g.double() * torch.from_numpy(d).cuda()).sum(1)
    quotient = (value(base + step) - value(base - step)) / (2 * s)
    # along: a sum of vocab fp32 gradients of total size at most 2 (1 + log vocab)
    tol = 6 * e_of(vocab) * (1 + np.log(vocab)) / s + 8 * s * s / 6 * (1 + np.log(vocab))
    assert float((along - quotient).abs().max()) <= tol


@pytest.mark.parametrize("rows", [0, 1, 2, 151, 152, 700, 5000])
def test_rows(nsm, rows):
    # every number of rows gives each row what it gets alone
    vocab = 515
    x = torch.randn(max(rows, 1), vocab, generator=torch.Generator().manual_seed(rows)).mul(3).bfloat16().cuda()[:rows]
    tokens = torch.arange(rows, device="cuda") % vocab
    teacher, index = torch.topk(torch.randn(max(rows, 1), vocab, device="cuda")[:rows], 6) if rows else (
        torch.empty(0, 6, device="cuda"), torch.empty(0, 6, dtype=torch.int64, device="cuda"))
    o = outputs(rows, 4)
    nsm.logprobs(x, tokens, o["logprob"], o["entropy"], o["lse"], o["top_logprob"], o["top_index"])
    g, g2 = torch.empty_like(x), torch.empty_like(x)
    w = torch.full((rows,), 0.5, device="cuda")
    nsm.logprobs_grad(x, tokens, w, w, g)
    nsm.distill_grad(x, teacher, index, w, g2, o["loss"])
    for r in sorted({0, rows // 2, rows - 1}) if rows else []:
        one = outputs(1, 4)
        a, b = torch.empty_like(x[:1]), torch.empty_like(x[:1])
        s = slice(r, r + 1)
        nsm.logprobs(x[s], tokens[s], one["logprob"], one["entropy"], one["lse"], one["top_logprob"], one["top_index"])
        nsm.logprobs_grad(x[s], tokens[s], w[s], w[s], a)
        nsm.distill_grad(x[s], teacher[s], index[s], w[s], b, one["loss"])
        e = e_of(vocab)
        for n in ("logprob", "entropy", "lse", "loss", "top_logprob"):
            close(one[n], o[n][s].double().cpu().numpy(), 2 * e * 20, n)
        assert torch.equal(one["top_index"], o["top_index"][s])
        close(a, g[s].double().cpu().numpy(), 1e-6 + 2 * STEP["bf16"] * finite(g[s].double().cpu().numpy()), "gradient")
        close(b, g2[s].double().cpu().numpy(), 1e-6 + 2 * STEP["bf16"] * finite(g2[s].double().cpu().numpy()), "gradient")


def test_same_bits_again_and_on_another_stream(nsm):
    x, _ = on_gpu(make_rows(21, 40, 30011), "bf16")
    tokens = torch.from_numpy(make_tokens(2, 40, 30011)).cuda()
    w = torch.ones(40, device="cuda")
    torch.cuda.synchronize()
    results = []
    for stream in (None, None, torch.cuda.Stream()):
        o = outputs(40, 20)
        g = torch.empty_like(x)
        torch.cuda.synchronize()
        nsm.logprobs(x, tokens, o["logprob"], o["entropy"], o["lse"], o["top_logprob"], o["top_index"], stream=stream)
        nsm.logprobs_grad(x, tokens, w, w, g, stream=stream)
        torch.cuda.synchronize()
        results.append([o[n] for n in ("logprob", "entropy", "lse", "top_logprob", "top_index")] + [g])
    for other in results[1:]:
        for a, b in zip(results[0], other):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_in_a_graph(nsm):
    x, seen = on_gpu(make_rows(22, 6, 5000), "bf16")
    tokens = torch.arange(6, device="cuda")
    o = outputs(6, 3)
    g = torch.empty_like(x)
    w = torch.ones(6, device="cuda")

    def calls(stream):
        nsm.logprobs(x, tokens, o["logprob"], o["entropy"], o["lse"], o["top_logprob"], o["top_index"], stream=stream)
        nsm.logprobs_grad(x, tokens, w, None, g, stream=stream)

    s = torch.cuda.Stream()
    calls(s)
    torch.cuda.synchronize()
    first = [o["logprob"].clone(), o["top_index"].clone(), g.clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        calls(torch.cuda.current_stream())
    o["logprob"].zero_()
    g.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, [o["logprob"], o["top_index"], g]):
        assert torch.equal(a, b)


def test_offsets_past_32_bits(nsm):
    # rows far apart: the last one starts beyond 2^32 bytes and 2^31 elements
    vocab, rows, ld = 1003, 3, (1 << 30) + 5
    buf = torch.zeros((rows - 1) * ld + vocab + 8, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((rows, vocab), (ld, 1))
    values = make_rows(1, rows, vocab)
    x.copy_(torch.from_numpy(values).bfloat16())
    seen = x.double().cpu().numpy()
    tokens = np.array([3, 1002, 0])
    o = outputs(rows, 5)
    t = torch.from_numpy(tokens).cuda()
    nsm.logprobs(x, t, o["logprob"], o["entropy"], o["lse"], o["top_logprob"], o["top_index"])
    want = ref.logprobs(seen, tokens, 1.0, 5)
    close(o["logprob"], want["logprob"], 2 * e_of(vocab) + 4 * U * finite(want["logprob"]), "logprob")
    assert np.array_equal(o["top_index"].cpu().numpy(), want["top_index"])
    w = np.ones(rows, dtype=np.float32)
    nsm.logprobs_grad(x, t, torch.from_numpy(w).cuda(), None, x)  # in place
    g = ref.logprobs_grad(seen, tokens, w, None)
    close(x, g, 1.01 * STEP["bf16"] * finite(g) + 2 * e_of(vocab), "gradient")
    assert int(torch.count_nonzero(buf[vocab:ld])) == 0  # nothing was written between the rows


@pytest.mark.parametrize("dtype", list(TYPES))
def test_nothing_is_written_outside_the_rows(nsm, dtype):
    for vocab, pad, offset in ((1, 2, 1), (13, 3, 2), (1029, 5, 7), (8192, 8, 0)):
        rows = 5
        x, _ = on_gpu(make_rows(vocab, rows, vocab), dtype, pad, offset)
        buf = torch.full((rows * (vocab + pad) + offset + 16,), 3.0, dtype=TYPES[dtype], device="cuda")
        g = buf[offset:offset + rows * (vocab + pad)].view(rows, vocab + pad)[:, :vocab]
        w = torch.ones(rows, device="cuda")
        tokens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        nsm.logprobs_grad(x, tokens, w, w, g)
        whole = torch.ones_like(buf, dtype=torch.bool)
        whole[offset:offset + rows * (vocab + pad)].view(rows, vocab + pad)[:, :vocab] = False
        assert bool((buf[whole] == 3.0).all())
        teacher = torch.zeros(rows, 2, device="cuda")
        index = torch.tensor([[0, -1]] * rows, device="cuda")
        nsm.distill_grad(x, teacher, index, None, g)
        assert bool((buf[whole] == 3.0).all())


def test_vocabulary_at_the_limit(nsm):
    vocab = 1 << 20
    x = np.random.default_rng(1).normal(size=(2, vocab)) * 3
    check_logprobs(nsm, x, "fp32", np.array([vocab - 1, 0]), 1.0, 64)
    check_distill(nsm, x, "bf16", 32, 1.0, True)


def test_binding_refusals(nsm):
    x = torch.zeros(3, 10, device="cuda")
    t = torch.zeros(3, dtype=torch.int64, device="cuda")
    f = torch.zeros(3, device="cuda")
    for bad in (lambda: nsm.logprobs(x.double(), t, f), lambda: nsm.logprobs(x.t(), t, f),
                lambda: nsm.logprobs(x[0], t, f), lambda: nsm.logprobs(x, t[:2], f),
                lambda: nsm.logprobs(x, t.float(), f), lambda: nsm.logprobs(x, t, f.double()),
                lambda: nsm.logprobs(x, t.cpu(), f), lambda: nsm.logprobs(x, t, f[:2]),
                lambda: nsm.logprobs(x, t, f, top_logprob=torch.zeros(3, 2, device="cuda")),
                lambda: nsm.logprobs_grad(x, t, f, None, x.bfloat16()),
                lambda: nsm.logprobs_grad(x, t, f, None, None),
                lambda: nsm.distill(x, f, t, f), lambda: nsm.distill(x, x[:, :2], t[:, None], f),
                lambda: nsm.distill(x, x[:, :2], t[:, None].expand(3, 2).float(), f)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(nsm.NsmError):
        nsm.logprobs(x, t)  # nothing is asked for
    with pytest.raises(nsm.NsmError):
        nsm.logprobs(x, t, f, temperature=0.0)
    with pytest.raises(nsm.NsmError):
        nsm.logprobs_backward(x, t, f, None, torch.ones(3, device="cuda"), f, torch.empty_like(x))
    assert nsm.device_status() == nsm.NSM_OK
