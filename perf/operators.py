"""Cases that measure the library's vocabulary losses: the log probabilities of given tokens
(with entropy and top alternatives) and distillation from a teacher's top logits, each
forward, backward, and both in one call.

``listed()`` gives the named cases, ``draw(rng)`` one more of the same ranges.
``prepare(case, seed)`` makes what a training or scoring program holds before the call,
``run(state)`` makes the call: in plain torch operations on 32-bit values where ``own`` is
false, through the library where it is true.  ``exact(case, seed)`` computes the outputs in
64 bits from the definitions, and ``work(case)`` says what a pass cannot do without.

Definitions, for one row x of V logits at temperature t, y = x / t:
    lse     = log sum_v exp(y_v)
    q_v     = exp(y_v - lse)
    logprob = y_token - lse          (0 where the token is outside [0, V): no token)
    entropy = -sum_v q_v log q_v     (0 log 0 = 0)
    top     = the k largest logits, ties to the lowest index, as y_v - lse with index v;
              a logit of -inf is no alternative (-inf and index -1 fill up)
  and for a teacher's entries (score z_j, index i_j, j < K; entries whose index is outside
  [0, V) do not count), S = the set of their indexes:
    p_j     = softmax over the entries of z_j / t                              (tail off)
    p_j     = exp(z_j), z_j log probabilities, p_rest = max(0, 1 - sum_j p_j)  (tail on)
    rest    = log sum_{v not in S} q_v
    loss    = sum_j p_j (log p_j - log q_{i_j}) [+ p_rest (log p_rest - rest)]
  Gradients are those of sum_r (d_logprob_r logprob_r + d_entropy_r entropy_r) and of
  sum_r d_loss_r loss_r, as far as a logit of -inf can have one: it gets zero.  A row with
  no weight, no target or no finite logit gets zeros.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEVICE = "cuda"
# elements of one piece of the 64-bit computations
EXACT_PIECE = 1 << 26
# bytes of logits in the largest case
MOST_BYTES = 1 << 31


def _case(op, rows, vocab, dtype, name=None, k=0, pad=0, temperature=1.0, entropy=False, tail=False, masked=0.0,
          ignored=0.0, empty=False, wide_index=True):
    case = {"op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "k": k, "pad": pad, "temperature": temperature,
            "entropy": entropy, "tail": tail, "masked": masked, "ignored": ignored, "empty": empty,
            "wide_index": wide_index}
    if name is not None:
        case["name"] = name
    return case


def listed():
    return [
        # one token just sampled: its log probability and five alternatives, on the GPT-2
        # vocabulary (an odd number of columns); latency counts
        _case("logprobs", 1, 50257, "bf16", "score_one_token", k=5, entropy=True),
        # a prompt scored token by token with 20 alternatives, part of it padding
        _case("logprobs", 2048, 50257, "bf16", "score_prompts", k=20, entropy=True, ignored=0.1),
        # a teacher's pass over a large batch: no tokens, 64 top log probabilities a row
        _case("logprobs", 8192, 131072, "bf16", "teacher_targets", k=64, ignored=1.0),
        # the cross-entropy of a training step on the GPT-2 vocabulary, loss and gradient
        _case("logprobs_grad", 8192, 50257, "bf16", "cross_entropy_step", ignored=0.05),
        # a small policy-gradient step in fp32 with an entropy bonus, masked actions, rows
        # that are a view of a wider buffer, and a row that the mask leaves empty
        _case("logprobs_grad", 257, 32003, "fp32", "policy_step_ragged", pad=5, temperature=0.7, entropy=True,
              masked=0.1, empty=True),
        # the backward pass alone where the weights depend on the log probabilities
        _case("logprobs_backward", 4096, 100003, "fp16", "policy_backward", entropy=True, ignored=0.05),
        # the same for one short sequence
        _case("logprobs_backward", 33, 50257, "bf16", "policy_backward_short", entropy=False, temperature=1.3),
        # the distillation loss over a validation batch
        _case("distill", 1024, 50257, "bf16", "distill_eval", k=32, temperature=2.0),
        # the same for a few rows in fp32 with the rest of the teacher's mass
        _case("distill", 4, 131072, "fp32", "distill_eval_few", k=128, tail=True, wide_index=False),
        # a distillation step on a large batch and vocabulary, the largest case
        _case("distill_grad", 8192, 131072, "bf16", "distill_step", k=64, tail=True, wide_index=False),
        # a byte-level student: many short rows
        _case("distill_grad", 16384, 259, "bf16", "distill_step_bytes", k=8, temperature=1.5),
        # the distillation's backward pass alone, fp32, an odd vocabulary
        _case("distill_backward", 1000, 65537, "fp32", "distill_backward", k=16, tail=True, ignored=0.05),
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs_grad", "logprobs_backward", "distill", "distill_grad", "distill_backward"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    size = 4 if dtype == "fp32" else 2
    vocab = _log_uniform(rng, 256, 200000)
    pad = rng.choice([0, 0, rng.randint(1, 16)])
    rows = _log_uniform(rng, 1, max(1, min(16384, MOST_BYTES // ((vocab + pad) * size))))
    k = rng.randint(0, 64) if op == "logprobs" else rng.randint(1, 128) if op.startswith("distill") else 0
    return _case(op, rows, vocab, dtype, k=k, pad=pad, temperature=rng.choice([1.0, 1.0, 0.7, 2.0]),
                 entropy=rng.random() < 0.5 and op.startswith("logprobs"),
                 tail=rng.random() < 0.5 and op.startswith("distill"), masked=rng.choice([0.0, 0.0, 0.05]),
                 ignored=rng.choice([0.0, 0.1]), empty=rng.random() < 0.25, wide_index=rng.random() < 0.5)


def prepare(case, seed):
    rows, vocab, t = case["rows"], case["vocab"], case["temperature"]
    dtype = DTYPES[case["dtype"]]
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=DEVICE)

    # a model's logits: a bell with a few units of spread, in half of the rows one token far
    # ahead; masked columns at -inf, and one row with nothing left where the case says so
    x = torch.randn(rows, vocab, generator=g, device=DEVICE).mul_(2.5)
    peak = torch.randint(0, vocab, (rows,), generator=g, device=DEVICE)
    lead = torch.where(uniform(rows) < 0.5, 8 + 8 * uniform(rows), 2 + 2 * uniform(rows))
    x.scatter_add_(1, peak[:, None], lead[:, None])
    if case["masked"]:
        gone = uniform(vocab) < case["masked"]
        x.masked_fill_(gone, -math.inf)
    hidden = [rows // 2] if case["empty"] and rows >= 4 else []

    index_type = torch.int64 if case["wide_index"] else torch.int32
    buffer = torch.empty(rows, vocab + case["pad"], dtype=dtype, device=DEVICE)
    logits = buffer[:, :vocab]
    logits.copy_(x)
    logits[hidden] = -math.inf
    state = {"case": case, "logits": logits}

    def numbers(*shape):
        return torch.empty(*shape, dtype=torch.float32, device=DEVICE)

    live = uniform(rows) >= case["ignored"]
    count = max(1, int(live.sum()))
    # fp16 gradients are taken with a loss scale, as mixed-precision training does
    unit = 1.0 if dtype == torch.float16 else 1.0 / count
    if case["op"].startswith("logprobs"):
        near = uniform(rows) < 0.7
        token = torch.where(near, peak, torch.randint(0, vocab, (rows,), generator=g, device=DEVICE))
        state["tokens"] = torch.where(live, token, -100).to(index_type)
        state["logprob"] = numbers(rows)
        state["lse"] = numbers(rows)
        state["entropy"] = numbers(rows) if case["entropy"] else None
        if case["op"] == "logprobs":
            k = case["k"]
            state["top_logprob"] = numbers(rows, k) if k else None
            state["top_index"] = torch.empty(rows, k, dtype=torch.int32, device=DEVICE) if k else None
            return state
        # minus the mean log probability, weighted by advantages where there is an entropy bonus
        weight = torch.randn(rows, generator=g, device=DEVICE) if case["entropy"] else torch.ones(rows, device=DEVICE)
        state["d_logprob"] = -unit * weight * live
        state["d_entropy"] = torch.full((rows,), -0.05 * unit, device=DEVICE) * live if case["entropy"] else None
        if case["op"] == "logprobs_backward":  # what the forward pass left
            stats = _log_softmax_stats(logits, t)
            state["lse"], state["entropy"] = stats["lse"], stats["entropy"] if case["entropy"] else None
    else:
        k = min(case["k"], vocab)
        x.add_(torch.randn(rows, vocab, generator=g, device=DEVICE).mul_(1.2))  # the teacher's row
        teacher, index = torch.topk(x, k, dim=1)
        if case["tail"]:
            x.div_(t)
            teacher = teacher / t - torch.logsumexp(x, 1, keepdim=True)
        short = uniform(rows) < 0.05  # some teachers gave fewer entries
        drop = short[:, None] & (torch.arange(k, device=DEVICE) >= (k + 1) // 2)
        state["index"] = torch.where(drop, -1, index).to(index_type)
        state["teacher"] = teacher if case["tail"] else teacher.to(dtype)
        state["loss"] = numbers(rows)
        state["lse"] = numbers(rows)
        state["rest"] = numbers(rows) if case["tail"] else None
        if case["op"] == "distill":
            return state
        state["d_loss"] = torch.full((rows,), unit * t * t, device=DEVICE) * live
        if case["op"] == "distill_backward":
            plain = _distill_plain(logits, state["teacher"], state["index"], t, case["tail"])
            state["lse"], state["rest"] = plain["lse"], plain["rest"]
    state["d_logits"] = torch.empty(rows, vocab + case["pad"], dtype=dtype, device=DEVICE)[:, :vocab]
    return state


# ---------------------------------------------------------------- the plain form


def _log_softmax_stats(logits, t):
    """Every row's y, lse, q and entropy on 32-bit values; an empty row has lse -inf."""
    y = logits.float() / t
    top = y.amax(1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    total = (y - top).exp().sum(1).log()  # -inf where the row is empty
    lse = total + top[:, 0]
    log_q = (y - top) - torch.where(total == -math.inf, torch.zeros_like(total), total)[:, None]
    q = log_q.exp()
    entropy = -torch.where(y == -math.inf, torch.zeros_like(q), q * log_q).sum(1)
    return {"y": y, "lse": lse, "q": q, "log_q": log_q, "entropy": entropy}


def _top_plain(logits, s, k):
    """The k largest logits of each row, ties to the lowest index: whole-number keys that hold
    the value's order above the index's."""
    vocab = logits.shape[1]
    bits = (logits.float() + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    key = (order << 32) + (0x7FFFFFFF - torch.arange(vocab, device=logits.device))
    count = min(k, vocab)
    index = 0x7FFFFFFF - (torch.topk(key, count, dim=1).values & 0xFFFFFFFF)
    value = s["log_q"].gather(1, index)
    none = s["y"].gather(1, index) == -math.inf
    top_logprob = torch.full((logits.shape[0], k), -math.inf, device=logits.device)
    top_index = torch.full((logits.shape[0], k), -1, dtype=torch.int32, device=logits.device)
    top_logprob[:, :count] = torch.where(none, torch.full_like(value, -math.inf), value)
    top_index[:, :count] = torch.where(none, torch.full_like(index, -1), index).int()
    return top_logprob, top_index


def _logprobs_plain(state):
    case, logits, tokens = state["case"], state["logits"], state["tokens"].long()
    vocab = logits.shape[1]
    s = _log_softmax_stats(logits, case["temperature"])
    given = (tokens >= 0) & (tokens < vocab)
    at = tokens.clamp(0, vocab - 1)[:, None]
    logprob = s["log_q"].gather(1, at)[:, 0]
    out = {"logprob": torch.where(given, logprob, torch.zeros_like(logprob)), "lse": s["lse"]}
    if case["entropy"]:
        out["entropy"] = s["entropy"]
    if case["op"] == "logprobs" and case["k"]:
        out["top_logprob"], out["top_index"] = _top_plain(logits, s, case["k"])
    return out


def _logprobs_gradient_plain(state, lse=None, entropy=None):
    case, logits, tokens = state["case"], state["logits"], state["tokens"].long()
    vocab, t = logits.shape[1], case["temperature"]
    if lse is None:
        s = _log_softmax_stats(logits, t)
        lse, entropy, log_q, q = s["lse"], s["entropy"], s["log_q"], s["q"]
    else:
        log_q = logits.float() / t - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[:, None]
        q = log_q.exp()
    given = (tokens >= 0) & (tokens < vocab)
    weight = torch.where(given, state["d_logprob"], torch.zeros_like(lse))
    factor = weight[:, None].expand_as(q)
    live = weight != 0
    if state["d_entropy"] is not None:
        spread = torch.where(log_q == -math.inf, torch.zeros_like(log_q), log_q + entropy[:, None])
        factor = factor + state["d_entropy"][:, None] * spread
        live = live | (state["d_entropy"] != 0)
    grad = -q * factor
    # at the token itself 1 - q without cancellation
    at = tokens.clamp(0, vocab - 1)[:, None]
    own_log_q = log_q.gather(1, at)[:, 0]
    hit = grad.gather(1, at)[:, 0] + weight * q.gather(1, at)[:, 0] - weight * torch.expm1(own_log_q)
    hit = torch.where(own_log_q == -math.inf, torch.zeros_like(hit), hit)
    grad.scatter_(1, at, torch.where(given, hit, grad.gather(1, at)[:, 0])[:, None])
    grad = torch.where((live & (lse != -math.inf))[:, None], grad / t, torch.zeros_like(grad))
    return grad.to(logits.dtype)


def _distill_plain(logits, teacher, index, t, tail):
    """Loss, lse and rest of every row on 32-bit values, with what the gradient needs."""
    vocab = logits.shape[1]
    index = index.long()
    kept = (index >= 0) & (index < vocab)
    at = torch.where(kept, index, torch.full_like(index, vocab))  # one column more takes the others
    z = teacher.float()
    z = torch.where(kept, z if tail else z / t, torch.full_like(z, -math.inf))
    if tail:
        log_p = z
    else:
        top = z.amax(1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        log_p = torch.where(z == -math.inf, z, (z - top) - (z - top).exp().sum(1, keepdim=True).log())
    p = log_p.exp()
    y = logits.float() / t
    inside = torch.zeros(logits.shape[0], vocab + 1, dtype=torch.bool, device=logits.device)
    inside.scatter_(1, at, torch.ones_like(kept))
    inside = inside[:, :vocab]
    top = y.amax(1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = (y - top).exp()
    total = e.sum(1).log()
    lse = total + top[:, 0]
    rest = torch.where(inside, torch.zeros_like(e), e).sum(1).log()
    rest = torch.where(rest == -math.inf, rest, rest - total)
    picked = y.gather(1, at.clamp(max=vocab - 1))
    log_q = torch.where(picked == -math.inf, picked, (picked - top) - total[:, None])
    loss = torch.where(p > 0, p * (log_p - log_q), torch.zeros_like(p)).sum(1)
    # 1 - sum p without the largest p's cancellation
    largest, place = log_p.max(1)
    others = p.scatter(1, place[:, None], 0.0).sum(1)
    lacking = -torch.expm1(largest) - others if tail else torch.zeros_like(lse)
    p_rest = lacking.clamp(min=0)
    p_rest = torch.where(rest == -math.inf, torch.zeros_like(p_rest), p_rest)
    any_entry = kept.any(1) if tail else (p > 0).any(1)
    loss = loss + torch.where(p_rest > 0, p_rest * (p_rest.log() - rest), torch.zeros_like(p_rest))
    loss = torch.where(any_entry, loss, torch.zeros_like(loss))
    return {"loss": loss, "lse": lse, "rest": rest if tail else None, "y": y, "p": p, "log_p": log_p, "log_q": log_q,
            "at": at, "inside": inside, "p_rest": p_rest, "excess": p_rest - lacking, "any": any_entry}


def _distill_gradient_plain(state, plain):
    case, d_loss = state["case"], state["d_loss"]
    t, vocab = case["temperature"], state["logits"].shape[1]
    y, p, p_rest, excess = plain["y"], plain["p"], plain["p_rest"], plain["excess"][:, None]
    lse = torch.where(plain["lse"] == -math.inf, torch.zeros_like(plain["lse"]), plain["lse"])
    # sum p + p_rest is 1 + excess
    grad = (y - lse[:, None]).exp() * (1 + excess)
    if case["tail"]:
        rest = torch.where(plain["rest"] == -math.inf, torch.zeros_like(lse), plain["rest"])
        grad = grad - (y - (lse + rest)[:, None]).exp() * p_rest[:, None]
    # at the teacher's entries q - p without cancellation
    log_q, log_p = plain["log_q"], plain["log_p"]
    apart = torch.where(p > 0, p * torch.expm1(log_q - log_p), log_q.exp()) + log_q.exp() * excess
    apart = torch.where(log_q == -math.inf, torch.zeros_like(apart), apart)
    wide = torch.zeros(y.shape[0], vocab + 1, device=y.device).scatter_(1, plain["at"], apart)[:, :vocab]
    grad = torch.where(plain["inside"], wide, grad)
    live = plain["any"] & (d_loss != 0) & (plain["lse"] != -math.inf)
    grad = torch.where(live[:, None], grad * (d_loss / t)[:, None], torch.zeros_like(grad))
    return grad.to(state["logits"].dtype)


def _run_plain(state):
    case = state["case"]
    if case["op"] == "logprobs":
        return _logprobs_plain(state)
    if case["op"] == "logprobs_grad":
        return {**_logprobs_plain(state), "d_logits": _logprobs_gradient_plain(state)}
    if case["op"] == "logprobs_backward":
        return {"d_logits": _logprobs_gradient_plain(state, state["lse"], state["entropy"])}
    plain = _distill_plain(state["logits"], state["teacher"], state["index"], case["temperature"], case["tail"])
    if case["op"] == "distill_backward":
        # the forward pass's statistics stand for those of this one
        plain["lse"], plain["rest"] = state["lse"], state["rest"]
        picked = plain["y"].gather(1, plain["at"].clamp(max=plain["y"].shape[1] - 1))
        plain["log_q"] = torch.where(picked == -math.inf, picked, picked - state["lse"][:, None])
        return {"d_logits": _distill_gradient_plain(state, plain)}
    out = {"loss": plain["loss"], "lse": plain["lse"]}
    if case["tail"]:
        out["rest"] = plain["rest"]
    if case["op"] == "distill_grad":
        out["d_logits"] = _distill_gradient_plain(state, plain)
    return out


# ---------------------------------------------------------------- the library's calls


def _run_own(state):
    import newton_schulz_orthogonalized_gb300 as nsm

    s, case = state, state["case"]
    op, t = case["op"], case["temperature"]
    if op == "logprobs":
        nsm.logprobs(s["logits"], s["tokens"], s["logprob"], entropy=s["entropy"], lse=s["lse"],
                     top_logprob=s["top_logprob"], top_index=s["top_index"], temperature=t)
        names = ("logprob", "lse", "entropy", "top_logprob", "top_index")
    elif op == "logprobs_grad":
        nsm.logprobs_grad(s["logits"], s["tokens"], s["d_logprob"], s["d_entropy"], s["d_logits"], s["logprob"],
                          entropy=s["entropy"], lse=s["lse"], temperature=t)
        names = ("logprob", "lse", "entropy", "d_logits")
    elif op == "logprobs_backward":
        nsm.logprobs_backward(s["logits"], s["tokens"], s["lse"], s["entropy"], s["d_logprob"], s["d_entropy"],
                              s["d_logits"], temperature=t)
        names = ("d_logits",)
    elif op == "distill":
        nsm.distill(s["logits"], s["teacher"], s["index"], s["loss"], lse=s["lse"], rest=s["rest"], temperature=t,
                    tail=case["tail"])
        names = ("loss", "lse", "rest")
    elif op == "distill_grad":
        nsm.distill_grad(s["logits"], s["teacher"], s["index"], s["d_loss"], s["d_logits"], s["loss"], lse=s["lse"],
                         rest=s["rest"], temperature=t, tail=case["tail"])
        names = ("loss", "lse", "rest", "d_logits")
    else:
        nsm.distill_backward(s["logits"], s["teacher"], s["index"], s["lse"], s["rest"], s["d_loss"], s["d_logits"],
                             temperature=t, tail=case["tail"])
        names = ("d_logits",)
    return {n: s[n] for n in names if s[n] is not None}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    """Logits read once and gradients written once, with the rows' own numbers; per logit a
    subtraction, a product, an exponential and a sum, per gradient about as many."""
    size = 4 if case["dtype"] == "fp32" else 2
    cells = case["rows"] * case["vocab"]
    gradient = case["op"].endswith(("_grad", "_backward"))
    read = cells * size
    if case["op"].endswith("_backward"):
        read *= 1 - case["ignored"]
    per_row = 24 + (12 * case["k"] if case["k"] else 0)
    return {"bytes": int(read + (cells * size if gradient else 0) + case["rows"] * per_row),
            "flops": cells * (8 if case["op"].endswith("_grad") else 4)}


# ---------------------------------------------------------------- in 64 bits


def _exact_rows(case, s, rows):
    """The outputs of the rows in the slice ``rows``, from the definitions."""
    t, op = case["temperature"], case["op"]
    x = s["logits"][rows].double()
    n, vocab = x.shape
    zero = x.new_zeros(())
    y = x / t
    # a backward pass takes the forward's 32-bit statistics for what they are
    given_stats = op.endswith("_backward")
    lse = s["lse"][rows].double() if given_stats else torch.logsumexp(y, 1)
    dead = torch.isneginf(lse)
    q = (y - lse.masked_fill(dead, 0.0)[:, None]).exp()
    out = {}
    if op.startswith("logprobs"):
        tokens = s["tokens"][rows].long()
        given = (tokens >= 0) & (tokens < vocab)
        line = torch.arange(n, device=x.device)
        chosen = torch.zeros(n, vocab, dtype=torch.bool, device=x.device)
        chosen[line[given], tokens[given]] = True
        entropy = s["entropy"][rows].double() if given_stats and case["entropy"] else -torch.special.xlogy(q, q).sum(1)
        if op != "logprobs_backward":
            logprob = x.new_zeros(n)
            logprob[given] = y[line[given], tokens[given]] - lse[given]
            logprob[given & dead] = -math.inf
            out["logprob"], out["lse"] = logprob, lse
            if case["entropy"]:
                out["entropy"] = entropy
        if op == "logprobs":
            if case["k"]:
                k = case["k"]
                value, order = torch.sort(x, dim=1, descending=True, stable=True)
                value, order = value[:, :k], order[:, :k].int()
                lacking = k - value.shape[1]
                value = torch.nn.functional.pad(value, (0, lacking), value=-math.inf)
                order = torch.nn.functional.pad(order, (0, lacking), value=-1)
                gone = torch.isneginf(value)
                out["top_logprob"] = (value / t - lse.masked_fill(dead, 0.0)[:, None]).masked_fill(gone, -math.inf)
                out["top_index"] = order.masked_fill(gone, -1)
            return out
        # d logprob / d y = onehot - q,  d entropy / d y = -q (log q + entropy)
        a = s["d_logprob"][rows].double() * given
        grad = a[:, None] * ((chosen & ~torch.isneginf(y)).double() - q)
        if s["d_entropy"] is not None:
            grad -= s["d_entropy"][rows].double()[:, None] * (torch.special.xlogy(q, q) + q * entropy[:, None])
    else:
        index = s["index"][rows].long()
        z = s["teacher"][rows].double()
        kept = (index >= 0) & (index < vocab)
        target = x.new_zeros(n, vocab)
        member = torch.zeros(n, vocab, dtype=torch.bool, device=x.device)
        r, j = kept.nonzero(as_tuple=True)
        member[r, index[r, j]] = True
        z = z.masked_fill(~kept, -math.inf)
        p = z.exp() if case["tail"] else torch.softmax(z / t, 1)
        nothing = ~kept.any(1) if case["tail"] else torch.isneginf(z).all(1)
        p = p.masked_fill(nothing[:, None], 0.0)
        target[r, index[r, j]] = p[r, j]
        outside_mass = torch.where(member, zero, q).sum(1)
        if given_stats and case["tail"]:
            outside_mass = s["rest"][rows].double().exp()
        # log q where the target has mass; what is masked there has log q = -inf
        log_q = torch.where(torch.isneginf(y), y, y - lse[:, None])
        loss = torch.where(target > 0, target * (target.log() - log_q), zero).sum(1)
        if case["tail"]:
            p_rest = (1 - p.sum(1)).clamp(min=0)
            p_rest = p_rest.masked_fill(outside_mass == 0, 0.0)
            rest = outside_mass.log()
            loss = loss + torch.where(p_rest > 0, p_rest * (p_rest.log() - rest), zero)
        loss = loss.masked_fill(nothing, 0.0)
        if op != "distill_backward":
            out["loss"], out["lse"] = loss, lse
            if case["tail"]:
                out["rest"] = rest
        if op == "distill":
            return out
        # the target over all tokens: what the rest holds is spread as the student spreads it
        grad = q * p.sum(1, keepdim=True) - target.masked_fill(torch.isneginf(y), 0.0)
        if case["tail"]:
            spread = torch.where(member, zero, q) / outside_mass.clamp(min=1e-300)[:, None]
            grad = grad + p_rest[:, None] * (q - spread)
        grad = grad * s["d_loss"][rows].double()[:, None]
        grad = grad.masked_fill(nothing[:, None], 0.0)
    out["d_logits"] = (grad / t).masked_fill(dead[:, None], 0.0)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    step = max(1, EXACT_PIECE // case["vocab"])
    pieces = [_exact_rows(case, s, slice(a, a + step)) for a in range(0, case["rows"], step)]
    return {name: torch.cat([p[name] for p in pieces]) for name in pieces[0]}
