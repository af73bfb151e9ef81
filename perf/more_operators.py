"""Cases that measure what stands at the two ends of a model's vocabulary and before the
optimizer's step: penalties, biases and grammar masks on logits (and their backward pass), the
embedding lookup and its gradient, and the global norm of many gradients with clipping.

``listed()`` gives the named cases, ``draw(rng)`` one more of the same ranges.
``prepare(case, seed)`` makes what a training or serving program holds before the call,
``run(state)`` makes the call: in plain torch operations on 32-bit values where ``own`` is
false, through the library where it is true.  ``exact(case, seed)`` computes the outputs in
64 bits from the definitions, and ``work(case)`` says what a pass cannot do without.

Definitions.
  adjust     for a row x of V logits, with c_v the number of times token v occurs in the row's
             history (its first `length` tokens; tokens outside [0, V) do not count):
                 a_v = x_v / repetition if x_v > 0, else x_v * repetition   where c_v > 0
                 a_v = x_v                                                  elsewhere
                 out_v = a_v - (frequency c_v + presence [c_v > 0]) + sum_{j: index_j = v} bias_j
                 out_v = -inf where the row's mask has bit v clear
  adjust_backward   d_logits_v = d_out_v d a_v / d x_v, 0 where the mask has bit v clear
  embedding  out_r = scale weight[token_r], 0 where the token is outside [0, V)
  embedding_backward   d_weight[v] (+)= scale sum_{r: token_r = v} d_out_r
  grad_norm  norm = sqrt(sum of all squares), norms = the same of each tensor
  clip_grads out = grads min(1, max_norm / norm), with norm and norms as above
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
DEVICE = "cuda"
# elements of one piece of the 64-bit computations
EXACT_PIECE = 1 << 26

# tables of gradients, as (how often, elements): the library's own workloads
TABLES = {
    # 4 matrices of 128 x 256 and a vector
    "tiny": [(4, 128 * 256), (1, 256)],
    # 12 layers of hidden 768 with their norms and biases, two embeddings and the head
    "gpt2small": [(12, 3 * 768 * 768), (12, 768 * 768), (24, 4 * 768 * 768), (72, 768), (12, 3 * 768), (12, 4 * 768),
                  (2, 50257 * 768), (1, 1024 * 768)],
    # 8 layers of hidden 4096
    "llama7b_layers": [(16, 4096 * 4096), (16, 1024 * 4096), (24, 11008 * 4096)],
}


def _adjust(op, rows, vocab, dtype, name=None, out="", length=0, sequences=0, penalties=False, bias=0, masks=0,
            allowed=1.0, pad=0, wide=True):
    """`sequences`: 0 for a history per row, else the rows are the positions of that many
    sequences and a row's history is what comes before it; `masks`: rows of the mask table."""
    case = {"op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "out": out or dtype, "length": length,
            "sequences": sequences, "penalties": penalties, "bias": bias, "masks": masks, "allowed": allowed, "pad": pad,
            "wide": wide}
    return case if name is None else {**case, "name": name}


def _embed(op, rows, vocab, cols, weight, out, name=None, scale=1.0, ignored=0.0, skew=4.0, accumulate=False, pad=0,
           wide=True):
    """`skew`: tokens are vocab u^skew for u uniform, so that 4 makes one in some 15 the same."""
    case = {"op": op, "rows": rows, "vocab": vocab, "cols": cols, "weight": weight, "out": out, "scale": scale,
            "ignored": ignored, "skew": skew, "accumulate": accumulate, "pad": pad, "wide": wide}
    return case if name is None else {**case, "name": name}


def _norm(op, table, dtype, name=None, out="", tensors=0, elements=0, gap=0, max_norm=1.0):
    """`table`: a name of TABLES, or "drawn" for `tensors` of unequal sizes with `elements` in
    all; `gap`: elements between one tensor and the next (0: each on a multiple of 64)."""
    case = {"op": op, "table": table, "dtype": dtype, "out": out or dtype, "tensors": tensors, "elements": elements,
            "gap": gap, "max_norm": max_norm}
    return case if name is None else {**case, "name": name}


def listed():
    return [
        # one token about to be sampled: its history's penalties, a few biases, a grammar; latency counts
        _adjust("adjust", 1, 50257, "bf16", "adjust_one_token", out="fp32", length=700, penalties=True, bias=4, masks=1,
                allowed=0.05),
        # a decoding batch on a large vocabulary, every request with its own history and grammar
        _adjust("adjust", 256, 131072, "bf16", "adjust_batch", out="fp32", length=4096, penalties=True, bias=16, masks=256,
                allowed=0.5, wide=False),
        # a policy's training step under the penalties that its samples were drawn with: the rows are
        # positions of sequences, each one's history what comes before it
        _adjust("adjust", 8192, 50257, "bf16", "adjust_policy", length=1024, sequences=8, penalties=True),
        # its backward pass in fp32 under a grammar with a few states, rows a view of a wider buffer
        _adjust("adjust_backward", 2049, 65537, "fp32", "adjust_policy_backward", length=683, sequences=3, penalties=True,
                masks=24, allowed=0.5, pad=3),
        # one token's row of an fp32 embedding as bf16 activations
        _embed("embedding", 1, 50257, 768, "fp32", "bf16", "embed_one_token", scale=768 ** 0.5, wide=False),
        # a batch of prompts
        _embed("embedding", 65536, 100003, 2048, "bf16", "bf16", "embed_prompts", ignored=0.05),
        # the gradient of one short sequence added to a tied head's, odd sizes
        _embed("embedding_backward", 257, 32003, 769, "fp32", "fp32", "embed_grad_short", accumulate=True, scale=0.5),
        # a training step's on the GPT-2 vocabulary, with one token in 15 the same
        _embed("embedding_backward", 16384, 50257, 768, "bf16", "bf16", "embed_grad_step", ignored=0.05),
        # a large batch, vocabulary and width: the gradient's 1 GB is written whole
        _embed("embedding_backward", 65536, 131072, 4096, "bf16", "bf16", "embed_grad_large"),
        # the smallest table's norm, with each tensor's
        _norm("grad_norm", "tiny", "bf16", "norm_tiny"),
        # a small model's gradients clipped into its optimizer's packed slots
        _norm("clip_grads", "gpt2small", "bf16", "clip_gpt2small"),
        # fp32 gradients of some large layers clipped into bf16 slots, the largest case
        _norm("clip_grads", "llama7b_layers", "fp32", "clip_llama7b_layers", out="bf16"),
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["adjust", "adjust_backward", "embedding", "embedding_backward", "grad_norm", "clip_grads"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    wide = rng.random() < 0.5
    pad = rng.choice([0, 0, rng.randint(1, 16)])
    if op.startswith("adjust"):
        vocab = _log_uniform(rng, 256, 200000)
        rows = _log_uniform(rng, 1, max(1, min(8192, (1 << 28) // vocab)))
        sequences = rng.choice([0, max(1, rows // 500)])
        length = -(-rows // sequences) if sequences else rng.choice([0, _log_uniform(rng, 1, 4096)])
        return _adjust(op, rows, vocab, dtype, out=rng.choice([dtype, "fp32"]), length=length, sequences=sequences,
                       penalties=length > 0, bias=rng.choice([0, rng.randint(1, 64)]) if op == "adjust" else 0,
                       masks=rng.choice([0, rng.randint(1, min(rows, 64))]), allowed=rng.choice([0.02, 0.5, 0.95]), pad=pad,
                       wide=wide)
    if op.startswith("embedding"):
        vocab, cols = _log_uniform(rng, 256, 200000), _log_uniform(rng, 16, 4096)
        return _embed(op, _log_uniform(rng, 1, 65536), min(vocab, (1 << 28) // cols), cols, rng.choice(["bf16", "fp32", dtype]),
                      dtype, scale=rng.choice([1.0, cols ** 0.5]), ignored=rng.choice([0.0, 0.1]),
                      skew=rng.choice([1.0, 4.0]), accumulate=rng.random() < 0.3 and op == "embedding_backward", pad=pad,
                      wide=wide)
    tensors = _log_uniform(rng, 1, 400)
    return _norm(op, "drawn", dtype, out=rng.choice([dtype, "bf16"]), tensors=tensors,
                 elements=max(tensors, _log_uniform(rng, 1000, 1 << 29)), gap=rng.choice([0, 0, rng.randint(1, 9)]),
                 max_norm=rng.choice([1.0, 1.0, 1e6]))


# ---------------------------------------------------------------- inputs


def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _matrix(rows, cols, pad, dtype):
    return torch.empty(rows, cols + pad, dtype=DTYPES[dtype], device=DEVICE)[:, :cols]


def _skewed(g, shape, vocab, skew):
    u = torch.rand(*shape, generator=g, device=DEVICE, dtype=torch.float64)
    return (vocab * u ** skew).long().clamp_(max=vocab - 1)


def _prepare_adjust(case, g):
    rows, vocab, length = case["rows"], case["vocab"], case["length"]
    index_type = torch.int64 if case["wide"] else torch.int32
    logits = _matrix(rows, vocab, case["pad"], case["dtype"])
    logits.copy_(torch.randn(rows, vocab, generator=g, device=DEVICE).mul_(3.0))
    state = {"logits": logits, "history": None, "length": None, "history_row": None, "mask": None, "mask_row": None,
             "repetition": None, "frequency": None, "presence": None, "bias_index": None, "bias": None}

    def per_row(low, high):
        return low + (high - low) * torch.rand(rows, generator=g, device=DEVICE)

    if length:
        lines = case["sequences"] or rows
        history = _skewed(g, (lines, length), vocab, 3.0)
        # a few places hold padding
        history[torch.rand(lines, length, generator=g, device=DEVICE) < 0.02] = -1
        state["history"] = history.to(index_type)
        if case["sequences"]:
            at = torch.arange(rows, device=DEVICE)
            state["history_row"] = torch.div(at, length, rounding_mode="floor").int()
            state["length"] = (at % length).int()
        else:
            state["length"] = torch.randint(0, length + 1, (rows,), generator=g, device=DEVICE).int()
            state["length"][0] = length
        state["repetition"] = per_row(1.0, 1.5)
        if case["op"] == "adjust":
            state["frequency"], state["presence"] = per_row(0.0, 0.5), per_row(-0.5, 1.0)
    if case["bias"]:
        state["bias_index"] = torch.randint(-1, vocab, (rows, case["bias"]), generator=g, device=DEVICE).to(index_type)
        state["bias"] = torch.randn(rows, case["bias"], generator=g, device=DEVICE).mul_(4.0)
    if case["masks"]:
        words = (vocab + 31) // 32
        bits = torch.rand(case["masks"], words * 32, generator=g, device=DEVICE) < case["allowed"]
        packed = (bits.view(case["masks"], words, 32).long() << torch.arange(32, device=DEVICE)).sum(2)
        state["mask"] = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).int()
        if case["masks"] != rows:  # rows share the table's, and some have no grammar
            state["mask_row"] = torch.randint(-1, case["masks"], (rows,), generator=g, device=DEVICE).int()
    if case["op"] == "adjust":
        state["result"] = _matrix(rows, vocab, case["pad"], case["out"])
    else:
        state["d_out"] = _matrix(rows, vocab, case["pad"], case["out"])
        state["d_out"].copy_(torch.randn(rows, vocab, generator=g, device=DEVICE))
        state["result"] = _matrix(rows, vocab, case["pad"], case["dtype"])
    return state


def _prepare_embedding(case, g):
    rows, vocab, cols = case["rows"], case["vocab"], case["cols"]
    tokens = _skewed(g, (rows,), vocab, case["skew"])
    tokens[torch.rand(rows, generator=g, device=DEVICE) < case["ignored"]] = -100
    state = {"tokens": tokens.to(torch.int64 if case["wide"] else torch.int32)}
    weight = _matrix(vocab, cols, case["pad"], case["weight"])
    out = _matrix(rows, cols, case["pad"], case["out"])
    if case["op"] == "embedding":
        weight.copy_(torch.randn(vocab, cols, generator=g, device=DEVICE).mul_(0.02))
        return {**state, "weight": weight, "result": out}
    out.copy_(torch.randn(rows, cols, generator=g, device=DEVICE).mul_(0.01))
    weight.zero_()
    if case["accumulate"]:  # the head's gradient is there already
        weight.copy_(torch.randn(vocab, cols, generator=g, device=DEVICE).mul_(0.01))
    return {**state, "d_out": out, "result": weight}


def _sizes(case):
    """Elements of each tensor of the case's table."""
    if case["table"] != "drawn":
        return [size for count, size in TABLES[case["table"]] for _ in range(count)]
    # unequal ones: each weighs a few times what the one before it does, over three decades
    weights = [10 ** (3 * ((7 * i + 3) % case["tensors"]) / case["tensors"]) for i in range(case["tensors"])]
    total = sum(weights)
    return [max(1, int(case["elements"] * w / total)) for w in weights]


def _offsets(case):
    offsets, at = [], 0
    for size in _sizes(case):
        offsets.append(at)
        at += size + case["gap"] if case["gap"] else -(-size // 64) * 64
    return offsets, at


def _views(case, buffer):
    return [buffer[a:a + n] for a, n in zip(_offsets(case)[0], _sizes(case))]


def _prepare_norm(case, g):
    offsets, total = _offsets(case)
    buffer = torch.empty(total, dtype=DTYPES[case["dtype"]], device=DEVICE)
    buffer.normal_(generator=g)
    grads = _views(case, buffer)
    # gradients of one model differ by some orders of magnitude
    size = 10 ** (-1 - 2 * torch.rand(len(grads), generator=g, device=DEVICE))
    for x, s in zip(grads, size.to(buffer.dtype)):
        x.mul_(s)
    state = {"grads": grads, "norm": torch.empty(1, device=DEVICE), "norms": torch.empty(len(grads), device=DEVICE)}
    if case["op"] == "clip_grads":
        # the optimizer's packed slots; what lies between them is left as it is
        state["packed"] = torch.zeros(total, dtype=DTYPES[case["out"]], device=DEVICE)
        state["slots"] = _views(case, state["packed"])
    return state


def prepare(case, seed):
    make = {"a": _prepare_adjust, "e": _prepare_embedding}.get(case["op"][0], _prepare_norm)
    return {"case": case, **make(case, _generator(seed))}


# ---------------------------------------------------------------- the plain form


def _counts_plain(s):
    """How often each token occurs in each row's history, rows x vocab; None without one."""
    case, history = s["case"], s["history"]
    if history is None:
        return None
    rows, vocab = case["rows"], case["vocab"]
    line = s["history_row"].long() if s["history_row"] is not None else torch.arange(rows, device=DEVICE)
    tokens = history.long()[line]
    place = torch.arange(tokens.shape[1], device=DEVICE)
    kept = (tokens >= 0) & (tokens < vocab) & (place < s["length"].long()[:, None])
    tokens = torch.where(kept, tokens, torch.full_like(tokens, vocab))  # one column more takes the others
    counts = torch.zeros(rows, vocab + 1, device=DEVICE)
    return counts.scatter_add_(1, tokens, torch.ones(1, 1, device=DEVICE).expand(tokens.shape))[:, :vocab]


def _banned_plain(s):
    """Which logits the rows' masks ban; None without a mask."""
    case, mask = s["case"], s["mask"]
    if mask is None:
        return None
    v = torch.arange(case["vocab"], device=DEVICE)
    banned = ((mask[:, v // 32] >> (v % 32).int()) & 1) == 0
    if s["mask_row"] is None:
        return banned
    return banned[s["mask_row"].clamp(min=0).long()] & (s["mask_row"] >= 0)[:, None]


def _adjust_plain(s):
    case = s["case"]
    x = s["logits"].float()
    counts, banned = _counts_plain(s), _banned_plain(s)
    if counts is not None:
        repetition = s["repetition"][:, None]
        x = torch.where(counts > 0, torch.where(x > 0, x / repetition, x * repetition), x)
        x = x - (s["frequency"][:, None] * counts + s["presence"][:, None] * (counts > 0))
    if s["bias"] is not None:
        index = s["bias_index"].long()
        kept = (index >= 0) & (index < case["vocab"])
        x = x.scatter_add(1, torch.where(kept, index, 0), torch.where(kept, s["bias"], 0.0))
    if banned is not None:
        x = x.masked_fill(banned, -math.inf)
    return s["result"].copy_(x)


def _adjust_backward_plain(s):
    grad = s["d_out"].float()
    counts, banned = _counts_plain(s), _banned_plain(s)
    if counts is not None:
        repetition = s["repetition"][:, None]
        grad = torch.where(counts > 0, torch.where(s["logits"] > 0, grad / repetition, grad * repetition), grad)
    if banned is not None:
        grad = grad.masked_fill(banned, 0.0)
    return s["result"].copy_(grad)


def _embedding_plain(s):
    case, tokens = s["case"], s["tokens"].long()
    kept = (tokens >= 0) & (tokens < case["vocab"])
    rows = s["weight"][tokens.clamp(0, case["vocab"] - 1)].float() * case["scale"]
    return s["result"].copy_(torch.where(kept[:, None], rows, 0.0))


def _embedding_backward_plain(s):
    case, tokens = s["case"], s["tokens"].long()
    kept = (tokens >= 0) & (tokens < case["vocab"])
    sums = torch.zeros(case["vocab"] + 1, case["cols"], device=DEVICE)  # one row more takes the others
    sums.index_add_(0, torch.where(kept, tokens, case["vocab"]), s["d_out"].float())
    sums = sums[:-1] * case["scale"]
    if case["accumulate"]:
        sums += s["result"]
    return s["result"].copy_(sums)


def _norm_plain(s):
    squares = torch.stack([g.float().square().sum() for g in s["grads"]])
    s["norms"].copy_(squares.sqrt())
    s["norm"].copy_(squares.sum().sqrt())
    out = {"norm": s["norm"], "norms": s["norms"]}
    if s["case"]["op"] == "clip_grads":
        factor = (s["case"]["max_norm"] / s["norm"]).clamp(max=1.0)
        out["packed"] = s["packed"]
        [slot.copy_(g.float() * factor) for slot, g in zip(s["slots"], s["grads"])]
    return out


PLAIN = {"adjust": _adjust_plain, "adjust_backward": _adjust_backward_plain, "embedding": _embedding_plain,
         "embedding_backward": _embedding_backward_plain, "grad_norm": _norm_plain, "clip_grads": _norm_plain}


# ---------------------------------------------------------------- the library's calls


def _run_own(s):
    import newton_schulz_orthogonalized_gb300 as nsm

    case = s["case"]
    op = case["op"]
    if op == "adjust":
        nsm.adjust_logits(s["logits"], s["result"], history=s["history"], length=s["length"], history_row=s["history_row"],
                          repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                          bias_index=s["bias_index"], bias=s["bias"], mask=s["mask"], mask_row=s["mask_row"])
        return s["result"]
    if op == "adjust_backward":
        nsm.adjust_logits_backward(s["logits"], s["d_out"], s["result"], history=s["history"], length=s["length"],
                                   history_row=s["history_row"], repetition=s["repetition"], mask=s["mask"],
                                   mask_row=s["mask_row"])
        return s["result"]
    if op == "embedding":
        nsm.embedding(s["weight"], s["tokens"], s["result"], scale=case["scale"])
        return s["result"]
    # a program keeps the workspace, and the table of gradients whose places do not change
    if op == "embedding_backward":
        if "workspace" not in s:
            s["workspace"] = torch.empty(nsm.embedding_workspace_bytes(case["rows"], case["vocab"], case["cols"]),
                                         dtype=torch.uint8, device=DEVICE)
        nsm.embedding_backward(s["d_out"], s["tokens"], s["result"], s["workspace"], scale=case["scale"],
                               accumulate=case["accumulate"])
        return s["result"]
    if "table" not in s:
        s["table"] = nsm.GradTable(s["grads"], s.get("slots"))
        s["workspace"] = torch.empty(s["table"].workspace_bytes, dtype=torch.uint8, device=DEVICE)
    if op == "grad_norm":
        nsm.grad_norm(s["table"], s["norm"], s["norms"], workspace=s["workspace"])
        return {"norm": s["norm"], "norms": s["norms"]}
    nsm.clip_grads(s["table"], case["max_norm"], s["norm"], s["norms"], workspace=s["workspace"])
    return {"norm": s["norm"], "norms": s["norms"], "packed": s["packed"]}


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


def work(case):
    """Inputs read once and outputs written once.  Logits that a mask bans need not be read;
    of an embedding's gradient the rows without a token are written too, unless it adds to
    what is there.  Clipping reads the gradients twice: the norm comes before the factor."""
    op = case["op"]
    if op.startswith("adjust"):
        cells = case["rows"] * case["vocab"]
        read = SIZES[case["dtype"] if op == "adjust" else case["out"]] * (case["allowed"] if case["masks"] else 1.0)
        write = SIZES[case["out"] if op == "adjust" else case["dtype"]]
        index = 8 if case["wide"] else 4
        rest = (case["sequences"] or case["rows"]) * case["length"] * index + case["rows"] * case["bias"] * (index + 4)
        return {"bytes": int(cells * (read + write) + rest + case["masks"] * ((case["vocab"] + 31) // 32) * 4), "flops": cells}
    if op.startswith("embedding"):
        # tokens = vocab u^skew: the share of the vocabulary that the rows reach
        live = case["rows"] * (1 - case["ignored"])
        reached, top = 0.0, 64
        for i in range(top):  # slices of u; each spreads over its own tokens
            slots = max(1.0, case["vocab"] * (((i + 1) / top) ** case["skew"] - (i / top) ** case["skew"]))
            reached += slots * -math.expm1(-live / top / slots)
        reached = min(reached, live)
        tokens = case["rows"] * (8 if case["wide"] else 4)
        if op == "embedding":
            read, write = reached * SIZES[case["weight"]], case["rows"] * SIZES[case["out"]]
        else:
            read = live * SIZES[case["out"]] + (reached * SIZES[case["weight"]] if case["accumulate"] else 0)
            write = (reached if case["accumulate"] else case["vocab"]) * SIZES[case["weight"]]
        return {"bytes": int(tokens + (read + write) * case["cols"]), "flops": int(live * case["cols"])}
    elements = sum(_sizes(case))
    size = SIZES[case["dtype"]]
    if op == "clip_grads":
        return {"bytes": elements * (2 * size + SIZES[case["out"]]), "flops": 3 * elements}
    return {"bytes": elements * size + 4, "flops": 2 * elements}


# ---------------------------------------------------------------- in 64 bits


def _exact_adjust(case, s, first, last):
    """Rows first to last, one after the other's history counted over all tokens."""
    vocab, rows = case["vocab"], last - first
    part = slice(first, last)
    x = s["logits"][part].double()
    backward = case["op"] == "adjust_backward"
    y = s["d_out"][part].double() if backward else x
    if s["history"] is not None:
        line = s["history_row"][part].long() if s["history_row"] is not None else torch.arange(first, last, device=DEVICE)
        held = s["history"][line].long()
        held[torch.arange(held.shape[1], device=DEVICE) >= s["length"][part].long()[:, None]] = -1
        r, j = ((held >= 0) & (held < vocab)).nonzero(as_tuple=True)
        count = torch.bincount(r * vocab + held[r, j], minlength=rows * vocab).view(rows, vocab)
        seen = count.bool()
        theta = s["repetition"][part].double()[:, None].expand(rows, vocab)
        factor = torch.where(x > 0, theta.reciprocal(), theta)
        y = torch.where(seen, y * factor, y)
        if not backward:
            y = y - s["frequency"][part].double()[:, None] * count
            y = y - torch.where(seen, s["presence"][part].double()[:, None], y.new_zeros(()))
    if s["bias"] is not None:
        index = s["bias_index"][part].long()
        r, j = ((index >= 0) & (index < vocab)).nonzero(as_tuple=True)
        y = y.index_put((r, index[r, j]), s["bias"][part].double()[r, j], accumulate=True)
    if s["mask"] is not None:
        which = s["mask_row"][part].long() if s["mask_row"] is not None else torch.arange(first, last, device=DEVICE)
        words = s["mask"][which.clamp(min=0)].long() & 0xFFFFFFFF
        bit = words[:, :, None].bitwise_right_shift(torch.arange(32, device=DEVICE)).bitwise_and(1).flatten(1)[:, :vocab]
        y = torch.where((bit == 1) | (which < 0)[:, None], y, y.new_full((), 0.0 if backward else -math.inf))
    return y


def _exact_embedding(case, s, first, last):
    """Columns first to last."""
    tokens, part = s["tokens"].long(), slice(first, last)
    row = ((tokens >= 0) & (tokens < case["vocab"])).nonzero()[:, 0]
    scale = float(case["scale"])
    if case["op"] == "embedding":
        out = torch.zeros(case["rows"], last - first, dtype=torch.float64, device=DEVICE)
        out[row] = s["weight"][:, part].double()[tokens[row]] * scale
        return out
    out = torch.zeros(case["vocab"], last - first, dtype=torch.float64, device=DEVICE)
    out.index_put_((tokens[row],), s["d_out"][:, part].double()[row] * scale, accumulate=True)
    return out + s["result"][:, part].double() if case["accumulate"] else out


def _exact_norm(case, s):
    norms = torch.stack([torch.linalg.vector_norm(g, dtype=torch.float64) for g in s["grads"]])
    norm = torch.linalg.vector_norm(norms)
    out = {"norm": norm[None], "norms": norms}
    if case["op"] == "clip_grads":
        factor = min(1.0, case["max_norm"] / float(norm))
        out["packed"] = torch.zeros(s["packed"].shape, dtype=torch.float64, device=DEVICE)
        for at, g in zip(_views(case, out["packed"]), s["grads"]):
            at.copy_(g)
            at.mul_(factor)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("adjust"):
        step = max(1, EXACT_PIECE // case["vocab"])
        return torch.cat([_exact_adjust(case, s, a, min(a + step, case["rows"])) for a in range(0, case["rows"], step)])
    if case["op"].startswith("embedding"):
        step = max(1, EXACT_PIECE // max(case["vocab"], case["rows"]))
        return torch.cat([_exact_embedding(case, s, a, min(a + step, case["cols"])) for a in range(0, case["cols"], step)], 1)
    return _exact_norm(case, s)
