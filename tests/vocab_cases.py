"""Cases of the vocabulary losses run through both builds of the library, for
tests/test_gpu_vocab_checked.py.

`run(nsm)` runs every case on cuda:0 and returns the outputs (name -> numpy array of bytes)
and the device status after each case.  The cases reach every kernel: rows in one warp's
registers, a block or a cluster per row, rows kept in shared memory, rows too long for that,
pieces of rows in the backward passes; the three types, odd vocabularies, rows that are views
of wider buffers, gradients aligned otherwise than their logits and in place; alternatives in
one warp, in a block and gathered from a cluster, with ties and where few are left.

Run as a script (`python tests/vocab_cases.py OUT.npz`), it writes the outputs to OUT.npz and
the statuses to OUT.json; with NSM_CHECKED=1 in the environment the binding loads the
bounds-checked build.
"""

from __future__ import annotations

import json
import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

# (rows, vocab, type, row padding, first element)
SHAPES = [(1, 1, "bf16", 0, 0), (5, 3, "fp32", 1, 1), (40, 259, "bf16", 0, 3), (9, 1000, "fp16", 3, 0),
          (7, 1017, "fp32", 0, 2), (33, 2041, "bf16", 7, 1), (6, 2050, "bf16", 0, 0), (20, 8001, "fp16", 0, 5),
          (3, 50257, "bf16", 0, 0), (300, 50257, "bf16", 0, 1), (2, 131072, "fp32", 4, 0), (170, 32003, "fp32", 5, 0),
          (2200, 50257, "bf16", 0, 0), (2, 1 << 20, "fp32", 0, 0)]


def _inputs(torch, rows, vocab, dtype, pad, first):
    g = torch.Generator(device="cuda").manual_seed(rows * 1000003 + vocab)
    kinds = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
    buf = torch.zeros(rows * (vocab + pad) + first + 8, dtype=kinds[dtype], device="cuda")
    x = buf[first:first + rows * (vocab + pad)].view(rows, vocab + pad)[:, :vocab]
    x.copy_(torch.randn(rows, vocab, generator=g, device="cuda") * 3)
    if vocab > 8:
        x[0, 3:7] = -float("inf")
    if rows > 2:
        x[1] = -float("inf")
        x[2] = 0.25
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    tokens[::4] = -100
    k = min(17, vocab)
    teacher, index = torch.topk(torch.randn(rows, vocab, generator=g, device="cuda") - 9, k)
    index[::3, -1] = index[::3, 0]
    index[1::3, 0] = -1
    weight = torch.randn(rows, generator=g, device="cuda")
    weight[-1] = 0
    return x, tokens, teacher, index, weight


def run(nsm):
    import torch
    out, status = {}, {}

    def keep(case, **tensors):
        torch.cuda.synchronize()
        for n, t in tensors.items():
            out[f"{case}.{n}"] = t.contiguous().view(torch.uint8).cpu().numpy()
        status[case] = tuple(int(v) for v in nsm.device_status_detail())

    for rows, vocab, dtype, pad, first in SHAPES:
        name = f"{rows}x{vocab}.{dtype}.{pad}.{first}"
        x, tokens, teacher, index, weight = _inputs(torch, rows, vocab, dtype, pad, first)

        def f(*shape):
            return torch.zeros(*(shape or (rows,)), device="cuda")

        for k in sorted({1, min(20, vocab), 128}):
            a = {"logprob": f(), "entropy": f(), "lse": f(), "top_logprob": f(rows, k),
                 "top_index": torch.zeros(rows, k, dtype=torch.int32, device="cuda")}
            nsm.logprobs(x, tokens, **a)
            keep(f"{name}.top{k}", **a)
        a = {"logprob": f(), "lse": f()}
        nsm.logprobs(x, tokens, **a, temperature=0.7)
        keep(f"{name}.logprobs", **a)
        ent = f()
        nsm.logprobs(x, None, entropy=ent)
        other = torch.zeros(rows * (vocab + 3) + 8, dtype=x.dtype, device="cuda")[1:1 + rows * (vocab + 3)]
        other = other.view(rows, vocab + 3)[:, :vocab]  # aligned otherwise
        same = torch.empty_like(x)
        for h in (None, weight):
            g1, a = torch.empty_like(x), {"logprob": f(), "lse": f()}
            nsm.logprobs_grad(x, tokens, weight, h, g1, **a)
            nsm.logprobs_grad(x, tokens, weight, h, other)
            keep(f"{name}.grad{h is not None}", gradient=g1, shifted=other, **a)
            nsm.logprobs(x, None, lse=a["lse"])
            nsm.logprobs_backward(x, tokens, a["lse"], ent, weight, h, same)
            nsm.logprobs_backward(x, tokens, a["lse"], ent, weight, h, other)
            keep(f"{name}.backward{h is not None}", gradient=same, shifted=other)
        for tail in (False, True):
            a = {"loss": f(), "lse": f(), "rest": f()}
            nsm.distill(x, teacher, index, **a, tail=tail)
            keep(f"{name}.distill{tail}", **a)
            g1 = torch.empty_like(x)
            nsm.distill_grad(x, teacher, index, weight, g1, tail=tail)
            nsm.distill_grad(x, teacher, index, weight, other, tail=tail)
            keep(f"{name}.distill_grad{tail}", gradient=g1, shifted=other)
            nsm.distill_backward(x, teacher, index, a["lse"], a["rest"], weight, same, tail=tail)
            nsm.distill_backward(x, teacher, index, a["lse"], a["rest"], weight, other, tail=tail)
            keep(f"{name}.distill_backward{tail}", gradient=same, shifted=other)
        y = x.clone() if x.is_contiguous() else x
        nsm.distill_grad(y, teacher, index, weight, y, tail=True)
        nsm.logprobs_grad(y, tokens, weight, None, y)
        keep(f"{name}.in_place", gradient=y)
    return out, status


if __name__ == "__main__":
    import newton_schulz_orthogonalized_gb300 as nsm_module
    outputs, statuses = run(nsm_module)
    np.savez(sys.argv[1], **outputs)
    with open(os.path.splitext(sys.argv[1])[0] + ".json", "w") as fh:
        json.dump({"checked": nsm_module.checked_build(), "status": {k: list(v) for k, v in statuses.items()}}, fh)
