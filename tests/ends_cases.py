"""Cases of the logit adjustments, the embedding with its gradient and the gradients' norm and clipping,
run through both builds of the library, for tests/test_gpu_ends_checked.py.

`run(nsm)` runs every case on cuda:0 and returns the outputs (name -> numpy array of bytes) and the
device status after each case.  The cases reach every kernel and path: slices inside a row and at its ends,
histories of one row and of many, biases, masks, in place and not, the three types; sorts by one block
and by tiles, tokens in one piece, two and many, rows that are cleared beside the sort and after it,
every alignment; few chunks and many, one type and several, sums that fp32 does not hold.

Run as a script (`python tests/ends_cases.py OUT.npz`), it writes the outputs to OUT.npz and the
statuses to OUT.json; with NSM_CHECKED=1 in the environment the binding loads the bounds-checked
build.
"""

from __future__ import annotations

import json
import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

# rows, vocab, type, tokens of history, its rows (0: one per row), biases, masks, padding, first element
ADJUST = [(1, 1, "bf16", 3, 0, 1, 1, 0, 0), (3, 31, "fp16", 1, 0, 0, 3, 0, 1), (5, 33, "fp32", 40, 2, 0, 0, 0, 3),
          (40, 4099, "bf16", 257, 3, 5, 2, 1, 5), (3, 8192, "bf16", 64, 0, 0, 3, 0, 0), (700, 20011, "fp16", 300, 2, 0, 0, 0, 0),
          (9, 50257, "bf16", 700, 0, 4, 9, 0, 0), (300, 32003, "fp32", 100, 1, 3, 2, 5, 2), (1, 1 << 20, "fp32", 100, 0, 1024, 1, 0, 0)]
# rows, vocab, cols, weight, rows' type, padding, first element, skew of the tokens
EMBED = [(1, 1, 1, "bf16", "fp32", 0, 0, 1), (33, 17, 8, "bf16", "bf16", 0, 0, 1), (257, 1023, 33, "fp32", "fp32", 0, 3, 4),
         (1025, 50257, 256, "bf16", "bf16", 0, 1, 4), (4096, 300, 264, "fp16", "fp32", 8, 0, 6), (9000, 70000, 771, "bf16", "fp16", 0, 0, 4),
         (70001, 1500, 16, "fp32", "bf16", 0, 0, 30), (600, 1 << 21, 8, "bf16", "bf16", 0, 0, 1), (64, 10, 4104, "bf16", "bf16", 0, 0, 1)]
# sizes of the tensors, their types in turn, elements between them, a factor
GRADS = [([1], ("fp32",), 0, 1.0), ([5, 0, 3, 40000], ("bf16", "fp32"), 1, 1.0), ([300001, 77, 16384, 5] * 4, ("bf16",), 3, 1.0),
         ([1000003, 40000], ("fp32",), 0, 1.0), ([99999] * 30, ("fp16", "fp32", "bf16"), 5, 1.0), ([33] * 1300, ("bf16",), 0, 1.0),
         ([1000003, 17], ("fp32",), 1, 1e30), ([900000, 5000], ("bf16",), 1, 1e-30)]


def run(nsm):
    import torch
    kinds = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
    out, status = {}, {}

    def keep(case, **tensors):
        torch.cuda.synchronize()
        for n, t in tensors.items():
            out[f"{case}.{n}"] = t.contiguous().view(torch.uint8).cpu().numpy()
        status[case] = tuple(int(v) for v in nsm.device_status_detail())

    def view(rows, cols, dtype, pad, first, values=None):
        buf = torch.zeros(rows * (cols + pad) + first + 8, dtype=kinds[dtype], device="cuda")
        v = buf[first:first + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        if values is not None:
            v.copy_(values)
        return v

    for rows, vocab, dtype, length, lines, k, masks, pad, first in ADJUST:
        name = f"adjust.{rows}x{vocab}.{dtype}"
        g = torch.Generator(device="cuda").manual_seed(rows + vocab)
        x = view(rows, vocab, dtype, pad, first, torch.randn(rows, vocab, generator=g, device="cuda") * 3)
        back = {"history": torch.randint(-2, vocab + 2, (lines or rows, length), generator=g, device="cuda"),
                "length": torch.randint(0, length + 1, (rows,), generator=g, device="cuda").int(),
                "repetition": 0.7 + torch.rand(rows, generator=g, device="cuda")}
        if lines:  # positions of sequences
            back["length"] = (torch.arange(rows, device="cuda") % (length + 1)).int()
            back["history_row"] = (torch.arange(rows, device="cuda") * lines // rows).int()
        if masks:
            back["mask"] = torch.randint(-2 ** 31, 2 ** 31, (masks, (vocab + 31) // 32), generator=g, device="cuda").int()
            if masks != rows:
                back["mask_row"] = torch.randint(-1, masks, (rows,), generator=g, device="cuda").int()
        kw = dict(back, frequency=torch.rand(rows, generator=g, device="cuda"), presence=torch.rand(rows, generator=g, device="cuda"))
        if k:
            kw["bias_index"] = torch.randint(-1, vocab + 1, (rows, k), generator=g, device="cuda")
            kw["bias"] = torch.randn(rows, k, generator=g, device="cuda")
        a, b = view(rows, vocab, dtype, pad, first), view(rows, vocab, "fp32", pad, 1)
        nsm.adjust_logits(x, a, **kw)
        nsm.adjust_logits(x, b, **kw)
        d, e = view(rows, vocab, dtype, pad, first), view(rows, vocab, dtype, pad, first + 1)
        nsm.adjust_logits_backward(x, x.clone(), d, **back)
        nsm.adjust_logits_backward(x, torch.ones(rows, vocab, device="cuda"), e, **back)
        y = x.clone()
        nsm.adjust_logits(y, y, **kw)
        keep(name, a=a, b=b, d=d, e=e, in_place=y)

    for rows, vocab, cols, w_type, o_type, pad, first, skew in EMBED:
        name = f"embedding.{rows}x{vocab}x{cols}"
        g = torch.Generator(device="cuda").manual_seed(rows + vocab)
        tokens = (vocab * torch.rand(rows, generator=g, device="cuda") ** skew).long()
        tokens[::7] = -100
        w = view(vocab, cols, w_type, pad, first, torch.randn(vocab, cols, generator=g, device="cuda"))
        o = view(rows, cols, o_type, pad, first)
        nsm.embedding(w, tokens, o, scale=1.5)
        d_out = view(rows, cols, o_type, pad, first + 1, torch.randn(rows, cols, generator=g, device="cuda"))
        ws = torch.empty(nsm.embedding_workspace_bytes(rows, vocab, cols), dtype=torch.uint8, device="cuda")
        d_w = view(vocab, cols, w_type, pad, first, torch.ones(vocab, cols, device="cuda"))
        nsm.embedding_backward(d_out, tokens, d_w, ws, scale=0.5)
        nsm.embedding_backward(d_out, tokens.int(), w, ws, accumulate=True)
        keep(name, out=o, d=d_w, added=w)

    for sizes, types, gap, factor in GRADS:
        name = f"grads.{len(sizes)}of{sum(sizes)}.{factor}"
        g = torch.Generator(device="cuda").manual_seed(len(sizes))
        grads = []
        for i, n in enumerate(sizes):
            t = view(1, n, types[i % len(types)], 0, gap)[0] if n else torch.empty(0, device="cuda")
            t.copy_(torch.randn(n, generator=g, device="cuda") * factor)
            grads.append(t)
        slots = [torch.zeros(n + 8, dtype=torch.bfloat16, device="cuda")[i % 3:i % 3 + n] for i, n in enumerate(sizes)]
        table, norm, norms = nsm.GradTable(grads, slots), torch.empty(1, device="cuda"), torch.empty(len(sizes), device="cuda")
        ws = torch.empty(table.workspace_bytes, dtype=torch.uint8, device="cuda")
        nsm.grad_norm(table, norm, norms, workspace=ws)
        norm0, norms0 = norm.clone(), norms.clone()
        nsm.clip_grads(table, 0.75, norm, norms, workspace=ws)
        nsm.clip_grads(grads, 0.75, workspace=ws)
        keep(name, norm=norm0, norms=norms0, again=norm, each=norms, slots=torch.cat(slots), grads=torch.cat([t.float() for t in grads]))
    return out, status


if __name__ == "__main__":
    import newton_schulz_orthogonalized_gb300 as nsm_module
    outputs, statuses = run(nsm_module)
    np.savez(sys.argv[1], **outputs)
    with open(os.path.splitext(sys.argv[1])[0] + ".json", "w") as fh:
        json.dump({"checked": nsm_module.checked_build(), "status": {k: list(v) for k, v in statuses.items()}}, fh)
