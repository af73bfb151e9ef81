"""Distils a small language model head from a teacher, with this library from the logits on:
the teacher's top log probabilities (logprobs), the student's loss and gradient in one pass
(distill_grad, or logprobs_grad for the plain cross-entropy), and the optimizer step
(MuonAdamW: Muon for the hidden matrices, AdamW for the embedding and the head).

    python examples/distill_finetune.py [--steps 40] [--loss distill|ce] [--vocab 5003]

PyTorch does the model's own products and carries the logits' gradient back through them
(``logits.backward(d_logits)``).  The data are synthetic: random contexts whose next tokens are
drawn from the teacher.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_schulz_orthogonalized_gb300 as nsm  # noqa: E402


class Model(torch.nn.Module):
    """Two embedded context tokens, a gated hidden layer, a head over the vocabulary."""

    def __init__(self, vocab: int, width: int, seed: int, scale: float):
        super().__init__()
        g = torch.Generator(device="cuda").manual_seed(seed)

        def matrix(rows, cols, size):
            return torch.nn.Parameter((torch.randn(rows, cols, generator=g, device="cuda") * size).bfloat16())

        self.embed_tokens = matrix(vocab, width, 1.0)
        self.up = matrix(4 * width, 2 * width, (2 * width) ** -0.5)
        self.gate = matrix(4 * width, 2 * width, (2 * width) ** -0.5)
        self.down = matrix(width, 4 * width, (4 * width) ** -0.5)
        self.lm_head = matrix(vocab, width, scale * width ** -0.5)

    def forward(self, context):
        x = torch.nn.functional.embedding(context, self.embed_tokens).flatten(1)
        h = (torch.nn.functional.silu(x @ self.gate.T) * (x @ self.up.T)) @ self.down.T
        return torch.nn.functional.layer_norm(h, h.shape[1:]) @ self.lm_head.T


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--loss", choices=("distill", "ce"), default="distill")
    ap.add_argument("--vocab", type=int, default=5003)
    ap.add_argument("--width", type=int, default=128)
    ap.add_argument("--rows", type=int, default=1024)
    ap.add_argument("--top", type=int, default=32)
    ap.add_argument("--temperature", type=float, default=1.0)
    a = ap.parse_args(argv)

    teacher = Model(a.vocab, a.width, seed=1, scale=3.0)
    student = Model(a.vocab, a.width, seed=2, scale=0.5)
    student.embed_tokens.data.copy_(teacher.embed_tokens.data)
    named = dict(student.named_parameters())
    opt = nsm.MuonAdamW([(n, tuple(p.shape)) for n, p in named.items()], muon_lr=0.02, adam_lr=2e-3)
    for n, p in named.items():
        opt.param(n).copy_(p.data)

    def numbers(*shape, dtype=torch.float32):
        return torch.empty(*(shape or (a.rows,)), dtype=dtype, device="cuda")

    top_logprob, top_index = numbers(a.rows, a.top), numbers(a.rows, a.top, dtype=torch.int32)
    loss, logprob, entropy = numbers(), numbers(), numbers()
    weight = torch.full((a.rows,), 1.0 / a.rows, device="cuda")
    contexts = torch.Generator(device="cuda").manual_seed(3)
    history = []
    for step in range(a.steps):
        context = torch.randint(0, a.vocab, (a.rows, 2), generator=contexts, device="cuda")
        with torch.no_grad():
            # what a teacher leaves for its student: k log probabilities and tokens a row
            teacher_logits = teacher(context)
            nsm.logprobs(teacher_logits, None, top_logprob=top_logprob, top_index=top_index,
                         temperature=a.temperature)
            tokens = torch.multinomial(torch.softmax(teacher_logits.float(), 1), 1, generator=contexts)[:, 0]
        logits = student(context)
        d_logits = torch.empty_like(logits)
        if a.loss == "distill":
            nsm.distill_grad(logits.detach(), top_logprob, top_index, weight, d_logits, loss,
                             temperature=a.temperature, tail=True)
        else:
            nsm.logprobs_grad(logits.detach(), tokens, -weight, None, d_logits, logprob)
            loss = -logprob
        logits.backward(d_logits)
        nsm.logprobs(logits.detach(), tokens, logprob, entropy)
        history.append((float(loss.mean()), float(logprob.mean()), float(entropy.mean())))
        for n, p in named.items():
            opt.grad(n).copy_(p.grad)
            p.grad = None
        opt.step()
        for n, p in named.items():
            p.data.copy_(opt.param(n))
        if step % max(1, a.steps // 8) == 0 or step == a.steps - 1:
            print(f"step {step:4d}  {a.loss} {history[-1][0]:8.4f}  log probability of the teacher's tokens "
                  f"{history[-1][1]:8.4f}  entropy {history[-1][2]:7.4f}")
    status = nsm.device_status()
    if status != nsm.NSM_OK:
        raise RuntimeError(f"device status {status}")
    return history


if __name__ == "__main__":
    main()
