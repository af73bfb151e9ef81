"""Launches of the vocabulary losses at every size of their shared memory: a block's default
limit is 48 KB for what a kernel declares and what a launch adds together, and a kernel's
limit belongs to the whole process, threads and earlier calls alike.  Each group runs in a
process of its own, so that no other call has raised a limit before."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _in_a_process(code):
    proc = subprocess.run([sys.executable, "-c", code], cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                          text=True, timeout=300)
    assert proc.returncode == 0, proc.stdout[-4000:]


HEAD = """
import torch
import newton_schulz_orthogonalized_gb300 as nsm
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
refused = []

def rows_of(rows, vocab, dtype):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    return torch.randn(rows, vocab, generator=g, device="cuda").to(TYPES[dtype])

def numbers(*shape):
    return torch.empty(*shape, device="cuda")

def attempt(what, call):
    try:
        call()
    except nsm.NsmError as e:
        refused.append((what, str(e)))
        return False
    return True

def near(got, want, vocab):
    # twice the relative error of a sum of exponentials over the row, as in test_gpu_vocab_loss.py
    tol = 2 * (108 + vocab / 256) * 2.0 ** -24 + 8 * 2.0 ** -24 * want.abs()
    assert bool(((got.double() - want).abs() <= tol).all()), (got, want)
"""

# rows and columns whose block takes somewhat less than 48 KB beside what the kernel declares
GRADIENTS = [(1100, 24410, "bf16"), (1100, 24500, "fp16"), (1100, 24553, "bf16"), (1100, 49000, "bf16"), (300, 97900, "bf16"),
             (1, 196000, "bf16"), (1, 196473, "fp16"), (1100, 12250, "fp32"), (1100, 24500, "fp32"), (300, 49000, "fp32"),
             (1, 97900, "fp32"), (1, 98237, "fp32")]


def test_gradients_just_under_the_default_limit():
    _in_a_process(HEAD + f"""
for rows, vocab, dtype in {GRADIENTS!r}:
    x = rows_of(rows, vocab, dtype)
    tokens = torch.arange(rows, device="cuda") % vocab
    w = torch.ones(rows, device="cuda")
    log_q = torch.log_softmax(x[-1].double(), 0)
    g, logprob, entropy = torch.empty_like(x), numbers(rows), numbers(rows)
    for h in (None, w):
        if attempt(("logprobs_grad", rows, vocab, dtype, h is not None),
                   lambda: nsm.logprobs_grad(x, tokens, w, h, g, logprob, entropy if h is not None else None)):
            near(logprob[-1], log_q[tokens[-1]], vocab)
    index = torch.arange(5, device="cuda").repeat(rows, 1)
    teacher = torch.zeros(rows, 5, device="cuda")
    loss = numbers(rows)
    if attempt(("distill_grad", rows, vocab, dtype), lambda: nsm.distill_grad(x, teacher, index, w, g, loss)):
        near(loss[-1], -(log_q[:5].mean() + torch.log(torch.tensor(5.0, dtype=torch.float64, device="cuda"))), vocab)
assert not refused, refused
assert nsm.device_status() == 0
""")


def test_forward_passes_just_under_the_default_limit():
    _in_a_process(HEAD + """
for rows, vocab in ((320, 196000), (160, 392000)):
    x = rows_of(rows, vocab, "fp32")
    index = torch.arange(5, device="cuda").repeat(rows, 1)
    teacher, loss = torch.zeros(rows, 5, device="cuda"), numbers(rows)
    if attempt(("distill", rows, vocab), lambda: nsm.distill(x, teacher, index, loss)):
        log_q = torch.log_softmax(x[-1].double(), 0)
        near(loss[-1], -(log_q[:5].mean() + torch.log(torch.tensor(5.0, dtype=torch.float64, device="cuda"))), vocab)
    del x
for rows, vocab, k, dtype in ((100, 256000, 128, "fp32"), (80, 262000, 106, "fp32"), (2, (1 << 20) - 8, 64, "fp32"),
                              (1, 819200, 128, "fp32"), (60, (1 << 20) - 16, 64, "fp16")):
    x = rows_of(rows, vocab, dtype)
    top, where, entropy = numbers(rows, k), torch.empty(rows, k, dtype=torch.int32, device="cuda"), numbers(rows)
    for e in (None, entropy):
        if attempt(("logprobs", rows, vocab, k, dtype, e is not None),
                   lambda: nsm.logprobs(x, None, entropy=e, top_logprob=top, top_index=where)):
            log_q = torch.log_softmax(x[-1].double(), 0)
            near(top[-1], torch.topk(log_q, k).values, vocab)
assert not refused, refused
assert nsm.device_status() == 0
""")


def test_threads_with_rows_of_different_lengths():
    # the same kernels with 65 and 100 KB of shared memory from two threads at once
    _in_a_process(HEAD + """
import threading
errors = []

def work(vocab, start):
    try:
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            x = rows_of(1, vocab, "bf16")
            tokens, w = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.ones(1, device="cuda")
            index, teacher = torch.zeros(1, 1, dtype=torch.int64, device="cuda"), torch.zeros(1, 1, device="cuda")
            g = torch.empty_like(x)
            torch.cuda.current_stream().synchronize()
            start.wait()
            for i in range(3000):
                nsm.logprobs_grad(x, tokens, w, None, g)
                nsm.distill_grad(x, teacher, index, w, g)
                if i % 200 == 0:
                    torch.cuda.current_stream().synchronize()
            torch.cuda.current_stream().synchronize()
    except Exception as e:
        errors.append((vocab, repr(e)))

start = threading.Barrier(2)
threads = [threading.Thread(target=work, args=(vocab, start)) for vocab in (262144, 400000)]
for t in threads:
    t.start()
for t in threads:
    t.join()
assert not errors, errors
assert nsm.device_status() == 0
""")
