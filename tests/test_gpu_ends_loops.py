"""The logit adjustments and the embedding lookup where a block takes several slices or units after one
another, against plain forms in 64 bits: the next slice under way, counts that go back to zero or on to the
next row of a sequence, and the first and last rounds of the loops."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

from oracle import adjust_ref as ref  # noqa: E402


def _torch():
    import torch
    return torch


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_orthogonalized_gb300 as m
    m.lib()
    return m


KINDS = {"bf16": "bfloat16", "fp16": "float16", "fp32": "float32"}
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}  # torch.finfo(t).eps / 2
LEAST = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}   # half the least subnormal


def _dtype(name):
    return getattr(_torch(), KINDS[name])


def _view(rows, cols, dtype, pad, first):
    torch = _torch()
    buf = torch.full((rows * (cols + pad) + first + 8,), 7.0, dtype=_dtype(dtype), device="cuda")
    return buf[first:first + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], buf


def _counts(rows, vocab, history, length=None, history_row=None):
    """How often each row's history holds each token, a place of the histories at a time."""
    torch = _torch()
    r = torch.arange(rows, device="cuda")
    line = r if history_row is None else history_row.long()
    n = torch.full((rows,), history.shape[1], device="cuda") if length is None else length.long().clamp(0, history.shape[1])
    n = torch.where((line >= 0) & (line < len(history)), n, 0)
    line = line.clamp(0, len(history) - 1)
    counts = torch.zeros(rows, vocab, dtype=torch.float64, device="cuda")
    for j in range(history.shape[1]):
        token = history[line, j].long()
        counts[r, token.clamp(0, vocab - 1)] += ((j < n) & (token >= 0) & (token < vocab)).double()
    return counts


def _allowed(rows, vocab, mask=None, mask_row=None):
    torch = _torch()
    if mask is None:
        return torch.ones(rows, vocab, dtype=torch.bool, device="cuda")
    line = torch.arange(rows, device="cuda") if mask_row is None else mask_row.long()
    v = torch.arange(vocab, device="cuda")
    bits = (mask.long()[:, v // 32] >> (v % 32) & 1).bool()
    return bits[line.clamp(0, len(mask) - 1)] | ((line < 0) | (line >= len(mask)))[:, None]


def _pick(kw, *names):
    return {n: kw[n] for n in names if n in kw}


def _slope(x, kw, counts):
    """What a logit is multiplied by."""
    torch = _torch()
    theta = kw["repetition"].double()[:, None]
    return torch.where(counts > 0, torch.where(x.double() > 0, 1 / theta, theta), torch.ones_like(counts))


def _adjust(x, kw):
    """(the adjusted logits, the sum of the sizes of what was added to each)"""
    torch = _torch()
    rows, vocab = x.shape
    counts = _counts(rows, vocab, **_pick(kw, "history", "length", "history_row"))
    a = x.double() * _slope(x, kw, counts)
    frequency, presence = kw["frequency"].double()[:, None], kw["presence"].double()[:, None]
    seen = counts > 0
    out = a - torch.where(seen, frequency * counts + presence, 0.0)
    size = a.abs() + torch.where(seen, frequency.abs() * counts + presence.abs(), 0.0)
    if "bias" in kw:
        r = torch.arange(rows, device="cuda")
        for j in range(kw["bias"].shape[1]):
            v = kw["bias_index"][:, j].long()
            b = torch.where((v >= 0) & (v < vocab), kw["bias"][:, j].double(), 0.0)
            out[r, v.clamp(0, vocab - 1)] += b
            size[r, v.clamp(0, vocab - 1)] += b.abs()
    return torch.where(_allowed(rows, vocab, **_pick(kw, "mask", "mask_row")), out, -float("inf")), size


def _sequences(rows, vocab, dtype, length, kind, seed, pad, first):
    """Rows that are the positions of sequences of 37: histories that grow by a token a row, stay, fall back,
    hold nothing, are none, and begin anew with a sequence."""
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = torch.arange(rows, device="cuda")
    lines = rows if kind == "own" else (rows + 36) // 37
    x, _ = _view(rows, vocab, dtype, pad, first)
    x.copy_(torch.randn(rows, vocab, generator=g, device="cuda") * 3)
    kw = {"history": torch.randint(-2, vocab + 2, (lines, length), generator=g, device="cuda").to(torch.int32 if seed % 2 else torch.int64)}
    kw["history"][:, 3::4] = kw["history"][:, :1].clone()  # a token again and again
    if vocab > 5000:  # tokens at the slices' ends
        kw["history"][:, 1::8] = (kw["history"][:, 1::8].clamp(0, vocab - 1) // 2048 * 2048 + kw["history"][:, 1::8] % 9 - 8).clamp(-1, vocab)
    at = r % 37 + 1
    at = torch.where(r % 5 == 4, at - 1, at)        # as the row before
    at = torch.where(r % 11 == 7, at // 2, at)      # shorter than that
    at = torch.where(r % 29 == 3, -1, at)           # nothing
    at = torch.where(r % 23 == 9, length + 5, at)   # all there is
    kw["length"] = at.int()
    if kind != "own":
        line = r // 37
        line = torch.where(r % 101 == 50, -1, line)
        kw["history_row"] = torch.where(r % 103 == 60, lines, line).int()
    kw["repetition"] = 0.7 + torch.rand(rows, generator=g, device="cuda")
    kw["frequency"] = torch.rand(rows, generator=g, device="cuda") - 0.3
    kw["presence"] = torch.rand(rows, generator=g, device="cuda") - 0.5
    if kind == "biases":
        kw["bias_index"] = torch.randint(-1, vocab + 1, (rows, 3), generator=g, device="cuda")
        kw["bias_index"][:, 2] = kw["bias_index"][:, 0].clone()
        kw["bias"] = torch.randn(rows, 3, generator=g, device="cuda")
    if kind in ("masks", "biases"):
        kw["mask"] = torch.randint(-2 ** 31, 2 ** 31, (7, (vocab + 31) // 32), generator=g, device="cuda").int()
        kw["mask"][2], kw["mask"][4] = 0, -1
        kw["mask_row"] = (r * 5 % 8 - 1).int()
    return x, kw


# type, vocabulary, slices of 4096 or (fp32) 2048 logits that it has with room for any alignment, times that a
# block comes round (rows that share a history are taken one after the other, as many as a quarter of that and four at most)
SHAPES = [("bf16", 61, 1, 3), ("bf16", 61, 1, 17), ("fp16", 4099, 2, 9), ("bf16", 8190, 3, 17), ("fp32", 97, 1, 13), ("fp32", 2049, 2, 17),
          ("fp32", 4097, 3, 9)]


@pytest.mark.parametrize("kind", ["history", "masks", "biases", "own"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_many_slices_a_block(nsm, shape, kind):
    torch = _torch()
    dtype, vocab, slices, rounds = shape
    resident = torch.cuda.get_device_properties(0).multi_processor_count * (8 if dtype == "fp32" else 7)
    rows = resident * rounds // slices + 3
    pad, first = (1, 3) if kind != "own" else (0, 0)
    x, kw = _sequences(rows, vocab, dtype, 41, kind, rows + len(kind), pad, first)
    want, size = _adjust(x, kw)
    banned = torch.isneginf(want)
    k = 3 if kind == "biases" else 0

    def near(got, out_type):
        assert torch.equal(torch.isneginf(got), banned)
        # fp32: quotient or product, penalty, difference, one sum per bias; then one rounding
        tol = (3 + k) * 2.0 ** -24 * size + HALF_STEP[out_type] * want.abs() + LEAST[out_type]
        assert bool((banned | ((got.double() - want).abs() <= tol * 1.0001)).all())

    for out_type, out_pad, out_first in ((dtype, pad, first), ("fp32", 0, 0)):
        out, buf = _view(rows, vocab, out_type, out_pad, out_first)
        nsm.adjust_logits(x, out, **kw)
        near(out, out_type)
        if out_type == dtype:  # in place the same bits
            y, _ = _view(rows, vocab, dtype, pad, first)
            y.copy_(x)
            nsm.adjust_logits(y, y, **kw)
            assert torch.equal(y, out)
        out.fill_(7.0)
        assert bool((buf == 7.0).all())
    # the plain form above is the oracle's: a few rows of it
    some = list(range(12)) + [rows - 1]
    part = {n: t[some].cpu().numpy() if n not in ("history", "mask") or (n == "history" and kind == "own") else t.cpu().numpy()
            for n, t in kw.items()}
    w, _ = ref.adjust(x[some].double().cpu().numpy(), **part)
    assert np.allclose(w, want[some].cpu().numpy(), rtol=1e-12, atol=1e-12)

    back = _pick(kw, "history", "length", "history_row", "repetition", "mask", "mask_row")
    del want, size
    slope = _slope(x, kw, _counts(rows, vocab, **_pick(kw, "history", "length", "history_row")))
    slope.masked_fill_(banned, 0.0)
    for d_type, d_pad, d_first in ((dtype, pad, first), ("fp32", 0, 1)):
        d_out, _ = _view(rows, vocab, d_type, d_pad, d_first)
        d_out.copy_(torch.randn(rows, vocab, generator=torch.Generator(device="cuda").manual_seed(vocab), device="cuda"))
        d_x, buf = _view(rows, vocab, dtype, pad, first)
        nsm.adjust_logits_backward(x, d_out, d_x, **back)
        exact = d_out.double() * slope
        # one quotient or product in fp32, one rounding
        assert bool(((d_x.double() - exact).abs() <= ((2.0 ** -24 + HALF_STEP[dtype]) * exact.abs() + LEAST[dtype]) * 1.0001).all())
        if d_type == dtype:
            nsm.adjust_logits_backward(x, d_out, d_out, **back)
            assert torch.equal(d_out, d_x)
        d_x.fill_(7.0)
        assert bool((buf == 7.0).all())
    assert nsm.device_status() == nsm.NSM_OK


# rows, vocab, cols, weight, rows' type, elements between rows, first one: all of more units than 2432 blocks take at once
LOOKUPS = [(30011, 5003, 769, "fp32", "bf16", 0, 0), (40003, 5003, 768, "bf16", "bf16", 0, 0), (20001, 1009, 2048, "fp16", "fp32", 3, 1),
           (2600003, 999, 8, "bf16", "fp16", 0, 0), (1300001, 70001, 9, "fp32", "fp32", 1, 3), (400009, 257, 250, "bf16", "fp32", 6, 0)]


@pytest.mark.parametrize("case", LOOKUPS, ids=lambda c: "x".join(map(str, c)))
def test_many_units_a_lane(nsm, case):
    torch = _torch()
    rows, vocab, cols, w_type, o_type, pad, first = case
    g = torch.Generator(device="cuda").manual_seed(rows)
    tokens = torch.randint(-1, vocab + 1, (rows,), generator=g, device="cuda").to(torch.int32 if rows % 3 else torch.int64)
    w, _ = _view(vocab, cols, w_type, pad, first)
    w.copy_(torch.randn(vocab, cols, generator=g, device="cuda"))
    live = (tokens >= 0) & (tokens < vocab)
    exact = torch.where(live[:, None], w[tokens.long().clamp(0, vocab - 1)].double(), 0.0)
    for scale in (1.0, -3.7):
        out, buf = _view(rows, cols, o_type, pad, first)
        nsm.embedding(w, tokens, out, scale=scale)
        want = exact * float(np.float32(scale))
        if scale == 1.0:
            assert torch.equal(out, exact.to(out.dtype))
        # one product in fp32, one rounding
        assert bool(((out.double() - want).abs() <= ((2.0 ** -24 + HALF_STEP[o_type]) * want.abs() + LEAST[o_type]) * 1.0001).all())
        out.fill_(7.0)
        assert bool((buf == 7.0).all())
    assert nsm.device_status() == nsm.NSM_OK
