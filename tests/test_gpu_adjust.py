"""Penalties, biases and masks on logits on the GPU against the float64 oracle."""

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
LEAST = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}            # half the least subnormal


def _dtype(name):
    return getattr(_torch(), KINDS[name])


def _view(rows, cols, dtype, pad=0, first=0, fill=7.0):
    """A rows x cols view of a wider buffer that begins `first` elements in; (view, buffer)."""
    torch = _torch()
    buf = torch.full((rows * (cols + pad) + first + 8,), fill, dtype=_dtype(dtype), device="cuda")
    return buf[first:first + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], buf


def _inputs(rows, vocab, dtype, seed, length, lines=None, k=0, masks=0, allowed=0.5, wide=True, pad=0, first=0):
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(seed)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    x, _ = _view(rows, vocab, dtype, pad, first)
    x.copy_(torch.randn(rows, vocab, generator=g, device="cuda") * 3)
    x[0, vocab // 2] = 0.0
    kw = {}
    kind = torch.int64 if wide else torch.int32
    if length:
        kw["history"] = torch.randint(-2, vocab + 2, (lines or rows, length), generator=g, device="cuda").to(kind)
        kw["history"][:, ::3] = kw["history"][:, :1].clone()  # one token many times
        kw["length"] = torch.randint(-1, length + 3, (rows,), generator=g, device="cuda").int()
        kw["length"][0] = length
        if lines:
            kw["history_row"] = torch.randint(-1, lines + 1, (rows,), generator=g, device="cuda").int()
            kw["history_row"][0] = 0
        kw["repetition"], kw["frequency"], kw["presence"] = 0.7 + uniform(rows), uniform(rows) - 0.3, uniform(rows) - 0.5
    if k:
        kw["bias_index"] = torch.randint(-1, vocab + 1, (rows, k), generator=g, device="cuda").to(kind)
        kw["bias_index"][:, -1] = kw["bias_index"][:, 0].clone()  # the same index twice
        kw["bias"] = torch.randn(rows, k, generator=g, device="cuda") * 4
    if masks:
        bits = (torch.rand(masks, (vocab + 31) // 32, 32, generator=g, device="cuda") < allowed).long()
        words = (bits << torch.arange(32, device="cuda")).sum(2)
        kw["mask"] = torch.where(words >= 1 << 31, words - (1 << 32), words).int()
        kw["mask"][0] = 0  # a row that allows nothing
        if masks != rows:
            kw["mask_row"] = torch.randint(-1, masks + 1, (rows,), generator=g, device="cuda").int()
            kw["mask_row"][0] = 0
    return x, kw


def _host(kw):
    return {n: t.cpu().numpy() for n, t in kw.items()}


def _back(kw):
    return {n: t for n, t in kw.items() if n not in ("frequency", "presence", "bias_index", "bias")}


def _forward_near(got, x, kw, out):
    want, size = ref.adjust(x.double().cpu().numpy(), **_host(kw))
    got = got.double().cpu().numpy()
    k = kw["bias"].shape[1] if "bias" in kw else 0
    # fp32: quotient or product, penalty (a fused one), difference, one sum per bias; then one rounding
    tol = (3 + k) * 2.0 ** -24 * size + HALF_STEP[out] * np.abs(want) + LEAST[out]
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    fine = np.isfinite(want)
    assert np.all(np.abs(got[fine] - want[fine]) <= tol[fine] * 1.0001)


def _backward_near(got, x, d_out, kw, out):
    want = ref.adjust_backward(x.double().cpu().numpy(), d_out.double().cpu().numpy(), **_host(_back(kw)))
    got = got.double().cpu().numpy()
    tol = (2.0 ** -24 + HALF_STEP[out]) * np.abs(want) + LEAST[out]
    assert np.all(np.abs(got - want) <= tol * 1.0001)
    assert np.array_equal(got == 0, want == 0) or out == "fp16"


# rows, vocab, type, tokens of history, its rows (0: one per row), biases, masks, padding, first element
CASES = [(1, 1, "bf16", 3, 0, 1, 1, 0, 0), (2, 7, "fp32", 5, 0, 2, 2, 1, 1), (3, 31, "fp16", 1, 0, 0, 3, 0, 1),
         (3, 32, "bf16", 0, 0, 4, 3, 3, 0), (5, 33, "fp32", 40, 2, 0, 0, 0, 3), (4, 1000, "bf16", 257, 3, 5, 2, 0, 5),
         (2, 8185, "fp16", 300, 0, 3, 2, 2, 7), (3, 8192, "bf16", 64, 0, 0, 5, 0, 0), (3, 8193, "fp32", 1000, 0, 6, 3, 7, 2),
         (2, 16377, "bf16", 100, 1, 9, 2, 0, 3), (5, 50257, "bf16", 700, 0, 4, 5, 0, 0), (2, 65537, "fp32", 2000, 2, 300, 1, 3, 1),
         (2, 131072, "fp16", 5000, 0, 16, 2, 0, 0), (1, 1 << 20, "bf16", 100, 0, 1024, 1, 0, 0), (40, 259, "fp16", 9, 7, 3, 4, 1, 0)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("wide", [True, False])
def test_forward_and_backward(nsm, case, wide):
    torch = _torch()
    rows, vocab, dtype, length, lines, k, masks, pad, first = case
    x, kw = _inputs(rows, vocab, dtype, rows * 1000 + vocab, length, lines, k, masks, wide=wide, pad=pad, first=first)
    x0 = x.clone()
    for out_type, out_first in ((dtype, first), ("fp32", 0), (dtype, first + 1)):
        out, buf = _view(rows, vocab, out_type, pad, out_first)
        nsm.adjust_logits(x, out, **kw)
        _forward_near(out, x, kw, out_type)
        out.fill_(7.0)
        assert bool((buf == 7.0).all())  # nothing beside the rows
    assert torch.equal(x, x0)
    g = torch.Generator(device="cuda").manual_seed(vocab)
    for d_type, d_first in ((dtype, first), ("fp32", 1)):
        d_out, _ = _view(rows, vocab, d_type, pad, d_first)
        d_out.copy_(torch.randn(rows, vocab, generator=g, device="cuda"))
        d_x, buf = _view(rows, vocab, dtype, pad, first)
        nsm.adjust_logits_backward(x, d_out, d_x, **_back(kw))
        _backward_near(d_x, x, d_out, kw, dtype)
        d_x.fill_(7.0)
        assert bool((buf == 7.0).all())


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_in_place_gives_the_same_bits(nsm, case):
    torch = _torch()
    rows, vocab, dtype, length, lines, k, masks, pad, first = case
    x, kw = _inputs(rows, vocab, dtype, rows + vocab, length, lines, k, masks, pad=pad, first=first)
    out, again = torch.empty_like(x), torch.empty_like(x)
    nsm.adjust_logits(x, out, **kw)
    nsm.adjust_logits(x, again, **kw)
    assert torch.equal(out, again)
    y, buf = _view(rows, vocab, dtype, pad, first)
    y.copy_(x)
    nsm.adjust_logits(y, y, **kw)
    assert torch.equal(y, out)
    d_out = torch.randn(rows, vocab, device="cuda").to(x.dtype)
    d_x = torch.empty_like(x)
    nsm.adjust_logits_backward(x, d_out, d_x, **_back(kw))
    y.copy_(d_out)
    nsm.adjust_logits_backward(x, y, y, **_back(kw))
    assert torch.equal(y, d_x)
    y.fill_(7.0)
    assert bool((buf == 7.0).all())


def test_only_what_is_asked_for(nsm):
    """Each part alone, and none: a copy, in the other type too."""
    torch = _torch()
    x, kw = _inputs(6, 5003, "bf16", 5, 50, 0, 7, 6)
    groups = [(), ("mask",), ("bias", "bias_index"), ("history", "repetition"), ("history", "frequency"), ("history", "presence"),
              ("history",), ("history", "length", "presence"), ("mask", "bias", "bias_index")]
    for names in groups:
        part = {n: kw[n] for n in names}
        for out_type in ("bf16", "fp32"):
            out = torch.empty(6, 5003, dtype=_dtype(out_type), device="cuda")
            nsm.adjust_logits(x, out, **part)
            _forward_near(out, x, part, out_type)
            if not names or names == ("history",):
                assert torch.equal(out, x.to(out.dtype))
        d = torch.empty_like(x)
        nsm.adjust_logits_backward(x, x, d, **_back(part))
        _backward_near(d, x, x, part, "bf16")
    d = torch.empty_like(x)
    nsm.adjust_logits_backward(None, x, d, mask=kw["mask"])
    _backward_near(d, x, x, {"mask": kw["mask"]}, "bf16")


def test_tables_with_row_strides(nsm):
    """Histories, biases and masks that are views of wider buffers, and begin anywhere."""
    torch = _torch()
    x, kw = _inputs(7, 9001, "bf16", 21, 301, 3, 6, 4)

    def strided(t, first, pad):
        buf = torch.full((t.shape[0] * (t.shape[1] + pad) + first,), 5, dtype=t.dtype, device="cuda")
        v = buf[first:].view(t.shape[0], t.shape[1] + pad)[:, :t.shape[1]]
        v.copy_(t)
        return v

    want, d_want = torch.empty(7, 9001, device="cuda"), torch.empty_like(x)
    nsm.adjust_logits(x, want, **kw)
    nsm.adjust_logits_backward(x, x, d_want, **_back(kw))
    for first, pad in ((1, 0), (0, 3), (3, 5)):
        for wide in (True, False):
            other = dict(kw)
            for n in ("history", "bias_index"):
                other[n] = strided(kw[n].long() if wide else kw[n].int(), first, pad)
            other["bias"], other["mask"] = strided(kw["bias"], first, pad), strided(kw["mask"], first, pad)
            out, d = torch.empty_like(want), torch.empty_like(x)
            nsm.adjust_logits(x, out, **other)
            nsm.adjust_logits_backward(x, x, d, **_back(other))
            assert torch.equal(out, want) and torch.equal(d, d_want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_values_that_are_no_numbers(nsm, dtype):
    """A banned token is -inf (its gradient 0) whatever stood there; infinities keep their sign."""
    torch = _torch()
    inf, nan = float("inf"), float("nan")
    lowest = torch.finfo(_dtype(dtype)).min
    x = torch.tensor([[nan, inf, -inf, lowest, 1.0, -1.0, nan, inf, -inf, lowest, 1.0, -1.0]], device="cuda").to(_dtype(dtype))
    history = torch.arange(12, device="cuda")[None]
    theta = torch.tensor([2.0], device="cuda")
    mask = torch.tensor([[0b111111000000]], dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    nsm.adjust_logits(x, out, history=history, repetition=theta, mask=mask)
    got = out[0].float().tolist()
    assert got[:6] == [-inf] * 6
    assert np.isnan(got[6]) and got[7:9] == [inf, -inf] and got[10:] == [0.5, -2.0]
    assert got[9] == -inf  # twice the lowest value: past the type's range
    d = torch.empty_like(x)
    nsm.adjust_logits_backward(x, torch.full_like(x, nan), d, mask=mask)
    assert d[0, :6].tolist() == [0.0] * 6 and bool(d[0, 6:].isnan().all())
    ones = torch.ones_like(x)
    nsm.adjust_logits_backward(x, ones, d, history=history, repetition=theta)
    assert d[0].float().tolist() == [2.0, 0.5, 2.0, 2.0, 0.5, 2.0] * 2


def test_long_history_and_empty_ones(nsm):
    torch = _torch()
    n = 200001
    history = torch.zeros(1, n, dtype=torch.int32, device="cuda")
    history[0, -1] = 5
    x = torch.zeros(4, 9, device="cuda")
    length = torch.tensor([n, n - 1, 0, -7], dtype=torch.int32, device="cuda")
    f = torch.full((4,), 0.5, device="cuda")
    out = torch.empty_like(x)
    nsm.adjust_logits(x, out, history=history, length=length, history_row=torch.zeros(4, dtype=torch.int32, device="cuda"), frequency=f)
    want = torch.zeros(4, 9, device="cuda")
    want[0, 0], want[0, 5], want[1, 0] = -0.5 * (n - 1), -0.5, -0.5 * (n - 1)
    assert torch.equal(out, want)
    # no tokens at all, and no rows
    nsm.adjust_logits(x, out, history=history[:, :0].expand(4, 0), frequency=f)
    assert torch.equal(out, x)
    nsm.adjust_logits(x[:0], out[:0])


def test_captured_and_replayed_on_another_stream(nsm):
    torch = _torch()
    x, kw = _inputs(9, 20011, "bf16", 77, 333, 2, 5, 3)
    out = torch.empty(9, 20011, device="cuda")
    want = torch.empty_like(out)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    nsm.adjust_logits(x, out, **kw, stream=stream)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nsm.adjust_logits(x, out, **kw)
    for seed in (1, 2):
        x.copy_(torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        kw["history"].copy_(torch.randint(0, 20011, kw["history"].shape, device="cuda"))
        graph.replay()
        nsm.adjust_logits(x, want, **kw)
        assert torch.equal(out, want)
        _forward_near(out, x, kw, "fp32")


def test_versions_and_autograd(nsm):
    """Torch knows what was written, and the pair is a differentiable function's two halves."""
    torch = _torch()
    x, kw = _inputs(4, 301, "fp32", 3, 20, 0, 3, 4, allowed=0.9)
    kw["mask"][0] = -1

    class Adjust(torch.autograd.Function):
        @staticmethod
        def forward(ctx, z):
            out = torch.empty_like(z)
            nsm.adjust_logits(z, out, **kw)
            ctx.save_for_backward(z)
            return out

        @staticmethod
        def backward(ctx, d_out):
            d = torch.empty_like(d_out)
            nsm.adjust_logits_backward(ctx.saved_tensors[0], d_out.contiguous(), d, **_back(kw))
            return d

    z = x.clone().requires_grad_(True)
    w = torch.randn(4, 301, device="cuda")
    out = Adjust.apply(z)
    torch.where(out == -float("inf"), torch.zeros_like(out), out).mul(w).sum().backward()
    step = 2.0 ** -6
    for r, v in ((0, 3), (1, 100), (2, 7), (3, 300), (0, int(kw["history"][0, 0].clamp(0, 300)))):
        def value(d):
            y = x.contiguous().clone()
            y[r, v] += d
            o = torch.empty_like(y)
            nsm.adjust_logits(y, o, **kw)
            return torch.where(o == -float("inf"), torch.zeros_like(o), o).double().mul(w.double()).sum()
        if abs(float(x[r, v])) > step:  # linear there: what is left is the rounding of two values
            slope = float(value(step) - value(-step)) / (2 * step)
            assert abs(slope - float(z.grad[r, v])) <= 2.0 ** -24 * 200 / step
    before = out._version
    nsm.adjust_logits(x, out.detach(), **kw)
    assert out._version > before
