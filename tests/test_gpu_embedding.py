"""The embedding lookup and its gradient on the GPU against the float64 oracle."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

from oracle import embedding_ref as ref  # noqa: E402


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


def _view(rows, cols, dtype, pad=0, first=0, fill=7.0):
    """A rows x cols view of a wider buffer that begins `first` elements in; (view, buffer)."""
    torch = _torch()
    buf = torch.full((rows * (cols + pad) + first + 8,), fill, dtype=_dtype(dtype), device="cuda")
    return buf[first:first + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], buf


def _tokens(rows, vocab, wide, seed, kind):
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "same":
        t = torch.full((rows,), vocab - 1, device="cuda")
    elif kind == "none":
        t = torch.randint(vocab, vocab + 9, (rows,), generator=g, device="cuda")
    elif kind == "skew":
        t = (vocab * torch.rand(rows, generator=g, device="cuda") ** 4).long()
    else:
        t = torch.randint(-2, vocab + 2, (rows,), generator=g, device="cuda")
    if kind == "skew" and rows > 4:
        t[::5] = -100
    return t.long() if wide else t.int()


def _workspace(nsm, rows, vocab, cols):
    torch = _torch()
    return torch.full((nsm.embedding_workspace_bytes(rows, vocab, cols),), 0xff, dtype=torch.uint8, device="cuda")


# rows, vocab, cols, weight, rows' type, padding, first element, tokens
CASES = [(1, 1, 1, "bf16", "fp32", 0, 0, "any"), (3, 5, 7, "fp32", "bf16", 1, 1, "any"), (33, 17, 8, "bf16", "bf16", 0, 0, "any"),
         (100, 3, 24, "fp16", "fp16", 0, 0, "any"), (257, 1023, 33, "fp32", "fp32", 0, 3, "skew"), (31, 1024, 100, "bf16", "fp32", 4, 0, "any"),
         (1000, 32003, 769, "fp32", "fp32", 0, 0, "skew"), (1025, 50257, 256, "bf16", "bf16", 0, 1, "skew"), (2048, 300, 264, "fp16", "fp32", 8, 0, "skew"),
         (4097, 259, 128, "bf16", "bf16", 0, 0, "skew"), (1500, 77, 520, "fp32", "bf16", 0, 2, "same"), (3000, 9, 64, "bf16", "fp16", 0, 0, "same"),
         (40, 65, 48, "fp32", "fp32", 0, 0, "none"), (70001, 1500, 16, "fp32", "bf16", 0, 0, "skew"), (600, 1 << 21, 8, "bf16", "bf16", 0, 0, "any"),
         (64, 10, 4104, "bf16", "bf16", 0, 0, "any")]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("wide", [True, False])
def test_lookup(nsm, case, wide):
    torch = _torch()
    rows, vocab, cols, w_type, o_type, pad, first, kind = case
    tokens = _tokens(rows, vocab, wide, rows + vocab, kind)
    w, _ = _view(vocab, cols, w_type, pad, first)
    w.copy_(torch.randn(vocab, cols, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda"))
    for scale in (1.0, -3.7):
        out, buf = _view(rows, cols, o_type, pad, first)
        nsm.embedding(w, tokens, out, scale=scale)
        # the scale is an fp32 number; one product, one rounding
        want = ref.embedding(w.double().cpu().numpy(), tokens.cpu().numpy(), float(np.float32(scale)))
        got = out.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= ((2.0 ** -24 + HALF_STEP[o_type]) * np.abs(want) + LEAST[o_type]) * 1.0001)
        out.fill_(7.0)
        assert bool((buf == 7.0).all())


def _sum_near(got, d_out, tokens, vocab, scale, old, out_type):
    want, size, count = ref.embedding_backward(d_out.double().cpu().numpy(), tokens.cpu().numpy(), vocab, float(np.float32(scale)),
                                               None if old is None else old.double().cpu().numpy())
    got = got.double().cpu().numpy()
    # n sums, the scale's product and the sum with what was there, of relative size 2^-24 each; one rounding
    tol = (count[:, None] + 2) * 2.0 ** -24 * size + HALF_STEP[out_type] * np.abs(want) + LEAST[out_type]
    assert np.all(np.abs(got - want) <= tol * 1.0001), np.max(np.abs(got - want) / tol)
    if old is None:
        assert np.all(got[count == 0] == 0.0)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("wide", [True, False])
def test_gradient(nsm, case, wide):
    torch = _torch()
    rows, vocab, cols, w_type, o_type, pad, first, kind = case
    tokens = _tokens(rows, vocab, wide, rows + vocab, kind)
    g = torch.Generator(device="cuda").manual_seed(rows)
    d_out, _ = _view(rows, cols, o_type, pad, first)
    d_out.copy_(torch.randn(rows, cols, generator=g, device="cuda"))
    ws = _workspace(nsm, rows, vocab, cols)
    for scale, accumulate, w_first in ((1.0, False, first), (0.37, False, first + 1), (-1.5, True, first)):
        d_w, buf = _view(vocab, cols, w_type, pad, w_first)
        old = None
        if accumulate:
            d_w.copy_(torch.randn(vocab, cols, generator=g, device="cuda"))
            old = d_w.clone()
        nsm.embedding_backward(d_out, tokens, d_w, ws, scale=scale, accumulate=accumulate)
        _sum_near(d_w, d_out, tokens, vocab, scale, old, w_type)
        # the same again, from another workspace's leavings
        first_bits = d_w.clone()
        if accumulate:
            d_w.copy_(old)
        ws.random_(0, 256)
        nsm.embedding_backward(d_out, tokens, d_w, ws, scale=scale, accumulate=accumulate)
        assert torch.equal(d_w, first_bits)
        d_w.fill_(7.0)
        assert bool((buf == 7.0).all())


def test_no_rows(nsm):
    torch = _torch()
    w = torch.randn(50, 12, device="cuda")
    none, tokens = torch.empty(0, 12, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    nsm.embedding(w, tokens, none)
    ws = _workspace(nsm, 0, 50, 12)
    kept = w.clone()
    nsm.embedding_backward(none, tokens, w, ws, accumulate=True)
    assert torch.equal(w, kept)
    nsm.embedding_backward(none, tokens, w, ws)
    assert bool((w == 0).all())


def test_rows_of_weight_past_32_bit_offsets(nsm):
    """Offsets of rows beyond 2^31 elements."""
    torch = _torch()
    vocab, cols = 600000, 4096
    w = torch.zeros(vocab, cols, dtype=torch.bfloat16, device="cuda")
    w[-1] = 3.0
    tokens = torch.tensor([vocab - 1, 0, vocab - 1], device="cuda")
    out = torch.empty(3, cols, device="cuda")
    nsm.embedding(w, tokens, out)
    assert out[:, 0].tolist() == [3.0, 0.0, 3.0]
    d = torch.ones(3, cols, dtype=torch.bfloat16, device="cuda")
    nsm.embedding_backward(d, tokens, w, _workspace(nsm, 3, vocab, cols))
    assert float(w[-1].float().min()) == 2.0 and float(w[0].float().max()) == 1.0 and float(w[1:-1].abs().max()) == 0.0


def test_values_that_are_no_numbers_stay_in_their_rows(nsm):
    torch = _torch()
    d = torch.ones(5, 16, device="cuda")
    d[1], d[3] = float("nan"), float("inf")
    tokens = torch.tensor([0, -1, 2, 4, 0], device="cuda")
    w = torch.empty(6, 16, device="cuda")
    nsm.embedding_backward(d, tokens, w, _workspace(nsm, 5, 6, 16))
    assert w[:, 0].tolist() == [2.0, 0.0, 1.0, 0.0, float("inf"), 0.0]


def test_gradient_against_differences(nsm):
    """sum(lookup * d_out) is linear in the weight: its slope is the gradient."""
    torch = _torch()
    tokens = _tokens(300, 40, True, 1, "skew")
    w = torch.randn(40, 24, device="cuda")
    d_out = torch.randn(300, 24, device="cuda")
    g = torch.empty_like(w)
    nsm.embedding_backward(d_out, tokens, g, _workspace(nsm, 300, 40, 24), scale=1.25)

    def value(z):
        out = torch.empty(300, 24, device="cuda")
        nsm.embedding(z, tokens, out, scale=1.25)
        return out.double().mul(d_out.double()).sum()

    for v, c in ((0, 0), (1, 23), (39, 5), (7, 7)):
        up, down = w.clone(), w.clone()
        up[v, c] += 1.0
        down[v, c] -= 1.0
        # 300 rows' rounded products, each at most some 2^-24 of 1.25 (|w| + 1) |d|
        assert abs(float(value(up) - value(down)) / 2 - float(g[v, c])) <= 300 * 2.0 ** -24 * 100


def test_captured_and_replayed(nsm):
    """Two captured calls that share a workspace, replayed with other tokens and between eager calls."""
    torch = _torch()
    rows, vocab, cols = 3000, 2000, 96
    tokens = _tokens(rows, vocab, True, 5, "skew")
    d_out = torch.randn(rows, cols, device="cuda").bfloat16()
    a, b = torch.empty(vocab, cols, dtype=torch.bfloat16, device="cuda"), torch.zeros(vocab, cols, device="cuda")
    ws = _workspace(nsm, rows, vocab, cols)
    nsm.embedding_backward(d_out, tokens, a, ws)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        nsm.embedding_backward(d_out, tokens, a, ws)
    with torch.cuda.graph(graphs[1]):
        nsm.embedding_backward(d_out, tokens, b, ws, accumulate=True)
    for seed in (1, 2):
        tokens.copy_(_tokens(rows, vocab, True, seed, "skew"))
        b.zero_()
        graphs[0].replay()
        graphs[1].replay()
        _sum_near(a, d_out, tokens, vocab, 1.0, None, "bf16")
        _sum_near(b, d_out, tokens, vocab, 1.0, None, "fp32")
        c = torch.empty_like(a)
        nsm.embedding_backward(d_out, tokens, c, ws)
        assert torch.equal(a, c)


def test_two_streams_with_a_workspace_each(nsm):
    torch = _torch()
    rows, vocab, cols = 20000, 3000, 128
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    tokens = [_tokens(rows, vocab, True, i, "skew") for i in range(2)]
    d_out = [torch.randn(rows, cols, device="cuda") for _ in range(2)]
    out = [torch.empty(vocab, cols, device="cuda") for _ in range(2)]
    ws = [_workspace(nsm, rows, vocab, cols) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            nsm.embedding_backward(d_out[i], tokens[i], out[i], ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        _sum_near(out[i], d_out[i], tokens[i], vocab, 1.0, None, "fp32")


def test_workspace_refusals(nsm):
    torch = _torch()
    d, t, w = torch.zeros(9, 8, device="cuda"), torch.zeros(9, dtype=torch.int64, device="cuda"), torch.zeros(5, 8, device="cuda")
    ws = _workspace(nsm, 9, 5, 8)
    for bad in (None, ws[:-256], ws[1:]):
        with pytest.raises(nsm.NsmError):
            nsm.embedding_backward(d, t, w, bad)
    with pytest.raises(ValueError):
        nsm.embedding_backward(d, t, w, torch.zeros(ws.numel(), dtype=torch.uint8))
    with pytest.raises(nsm.NsmError):
        nsm.embedding_backward(d, t, w, w.view(torch.uint8).view(-1))


@pytest.mark.parametrize("rows,vocab,cols", [(9000, 300000, 24), (5000, (1 << 28) + 5, 1)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_of_more_sorting_passes(nsm, rows, vocab, cols, accumulate):
    """Vocabularies whose tokens take three and four digits."""
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(rows)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    tokens[: rows // 3] = tokens[-(rows // 3):] // 4096 * 4096 % vocab  # some tokens several times
    tokens[::11] = -100
    d_out = torch.randn(rows, cols, generator=g, device="cuda")
    w = torch.full((vocab, cols), 0.5, dtype=torch.bfloat16, device="cuda")
    nsm.embedding_backward(d_out, tokens, w, _workspace(nsm, rows, vocab, cols), accumulate=accumulate)
    live = tokens >= 0
    some, place = torch.unique(tokens[live], return_inverse=True)
    start = 0.5 if accumulate else 0.0
    got = w[some]
    _sum_near(got, d_out[live], place, len(some), 1.0, torch.full_like(got, 0.5) if accumulate else None, "bf16")
    w[some] = start
    assert bool((w == start).all())
