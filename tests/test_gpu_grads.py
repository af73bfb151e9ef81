"""The norm of many gradients and clipping on the GPU against the float64 oracle."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

from oracle import grads_ref as ref  # noqa: E402


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
# A chunk's 16384 squares: at most 10 in each of a thread's 8 running sums (fused: one rounding
# each), 3 sums of those, 5 within a warp, 8 of the warps; scaled ones two products more.  The rest is 64-bit.  The
# root halves it and is rounded to fp32.
NORM_TOL = (10 + 3 + 5 + 8 + 2) / 2 * 2.0 ** -24 + 2 * 2.0 ** -24


def _dtype(name):
    return getattr(_torch(), KINDS[name])


def _pieces(sizes, dtypes, gap, seed, scale=1.0):
    """Tensors of these sizes out of one buffer per type, `gap` elements apart; and the buffers."""
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(seed)
    buffers, tensors, at = {}, [], {}
    for d in set(dtypes):
        total = sum(n + gap for n, t in zip(sizes, dtypes) if t == d) + gap + 8
        buffers[d], at[d] = torch.full((total,), 7.0, dtype=_dtype(d), device="cuda"), gap
    for i, (n, d) in enumerate(zip(sizes, dtypes)):
        t = buffers[d][at[d]:at[d] + n]
        t.copy_(torch.randn(n, generator=g, device="cuda") * scale * 10.0 ** -(i % 4))
        tensors.append(t)
        at[d] += n + gap
    return tensors, buffers


def _host(tensors):
    return [t.double().cpu().numpy() for t in tensors]


def _near(got, want, tol=NORM_TOL):
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    assert np.all(np.abs(got - want) <= tol * np.abs(want) + 2.0 ** -150), (got, want)


SIZES = [[1], [5, 0, 3], [7, 8, 9, 16384, 16385, 1, 0], [100003], [16384 * 3], [256] * 200, [1 << 20, 17, 40000, 3] * 5,
         [33] * 1300, [0, 0], [11008 * 64 + 5, 1000003]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}of{sum(s)}")
@pytest.mark.parametrize("types", [("bf16",), ("fp16",), ("fp32",), ("fp32", "bf16", "fp16")], ids="-".join)
@pytest.mark.parametrize("gap", [0, 1, 8])
def test_norm_and_clip(nsm, sizes, types, gap):
    torch = _torch()
    dtypes = [types[i % len(types)] for i in range(len(sizes))]
    grads, buffers = _pieces(sizes, dtypes, gap, len(sizes) + gap)
    norm, norms = torch.empty(1, device="cuda"), torch.empty(len(sizes), device="cuda")
    table = nsm.GradTable(grads)
    ws = torch.full((table.workspace_bytes,), 0xff, dtype=torch.uint8, device="cuda")
    nsm.grad_norm(table, norm, norms, workspace=ws)
    host = _host(grads)
    want, each = ref.grad_norm(host)
    _near(norm.item(), want)
    _near(norms.cpu(), each)
    total = torch.empty((), device="cuda")
    nsm.grad_norm(grads, total, workspace=ws)
    assert float(total) == float(norm)
    for out_types in (types, ("bf16",), ("fp32",), ("fp16",)):
        for limit in (want * 0.37 or 1.0, want * 2 + 1):
            out, out_buffers = _pieces(sizes, [out_types[i % len(out_types)] for i in range(len(sizes))], 1, 1)
            for o in out:
                o.fill_(5.0)
            norm.zero_()
            norms.zero_()
            nsm.clip_grads(nsm.GradTable(grads, out), float(np.float32(limit)), norm, norms, workspace=ws)
            _near(norm.item(), want)
            _near(norms.cpu(), each)
            clipped, _, _ = ref.clip_grads(host, float(np.float32(limit)))
            for i, (o, c) in enumerate(zip(out, clipped)):
                d = out_types[i % len(out_types)]
                # the norm's error, the factor's rounding, the product's, the result's
                tol = (NORM_TOL + 2 * 2.0 ** -24 + HALF_STEP[d]) * np.abs(c) + LEAST[d]
                assert np.all(np.abs(o.double().cpu().numpy() - c) <= tol * 1.0001)
                o.fill_(7.0)
            for b in out_buffers.values():
                assert bool((b == 7.0).all())
    # in place gives the same bits, and a norm within the limit changes nothing
    same = [torch.empty_like(t) for t in grads]
    limit = float(np.float32(want * 0.6 or 1.0))
    nsm.clip_grads(nsm.GradTable(grads, same), limit, None, None, workspace=ws)
    nsm.clip_grads(table, limit * 1e6, workspace=ws)
    for t, h in zip(grads, host):
        assert np.array_equal(t.double().cpu().numpy(), h)
    nsm.clip_grads(table, limit, norm, workspace=ws)
    _near(norm.item(), want)
    for t, s in zip(grads, same):
        assert torch.equal(t, s)
        t.fill_(7.0)
    for b in buffers.values():
        assert bool((b == 7.0).all())


@pytest.mark.parametrize("dtype,scale", [("fp32", 1e30), ("fp32", 1e-30), ("fp32", 1e-42), ("bf16", 1e37), ("bf16", 1e-37),
                                         ("fp32", 1e-12), ("fp16", 6e4), ("fp16", 1e-7)])
def test_squares_leave_no_range(nsm, dtype, scale):
    torch = _torch()
    grads, _ = _pieces([40000, 3, 16384, 77], [dtype] * 4, 1, 9)
    for t in grads:
        t.copy_((t.float().clamp(-1, 1).double() * scale))
    grads.append(torch.zeros(50000, dtype=_dtype(dtype), device="cuda"))
    norm, norms = torch.empty(1, device="cuda"), torch.empty(5, device="cuda")
    table = nsm.GradTable(grads)
    ws = torch.empty(table.workspace_bytes, dtype=torch.uint8, device="cuda")
    nsm.grad_norm(table, norm, norms, workspace=ws)
    want, each = ref.grad_norm(_host(grads))
    least = 2.0 ** -149  # of a subnormal norm
    if want > torch.finfo(torch.float32).max:  # sqrt(40000 and more) 1e37 is past fp32's range: +inf, as documented
        assert norm.item() == float("inf")
    else:
        assert abs(norm.item() - want) <= NORM_TOL * want + least
    each = np.where(each > torch.finfo(torch.float32).max, np.inf, each)
    assert np.array_equal(np.isinf(each), norms.isinf().cpu().numpy())
    fine = np.isfinite(each)
    assert np.all(np.abs(norms.double().cpu().numpy()[fine] - each[fine]) <= NORM_TOL * each[fine] + least)
    out = [torch.empty(t.shape, device="cuda") for t in grads]
    limit = float(np.float32(max(want * 1e-9, 1e-37) if scale > 1 else want / 3))
    if limit < 1e-30 and scale < 1:
        return
    nsm.clip_grads(nsm.GradTable(grads, out), limit, norm, workspace=ws)
    for o, c in zip(out, ref.clip_grads(_host(grads), limit)[0]):
        assert np.all(np.abs(o.double().cpu().numpy() - c) <= (NORM_TOL + 3 * 2.0 ** -24) * np.abs(c) + least)


def test_norm_past_fp32_and_a_tiny_factor(nsm):
    """The norm of these is past fp32's range; the factor is below it, the clipped ones are not."""
    torch = _torch()
    g = torch.full((1 << 20,), 3e38, device="cuda")
    out, norm = torch.empty_like(g), torch.empty(1, device="cuda")
    table = nsm.GradTable([g], [out])
    ws = torch.empty(table.workspace_bytes, dtype=torch.uint8, device="cuda")
    nsm.clip_grads(table, 1.0, norm, workspace=ws)
    assert norm.item() == float("inf")
    want = 1.0 / 1024
    assert float((out.double() - want).abs().max()) <= (NORM_TOL + 3 * 2.0 ** -24) * want


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_no_number_leaves_the_gradients(nsm, value):
    torch = _torch()
    grads, _ = _pieces([100, 40000], ["bf16", "fp32"], 0, 4)
    grads[1][33333] = value
    kept = [t.clone() for t in grads]
    norm, norms = torch.empty(1, device="cuda"), torch.empty(2, device="cuda")
    out = [torch.empty_like(t) for t in grads]
    ws = torch.empty(nsm.GradTable(grads).workspace_bytes, dtype=torch.uint8, device="cuda")
    for table in (nsm.GradTable(grads, out), nsm.GradTable(grads)):
        nsm.clip_grads(table, 1e-3, norm, norms, workspace=ws)
        for got in (norm[0], norms[1]):
            assert bool(got.isnan()) if value != value else float(got) == float("inf")
        assert bool(norms[0].isfinite())
        for t, k in zip(table.out or grads, kept):
            assert torch.equal(t.nan_to_num(123.0, 4.0, 5.0), k.nan_to_num(123.0, 4.0, 5.0))


def test_same_bits_every_time_and_captured(nsm):
    torch = _torch()
    grads, _ = _pieces([300001, 77, 16384, 5] * 4, ["bf16", "fp32"] * 8, 3, 8)
    out = [torch.empty_like(t) for t in grads]
    table = nsm.GradTable(grads, out)
    ws = torch.empty(table.workspace_bytes, dtype=torch.uint8, device="cuda")
    norm = torch.empty(1, device="cuda")
    nsm.clip_grads(table, 0.5, norm, workspace=ws)
    bits, first = [o.clone() for o in out], float(norm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nsm.clip_grads(table, 0.5, norm, workspace=ws)
    for _ in range(3):
        ws.random_(0, 256)
        norm.zero_()
        graph.replay()
        assert float(norm) == first and all(torch.equal(o, b) for o, b in zip(out, bits))
    for t in grads:
        t.mul_(3.0)
    graph.replay()
    _near(norm.item(), ref.grad_norm(_host(grads))[0])


def test_more_than_2_31_elements(nsm):
    torch = _torch()
    n = (1 << 31) + 4099
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-1], g[0], g[1 << 31] = 3.0, 4.0, 12.0
    norm = torch.empty(1, device="cuda")
    table = nsm.GradTable([g])
    ws = torch.empty(table.workspace_bytes, dtype=torch.uint8, device="cuda")
    nsm.clip_grads(table, 6.5, norm, workspace=ws)
    assert norm.item() == 13.0 and [float(g[i]) for i in (-1, 0, 1 << 31)] == [1.5, 2.0, 6.0]


def test_more_sums_than_a_block_adds(nsm):
    """Many launches, whose blocks' sums one launch adds first; in place and to slots."""
    torch = _torch()
    n, size = 8000, 20000
    buffer = torch.randn(n * size, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    grads = list(buffer.view(n, size))
    slots = torch.empty(n, size, dtype=torch.bfloat16, device="cuda")
    table = nsm.GradTable(grads, list(slots))
    norm, norms = torch.empty(1, device="cuda"), torch.empty(n, device="cuda")
    ws = torch.empty(table.workspace_bytes, dtype=torch.uint8, device="cuda")
    nsm.clip_grads(table, 2.0, norm, norms, workspace=ws)
    each = torch.linalg.vector_norm(buffer.view(n, size), dim=1, dtype=torch.float64)
    want = float(torch.linalg.vector_norm(each))
    _near(norm.item(), want)
    _near(norms.cpu(), each.cpu())
    clipped = buffer.view(n, size).double() * (2.0 / want)
    assert bool(((slots.double() - clipped).abs() <= (NORM_TOL + 2 * 2.0 ** -24 + 2.0 ** -8) * clipped.abs() * 1.0001 + LEAST["bf16"]).all())
    norm.zero_()
    nsm.clip_grads(grads, 2.0, norm, workspace=ws)
    _near(norm.item(), want)
    assert torch.equal(buffer.view(n, size), slots)


@pytest.mark.parametrize("captured", [False, True])
def test_first_clip_on_a_stream_of_its_own(nsm, captured):
    """While the current stream is behind: nothing that it still has to do is the clip's."""
    torch = _torch()
    opt = nsm.MuonAdamW([("layers.0.proj.weight", (64, 96)), ("norm.bias", (64,))])
    opt.grad("layers.0.proj.weight").fill_(0.5)
    opt.grad("norm.bias").fill_(2.0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            norm = opt.clip(1.0)
        opt.grad_norms.zero_()
        norm.zero_()
        graph.replay()
    else:
        torch.cuda._sleep(100_000_000)
        norm = opt.clip(1.0, stream=side.cuda_stream)
    torch.cuda.synchronize()
    _near(norm.item(), (64 * 96 * 0.25 + 64 * 4.0) ** 0.5)
    _near(opt.grad_norms.cpu(), [(64 * 96 * 0.25) ** 0.5, 16.0])


def test_refusals(nsm):
    torch = _torch()
    a, b = torch.zeros(100, device="cuda"), torch.zeros(100, device="cuda")
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    norm = torch.empty(1, device="cuda")

    def refused(table, **kw):
        with pytest.raises((nsm.NsmError, ValueError)):
            nsm.clip_grads(table, 1.0, kw.pop("norm", norm), workspace=kw.pop("workspace", ws), **kw)

    refused([a, a])                                   # twice in place
    refused(nsm.GradTable([a, b], [b, a]))            # one's place is another's input
    refused(nsm.GradTable([a[:50]], [a[25:75]]))
    refused([a], norm=a[3:4])
    refused([a], workspace=None)
    refused([a], workspace=ws[:8])
    refused([a], workspace=ws[1:])
    refused([a], norms=torch.empty(2, device="cuda"))
    refused([a], norm=torch.empty(1))
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(nsm.NsmError):
            nsm.clip_grads([a], bad, norm, workspace=ws)
    nsm.grad_norm([a, a, a[3:]], norm, workspace=ws)  # read twice: counted twice
    nsm.clip_grads(nsm.GradTable([a, b], [a, b]), 1.0, norm, workspace=ws)
    for bad in ([], [a.cpu()], [a.long()], [a.view(10, 10).T], [torch.zeros(3, 4, device="cuda")[:, :2]]):
        with pytest.raises(ValueError):
            nsm.GradTable(bad)
    for bad in ([b[:99]], [b, b], [b.cpu()]):
        with pytest.raises(ValueError):
            nsm.GradTable([a], bad)


def _named():
    return [("model.embed_tokens.weight", (97, 32)), ("layers.0.proj.weight", (128, 64)), ("layers.1.proj.weight", (40, 200)),
            ("norm.weight", (33,)), ("lm_head.weight", (97, 32))]


def test_optimizer_clips_its_slots(nsm):
    """MuonAdamW: clipping the slots, clipping gradients into them, and a step that clips first."""
    torch = _torch()
    opts = [nsm.MuonAdamW(_named(), adam_lr=1e-2) for _ in range(3)]
    g = torch.Generator(device="cuda").manual_seed(2)
    grads = {n: torch.randn(s, generator=g, device="cuda") * 3 for n, s in _named()}
    for o in opts:
        for n, _ in _named():
            o.param(n).copy_(torch.full(o.param(n).shape, 0.5))
            o.grad(n).copy_(grads[n])
    norm, each = ref.grad_norm(_host([opts[0].grad(n) for n in opts[0].muon_names + opts[0].adam_names]))
    got = opts[0].clip(1.5)
    _near(got.item(), norm)
    _near(opts[0].grad_norms.cpu(), each)
    for n, _ in _named():
        want = opts[1].grad(n).double() * min(1.0, 1.5 / norm)
        assert float((opts[0].grad(n).double() - want).abs().max()) <= (NORM_TOL + 2 * 2.0 ** -24 + 2.0 ** -8) * float(want.abs().max())
    # a step that clips is clipping and a step
    opts[0].step()
    opts[1].step(max_norm=1.5)
    for n, _ in _named():
        assert torch.equal(opts[0].param(n), opts[1].param(n))
    # fp32 gradients into the slots: their own norm, rounded once
    own, _ = ref.grad_norm(_host([grads[n] for n in grads]))
    _near(opts[2].clip(1.5, grads).item(), own)
    for n, _ in _named():
        want = grads[n].double() * (1.5 / own)
        tol = (NORM_TOL + 2 * 2.0 ** -24 + 2.0 ** -8) * want.abs() + LEAST["bf16"]
        assert bool(((opts[2].grad(n).double() - want).abs() <= tol * 1.0001).all())
    with pytest.raises(ValueError):
        opts[2].clip(1.5, {n: grads[n] for n in list(grads)[1:]})
    with pytest.raises(ValueError):
        opts[2].clip(1.5, {**grads, "norm.weight": grads["lm_head.weight"]})
    assert nsm.device_status() == nsm.NSM_OK
