"""The embedding lookup and its gradient, without a GPU: the float64 oracle against central
differences, the workspace's size, and every refusal of the C ABI and of the binding (all of
them are returned before a CUDA call)."""

import os

import numpy as np
import pytest

from oracle import embedding_ref as ref
from test_adjust import OnDevice, stub  # noqa: F401


def test_oracle_gradient_against_differences():
    rng = np.random.default_rng(1)
    w, d = rng.normal(size=(6, 3)), rng.normal(size=(11, 3))
    tokens = [0, 5, 5, -1, 6, 2, 0, 5, 3, -100, 0]
    g, size, count = ref.embedding_backward(d, tokens, 6, 0.7)
    assert count.tolist() == [3, 0, 1, 1, 0, 3] and np.all(size >= np.abs(g) - 1e-15)
    for v in range(6):
        for c in range(3):
            up, down = w.copy(), w.copy()
            up[v, c] += 1
            down[v, c] -= 1
            slope = np.sum((ref.embedding(up, tokens, 0.7) - ref.embedding(down, tokens, 0.7)) * d) / 2
            assert abs(slope - g[v, c]) < 1e-12


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_orthogonalized_gb300 as m
    if not os.path.exists(m.LIB_PATH):
        from newton_schulz_orthogonalized_gb300 import _build
        _build.build()
    m.lib()
    return m


W, T, O, S = 0x100000000, 0x200000000, 0x300000000, 0x400000000


def _lookup(nsm, w=W, dtype=0, vocab=50, cols=20, ldw=20, tokens=T, wide=1, rows=7, scale=1.0, out=O, out_dtype=2, ldo=20):
    return nsm.lib().nsm_embedding(w, dtype, vocab, cols, ldw, tokens, wide, rows, scale, out, out_dtype, ldo, None)


def _backward(nsm, d=O, dtype=2, rows=7, cols=20, ldg=20, tokens=T, wide=1, vocab=50, scale=1.0, accumulate=0, w=W, w_dtype=0,
              ldw=20, ws=S, ws_bytes=1 << 24):
    return nsm.lib().nsm_embedding_backward(d, dtype, rows, cols, ldg, tokens, wide, vocab, scale, accumulate, w, w_dtype, ldw, ws,
                                            ws_bytes, None)


def test_refusals(nsm):
    E = nsm
    for call in (_lookup, _backward):
        for bad in (dict(w=0), dict(tokens=0), dict(out=0) if call is _lookup else dict(d=0)):
            assert call(nsm, **bad) == E.NSM_ERR_NULL, bad
        for bad in (dict(rows=-1), dict(rows=1 << 31), dict(vocab=0), dict(vocab=(1 << 30) + 1), dict(cols=0),
                    dict(cols=(1 << 20) + 1), dict(ldw=19), dict(ldw=1 << 58)):
            assert call(nsm, **{**bad, **({"ws_bytes": 1 << 62} if call is _backward else {})}) == E.NSM_ERR_SHAPE, bad
        for bad in (dict(dtype=3), dict(dtype=-1), dict(scale=float("nan")), dict(scale=float("inf"))):
            assert call(nsm, **bad) == E.NSM_ERR_ARG, bad
        for bad in (dict(w=W + 1), dict(tokens=T + 4)):
            assert call(nsm, **bad) == E.NSM_ERR_ALIGN, bad
    assert _lookup(nsm, ldo=19) == E.NSM_ERR_SHAPE and _backward(nsm, ldg=19) == E.NSM_ERR_SHAPE
    assert _lookup(nsm, out_dtype=5) == E.NSM_ERR_ARG and _backward(nsm, w_dtype=5) == E.NSM_ERR_ARG
    assert _lookup(nsm, out=O + 2) == E.NSM_ERR_ALIGN and _backward(nsm, d=O + 2) == E.NSM_ERR_ALIGN
    # overlaps: what is written against everything else
    for bad in (dict(out=W), dict(out=W + 1996), dict(out=T)):
        assert _lookup(nsm, **bad) == E.NSM_ERR_ARG, bad
    for bad in (dict(w=O), dict(w=T), dict(ws=W), dict(ws=O), dict(ws=T)):
        assert _backward(nsm, **bad) == E.NSM_ERR_ARG, bad
    assert _backward(nsm, ws=0) == E.NSM_ERR_WORKSPACE
    assert _backward(nsm, ws_bytes=100) == E.NSM_ERR_WORKSPACE
    assert _backward(nsm, ws=S + 16) == E.NSM_ERR_ALIGN
    assert _lookup(nsm, rows=0, tokens=0, out=0) == E.NSM_OK
    assert _backward(nsm, rows=0, tokens=0, d=0, accumulate=1) == E.NSM_OK
    assert nsm.last_launch_count() == 0


def test_workspace_bytes(nsm):
    small = nsm.embedding_workspace_bytes(1, 1, 1)
    assert 0 < small < 1 << 16
    last = 0
    for rows in (1, 100, 1000, 16384, 65536, 1 << 20):
        b = nsm.embedding_workspace_bytes(rows, 50257, 768)
        assert b >= last and b % 256 == 0
        # pairs twice, a number per token, two rows of fp32 sums (with room for any alignment) per piece of the
        # sorted entries: pieces of 32, or shorter ones, no more than twice the 2432 / 3 that are wanted
        assert b <= 16 * rows + 4 * 50257 + 2 * (rows // 32 + 2 * 2432 // 3 + 2) * 1024 * 4 + (1 << 20)
        last = b
    for bad in ((-1, 5, 5), (5, 0, 5), (5, 5, 0), (1 << 31, 5, 5), (5, 1 << 31, 5), (5, 5, 1 << 21)):
        with pytest.raises(nsm.NsmError):
            nsm.embedding_workspace_bytes(*bad)


def test_binding_refusals(nsm, stub):  # noqa: F811
    import torch
    f32, bf, i64, u8 = torch.float32, torch.bfloat16, torch.int64, torch.uint8
    D = OnDevice
    ws = D((4096,), u8)
    nsm.embedding(D((50, 20), f32), D((7,), i64), D((7, 20), bf))
    nsm.embedding_backward(D((7, 20), bf), D((7,), torch.int32), D((50, 20), f32), ws)
    ran = len(stub.calls)
    for w, t, o in ((D((50, 20), f32, 1), D((7,), i64), D((7, 20), bf)), (D((50, 20), f32, -1), D((7,), i64), D((7, 20), bf)),
                    (D((50,), f32), D((7,), i64), D((7, 20), bf)), (D((50, 20), torch.int8), D((7,), i64), D((7, 20), bf)),
                    (D((50, 20), f32), D((7,), f32), D((7, 20), bf)), (D((50, 20), f32), D((7, 1), i64), D((7, 20), bf)),
                    (D((50, 20), f32), D((7,), i64, 1), D((7, 20), bf)), (D((50, 20), f32), D((7,), i64), D((7, 21), bf)),
                    (D((50, 20), f32), D((7,), i64), D((6, 20), bf)), (D((50, 20), f32), D((7,), i64), D((7, 20), bf, 1)),
                    (D((50, 20), f32, 0, (1, 50)), D((7,), i64), D((7, 20), bf)),
                    (D((50, 20), f32), D((7,), i64), D((7, 20), bf, 0, (1, 7)))):
        with pytest.raises(ValueError):
            nsm.embedding(w, t, o)
        with pytest.raises(ValueError):
            nsm.embedding_backward(o, t, w, ws)
    for bad in (D((4096,), u8, 1), D((4096,), u8, -1), D((64, 32), u8, 0, (1, 64))):
        with pytest.raises(ValueError):
            nsm.embedding_backward(D((7, 20), bf), D((7,), i64), D((50, 20), f32), bad)
    assert len(stub.calls) == ran
