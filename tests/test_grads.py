"""The norm of many gradients and clipping, without a GPU: the float64 oracle, and every refusal
of the C ABI and of the binding (all of them are returned before a CUDA call)."""

import ctypes
import os

import numpy as np
import pytest

from oracle import grads_ref as ref
from test_adjust import OnDevice, stub  # noqa: F401


def test_oracle():
    grads = [np.array([3.0, 4.0]), np.zeros((0,)), np.array([[12.0]])]
    norm, each = ref.grad_norm(grads)
    assert norm == 13.0 and each.tolist() == [5.0, 0.0, 12.0]
    out, _, _ = ref.clip_grads(grads, 6.5)
    assert out[0].tolist() == [1.5, 2.0] and out[2].tolist() == [[6.0]]
    assert ref.clip_grads(grads, 13.0)[0][0].tolist() == [3.0, 4.0]
    assert abs(ref.grad_norm([np.full(4, 1e200)])[0] / 2e200 - 1) < 1e-15
    assert ref.grad_norm([np.array([1.0, np.inf])])[0] == np.inf and np.isnan(ref.grad_norm([np.array([np.nan, np.inf])])[0])


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_orthogonalized_gb300 as m
    if not os.path.exists(m.LIB_PATH):
        from newton_schulz_orthogonalized_gb300 import _build
        _build.build()
    m.lib()
    return m


A, B, C, N, S = 0x100000000, 0x200000000, 0x300000000, 0x400000000, 0x500000000


def _args(places, numels, dtypes):
    return (ctypes.c_void_p * len(places))(*places), (ctypes.c_int64 * len(numels))(*numels), (ctypes.c_int32 * len(dtypes))(*dtypes)


def _clip(nsm, grads=(A, B, 0), numels=(100, 200, 0), dtypes=(0, 2, 1), n=3, out=None, out_dtypes=(0, 0, 0), max_norm=1.0, norm=N,
          norms=N + 0x100, ws=S, ws_bytes=4096, norm_only=False):
    g, k, t = _args(grads, numels, dtypes)
    if norm_only:
        return nsm.lib().nsm_grad_norm(g, k, t, n, norm, norms, ws, ws_bytes, None)
    o, _, ot = _args(out or grads, numels, out_dtypes)
    return nsm.lib().nsm_clip_grads(g, k, t, n, o if out else None, ot if out else None, max_norm, norm, norms, ws, ws_bytes, None)


@pytest.mark.parametrize("norm_only", [False, True])
def test_refusals(nsm, norm_only):
    E = nsm

    def call(**kw):
        return _clip(nsm, norm_only=norm_only, **kw)

    assert call(grads=(0, B, 0)) == E.NSM_ERR_NULL
    for bad in (dict(n=0), dict(n=-1), dict(n=(1 << 20) + 1), dict(numels=(100, -1, 0)), dict(numels=(100, 1 << 45, 0)),
                dict(numels=(1 << 44, 1 << 44, 1 << 44))):
        assert call(**bad) == E.NSM_ERR_SHAPE, bad
    for bad in (dict(dtypes=(0, 3, 1)), dict(dtypes=(0, -1, 1)), dict(norm=A), dict(norm=B + 796), dict(norms=A), dict(ws=A),
                dict(norms=N - 4), dict(norm=S)):
        assert call(**bad) == E.NSM_ERR_ARG, bad
    for bad in (dict(grads=(A + 1, B, 0)), dict(grads=(A, B + 2, 0)), dict(norm=N + 2), dict(norms=N + 1), dict(ws=S + 16)):
        assert call(**bad) == E.NSM_ERR_ALIGN, bad
    for bad in (dict(ws=0), dict(ws_bytes=8)):
        assert call(**bad) == E.NSM_ERR_WORKSPACE, bad
    L = nsm.lib()
    g, k, t = _args((A,), (5,), (0,))
    if norm_only:
        assert L.nsm_grad_norm(g, k, t, 1, None, None, S, 4096, None) == E.NSM_ERR_NULL
        assert L.nsm_grad_norm(None, k, t, 1, N, None, S, 4096, None) == E.NSM_ERR_NULL
        assert L.nsm_grad_norm(g, None, t, 1, N, None, S, 4096, None) == E.NSM_ERR_NULL
        assert L.nsm_grad_norm(g, k, None, 1, N, None, S, 4096, None) == E.NSM_ERR_NULL
    else:
        assert L.nsm_clip_grads(g, k, t, 1, g, None, 1.0, N, None, S, 4096, None) == E.NSM_ERR_NULL


def test_clip_refusals(nsm):
    E = nsm
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert _clip(nsm, max_norm=bad) == E.NSM_ERR_ARG
    for bad in (dict(grads=(A, A, 0), dtypes=(0, 0, 0)), dict(grads=(A, A + 100, 0)), dict(out=(B, C, 0)), dict(out=(C, C + 100, 0)),
                dict(out=(A + 2, C, 0)), dict(out=(C, B, 0)), dict(out=(C, N, 0)), dict(out=(C, S, 0)), dict(out_dtypes=(0, 7, 0), out=(C, C + 0x1000, 0))):
        assert _clip(nsm, **bad) == E.NSM_ERR_ARG, bad
    assert _clip(nsm, out=(C, 0, 0)) == E.NSM_ERR_NULL
    assert _clip(nsm, out=(C, C + 0x1001, 0)) == E.NSM_ERR_ALIGN


def test_timing_kinds(nsm):
    for kind in (nsm.KIND_ADJUST, nsm.KIND_EMBEDDING, nsm.KIND_GRADS):
        assert nsm.timing_read(kind) == (0.0, 0, 0.0) and kind in nsm.KIND_NAMES
    with pytest.raises(nsm.NsmError):
        nsm.timing_read(max(nsm.KIND_NAMES) + 1)


def test_workspace_bytes(nsm):
    k = (ctypes.c_int64 * 3)(0, 1, 1 << 30)
    b = nsm.lib().nsm_grad_workspace_bytes(k, 3)
    assert 0 < b <= ((1 << 30) // 16384 + 3) * 8 + 1024
    assert nsm.lib().nsm_grad_workspace_bytes(k, 0) == 0 and nsm.lib().nsm_grad_workspace_bytes(None, 3) == 0


def test_binding_refusals(nsm, stub):  # noqa: F811
    import torch
    f32, bf, u8 = torch.float32, torch.bfloat16, torch.uint8
    D = OnDevice
    g = [D((5, 20), f32), D((7,), bf)]
    ws = D((4096,), u8)
    table = nsm.GradTable(g, [D((100,), bf), D((7,), bf)])
    nsm.grad_norm(table, D((1,), f32), D((2,), f32), workspace=ws)
    nsm.clip_grads(g, 1.0, D((), f32), workspace=ws)
    ran = [c for c in stub.calls if not c.endswith("_bytes")]
    for bad in (dict(norm=D((2,), f32)), dict(norm=D((1,), bf)), dict(norm=D((1,), f32, 1)), dict(norm=D((1,), f32), norms=D((3,), f32)),
                dict(norm=D((1,), f32), workspace=D((4096,), u8, -1))):
        for call in (lambda **kw: nsm.grad_norm(g, **kw), lambda **kw: nsm.clip_grads(table, 1.0, **kw)):
            with pytest.raises(ValueError):
                call(**{"workspace": ws, **bad})
    for bad in ([], [D((5,), torch.int32)], [D((5,), f32), D((5,), f32, 1)], [D((5,), f32, -1)], [D((4, 4), f32, 0, (1, 4))]):
        with pytest.raises(ValueError):
            nsm.GradTable(bad)
    for bad in ([D((99,), bf), D((7,), bf)], [D((100,), bf)], [D((100,), bf), D((7,), torch.int8)], [D((100,), bf), D((7,), bf, 1)]):
        with pytest.raises(ValueError):
            nsm.GradTable(g, bad)
    other = nsm.GradTable([D((5,), f32, 1)])
    with pytest.raises(ValueError):
        nsm.grad_norm(other, D((1,), f32, 1), workspace=D((4096,), u8, 1))
    assert [c for c in stub.calls if not c.endswith("_bytes")] == ran
