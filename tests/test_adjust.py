"""Penalties, biases and masks on logits, without a GPU: the float64 oracle against central
differences and by hand, and every refusal of the C ABI and of the binding (all of them are
returned before a CUDA call)."""

import os

import numpy as np
import pytest

from oracle import adjust_ref as ref


def test_oracle_by_hand():
    x = np.array([[2.0, -2.0, 0.0, 1.0, 5.0]])
    history = np.array([[1, 0, 0, 7, -1, 4]])
    got, _ = ref.adjust(x, history, np.array([5]), None, [2.0], [0.5], [0.25], np.array([[3, 3, 9, 0]]),
                        np.array([[1.0, 2.0, 4.0, 8.0]]), np.array([[0b01111]]))
    assert got.tolist() == [[1.0 - 1.25 + 8.0, -4.0 - 0.75, 0.0, 4.0, -np.inf]]


@pytest.mark.parametrize("theta", [0.5, 1.0, 1.7])
def test_oracle_gradient_against_differences(theta):
    rng = np.random.default_rng(int(theta * 10))
    x = rng.normal(size=(3, 41)) * 2
    history = rng.integers(-2, 45, size=(2, 30))
    row = np.array([1, 0, -1])
    mask = rng.integers(-2 ** 31, 2 ** 31, size=(3, 2)).astype(np.int32)
    d_out = rng.normal(size=x.shape)
    kw = dict(history=history, length=np.array([30, 4, 30]), history_row=row, mask=mask)
    g = ref.adjust_backward(x, d_out, repetition=[theta] * 3, **kw)

    def value(z):
        o, _ = ref.adjust(z, repetition=[theta] * 3, frequency=[0.3] * 3, presence=[0.1] * 3, **kw)
        return np.sum(np.where(np.isinf(o), 0.0, o) * d_out)

    step = 1e-4  # piecewise linear: exact away from the kink at 0
    for r, v in zip(*np.nonzero(np.abs(x) > 1e-3)):
        up, down = x.copy(), x.copy()
        up[r, v] += step
        down[r, v] -= step
        assert abs((value(up) - value(down)) / (2 * step) - g[r, v]) < 1e-8


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_orthogonalized_gb300 as m
    if not os.path.exists(m.LIB_PATH):
        from newton_schulz_orthogonalized_gb300 import _build
        _build.build()
    m.lib()
    return m


X, O, H, M, B, F = 0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000, 0x60000000


def _adjust(nsm, x=X, dtype=0, rows=4, vocab=100, ld=100, history=H, wide=1, hrows=4, hlen=10, ldh=10, length=F, hrow=0,
            rep=F + 0x100, freq=F + 0x200, pres=F + 0x300, bi=B, bw=1, ldbi=3, bias=B + 0x1000, ldb=3, k=3, mask=M, mrows=4,
            ldm=4, mrow=0, out=O, out_dtype=0, ldo=100):
    return nsm.lib().nsm_adjust_logits(x, dtype, rows, vocab, ld, history, wide, hrows, hlen, ldh, length, hrow, rep, freq, pres,
                                       bi, bw, ldbi, bias, ldb, k, mask, mrows, ldm, mrow, out, out_dtype, ldo, None)


def test_refusals(nsm):
    E = nsm
    for bad in (dict(x=0), dict(out=0), dict(bi=0), dict(bias=0), dict(history=0), dict(history=0, length=0, rep=0, freq=0),
                dict(history=0, hrow=F, rep=0, freq=0, pres=0), dict(mask=0, mrow=F)):
        assert _adjust(nsm, **bad) == E.NSM_ERR_NULL, bad
    for bad in (dict(dtype=3), dict(dtype=-1), dict(out_dtype=1), dict(dtype=2, out_dtype=0), dict(k=-1), dict(k=1025)):
        assert _adjust(nsm, **bad) == E.NSM_ERR_ARG, bad
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(vocab=0), dict(vocab=(1 << 20) + 1), dict(vocab=1 << 33), dict(ld=99),
                dict(ldo=99), dict(ld=1 << 61), dict(hrows=0), dict(hrows=3), dict(hlen=-1), dict(ldh=9), dict(mrows=0),
                dict(mrows=5), dict(ldm=3), dict(ldbi=2), dict(ldb=2)):
        assert _adjust(nsm, **bad) == E.NSM_ERR_SHAPE, bad
    for bad in (dict(x=X + 1), dict(out=O + 1), dict(out=O + 2, out_dtype=2), dict(history=H + 4), dict(bi=B + 4),
                dict(bias=B + 0x1002), dict(mask=M + 2), dict(length=F + 2), dict(rep=F + 1), dict(mrow=F + 3)):
        assert _adjust(nsm, **bad) == E.NSM_ERR_ALIGN, bad
    # what is written overlaps nothing, but the logits when they are the same rows
    for bad in (dict(out=X + 2), dict(out=X, ldo=101), dict(out=X, out_dtype=2), dict(out=H), dict(out=M), dict(out=B),
                dict(out=F), dict(out=F + 0x100)):
        assert _adjust(nsm, **bad) == E.NSM_ERR_ARG, bad
    assert _adjust(nsm, rows=0, x=0, out=0) == E.NSM_OK
    assert nsm.last_launch_count() == 0


def _backward(nsm, x=X, dtype=0, rows=4, vocab=100, ld=100, history=H, length=F, rep=F + 0x100, mask=M, d_out=B, d_dtype=0,
              ldg=100, d_logits=O, ldd=100):
    return nsm.lib().nsm_adjust_logits_backward(x, dtype, rows, vocab, ld, history, 1, 4, 10, 10, length, 0, rep, mask, 4, 4, 0,
                                                d_out, d_dtype, ldg, d_logits, ldd, None)


def test_backward_refusals(nsm):
    E = nsm
    for bad in (dict(x=0), dict(d_out=0), dict(d_logits=0), dict(history=0, length=0)):
        assert _backward(nsm, **bad) == E.NSM_ERR_NULL, bad
    for bad in (dict(dtype=4), dict(d_dtype=1), dict(dtype=2, d_dtype=0), dict(d_logits=B + 2), dict(d_logits=B, d_dtype=2),
                dict(d_logits=X)):
        assert _backward(nsm, **bad) == E.NSM_ERR_ARG, bad
    for bad in (dict(ld=99), dict(ldg=99), dict(ldd=99), dict(vocab=0)):
        assert _backward(nsm, **bad) == E.NSM_ERR_SHAPE, bad
    assert _backward(nsm, d_logits=O + 1) == E.NSM_ERR_ALIGN
    assert _backward(nsm, rows=0) == E.NSM_OK


class OnDevice:
    """What the binding asks of a tensor, for one on the GPU (no GPU is touched)."""

    def __init__(self, shape, dtype, device=0, stride=None):
        import torch
        t = torch.zeros(shape, dtype=dtype)
        self._t = t if stride is None else t.as_strided(shape, stride)
        self._device = device
        self.shape, self.dtype, self.device = self._t.shape, dtype, f"cuda:{device}"
        for n in ("stride", "data_ptr", "is_contiguous", "numel", "element_size"):
            setattr(self, n, getattr(self._t, n))

    def get_device(self):
        return self._device

    def __len__(self):
        return self.shape[0]


class Library:
    """Records calls in place of libnsmuon."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 1024 if name.endswith("_bytes") else 0
        return call


@pytest.fixture
def stub(nsm, monkeypatch):
    library = Library()
    nsm._torch_types()
    monkeypatch.setattr(nsm, "_torch_types", lambda: None)
    monkeypatch.setattr(nsm, "lib", lambda: library)
    monkeypatch.setattr(nsm, "_loss_stream", lambda stream, d: 0)
    monkeypatch.setattr(nsm, "_written", lambda *tensors: None)
    monkeypatch.setattr(nsm, "_current_device", lambda: 0)
    return library


def test_binding_refusals(nsm, stub):
    import torch
    bf, f32, i64, i32 = torch.bfloat16, torch.float32, torch.int64, torch.int32
    D = OnDevice

    def call(x=D((4, 100), bf), out=D((4, 100), bf), **kw):
        nsm.adjust_logits(x, out, **kw)

    def back(x=D((4, 100), bf), d_out=D((4, 100), bf), d_x=D((4, 100), bf), **kw):
        nsm.adjust_logits_backward(x, d_out, d_x, **kw)

    call()
    call(out=D((4, 100), f32), history=D((2, 9), i32), history_row=D((4,), i32), length=D((4,), i32), repetition=D((4,), f32),
         bias_index=D((4, 2), i64), bias=D((4, 2), f32), mask=D((4, 4), i32))
    back(d_out=D((4, 100), f32), history=D((4, 9), i64), repetition=D((4,), f32), mask=D((1, 4), i32), mask_row=D((4,), i32))
    back(x=None)
    ran = len(stub.calls)
    for bad in (dict(x=D((4, 100), bf, 1)), dict(x=D((4, 100), bf, -1)), dict(x=D((400,), bf)), dict(x=D((4, 100), torch.int8)),
                dict(out=D((4, 99), bf)), dict(out=D((4, 100), torch.float16)), dict(out=D((4, 100), bf, 1)),
                dict(out=D((4, 100), bf, 0, (1, 4))), dict(history=D((9,), i64)), dict(history=D((4, 9), f32)),
                dict(history=D((4, 9), i64, 1)), dict(history=D((4, 9), i64), length=D((4,), i64)),
                dict(history=D((4, 9), i64), length=D((3,), i32)), dict(history=D((4, 9), i64), history_row=D((4,), i64)),
                dict(history=D((4, 9), i64), repetition=D((4,), bf)), dict(history=D((4, 9), i64), presence=D((1,), f32)),
                dict(bias=D((4, 2), f32)), dict(bias_index=D((4, 2), i64)),
                dict(bias_index=D((4, 2), i64), bias=D((4, 3), f32)), dict(bias_index=D((4, 2), i64), bias=D((4, 2), bf)),
                dict(bias_index=D((4, 2), f32), bias=D((4, 2), f32)), dict(mask=D((4, 3), i32)), dict(mask=D((4, 4), i64)),
                dict(mask=D((4,), i32)), dict(mask=D((1, 4), i32), mask_row=D((4,), i64))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(x=None, history=D((4, 9), i64), repetition=D((4,), f32)), dict(d_x=D((4, 100), f32)),
                dict(d_out=D((4, 100), torch.float16)), dict(d_out=D((3, 100), bf)), dict(x=D((4, 100), bf, 1))):
        with pytest.raises(ValueError):
            back(**bad)
    assert len(stub.calls) == ran
