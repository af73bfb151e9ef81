"""MuonAdamW's state without a GPU: what a checkpoint holds, and calls on optimizers at the edge of
what they are made for."""

import io
import os

import pytest


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_orthogonalized_gb300 as m
    if not os.path.exists(m.LIB_PATH):
        from newton_schulz_orthogonalized_gb300 import _build
        _build.build()
    m.lib()
    return m


NAMED = [("layers.0.proj.weight", (128, 256)), ("layers.1.proj.weight", (300, 200)), ("norm.weight", (77,))]


def test_a_checkpoint_holds_its_tensors_and_no_more(nsm):
    """Saving a view writes all that its storage holds: none may be of the step's workspace."""
    import torch
    opt = nsm.MuonAdamW(NAMED, device="cpu")
    state = opt.state_dict()
    own = 0
    for key, t in state.items():
        if torch.is_tensor(t):
            assert t.untyped_storage().nbytes() == t.numel() * t.element_size(), key
            own += t.numel() * t.element_size()
    file = io.BytesIO()
    torch.save(state, file)
    assert own <= file.tell() < own + (1 << 16)  # and the names, sizes and headers
    assert state["muon_exponents"].tolist() == [nsm.EXPONENT_NONE] * 2
    opt._exponents().copy_(torch.tensor([3, -5]))
    other = nsm.MuonAdamW(NAMED, device="cpu")
    other.load_state_dict(opt.state_dict())
    assert other._exponents().tolist() == [3, -5]


def test_an_optimizer_without_parameters_clips_nothing(nsm):
    """An owner that got none: its norm is 0, and a step that clips is a step."""
    opt = nsm.MuonAdamW([], device="cpu")
    opt.step()
    opt.step(max_norm=1.0)
    assert opt.step_count == 2
    for grads in (None, {}):
        norm = opt.clip(2.0, grads)
        assert norm.tolist() == [0.0] and opt.grad_norms.numel() == 0
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(nsm.NsmError):
            opt.clip(bad)
    with pytest.raises(ValueError):
        opt.clip(1.0, {"a": None})


def test_clip_finds_slots_that_have_moved(nsm, monkeypatch):
    """The slots' buffers are plain tensors, whose memory a program may change between two clips, as between
    two steps: the kept table is of where they are."""
    import torch
    opt = nsm.MuonAdamW(NAMED, device="cpu")
    clipped = []
    monkeypatch.setattr(nsm, "GradTable", lambda grads, out=None: [t.data_ptr() for t in (out or grads)])
    monkeypatch.setattr(nsm, "clip_grads", lambda table, *args, **kw: clipped.append(table))
    grads = {n: torch.zeros(s) for n, s in NAMED}
    for move in (lambda: None, lambda: setattr(opt.muon_grads, "data", opt.muon_grads.clone()),
                 lambda: opt.adam_grads.set_(opt.adam_grads.clone()), lambda: setattr(opt, "muon_grads", opt.muon_grads.clone())):
        move()
        for given in (None, grads):
            opt.clip(1.0, given)
            assert clipped[-1] == [opt.grad(n).data_ptr() for n in opt.muon_names + opt.adam_names]
    opt.clip(1.0)
    assert clipped[-1] is clipped[-3]  # made once while they stay
