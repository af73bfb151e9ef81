"""A checkpoint resumes to the same bits whatever the memory held that a new optimizer's workspace gets:
the step keeps an exponent per matrix there, which a new optimizer begins without and a checkpoint
carries."""

import pytest

pytestmark = pytest.mark.gpu

NAMED = [(f"layers.{i}.proj.weight", s) for i, s in enumerate([(128, 256), (300, 200), (256, 512)])]


def _steps(opt, first, count):
    import torch
    for k in range(first, first + count):
        g = torch.Generator(device="cuda").manual_seed(k)
        for n, _ in NAMED:
            # entries far below their matrix's largest, which a small exponent would store as subnormals
            t = torch.randn(opt.grad(n).shape, generator=g, device="cuda")
            t.mul_(2.0 ** torch.randint(-24, 1, t.shape, generator=g, device="cuda"))
            t[0, 0] = 24.0
            opt.grad(n).copy_(t)
        opt.step()


def _new(torch, nsm, monkeypatch, left):
    """An optimizer whose workspace's memory held `left`."""
    with monkeypatch.context() as m:
        empty = torch.empty
        m.setattr(torch, "empty", lambda *a, **kw: empty(*a, **kw).fill_(left))
        return nsm.MuonAdamW(NAMED)


@pytest.mark.parametrize("left", [0, 5, 255])
def test_resume_whatever_the_memory_held(monkeypatch, left):
    import torch

    import newton_schulz_orthogonalized_gb300 as nsm
    opt, same = _new(torch, nsm, monkeypatch, 0), _new(torch, nsm, monkeypatch, left)
    for o in (opt, same):
        for n, _ in NAMED:
            o.param(n).copy_(torch.full(o.param(n).shape, 0.1))
        _steps(o, 0, 2)
    assert torch.equal(opt.muon_params, same.muon_params)
    saved = {k: (v.cpu().clone() if torch.is_tensor(v) else v) for k, v in opt.state_dict().items()}
    _steps(opt, 2, 2)
    fresh = _new(torch, nsm, monkeypatch, left)
    fresh.load_state_dict(saved)
    _steps(fresh, 2, 2)
    for key in ("muon_params", "muon_momentum"):
        assert torch.equal(getattr(fresh, key), getattr(opt, key)), key
    # a checkpoint without the exponents: as from a new optimizer, the same whatever the memory held
    old = {k: v for k, v in saved.items() if k != "muon_exponents"}
    runs = []
    for value in (left, 0):
        o = _new(torch, nsm, monkeypatch, value)
        _steps(o, 7, 1)
        o.load_state_dict(old)
        _steps(o, 2, 1)
        runs.append(o)
    assert torch.equal(runs[0].muon_params, runs[1].muon_params)
