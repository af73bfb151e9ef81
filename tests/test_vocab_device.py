"""The binding's check that the logits are on the current device: the library launches there,
on the stream that the binding takes from the logits' device.  Tensors of another device are
stood in for (no GPU is touched)."""

import pytest
import torch


class OnDevice:
    """What the binding asks of a tensor, for one that is on GPU `device`."""
    is_cuda = True

    def __init__(self, shape, dtype, device):
        self._t, self._device = torch.zeros(shape, dtype=dtype), device
        self.shape, self.dtype, self.device = self._t.shape, dtype, f"cuda:{device}"
        self.dim, self.stride, self.data_ptr = self._t.dim, self._t.stride, self._t.data_ptr
        self.is_contiguous = self._t.is_contiguous

    def get_device(self):
        return self._device


class Library:
    """Records calls in place of libnsmuon."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


def _calls(nsm, device):
    x, g = OnDevice((3, 10), torch.float32, device), OnDevice((3, 10), torch.float32, device)
    t, f = OnDevice((3,), torch.int64, device), OnDevice((3,), torch.float32, device)
    z, i = OnDevice((3, 2), torch.float32, device), OnDevice((3, 2), torch.int32, device)
    return {"nsm_logprobs": lambda: nsm.logprobs(x, t, f), "nsm_logprobs_grad": lambda: nsm.logprobs_grad(x, t, f, None, g),
            "nsm_logprobs_backward": lambda: nsm.logprobs_backward(x, t, f, None, f, None, g),
            "nsm_distill": lambda: nsm.distill(x, z, i, f), "nsm_distill_grad": lambda: nsm.distill_grad(x, z, i, f, g),
            "nsm_distill_backward": lambda: nsm.distill_backward(x, z, i, f, None, f, g)}


NAMES = ["nsm_logprobs", "nsm_logprobs_grad", "nsm_logprobs_backward", "nsm_distill", "nsm_distill_grad", "nsm_distill_backward"]


@pytest.mark.parametrize("current,device", [(0, 1), (1, 0), (0, 0), (1, 1)])
@pytest.mark.parametrize("name", NAMES)
def test_logits_of_another_device_are_refused(monkeypatch, name, current, device):
    import newton_schulz_orthogonalized_gb300 as nsm
    library = Library()
    nsm._torch_types()
    monkeypatch.setattr(nsm, "_torch_types", lambda: None)
    monkeypatch.setattr(nsm, "lib", lambda: library)
    monkeypatch.setattr(nsm, "_loss_stream", lambda stream, d: 0)
    monkeypatch.setattr(nsm, "_written", lambda *tensors: None, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    monkeypatch.setattr(nsm, "_current_device", lambda: current, raising=False)
    call = _calls(nsm, device)[name]
    if device == current:
        call()
        assert library.calls == [name]
    else:
        with pytest.raises(ValueError, match="current"):
            call()
        assert library.calls == []
