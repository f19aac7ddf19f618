"""The binding of the log probabilities and of distillation without a GPU: a library that notes what it
is given, and host tensors that pass for the GPU's."""
import struct

import pytest
import torch
from torch.autograd import forward_ad
from torch.autograd.graph import saved_tensors_hooks
from torch.utils.checkpoint import checkpoint

from speculative_decoding_verification_66_gb300 import logprobs as lp


class OnGpu(torch.Tensor):
    is_cuda = True


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(rows, *args):
            self.calls.append((name, struct.unpack("@P5qif", rows), args))
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(lp._lib, "load_logprobs", lambda: lib)
    describe = lp._describe
    monkeypatch.setattr(lp, "_describe", lambda x, T: describe(x.as_subclass(OnGpu), T))
    monkeypatch.setattr(lp, "_on", lambda dev, stream, call, tensors: call(0))
    monkeypatch.setattr(lp, "_workspace", lambda *a: (None, 0))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    return lib


IDS, LOGP = torch.zeros(4, 3, dtype=torch.int32), torch.zeros(4, 3)
LOSSES = [lambda x: lp.sv_token_logprobs(x, IDS[:, 0].contiguous(), temperature=0.5).lse,
          lambda x: lp.sv_distill_loss(x, IDS, LOGP, temperature=0.5)]


@pytest.mark.parametrize("loss", LOSSES)
def test_the_backward_pass_reads_recomputed_logits(library, loss):
    made = []

    def f(x):
        made.append(x * 2.0)
        return loss(made[-1])

    x = torch.randn(4, 50).requires_grad_()
    checkpoint(f, x, use_reentrant=False).sum().backward()
    # (all of them are alive, so that each has a place of its own)
    assert len(made) == 2 and library.calls[-1][0].endswith("_backward")
    assert library.calls[0][1][0] == made[0].data_ptr()
    assert library.calls[-1][1][0] == made[1].data_ptr() != made[0].data_ptr()
    assert library.calls[-1][1][1:] == library.calls[0][1][1:]


@pytest.mark.parametrize("loss", LOSSES)
def test_the_backward_pass_reads_what_a_hook_has_kept(library, loss):
    room = torch.randn(4, 70)

    def pack(t):
        if t.shape == (4, 50):
            room[:, 5:55] = t.detach()
            return room[:, 5:55]
        return t

    x = torch.randn(4, 50).requires_grad_()
    with saved_tensors_hooks(pack, lambda t: t):
        y = loss(x * 2.0)
    y.sum().backward()
    name, rows, _ = library.calls[-1]
    assert name.endswith("_backward") and rows[0] == room[:, 5:].data_ptr()
    assert rows[1:6] == (1, 4, 0, 70, 50) and rows[7] == 0.5


@pytest.mark.parametrize("loss", LOSSES)
@pytest.mark.parametrize("reverse_too", [False, True])
def test_forward_mode_is_refused(library, loss, reverse_too):
    x = torch.randn(4, 50, requires_grad=reverse_too)
    with forward_ad.dual_level():
        with pytest.raises(NotImplementedError):
            loss(forward_ad.make_dual(x, torch.ones(4, 50)))
        assert not library.calls
        loss(x)  # (no tangent of its own)
    assert library.calls
