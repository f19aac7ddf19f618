"""The binding of the log probabilities and of distillation without a GPU: a library that notes what it
is given, and host tensors that pass for the GPU's."""
import random
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


def test_gradients_that_share_elements_with_the_logits_are_refused_and_no_others():
    """Against the sets of elements, for strides and offsets of all kinds. (Gradients whose rows overlap
    one another, or that have other strides between the logits' rows, are refused as well.)"""
    rng = random.Random(1)
    room, taken = torch.zeros(1000), 0
    for _ in range(20000):
        outer, inner, V = rng.randint(1, 4), rng.randint(1, 4), rng.randint(1, 9)
        s, t, a, b = rng.randint(0, 60), rng.randint(0, 60), rng.randint(0, 120), rng.randint(0, 120)
        logits, grad = (room.as_strided((outer, inner, V), (s, t, 1), at) for at in (a, b))
        step = [i * s + j * t for i in range(outer) for j in range(inner)]
        if any(abs(p - q) < V for n, p in enumerate(step) for q in step[:n]):
            continue
        if outer > 1 and inner > 1 and s < (inner - 1) * t + V and t < (outer - 1) * s + V:
            continue
        shared = any(abs(a + p - b - q) < V for p in step for q in step)
        try:
            lp._check_grad(grad, logits)
            assert a == b or not shared, (outer, inner, V, s, t, a, b)
            taken += 1
        except ValueError:
            assert a != b and shared, (outer, inner, V, s, t, a, b)
    assert taken > 5000


def test_gradients_of_other_strides():
    room = torch.zeros(600)
    logits = room[:400].view(4, 100)[:, :40]
    lp._check_grad(room[400:560].view(4, 40), logits)
    with pytest.raises(ValueError):
        lp._check_grad(room[40:].as_strided((4, 40), (50, 1)), logits)
    # Where there is one row of a kind, its stride is nobody's.
    x = torch.zeros(1, 6, 50)
    lp._check_grad(x.as_strided((1, 6, 50), (7, 50, 1)), x)
    lp._check_grad(x[:, 2:3].as_strided((1, 1, 50), (1, 9, 1)), x[:, 2:3])
    with pytest.raises(ValueError):
        lp._check_grad(x[:, 1:5].as_strided((1, 4, 50), (7, 50, 1)), x[:, :4])


def test_all_that_a_call_writes_is_told_to_autograd(library):
    x, f32, i32 = torch.randn(4, 50), torch.float32, torch.int32

    def given(*names):
        shapes = dict(row_status=((4,), i32), row_stats=((4, lp.SV_ROW_STATS), f32), loss=((4,), f32),
                      grad=((4, 50), f32))
        return {n: torch.zeros(shapes[n][0], dtype=shapes[n][1]) for n in names}

    for leaf in (False, True):
        y = x.clone().requires_grad_(leaf)
        for call, names in ((lambda **kw: lp.sv_token_logprobs(y, **kw), ("row_status", "row_stats")),
                            (lambda **kw: lp.sv_distill_loss(y, IDS, LOGP, **kw), ("row_status",)),
                            (lambda **kw: lp.sv_distill(y, IDS, LOGP, **kw),
                             ("row_status", "row_stats", "loss", "grad")),
                            (lambda **kw: lp.sv_token_logprobs_backward(y, torch.zeros(4, 8), **kw), ("grad",)),
                            (lambda **kw: lp.sv_distill_backward(y, IDS, LOGP, torch.zeros(4, 8), LOGP[:, 0].contiguous(),
                                                                 **kw), ("grad",))):
            out = given(*names)
            call(**out)
            assert all(t._version == 1 for t in out.values()), names


@pytest.mark.parametrize("call", [lambda x, T: lp.sv_token_logprobs(x, temperature=T).lse,
                                  lambda x, T: lp.sv_distill_loss(x, IDS, LOGP, temperature=T)])
def test_the_backward_pass_has_the_forward_calls_temperature(library, call):
    T = torch.tensor(0.5)
    y = call(torch.randn(4, 50, requires_grad=True), T)
    T.fill_(2.0)
    y.sum().backward()
    assert [rows[7] for _, rows, _ in library.calls] == [0.5, 0.5]
