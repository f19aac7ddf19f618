"""Log probabilities and distillation inside autograd's other arrangements: activation checkpoints
and hooks for saved tensors, under which the backward pass is handed other logits than the forward
pass read, in another place."""
import pytest
import torch
from torch.autograd.graph import save_on_cpu, saved_tensors_hooks
from torch.utils.checkpoint import checkpoint

import speculative_decoding_verification_66_gb300 as sv
from test_gpu_distill import check, teacher
from test_gpu_logprobs import check_gradient, draw, draw_tokens

pytestmark = pytest.mark.gpu

ROWS, V = 12, 9001


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_logprobs()
    torch.cuda.set_device(0)


class LogProbs:
    def __init__(self, dtype):
        self.x, self.tokens = draw((ROWS, V), dtype, 3), draw_tokens((ROWS,), V)
        self.a, self.b = (torch.randn(ROWS, device="cuda") for _ in range(2))

    def loss(self, logits):
        r = sv.sv_token_logprobs(logits, self.tokens, temperature=0.8)
        return (self.a * r.logprobs + self.b * r.entropy).sum()

    def check(self, grad):
        check_gradient(grad, self.x, self.tokens, self.a, self.b, None, 0.8)


class Distillation:
    def __init__(self, dtype):
        x, self.ids, self.lp = teacher((ROWS,), V, 15, 3)
        self.x = x.to(draw((1, 1), dtype).dtype)
        self.w = torch.rand(ROWS, device="cuda")

    def loss(self, logits):
        return (self.w * sv.sv_distill_loss(logits, self.ids, self.lp, temperature=1.3,
                                            tail="bucket")).sum()

    def check(self, grad):
        check(self.x, self.ids, self.lp, 1.3, "bucket", None, grad, self.w)


def plain_gradient(op):
    x = op.x.detach().requires_grad_()
    return torch.autograd.grad(op.loss(x * 1.0), x)[0]


def junk(like):
    """Fills memory of logits that are gone."""
    return [torch.full_like(like, float("nan")) for _ in range(8)]


both = pytest.mark.parametrize("make", [LogProbs, Distillation])
types = pytest.mark.parametrize("dtype", ["bf16", "f32"])


@both
@types
@pytest.mark.parametrize("reentrant", [False, True])
def test_checkpoints(make, dtype, reentrant):
    op = make(dtype)
    want = plain_gradient(op)
    x = op.x.detach().requires_grad_()
    loss = checkpoint(lambda t: op.loss(t * 1.0), x, use_reentrant=reentrant)
    there = junk(op.x)
    grad, = torch.autograd.grad(loss, x) if not reentrant else (loss.backward(), x.grad)[1:]
    assert torch.equal(grad, want) and len(there) == 8
    op.check(grad)


def padded(t):
    room = torch.zeros(t.shape[0], t.shape[1] + 13, dtype=t.dtype, device=t.device)
    room[:, 3:t.shape[1] + 3] = t
    return room[:, 3:t.shape[1] + 3]


def transposed(t):
    return t.t().contiguous().t()


@both
@types
@pytest.mark.parametrize("copy", [torch.clone, padded, transposed])
def test_hooks_for_saved_tensors(make, dtype, copy):
    op = make(dtype)
    want = plain_gradient(op)
    x = op.x.detach().requires_grad_()
    with saved_tensors_hooks(lambda t: copy(t.detach()) if t.dim() == 2 else t, lambda t: t):
        logits = x * 1.0
        loss = op.loss(logits)
    logits.detach().fill_(float("nan"))
    del logits
    there = junk(op.x)
    grad, = torch.autograd.grad(loss, x)
    assert torch.equal(grad, want) and len(there) == 8
    op.check(grad)


@both
@types
def test_saved_on_the_host(make, dtype):
    op = make(dtype)
    want = plain_gradient(op)
    x = op.x.detach().requires_grad_()
    with save_on_cpu():
        loss = op.loss(x * 1.0)
    there = junk(op.x)
    grad, = torch.autograd.grad(loss, x)
    assert torch.equal(grad, want) and len(there) == 8
    op.check(grad)
