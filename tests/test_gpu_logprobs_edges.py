"""Log probabilities and distillation where a call is just inside of what is allowed, or just outside."""
import math

import pytest
import torch

import logprobs_util as u
import speculative_decoding_verification_66_gb300 as sv
from test_gpu_logprobs import check_gradient, draw, draw_tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_logprobs()
    torch.cuda.set_device(0)


def stats_of(x, tokens=None):
    stats = torch.empty(*x.shape[:-1], sv.SV_ROW_STATS, device="cuda")
    sv.sv_token_logprobs(x, tokens, row_stats=stats)
    return stats


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "f32"])
@pytest.mark.parametrize("V", [1000, 1024, 10007])
def test_backward_tokens_that_the_forward_call_did_not_have(dtype, V):
    """Tokens past the vocabulary, within the last turn and beyond it: NaN in their rows, and nothing
    behind them is written."""
    odd = [V, V + 1, V + 20, V + 500, V + 1023, V + 5000, 2 ** 31 - 1, -2, -2 ** 31, -1, V - 1, 0]
    tokens = torch.tensor(odd, dtype=torch.int32, device="cuda")
    x = draw((len(odd), V), dtype, V)
    a, b = (torch.randn(len(odd), device="cuda") for _ in range(2))
    room = torch.full((len(odd), V + 2048), 7.0, dtype=x.dtype, device="cuda")
    for stats in (stats_of(x), stats_of(x, draw_tokens((len(odd),), V, skip=0))):
        grad = sv.sv_token_logprobs_backward(x, stats, tokens=tokens, grad_logprobs=a, grad_entropy=b,
                                             grad=room[:, :V])
        check_gradient(grad, x, tokens, a, b, None, 1.0)
        assert grad[:9].isnan().all() and (grad[9] == 0).all() and grad[10:].isfinite().all()
        assert (room[:, V:] == 7.0).all()
    # Rows that the forward call was not asked of, or had a bad token of.
    first = torch.full((len(odd),), -1, dtype=torch.int32, device="cuda")
    first[10] = V
    grad = sv.sv_token_logprobs_backward(x, stats_of(x, first), tokens=tokens, grad_logprobs=a)
    assert grad[:9].isnan().all() and (grad[[9, 11]] == 0).all() and grad[10].isnan().all()


def test_tokens_of_inference_mode_changed_before_the_backward_pass():
    """(Nothing tells autograd of it.)"""
    V = 1000
    x = draw((3, V), "f32").requires_grad_()
    with torch.inference_mode():
        tokens = torch.zeros(3, dtype=torch.int32, device="cuda")
    r = sv.sv_token_logprobs(x, tokens)
    with torch.inference_mode():
        tokens.copy_(torch.tensor([V + 3, 5, -7], dtype=torch.int32))
    r.logprobs.sum().backward()
    assert x.grad[[0, 2]].isnan().all()
    check_gradient(x.grad[1:2], x[1:2], tokens[1:2], torch.ones(1, device="cuda"), None, None, 1.0)
