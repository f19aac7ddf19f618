"""Log probabilities and distillation where a call is just inside of what is allowed, or just outside."""
import math

import pytest
import torch

import logprobs_util as u
import speculative_decoding_verification_66_gb300 as sv
from test_gpu_distill import check as check_distillation
from test_gpu_distill import teacher
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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_largest_vocabulary_and_its_gradients(dtype):
    """2^31 - 1 tokens, nearly all of them masked, the gradient over the logits themselves."""
    V = 2 ** 31 - 1
    at = torch.tensor([0, 5, 1023, 1024, 2 ** 30 + 7, V - 9, V - 2, V - 1], device="cuda")
    some = draw((1, len(at)), dtype, 1)
    x = torch.empty(V, dtype=some.dtype, device="cuda")

    def others_are_zero(want):
        assert sum(int((part != 0).sum()) for part in x.split(1 << 28)) == int((want != 0).sum())

    for t in (3, 7):
        x.fill_(-math.inf)
        x[at] = some[0]
        token = at[t].to(torch.int32)
        stats = torch.empty(sv.SV_ROW_STATS, device="cuda")
        r = sv.sv_token_logprobs(x, token, row_stats=stats)
        w = u.logprobs(some, torch.tensor([t], device="cuda"))
        for name in ("logprobs", "entropy", "lse"):
            u.close(getattr(r, name), w[name][0], 1e-5, name)
        assert int(r.rank) == int(w["rank"])
        one = torch.ones((), device="cuda")
        grad = sv.sv_token_logprobs_backward(x, stats, tokens=token, grad_logprobs=one, grad=x)
        want = u.logprobs_grad(some, torch.tensor([t], device="cuda"), one[None], None, None)
        u.check_grad(grad[at], want[0], 1.0, len(at), 8.0)
        others_are_zero(want)
    x.fill_(-math.inf)
    x[at] = some[0]
    ids, lp = torch.tensor([5, 1, 2], device="cuda"), torch.tensor([-1.0, -2.0, -3.0], device="cuda")
    want, g, _ = u.distill(some, ids[None], lp[None])
    loss, grad = sv.sv_distill(x, at[ids].to(torch.int32), lp, grad=x)
    u.close(loss, want[0], 1e-5, "loss")
    u.check_grad(grad[at], g[0], 1.0, len(at), 8.0)
    others_are_zero(g)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "f32"])
def test_entropies_are_as_exact_wherever_the_largest_logit_is(dtype):
    """Rows of normal logits and one that has about half of the probability: in the first turn of its
    warp, whose sums are then relative to it throughout, or later, some 15 bits above what its lane has
    seen. What a lane adds after the largest logit is rounded relative to the sums at that time: no
    more than half a step of its logit's own share each, in both cases, and there are fewer of those
    additions in the second. So that one's root mean square error is at most the first one's, but for
    the sampling: 400 rows give either within 1 / sqrt(800), their ratio within 5 % (one standard
    deviation), 50 % are ten of those."""
    N, V = 400, 128256
    x = torch.randn((N, V), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    at = torch.randint(4200, 40000, (N, 1), generator=torch.Generator().manual_seed(5)).cuda()
    off = []
    for where in (torch.zeros_like(at), at):
        y = x.scatter(1, where, 12.5).to(u.DTYPES[dtype])
        r = sv.sv_token_logprobs(y)
        w = torch.cat([u.logprobs(rows)["entropy"] for rows in y.split(50)])
        off.append((r.entropy.double() - w).square().mean().sqrt().item())
    assert off[1] <= 1.5 * off[0], off


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [33, 2048, 70001])
def test_gradients_between_the_logits_rows(dtype, V):
    room = draw((5, 2, 3, V), dtype, V)
    x, out = room[:, 0], room[:, 1]
    tokens, a = draw_tokens((5, 3), V), torch.randn(5, 3, device="cuda")
    before = x.clone()
    grad = sv.sv_token_logprobs_backward(x, stats_of(x, tokens), tokens=tokens, grad_logprobs=a, grad=out)
    assert torch.equal(x, before)
    check_gradient(grad, x, tokens, a, None, None, 1.0)
    r = sv.sv_token_logprobs(0.9 * before, top_k=5)
    loss, grad = sv.sv_distill(x, r.top_tokens, r.top_logprobs, grad=out)
    check_distillation(before, r.top_tokens, r.top_logprobs, 1.0, "renormalise", loss, grad)
    assert torch.equal(x, before)


def test_a_gradient_in_place_by_another_view():
    x, tokens, a = draw((1, 6, 1000), "bf16"), draw_tokens((1, 6), 1000), torch.randn(1, 6, device="cuda")
    stats = stats_of(x, tokens)
    want = sv.sv_token_logprobs_backward(x, stats, tokens=tokens, grad_logprobs=a)
    view = x.as_strided((1, 6, 1000), (24, 1000, 1))
    assert torch.equal(sv.sv_token_logprobs_backward(x, stats, tokens=tokens, grad_logprobs=a, grad=view), want)


@pytest.mark.parametrize("V", [3001, 70001])
def test_probabilities_past_float32(V):
    """Logits of a hundred given for log probabilities: renormalised they are what they are; as they
    stand they have no sum."""
    x, ids, lp = teacher((6,), V, 5, 8, missing=0.0, none=0.0)
    lp[0, 2] = 100.0
    lp[1] = 88.0                             # each is in range, their sum is not
    lp[2, 0], lp[2, 1], ids[2, 1] = 88.5, 88.5, ids[2, 0].clone()
    lp[3] = torch.tensor([80.0, -3.0, -4.0, 60.0, 1.0])
    status = torch.empty(6, dtype=torch.int32, device="cuda")
    loss, grad = sv.sv_distill(x, ids, lp, tail="bucket", row_status=status)
    assert status.tolist() == [u.NONFINITE] * 3 + [0] * 3
    assert loss[:3].isnan().all() and grad[:3].isnan().all() and grad[3:].isfinite().all()
    want, g, _ = u.distill(x[3:], ids[3:], lp[3:], 1.0, "bucket")
    assert ((loss[3:] - want) / want).abs().max() < 1e-5   # (80 roundings of 2^-24 in a logarithm of 80)
    y = x.detach().requires_grad_()
    l2 = sv.sv_distill_loss(y, ids, lp, tail="bucket", row_status=status)
    l2.sum().backward()
    assert l2[:3].isnan().all() and y.grad[:3].isnan().all() and y.grad[3:].isfinite().all()
    assert status.tolist() == [u.NONFINITE] * 3 + [0] * 3
    loss, grad = sv.sv_distill(x, ids, lp, row_status=status)
    assert not status.any()
    check_distillation(x, ids, lp, 1.0, "renormalise", loss, grad)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [2.0 ** 117, 1e30, 1e-3, 1e-38])
def test_temperatures_at_their_ends(dtype, T):
    """Logits from end to end of the type, which differ by more than float32 holds; at the highest
    temperature they are some 2000 apart."""
    V = 5003
    big = float(torch.finfo(u.DTYPES[dtype]).max)
    x = draw((5, V), dtype, 7)
    x[0, ::3], x[0, 1] = -big, big
    x[1, ::2], x[1, 5] = -math.inf, 3.0
    x[2] = x[2] * (big / 32)
    x[3] = (x[3].float() * min(T, 1e36)).to(x.dtype)
    tokens = torch.tensor([1, 5, 77, 4000, V - 1], dtype=torch.int32, device="cuda")
    tokens[2], tokens[3] = x[2].argmax().int(), x[3].argmax().int()
    status = torch.full((5,), 77, dtype=torch.int32, device="cuda")
    y = x.detach().requires_grad_()
    r = sv.sv_token_logprobs(y, tokens, temperature=T, top_k=4, row_status=status)
    # (log-sum-exps past float32 are infinite)
    u.check_logprobs(x, tokens, T, 4, r, status)
    if T > 1e-30:
        a = torch.randn(5, device="cuda")
        g, = torch.autograd.grad(r.logprobs, y, a)
        # Beside what check_gradient allows, the token's own gradient a (1 - p) / T has three roundings of
        # 2^-24 in float32: the temperature's to float32, its inverse's, and the product's.
        want = u.logprobs_grad(x, tokens, a, None, None, T)
        w = u.logprobs(x, tokens, T)
        far = torch.where(w["p"] > 0, w["logp"].abs(), 0.0) + w["entropy"][:, None] + 1
        tol = (u.half_step(x.dtype) * (1 + 2 ** -6) + 3 * u.U) * want.abs() + 1e-38 \
            + 4 * u.sum_tol(V, 8.0) * w["p"] * a.double().abs()[:, None] * far / T
        u.close(g, want, tol, "grad")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "f32"])
@pytest.mark.parametrize("mask", ["-inf", "lowest"])
@pytest.mark.parametrize("V", [300, 70001])
def test_a_teacher_and_a_student_that_are_allowed_the_same_few_tokens(dtype, mask, V):
    """Where a mask leaves at most ten tokens, twenty entries have all of the teacher's probability, but
    for the rounding of their sum: nothing is left for the tokens that nobody may take."""
    N, dt = 300, u.DTYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(V)
    low = -math.inf if mask == "-inf" else -float(torch.finfo(dt).max)
    allowed = torch.randint(0, V, (N, 10), generator=g, device="cuda")
    there = torch.zeros(N, V, dtype=torch.bool, device="cuda").scatter_(1, allowed, True)
    target, x = (torch.randn((N, V), generator=g, device="cuda").mul_(2.5).to(dt).masked_fill_(~there, low)
                 for _ in range(2))
    r = sv.sv_token_logprobs(target, top_k=20)
    status = torch.empty(N, dtype=torch.int32, device="cuda")
    loss, grad = sv.sv_distill(x, r.top_tokens, r.top_logprobs, tail="bucket", row_status=status)
    assert not status.any()
    P = torch.zeros(N, V, dtype=torch.float64, device="cuda")
    P.scatter_add_(1, r.top_tokens.long(), r.top_logprobs.double().exp())
    logq = torch.log_softmax(x.double(), -1)
    want = (torch.special.xlogy(P, P) - torch.where(P > 0, P * logq, 0.0)).sum(-1)
    # (as in the other tests: the entries' probabilities by 2 roundings and their logarithms by one, log q
    # by its distance from the mean of some 20, and the sums)
    u.close(loss, want, u.sum_tol(V, 8.0) + 4 * u.U * (20 + 20 + want), "loss")
    q = logq.exp()
    # (the sum of P is 1 but for kRounding's 8 roundings, and stands before q)
    u.check_grad(grad, P.sum(-1, keepdim=True) * q - P, q * 20 + P, V, 8.0)
    y = x.detach().requires_grad_()
    l2 = sv.sv_distill_loss(y, r.top_tokens, r.top_logprobs, tail="bucket")
    l2.sum().backward()
    u.close(l2.detach(), want, u.sum_tol(V, 8.0) + 4 * u.U * (20 + 20 + want), "loss")
    u.check_grad(y.grad, P.sum(-1, keepdim=True) * q - P, q * 20 + P, V, 8.0)


@pytest.mark.parametrize("V", [300, 70001])
def test_what_a_teacher_leaves_to_masked_tokens_is_missed(V):
    """A rest above what roundings leave is the teacher's, and costs what it costs."""
    x = torch.full((2, V), -math.inf, device="cuda")
    x[:, :4] = 0.0
    x[1, 4:] = -500.0
    ids = torch.tensor([[0, 1, 2, 3]] * 2, dtype=torch.int32, device="cuda")
    for rest in (1e-3, 1e-5):
        lp = torch.full((2, 4), math.log((1 - rest) / 4), device="cuda")
        loss, grad = sv.sv_distill(x, ids, lp, tail="bucket")
        want, g, _ = u.distill(x, ids, lp, 1.0, "bucket")
        assert loss[0] == math.inf and grad.isfinite().all()
        # (four roundings of probabilities of 1/4, times the distance of 500)
        u.close(loss[1], want[1], 4 * u.U * 520 + u.sum_tol(V, 8.0), "loss")
