"""Rounds that report log probabilities and teach the draft's head: verification, log probabilities
and distillation together, as they would be used."""
import pytest
import torch

import logprobs_util as u
import speculative_decoding_verification_66_gb300 as sv
from speculative_decoding_verification_66_gb300.verify_round import Model, generate, learn_step
from test_gpu_verify_round import plain_logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load()
    sv.load_attention()
    sv.load_logprobs()
    torch.cuda.set_device(0)


def models(V, B, seeds=(1, 2)):
    return (Model(2, 256, 4, 2, V, B, 200, seed=seeds[0]), Model(1, 128, 2, 1, V, B, 200, seed=seeds[1]))


def test_emitted_tokens_come_with_their_log_probabilities():
    """Against a plain forward over the emitted tokens in 64 bits. The logits of its 16-bit path have
    standard deviation one and are off by some 20 roundings of the hidden state in quadrature
    (2^-8 / sqrt(3) each); a log probability by twice that. Five standard deviations."""
    B, L, K, V = 3, 23, 3, 512
    target, draft = models(V, B)
    g = torch.Generator(device="cuda").manual_seed(3)
    prompt = torch.randint(0, V, (B, L), dtype=torch.int32, device="cuda", generator=g)
    details = []
    out, kept, _ = generate(target, draft, prompt, 5, K, mode="sample", details=details)
    assert len(details) == 5 and all("loss" not in d for d in details)
    lp = torch.stack([d["logprobs"] for d in details])
    assert torch.equal(lp != 0, out >= 0)
    for b in range(B):
        rows = out[:, b] >= 0
        new = out[:, b][rows]
        whole = torch.cat([prompt[b], new])
        logits = plain_logits(target, whole[:-1])[L - 1:]
        want = torch.log_softmax(logits, -1).gather(1, new.long()[:, None])[:, 0]
        u.close(lp[:, b][rows], want, 2 * 5 * (20 * 4.0 ** -8 / 3) ** 0.5, "log probability")


@pytest.mark.parametrize("mode", ["greedy", "sample"])
def test_rounds_that_learn(mode):
    """What was verified is taught, up to the first draft that was not kept, and nothing else; what is
    emitted is still the target's."""
    B, L, K, V = 5, 20, 4, 1000
    target, draft = models(V, B)
    head = draft.head.clone()
    prompt = torch.randint(0, V, (B, L), dtype=torch.int32, device="cuda")
    details = []
    out, kept, _ = generate(target, draft, prompt, 4, K, mode, learn=0.25, top=16, details=details)
    assert torch.equal((out >= 0).sum(-1), kept + 1)
    for d, n in zip(details, kept):
        taught = torch.arange(K, device="cuda") <= n[:, None]
        assert d["loss"].isfinite().all() and torch.equal(d["loss"] > 0, taught)
    assert not torch.equal(head, draft.head) and draft.head.isfinite().all()
    first, _, _ = generate(target, models(V, B)[1], prompt, 1, K, "greedy")
    again, _, _ = generate(target, draft, prompt, 1, K, "greedy")
    assert torch.equal(first[0, :, 0], again[0, :, 0])


def test_a_step_is_the_gradients():
    """The head's step against autograd in 64 bits, from the same hidden states and teacher: the
    logits' gradient is rounded to bfloat16 before the product over the positions (2^-8 of each
    term), the product to bfloat16 (2^-8 of it), and torch lets its partial sums be rounded to
    bfloat16 as well (allow_bf16_reduced_precision_reduction: 2^-8 of the terms once more)."""
    B, K, V, width = 4, 3, 700, 128
    g = torch.Generator(device="cuda").manual_seed(5)
    head = (torch.randn(V, width, generator=g, device="cuda") * width ** -0.5).bfloat16()
    hidden = torch.randn(B, K, width, generator=g, device="cuda").bfloat16()
    logits = torch.randn(B, K, V, generator=g, device="cuda") * 2
    tokens = torch.zeros(B, K, dtype=torch.int32, device="cuda")
    tokens[1, 2], tokens[2, 1:] = -1, -1
    r = sv.sv_token_logprobs(logits, tokens, temperature=1.2, top_k=9)
    before = head.clone()
    loss, step = learn_step(head, hidden, r.top_tokens, r.top_logprobs, 0.5, temperature=1.2)
    x = hidden.double().reshape(B * K, width) @ before.double().t()
    want, dx, _ = u.distill(x, r.top_tokens.view(B * K, -1), r.top_logprobs.view(B * K, -1), 1.2,
                            "bucket")
    u.close(loss.view(-1), want, 1e-5, "loss")  # (float32 logits of 128 products)
    dx = dx / (tokens >= 0).sum()
    rows = hidden.double().reshape(B * K, width)
    bound = 2 * 2.0 ** -8 * (dx.abs().t() @ rows.abs()) + 2.0 ** -8 * (dx.t() @ rows).abs() + 1e-7
    u.close(step, dx.t() @ rows, 1.02 * bound, "step")
    u.close(head, before.double() - 0.5 * step.double(),
            2.0 ** -8 * (before.double().abs() + step.double().abs()), "head")
