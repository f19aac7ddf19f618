"""The operators together: rounds of speculative decoding with a paged cache, checked against a
plain forward over the tokens that they emitted."""
import pytest
import torch

import speculative_decoding_verification_66_gb300 as sv
from speculative_decoding_verification_66_gb300.verify_round import Model, generate

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load()
    sv.load_attention()
    torch.cuda.set_device(0)


def plain_logits(m, tokens):
    """Logits of every position of tokens [L], in 64 bits, by whole matrices."""
    w = [[x.double() for x in ws] for ws in (m.qkv, m.out, m.up, m.down)]

    def norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    x = m.embedding[tokens.long()].double()
    L, H, Hk, d = len(tokens), m.heads, m.kv_heads, m.d
    hidden = torch.ones(L, L, dtype=torch.bool, device=x.device).triu(1)
    for qkv, out, up, down in zip(*w):
        f = (norm(x) @ qkv.T).view(L, H + 2 * Hk, d)
        q, k, v = f[:, :H], f[:, H:H + Hk], f[:, H + Hk:]
        k, v = k.repeat_interleave(H // Hk, 1), v.repeat_interleave(H // Hk, 1)
        s = torch.einsum("qhd,khd->hqk", q, k) * d ** -0.5
        p = torch.softmax(s.masked_fill(hidden, -torch.inf), -1)
        x = x + torch.einsum("hqk,khd->qhd", p, v).reshape(L, -1) @ out.T
        x = x + torch.nn.functional.silu(norm(x) @ up.T) @ down.T
    return norm(x) @ m.head.double().T


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("same", [True, False])
def test_greedy_rounds_emit_the_targets_choices(e4m3, same):
    """Every emitted token is the target's best, up to what its 16- or 8-bit path may mix up;
    with the target as its own draft nearly everything is kept, with another draft nearly nothing."""
    B, L, K, V, rounds = 3, 37, 4, 512, 6
    make = lambda seed: Model(2, 256, 4, 2, V, B, 200, e4m3=e4m3, seed=seed)  # noqa: E731
    target, draft = make(1), make(1 if same else 2)
    prompt = torch.randint(0, V, (B, L), dtype=torch.int32, device="cuda",
                           generator=torch.Generator(device="cuda").manual_seed(3))
    out, kept, cached = generate(target, draft, prompt, rounds, K)
    mean = float(kept.float().mean())
    assert (kept >= 0).all() and (mean > 0.8 * K if same else mean < 1.0)
    assert torch.equal(cached, L - 1 + (kept + 1).sum(0).to(torch.int32))
    # Relative roundings of the hidden state, of root mean square 2^-8 / sqrt(3) at most in bfloat16
    # (about ten a layer) and 2^-4 / sqrt(3) in e4m3 (a layer's keys and values), independent of one
    # another; logits have standard deviation one, so the difference of two moves by sqrt(2) times
    # their sum in quadrature. Five standard deviations for some 10^5 comparisons.
    tol = 5 * 2 ** 0.5 * (20 * 4.0 ** -8 / 3 + (4 * 4.0 ** -4 / 3 if e4m3 else 0.0)) ** 0.5
    for b in range(B):
        new = [t for r in range(rounds) for t in out[r, b].tolist() if t >= 0]
        assert len(new) == int((kept[:, b] + 1).sum())
        whole = torch.cat([prompt[b], torch.tensor(new, dtype=torch.int32, device="cuda")])
        logits = plain_logits(target, whole[:-1])[L - 1:]
        best = logits.amax(-1)
        got = logits.gather(1, whole[L:].long()[:, None]).squeeze(1)
        assert (best - got <= tol).all(), float((best - got).max())


def test_sampled_rounds_run_and_keep_counts():
    B, L, K, V = 5, 20, 3, 300
    target = Model(2, 128, 2, 1, V, B, 100, seed=1)
    draft = Model(1, 128, 2, 1, V, B, 100, seed=2)
    prompt = torch.randint(0, V, (B, L), dtype=torch.int32, device="cuda")
    out, kept, cached = generate(target, draft, prompt, 4, K, mode="sample", temperature=1.3)
    assert ((kept >= 0) & (kept <= K)).all()
    assert torch.equal((out >= 0).sum(-1), kept + 1) and (out < V).all()
