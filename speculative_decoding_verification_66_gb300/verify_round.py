"""A whole round of speculative decoding on one GPU, from tokens to tokens.

A target and a draft transformer of random weights generate for a batch of
sequences. Every round the draft model proposes K tokens one at a time; the
target model runs once over the K + 1 new positions of every sequence: each of
its layers writes their keys and values into the paged cache (``sv_kv_append``)
and lets their queries attend to it (``sv_chunk_attention``); and the hidden
states go to ``spec_verify_lmhead``. What is rejected is taken back by passing
the shorter cached length to the next round: nothing is copied or cleared, and
no length ever comes to the host.

With ``--logprobs`` every emitted token comes with its log probability
(``sv_token_logprobs``); with ``--learn`` the draft model's head learns, after every
round, from what the target thought of the positions that it verified: the
target's top alternatives are the teacher of ``sv_distill``.

    python -m speculative_decoding_verification_66_gb300.verify_round --rounds 8 --learn 0.5
"""
from __future__ import annotations

import argparse
import time

import torch

from .api import spec_verify_lmhead, sv_lmhead_logits
from .attention import sv_chunk_attention, sv_kv_append, sv_kv_read
from .logprobs import sv_distill, sv_token_logprobs


class Model:
    """Pre-norm transformer layers without positions, of random weights, over a paged cache."""

    def __init__(self, layers, width, heads, kv_heads, vocab, batch, max_len, page=16,
                 e4m3=False, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            w = torch.empty(shape, device=device).normal_(generator=g) * shape[-1] ** -0.5
            return w.bfloat16()

        self.heads, self.kv_heads, self.d = heads, kv_heads, width // heads
        self.embedding = weight(vocab, width) * width ** 0.5
        self.qkv = [weight((heads + 2 * kv_heads) * self.d, width) for _ in range(layers)]
        self.out = [weight(width, width) for _ in range(layers)]
        self.up = [weight(2 * width, width) for _ in range(layers)]
        self.down = [weight(width, 2 * width) for _ in range(layers)]
        self.head = weight(vocab, width)
        pages = -(-max_len // page)
        # Sequence b's pages are spread over the pool.
        self.table = torch.arange(batch * pages, dtype=torch.int32, device=device) \
            .view(pages, batch).t().contiguous()
        shape = (layers, 2, batch * pages, page, kv_heads, self.d)
        self.pages = torch.empty(shape, device=device,
                                 dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16)
        self.exps = torch.empty(shape[:-1], dtype=torch.uint8, device=device) if e4m3 else None

    def cache(self, layer):
        exps = {} if self.exps is None else \
            dict(k_exps=self.exps[layer, 0], v_exps=self.exps[layer, 1])
        return (self.pages[layer, 0], self.pages[layer, 1], self.table), exps

    @staticmethod
    def norm(x):
        f = x.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def forward(self, tokens, cached, starts, chunk):
        """Final hidden states [N, width] of the packed new tokens; their keys and values are in
        the cache afterwards."""
        H, Hk, d = self.heads, self.kv_heads, self.d
        x = self.embedding[tokens.long()]
        for i in range(len(self.qkv)):
            cache, exps = self.cache(i)
            fused = torch.nn.functional.linear(self.norm(x), self.qkv[i]).view(-1, H + 2 * Hk, d)
            q, k, v = fused[:, :H], fused[:, H:H + Hk], fused[:, H + Hk:]
            sv_kv_append(k, v, *cache, cached, starts, **exps)
            y = sv_chunk_attention(q, *cache, cached, starts, **exps, max_chunk=chunk)
            x = x + torch.nn.functional.linear(y.view(x.shape), self.out[i])
            y = torch.nn.functional.linear(self.norm(x), self.up[i])
            x = x + torch.nn.functional.linear(torch.nn.functional.silu(y), self.down[i])
        return self.norm(x)


def ramp(batch, step, device):
    return torch.arange(0, batch * step + 1, step, dtype=torch.int32, device=device)


def learn_step(head, hidden, teacher_tokens, teacher_logprobs, rate, temperature=1.0, err=None):
    """One step of a draft model's head [V, width] towards a teacher's top alternatives
    [B, K, top] at the positions of its hidden states [B, K, width]; the unlisted tokens count as
    one outcome. The head is changed in place, by ``rate`` times the gradient of the mean divergence.
    Returns the divergences [B, K] before the step (0 where there is no teacher) and the gradient."""
    B, K, width = hidden.shape
    rows = hidden.reshape(B * K, width)
    logits = sv_lmhead_logits(rows, head, err=err).view(B, K, -1)
    taught = (teacher_tokens >= 0).any(-1)
    weights = taught / taught.sum().clamp(min=1)
    # (the logits are not needed again: their gradient takes their place)
    loss, grad = sv_distill(logits, teacher_tokens, teacher_logprobs, weights=weights,
                            temperature=temperature, tail="bucket", grad=logits)
    step = grad.view(B * K, -1).t().to(head.dtype) @ rows
    head.sub_(step, alpha=rate)
    return loss, step


def generate(target, draft, prompt, rounds, K, mode="greedy", temperature=1.0, seed=1, learn=0.0,
             top=32, details=None):
    """Rounds of K drafts for prompt [B, L] (L >= 2). Returns the emitted tokens [rounds, B, K + 1]
    (-1 where a round emitted fewer), the numbers of drafts kept [rounds, B] and the cached lengths.

    ``details``: a list that receives, for every round, a dict of the emitted tokens' ``logprobs``
    [B, K + 1] (0 behind the last one) and, where the draft's head learns (at rate ``learn``, from
    ``top`` alternatives of the target, up to the first position that was not kept), of its
    divergences ``loss`` [B, K]."""
    B, L = prompt.shape
    dev = prompt.device
    g = torch.Generator(device=dev).manual_seed(seed)
    zero = torch.zeros(B, dtype=torch.int32, device=dev)
    # The prompt but for its last token, which begins the first round.
    for model in (target, draft):
        model.forward(prompt[:, :-1].reshape(-1), zero, ramp(B, L - 1, dev), L - 1)
    cached = zero + (L - 1)
    last = prompt[:, -1].contiguous()
    one, chunk = ramp(B, 1, dev), ramp(B, K + 1, dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    emitted, kept = [], []
    for n in range(rounds):
        tokens, hidden = [last], []
        for i in range(K):
            h = draft.forward(tokens[-1], cached + i, one, 1)
            # (the verification's own LM head, so that both see the same distribution)
            logits = sv_lmhead_logits(h, draft.head, err=err)
            if mode == "greedy":
                x = logits.argmax(-1)
            else:
                x = torch.multinomial(torch.softmax(logits / temperature, -1), 1,
                                      generator=g).squeeze(1)
            hidden.append(h)
            tokens.append(x.to(torch.int32))
        # (the last draft's key and value, for the round that keeps all of them)
        draft.forward(tokens[-1], cached + K, one, 1)
        tokens = torch.stack(tokens, 1)  # [B, K + 1]
        h = target.forward(tokens.reshape(-1), cached, chunk, K + 1).view(B, K + 1, -1)
        out, accepted = spec_verify_lmhead(
            h, target.head, torch.stack(hidden, 1).contiguous(), draft.head,
            tokens[:, 1:].contiguous(), temperature, seed + n, mode)
        if learn or details is not None:
            # Rows behind the last emitted token (-1) are not read, and teach nothing.
            logits = sv_lmhead_logits(h.view(B * (K + 1), -1), target.head, err=err)
            r = sv_token_logprobs(logits.view(B, K + 1, -1), out, temperature=temperature,
                                  top_k=min(top, logits.shape[-1]) if learn else 0)
            report = {"logprobs": r.logprobs}
            if learn:
                report["loss"], _ = learn_step(
                    draft.head, torch.stack(hidden, 1), r.top_tokens[:, :K].contiguous(),
                    r.top_logprobs[:, :K].contiguous(), learn, temperature, err)
            if details is not None:
                details.append(report)
        emitted.append(out)
        kept.append(accepted)
        last = out.gather(1, accepted.long()[:, None]).squeeze(1)
        cached = cached + accepted + 1
    if int(err):
        raise RuntimeError("a wait of the LM head ran out")
    return torch.stack(emitted), torch.stack(kept), cached


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=500)
    ap.add_argument("--rounds", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--mode", choices=("greedy", "sample"), default="sample")
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="e4m3")
    ap.add_argument("--logprobs", action="store_true")
    ap.add_argument("--learn", type=float, default=0.0, metavar="RATE")
    a = ap.parse_args()
    V, max_len = 32000, a.prompt + a.rounds * (a.drafts + 1) + 1
    e4m3 = a.cache == "e4m3"
    target = Model(4, 1024, 8, 2, V, a.batch, max_len, page=64, e4m3=e4m3, seed=1)
    draft = Model(1, 512, 8, 2, V, a.batch, max_len, page=64, e4m3=e4m3, seed=2)
    prompt = torch.randint(0, V, (a.batch, a.prompt), dtype=torch.int32, device="cuda")
    generate(target, draft, prompt, 1, a.drafts, a.mode)  # warm-up
    torch.cuda.synchronize()
    details = [] if a.logprobs or a.learn else None
    t = time.perf_counter()
    out, kept, cached = generate(target, draft, prompt, a.rounds, a.drafts, a.mode, learn=a.learn,
                                 details=details)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    tokens = int((out >= 0).sum())
    starts = torch.zeros(a.batch + 1, dtype=torch.int32, device="cuda")
    starts[1:] = torch.cumsum(cached, 0)
    cache, exps = target.cache(0)
    k, _ = sv_kv_read(*cache, torch.zeros_like(cached), starts, int(starts[-1]), **exps)
    print(f"{a.batch} sequences, {a.rounds} rounds of {a.drafts} drafts: {tokens} tokens in "
          f"{t * 1e3:.1f} ms, {float(kept.float().mean()):.2f} drafts kept a round; the first "
          f"layer's keys read back: {tuple(k.shape)}")

    if details:
        lp = torch.stack([d["logprobs"] for d in details])
        print(f"mean log probability of an emitted token: {float(lp.sum()) / max(tokens, 1):.3f}")
    if a.learn:
        loss = [float(d["loss"].sum() / (d["loss"] != 0).sum().clamp(min=1)) for d in details]
        print(f"divergence of the draft from the target: {loss[0]:.4f} in the first round, "
              f"{loss[-1]:.4f} in the last")


if __name__ == "__main__":
    main()
