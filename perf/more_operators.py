"""What is measured of the log probabilities of given tokens and of the distillation from a
teacher's top logits.

Two operators over rows of logits, each with its backward pass. The first gives, for every row, the
log probability of a token, its place among the row's tokens, the row's entropy and log-sum-exp, and
the top alternatives with their log probabilities. The second takes such top alternatives as a
teacher's and gives the divergence of a student's rows from them, and its gradient. A draft model is
trained that way from what the target's verification computed.

A case is a dict:
  op      "logprobs": the first operator
          "logprobs_grad": log probabilities and entropy, and the logits' gradient from both
          "loss_grad": the second operator through autograd, loss and gradient
          "distill": its loss and gradient in one call, rows weighted
  B, R    sequences and rows of each; the logits are [B, R, V]
  V       vocabulary
  ragged  whether the sequences have from 1 to R rows in use; the others have no token (-1) or no
          teacher (-1 throughout)
  dtype   "bf16", "fp16" or "f32": logits and their gradient
  k       top alternatives (0: none), or entries of the teacher
  tokens  whether tokens are given (logprobs)
  temperature
  tail    what the second operator makes of the teacher's probability that is not listed:
          "renormalise" (the listed ones are scaled to sum 1) or "bucket" (the unlisted tokens are one
          outcome); "" otherwise
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}


def _case(name, op, B, R, V, ragged, dtype, k, temperature=1.0, tail="", tokens=True):
    c = dict(op=op, B=B, R=R, V=V, ragged=ragged, dtype=dtype, k=k, tokens=tokens,
             temperature=temperature, tail=tail)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # One user, one token, five alternatives shown: the call's latency.
        _case("logprobs 1 row, top 5", "logprobs", 1, 1, 128256, False, "bf16", 5),
        # A small verification batch in 32 bits; -1 behind what it emitted.
        _case("logprobs 8 x 5, f32, top 20", "logprobs", 8, 5, 32000, True, "f32", 20),
        # The headline verification batch: what it emitted, with alternatives, for its users.
        _case("logprobs 256 x 9, top 20", "logprobs", 256, 9, 128256, True, "bf16", 20, 0.7),
        # The target's rows become a teacher's: 128 tokens of each, and no token asked for.
        _case("teacher 32 x 17, top 128", "logprobs", 32, 17, 152064, False, "bf16", 128,
              tokens=False),
        # A prompt's tokens scored; rows of an odd vocabulary start anywhere.
        _case("score 2000 x 32003, fp16", "logprobs", 1, 2000, 32003, False, "fp16", 0),
        # Fine-tuning on given tokens with a bonus for entropy.
        _case("logprobs grad 2048", "logprobs_grad", 8, 256, 128256, True, "bf16", 0),
        # The same in 32 bits, with a small batch.
        _case("logprobs grad 300, f32", "logprobs_grad", 3, 100, 32000, False, "f32", 0, 0.8),
        # Distillation inside a model's own training loop: loss forward, gradient backward.
        _case("loss and backward 2048, k 64", "loss_grad", 8, 256, 128256, False, "bf16", 64,
              tail="renormalise"),
        # A draft head's training step on a big batch, loss and gradient at once.
        _case("distill 4096, k 32, bucket", "distill", 16, 256, 128256, False, "bf16", 32,
              tail="bucket"),
        # The positions of a long-draft batch in 32 bits, many teacher entries, softened.
        _case("distill 32 x 16, f32, k 128", "distill", 32, 16, 152064, True, "f32", 128, 2.0,
              tail="renormalise"),
        # An odd vocabulary and ragged sequences.
        _case("distill 7 x 100, fp16, k 20", "distill", 7, 100, 32003, True, "fp16", 20,
              tail="bucket"),
        # Online: after a small verification round the draft learns from it.
        _case("distill 8 x 4, k 10", "distill", 8, 4, 32000, True, "bf16", 10,
              tail="renormalise"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["logprobs", "logprobs", "logprobs_grad", "loss_grad", "distill", "distill"])
        V = rng.choice([32000, 128256, 152064, 32003, _log_int(rng, 200, 160000),
                        _log_int(rng, 200, 160000)])
        c = _case(None, op, _log_int(rng, 1, 256), _log_int(rng, 1, 2000), V, rng.random() < 0.6,
                  rng.choice(["bf16", "bf16", "fp16", "f32"]), 0,
                  rng.choice([1.0, 1.0, 0.7, round(rng.uniform(0.5, 2.0), 2)]))
        if op == "logprobs":
            c["k"] = rng.choice([0, 1, rng.randint(2, 20), _log_int(rng, 20, 128)])
            c["tokens"] = rng.random() < 0.8
        elif op != "logprobs_grad":
            c["k"] = _log_int(rng, 1, 128)
            c["tail"] = rng.choice(["renormalise", "bucket"])
        n = c["B"] * c["R"] * V
        # (the plain form of the top alternatives needs the most room and time for an element)
        if n <= (3e8 if c["k"] and op == "logprobs" else 5.2e8) and work(c)["bytes"] <= 2.0e9:
            return c


def _lengths(c):
    """Rows in use of every sequence, the same for every seed but for their order."""
    if not c["ragged"]:
        return [c["R"]] * c["B"]
    return [1 + round((c["R"] - 1) * ((b * 7 % c["B"]) / (c["B"] - 1) if c["B"] > 1 else 0.6))
            for b in range(c["B"])]


def work(case):
    c = case
    N, rows, V, k = c["B"] * c["R"], sum(_lengths(c)), c["V"], c["k"]
    es = 4 if c["dtype"] == "f32" else 2
    given = c["op"] != "logprobs" or c["tokens"]
    total = (rows if given else N) * V * es
    if c["op"] == "logprobs":
        # token in; log probability, rank, entropy and log-sum-exp out, and the alternatives
        total += N * ((12 if c["tokens"] else 0) + 8 + 8 * k)
        return {"bytes": total, "flops": 4.0 * (rows if given else N) * V}
    total += N * V * es  # the gradient, zeros too
    # token, two gradients in, log probability and entropy out; or the teacher and the weight in, the
    # loss out
    total += N * (20 if c["op"] == "logprobs_grad" else 8 + 8 * k)
    return {"bytes": total, "flops": 8.0 * rows * V}


def _slices(c, elements):
    """Ranges of rows of at most so many elements."""
    step = max(1, int(elements // c["V"]))
    return [slice(i, min(i + step, c["B"] * c["R"])) for i in range(0, c["B"] * c["R"], step)]


def _top(x, k):
    """Ids of the k largest of each row, in order, ties by the lowest index: the sort key is the
    number's bits, in an order that whole numbers have too, with the index below them."""
    bits = (x.float() + 0.0).view(torch.int32)  # (+ 0.0: there is one zero)
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    low = torch.arange(x.shape[-1] - 1, -1, -1, device=x.device)
    key = torch.topk(bits * (1 << 32) + low, k, sorted=True).values
    return x.shape[-1] - 1 - (key & 0xFFFFFFFF)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    B, R, V, T = c["B"], c["R"], c["V"], c["temperature"]
    N = B * R
    lens = torch.tensor(_lengths(c))[torch.randperm(B, generator=h)]
    used = (torch.arange(R) < lens[:, None]).view(N).cuda()
    logits = torch.empty((N, V), dtype=DTYPES[c["dtype"]], device="cuda")
    teacher = c["op"] in ("loss_grad", "distill")
    s = {"case": c}
    # The mean over the rows; with a loss scale that keeps float16's gradients in range.
    mean = 64.0 if c["dtype"] == "fp16" else 1.0 / N
    if teacher:
        ids = torch.full((N, c["k"]), -1, dtype=torch.int32, device="cuda")
        lp = torch.full((N, c["k"]), -math.inf, device="cuda")
    else:
        tokens = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    for r in _slices(c, 1 << 26):
        # A model's logits: normal, and a few tokens that the context calls for.
        x = torch.randn((r.stop - r.start, V), generator=g, device="cuda").mul_(2.5)
        at = torch.randint(0, V, (x.shape[0], 8), generator=g, device="cuda")
        x.scatter_add_(1, at, torch.rand(at.shape, generator=g, device="cuda").mul_(10.0))
        if not teacher:
            logits[r] = x
            # Tokens as a sampler draws them.
            noise = torch.rand(x.shape, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
            x.div_(T).sub_(noise.log_().neg_().log_())
            tokens[r] = torch.where(used[r], x.argmax(-1).to(torch.int32), tokens[r])
        else:
            top = _top(x, c["k"])
            p = torch.log_softmax(x / T, -1).gather(1, top)
            ids[r] = torch.where(used[r, None], top.to(torch.int32), ids[r])
            lp[r] = torch.where(used[r, None], p, lp[r])
            # A student that knows something of it.
            logits[r] = x.mul_(0.8).add_(torch.randn(x.shape, generator=g, device="cuda"))
    s["logits"] = logits.view(B, R, V)
    if teacher:
        s["teacher_tokens"], s["teacher_logprobs"] = ids.view(B, R, -1), lp.view(B, R, -1)
        s["weights"] = torch.rand((B, R), generator=g, device="cuda").add_(0.5).mul_(mean)
    else:
        s["tokens"] = tokens.view(B, R) if c["tokens"] else None
    if c["op"] == "logprobs_grad":
        # An advantage for each token, and a bonus for entropy.
        s["upstream"] = (torch.randn((B, R), generator=g, device="cuda").mul_(mean),
                         torch.full((B, R), 0.01 * mean, device="cuda"))
    if c["op"] in ("logprobs_grad", "loss_grad"):
        s["logits"].requires_grad_()
    return s


def _plain_logprobs(s):
    c = s["case"]
    raw = s["logits"].detach().float()
    x = raw / c["temperature"]
    top = x.amax(-1, keepdim=True)
    x = x - top
    e = x.exp()
    total = e.sum(-1, keepdim=True)
    logs = total.log()
    # (0 log 0 = 0, for logits of -inf)
    entropy = logs - (e * x.clamp(min=-3e38)).sum(-1, keepdim=True) / total
    out = {"entropy": entropy.squeeze(-1), "lse": (top + logs).squeeze(-1)}
    if c["tokens"]:
        none = s["tokens"] < 0
        t = s["tokens"].long().clamp(min=0).unsqueeze(-1)
        out["logprobs"] = (x.gather(-1, t) - logs).squeeze(-1)
    if c["op"] == "logprobs_grad":
        a, b = (u.unsqueeze(-1) for u in s["upstream"])
        # d log p_t = [v = t] - p_v;  d H = -p_v (log p_v + H)
        p = e.div_(total)
        grad = x.sub_(logs).clamp_(min=-3e38).add_(entropy).mul_(b).add_(a).mul_(p).neg_()
        grad.scatter_add_(-1, t, a).div_(c["temperature"])
        return {"logprobs": out["logprobs"].masked_fill(none, 0.0),
                "entropy": out["entropy"].masked_fill(none, 0.0),
                "grad": grad.masked_fill_(none.unsqueeze(-1), 0.0).to(s["logits"].dtype)}
    del e
    if c["tokens"]:
        own_logit = raw.gather(-1, t)
        i = torch.arange(c["V"], device=raw.device)
        ahead = (raw > own_logit) | ((raw == own_logit) & (i < t))
        out = {key: v.masked_fill(none, 0.0) for key, v in out.items()}
        out["rank"] = ahead.sum(-1, dtype=torch.int32).masked_fill(none, -1)
    if c["k"]:
        ids = _top(raw, c["k"])
        lp = x.gather(-1, ids) - logs
        out["top_tokens"], out["top_logprobs"] = ids.to(torch.int32), lp
        if c["tokens"]:
            out["top_tokens"] = out["top_tokens"].masked_fill(none.unsqueeze(-1), -1)
            out["top_logprobs"] = lp.masked_fill(none.unsqueeze(-1), -math.inf)
    return out


def _plain_distill(s):
    c = s["case"]
    T = c["temperature"]
    ids, lp = s["teacher_tokens"].long(), s["teacher_logprobs"]
    there = ids >= 0
    none = ~there.any(-1, keepdim=True)
    ids = ids.clamp(min=0)
    raw = s["logits"].detach().float()
    highest = raw.amax(-1, keepdim=True)
    # (64 bits for the few numbers of a row whose differences the loss is made of, and for sums)
    far = (raw.gather(-1, ids).double() - highest) / T
    x = (raw - highest).div_(T)
    del raw
    p = lp.double().exp().masked_fill(~there, 0.0)
    mass = p.sum(-1, keepdim=True)
    log_p = lp.double()
    rest = (1.0 - mass).clamp(min=0.0)
    if c["tail"] == "renormalise":
        p, log_p, rest = p / mass, log_p - mass.log(), torch.zeros_like(mass)
    e = x.exp()
    total = e.sum(-1, keepdim=True, dtype=torch.float64)
    log_q = far - total.log()
    loss = torch.where(p > 0, p * (log_p - log_q), 0.0).sum(-1, keepdim=True)
    grad = e * ((p.sum(-1, keepdim=True) + rest) / total).float()
    if c["tail"] == "bucket":
        # The unlisted tokens as one outcome.
        listed = torch.zeros(x.shape, dtype=torch.bool, device=x.device).scatter_(-1, ids, there)
        e = e.masked_fill_(listed, 0.0)
        others = e.sum(-1, keepdim=True, dtype=torch.float64)
        log_q = (others / total).log()
        loss = loss + torch.where(rest > 0, rest * (rest.log() - log_q), 0.0)
        grad.sub_(e.mul_((rest / others).float()))
    grad.scatter_add_(-1, ids, -p.float())
    grad.mul_((s["weights"] / T).unsqueeze(-1))
    return {"loss": loss.masked_fill(none, 0.0).squeeze(-1).float(),
            "grad": grad.masked_fill_(none, 0.0).to(s["logits"].dtype)}


def run(state):
    s = state
    c = s["case"]
    if not own:
        return (_plain_logprobs if c["op"].startswith("logprobs") else _plain_distill)(s)
    import speculative_decoding_verification_66_gb300 as sv
    if c["op"].startswith("logprobs"):
        r = sv.sv_token_logprobs(s["logits"], s["tokens"], temperature=c["temperature"],
                                 top_k=c["k"])
        if c["op"] == "logprobs_grad":
            grad, = torch.autograd.grad((r.logprobs, r.entropy), s["logits"], s["upstream"])
            return {"logprobs": r.logprobs.detach(), "entropy": r.entropy.detach(), "grad": grad}
        out = {"entropy": r.entropy, "lse": r.lse}
        if c["tokens"]:
            out.update(logprobs=r.logprobs, rank=r.rank)
        if c["k"]:
            out.update(top_tokens=r.top_tokens, top_logprobs=r.top_logprobs)
        return out
    teacher = (s["teacher_tokens"], s["teacher_logprobs"])
    if c["op"] == "loss_grad":
        loss = sv.sv_distill_loss(s["logits"], *teacher, temperature=c["temperature"],
                                  tail=c["tail"])
        grad, = torch.autograd.grad(loss, s["logits"], s["weights"])
        return {"loss": loss.detach(), "grad": grad}
    loss, grad = sv.sv_distill(s["logits"], *teacher, weights=s["weights"],
                               temperature=c["temperature"], tail=c["tail"])
    return {"loss": loss, "grad": grad}


def _exact_logprobs(c, s, r, x, out):
    tokens = s["tokens"].view(-1)[r] if c["tokens"] else None
    y = x.detach().requires_grad_(c["op"] == "logprobs_grad")
    z = y / c["temperature"]
    lse = torch.logsumexp(z, -1)
    logs = z - lse[:, None]
    entropy = -(logs.exp() * logs).sum(-1)
    got = {"entropy": entropy, "lse": lse}
    if c["tokens"]:
        t = tokens.long().clamp(min=0)[:, None]
        got["logprobs"] = logs.gather(1, t).squeeze(1)
        keep = (tokens >= 0).double()
        got = {key: v * keep for key, v in got.items()}
    if c["op"] == "logprobs_grad":
        a, b = (u.view(-1)[r].double() for u in s["upstream"])
        got["grad"], = torch.autograd.grad((got["logprobs"] * a + got["entropy"] * b).sum(), y)
        got.pop("lse")
    else:
        if c["tokens"]:
            mine = x.gather(1, t)
            rank = (x > mine).sum(-1)
            same = (x == mine).cumsum(-1).gather(1, t).squeeze(1) - 1
            got["rank"] = torch.where(tokens >= 0, rank + same, -1).to(torch.int32)
        if c["k"]:
            order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :c["k"]]
            lp = logs.gather(1, order)
            if c["tokens"]:
                order = order.masked_fill((tokens < 0)[:, None], -1)
                lp = lp.masked_fill((tokens < 0)[:, None], -math.inf)
            got["top_tokens"], got["top_logprobs"] = order.to(torch.int32), lp
    for key, v in got.items():
        out.setdefault(key, []).append(v.detach())


def _exact_distill(c, s, r, x, out):
    """Dense teacher distributions, and autograd in 64 bits."""
    ids, lp = s["teacher_tokens"].flatten(0, 1)[r], s["teacher_logprobs"].flatten(0, 1)[r]
    w = s["weights"].view(-1)[r].double()
    p = torch.zeros_like(x)
    listed = torch.zeros_like(x)
    row, col = (ids >= 0).nonzero(as_tuple=True)
    p.index_put_((row, ids[row, col].long()), lp[row, col].double().exp(), accumulate=True)
    listed[row, ids[row, col].long()] = 1.0
    active = listed.sum(-1) > 0
    mass = p.sum(-1)
    if c["tail"] == "renormalise":
        p /= torch.where(active, mass, 1.0)[:, None]
    y = x.detach().requires_grad_()
    logs = torch.log_softmax(y / c["temperature"], -1)
    loss = torch.special.xlogy(p, p).sum(-1) - (p * logs).sum(-1)
    if c["tail"] == "bucket":
        left = (1.0 - mass).clamp(min=0.0)
        q = torch.logsumexp(logs.masked_fill(listed > 0, -math.inf), -1)
        loss = loss + torch.special.xlogy(left, left) - torch.where(left > 0, left * q, 0.0)
    loss = torch.where(active, loss, 0.0)
    grad, = torch.autograd.grad((loss * w).sum(), y)
    out.setdefault("loss", []).append(loss.detach())
    out.setdefault("grad", []).append(torch.where(active[:, None], grad, 0.0))


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    rows = s["logits"].detach().view(-1, c["V"])
    out = {}
    for r in _slices(c, 1 << 25):
        (_exact_logprobs if c["op"].startswith("logprobs") else _exact_distill)(
            c, s, r, rows[r].double(), out)
    return {key: torch.cat(v).unflatten(0, (c["B"], c["R"])) for key, v in out.items()}
