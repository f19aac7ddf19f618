"""Plain forms in 64 bits of the log probabilities and of distillation, and the roundings that the
kernels are allowed.

Tolerances. u = 2^-24 is half a step of float32. A sum of n positive float32 terms that is built
serially by threads of n / 128 terms (at most; the kernels' threads have fewer) and then as a tree is
off by a random walk of its roundings, six standard deviations of which are 6 sqrt(n / 128) u, and
each term 2^t by 2^-22 (the exponential) and |t| ln 2 times 3 u (the difference, its product and the
factor's own rounding). Weighted by the terms' shares, |t| ln 2 averages to the entropy less the log
of the sum at most, so a log-sum-exp is off by SUM(V, H) = u (8 + 6 sqrt(V / 128) + 3 (H + 1)).
Gradients and probabilities are products of such terms, and are rounded to the logits' type by half a
step (float16: also 2^-25 of its own below its normal range).
"""
import math

import torch

U = 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
BAD_TOKEN, NONFINITE = 1, 2


def sum_tol(V, H=0.0):
    """Relative error of a row's sum, and so the absolute one of its logarithm."""
    return U * (8 + 6 * math.sqrt(V / 128) + 3 * (H + 1))


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def logprobs(x, tokens=None, temperature=1.0, k=0):
    """Everything of rows x [N, V], in 64 bits, with the status bits that the kernels give."""
    N, V = x.shape
    raw = x.double()
    top = raw.amax(-1)
    z = (raw - top[:, None]) / temperature  # (relative to the largest, however far from 0 it is)
    status = torch.where(top.isfinite(), 0, NONFINITE)  # (NaN, +inf, or -inf throughout)
    skipped = torch.zeros(N, dtype=torch.bool, device=x.device)
    t = torch.zeros(N, dtype=torch.long, device=x.device)
    if tokens is not None:
        t = tokens.long()
        skipped = t == -1
        bad = ((t < -1) | (t >= V))
        status = torch.where(bad, status | BAD_TOKEN, status)
        t = t.clamp(0, V - 1)
    status = torch.where(skipped, 0, status)
    total = torch.logsumexp(z, -1)
    lse = top / temperature + total
    logp = z - total[:, None]
    p = logp.exp()
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(-1)
    mine = raw.gather(1, t[:, None])
    at = torch.arange(V, device=x.device)
    rank = ((raw > mine) | ((raw == mine) & (at < t[:, None]))).sum(-1)
    order = torch.sort(raw + 0.0, dim=-1, descending=True, stable=True).indices[:, :k]
    out = {"logprobs": logp.gather(1, t[:, None])[:, 0], "entropy": entropy, "lse": lse,
           "rank": rank, "top_tokens": order, "top_logprobs": logp.gather(1, order)}
    whole = {"rank", "top_tokens"}
    for name, v in out.items():
        s = skipped.view(-1, *[1] * (v.dim() - 1))
        b = (status != 0).view(s.shape)
        none = -1 if name in whole else -math.inf if name == "top_logprobs" else 0.0
        v = torch.where(s, none, torch.where(b, -1 if name in whole else math.nan, v))
        out[name] = v
    return out | {"status": status.int(), "skipped": skipped, "p": p, "logp": logp}


def logprobs_grad(x, tokens, a, b, c, temperature=1.0):
    """Gradient of a . logprobs + b . entropy + c . lse (None: zero), by the formula."""
    r = logprobs(x, tokens, temperature)
    N, V = x.shape
    p, logp = r["p"], r["logp"]
    g = torch.zeros_like(p)
    if a is not None:
        hot = torch.zeros_like(p)
        hot[torch.arange(N, device=x.device), tokens.long().clamp(0, V - 1)] = 1.0
        g += a.double()[:, None] * (hot - p)
    if b is not None:
        h = -torch.where(p > 0, p * logp, 0.0).sum(-1, keepdim=True)
        g -= b.double()[:, None] * torch.where(p > 0, p * (logp + h), 0.0)
    if c is not None:
        g += c.double()[:, None] * p
    g /= temperature
    g = torch.where(r["skipped"][:, None], 0.0, g)
    return torch.where((r["status"] != 0)[:, None], math.nan, g)


def distill(x, ids, logp, temperature=1.0, tail="renormalise"):
    """loss [N], dloss/dx [N, V], status; 64 bits, by dense rows of teachers."""
    N, V = x.shape
    dev = x.device
    raw = x.double()
    ids = ids.long()
    lp = logp.double()
    there = ids != -1
    none = ~there.any(-1)
    status = torch.where(raw.amax(-1).isfinite(), 0, NONFINITE)
    lp_bad = lp.isnan() | (lp == math.inf)
    status = torch.where(none & ~lp_bad.any(-1), 0, status)
    status = torch.where(lp_bad.any(-1), status | NONFINITE, status)
    out = (ids < -1) | (ids >= V)
    status = torch.where(out.any(-1), status | BAD_TOKEN, status)
    use = there & ~out & ~lp_bad
    row = torch.arange(N, device=dev)[:, None].expand_as(ids)
    shift = torch.zeros(N, 1, dtype=torch.float64, device=dev)
    if tail == "renormalise":
        shift = torch.where(use, lp, -math.inf).amax(-1, keepdim=True)
        shift = torch.where(shift.isfinite(), shift, 0.0)
    P = torch.zeros(N, V, dtype=torch.float64, device=dev)
    P.index_put_((row[use], ids[use]), (lp - shift).exp()[use], accumulate=True)
    listed = torch.zeros_like(P)
    listed[row[use], ids[use]] = 1.0
    mass = P.sum(-1, keepdim=True)
    rest = torch.zeros_like(mass)
    if tail == "renormalise":
        status = torch.where(~none & (mass[:, 0] == 0) & (status == 0), NONFINITE, status)
        P = P / torch.where(mass > 0, mass, 1.0)
    else:
        rest = (1.0 - mass).clamp(min=0.0)
        rest = torch.where(listed.sum(-1, keepdim=True) == V, 0.0, rest)
    z = (raw - raw.amax(-1, keepdim=True)) / temperature
    logq = z - torch.logsumexp(z, -1, keepdim=True)
    q = logq.exp()
    loss = (torch.special.xlogy(P, P) - torch.where(P > 0, P * logq, 0.0)).sum(-1)
    M = P.sum(-1, keepdim=True) + rest
    g = M * q - P
    if tail == "bucket":
        log_o = torch.logsumexp(logq.masked_fill(listed > 0, -math.inf), -1, keepdim=True)
        loss = loss + torch.where(rest > 0, rest * (rest.log() - log_o), 0.0)[:, 0]
        g = g - torch.where((listed > 0) | (q == 0), 0.0, rest * (logq - log_o).exp())
    g = g / temperature
    bad = status != 0
    loss = torch.where(bad, math.nan, torch.where(none, 0.0, loss))
    g = torch.where(bad[:, None], math.nan, torch.where(none[:, None], 0.0, g))
    return loss, g, status.int()


def close(got, want, tol, what=""):
    """got is within tol (a number or array) of want; NaN and infinities in the same places."""
    # (what rounds to a number too large for its type is infinite)
    dt = got.dtype
    got, want = got.double(), torch.where(want.to(dt).isinf(), want.to(dt).double(), want.double())
    same = (got == want) | (got.isnan() & want.isnan())
    off = torch.where(same, 0.0, (got - want).abs())
    bad = ~(off <= tol)
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        limit = tol if not torch.is_tensor(tol) else float(tol.expand_as(want)[at])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at {at}: "
                             f"{float(got[at])!r} for {float(want[at])!r} (allowed {limit:.3g})")


def check_logprobs(x, tokens, temperature, k, r, status=None):
    """A TokenLogprobs r of x (any shape) against the plain form."""
    V = x.shape[-1]
    flat = x.reshape(-1, V)
    w = logprobs(flat, None if tokens is None else tokens.reshape(-1), temperature, k)
    H = torch.where(w["entropy"].isfinite(), w["entropy"], 0.0)
    top = flat.double().amax(-1)
    s = U * (8 + 6 * math.sqrt(V / 128)) + 3 * U * (H + 1)

    def size(v):
        return torch.where(v.isfinite(), v.abs(), 0.0)

    # A log probability: its own rounding and, by the factor's, that of its distance from the mean
    # log probability, which is the entropy.
    names = {"entropy": s * (1 + H) + U * H, "lse": s + 3 * U * (size(w["lse"]) + size(top) / temperature),
             "logprobs": s + 3 * U * (size(w["logprobs"]) + H),
             "top_logprobs": s[:, None] + 3 * U * (size(w["top_logprobs"]) + H[:, None])}
    for name, tol in names.items():
        got = getattr(r, name)
        if (name == "logprobs" and tokens is None) or (name == "top_logprobs" and not k):
            assert got is None
            continue
        assert got.shape[:x.dim() - 1] == x.shape[:-1] and got.dtype == torch.float32
        close(got.detach().reshape(w[name].shape), w[name], tol, name)
    if tokens is not None:
        assert r.rank.dtype == torch.int32 and torch.equal(r.rank.reshape(-1).long(), w["rank"])
    if k:
        assert torch.equal(r.top_tokens.reshape(-1, k).long(), w["top_tokens"])
    if status is not None:
        assert torch.equal(status.reshape(-1), w["status"])
    return w


def check_grad(got, want, scale, V, H, what="grad"):
    """A gradient against the formula's: rounded once to its type, after terms off by the sums'
    tolerance (scale: what they were multiplied with, [N, V] or less)."""
    dt = got.dtype
    tol = half_step(dt) * (1 + 2 ** -6) * torch.where(want.isfinite(), want.abs(), 0.0) \
        + 4 * sum_tol(V, H) * scale + (2.0 ** -25 if dt == torch.float16 else 1e-38)
    close(got.reshape(want.shape), want, tol, what)
