"""What is measured of the paged key/value cache and the attention over it.

Three operators: writing a chunk of new keys and values into the pages of a
cache (as they are, or quantised to e4m3 with a power-of-two exponent per
token and head), reading a range of tokens back, and the attention of a chunk
of new queries (a draft to be verified, a single token, a piece of a prompt)
over the cached tokens and the chunk itself.

A case is a dict:
  op        "append", "read" or "attention"
  B         sequences
  chunk     the longest chunk of new tokens (append, attention) or of tokens
            read back (read); ragged cases have chunks from 1 to this
  context   the longest cached length; ragged cases go from a quarter to this
  ragged    whether the lengths differ
  hq, hkv   query heads (attention) and key/value heads
  d         head size
  dtype     "bf16" or "fp16": queries, new keys and values, outputs
  cache     "16" (the cache holds dtype) or "e4m3"
  page      tokens in a page
  heads_first  whether a page holds its heads outermost
  window    0, or how many keys back a query sees
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(name, op, B, chunk, context, ragged, hq, hkv, d, dtype="bf16", cache="16", page=16,
          heads_first=False, window=0):
    c = dict(op=op, B=B, chunk=chunk, context=context, ragged=ragged, hq=hq, hkv=hkv, d=d,
             dtype=dtype, cache=cache, page=page, heads_first=heads_first, window=window)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # One user, one token: the call's latency.
        _case("decode 1 sequence", "attention", 1, 1, 700, False, 32, 8, 128),
        # A small server verifying 4 draft tokens a sequence.
        _case("verify 64 x 5", "attention", 64, 5, 4000, True, 32, 8, 128),
        # The headline verification batch (256 sequences, 8 drafts) on a quantised cache.
        _case("verify 256 x 9, e4m3", "attention", 256, 9, 6000, True, 32, 8, 128, cache="e4m3",
              page=64),
        # Long documents, 16 drafts, eight query heads to a key head.
        _case("verify 32 x 17, long", "attention", 32, 17, 32768, True, 64, 8, 128, page=64),
        # Many short chats on a small model without shared heads.
        _case("decode 512, d 64, fp16", "attention", 512, 1, 2000, True, 16, 16, 64, dtype="fp16",
              page=32, heads_first=True),
        # Few very long contexts, a token at a time.
        _case("decode 4, 131k, e4m3", "attention", 4, 1, 131000, False, 32, 8, 128, cache="e4m3",
              page=128, heads_first=True),
        # A piece of a long prompt.
        _case("prompt piece 2048", "attention", 1, 2048, 6000, False, 32, 8, 128, page=64),
        # Pieces of several prompts of odd lengths, seven heads to a key head, windowed.
        _case("ragged pieces, window", "attention", 12, 700, 3000, True, 28, 4, 128, cache="e4m3",
              window=1024),
        # The headline batch's new keys and values into the quantised cache, and back.
        _case("append 256 x 9, e4m3", "append", 256, 9, 2000, True, 0, 8, 128, cache="e4m3",
              page=64),
        # Whole prompts into a 16-bit cache.
        _case("append 4 x 8000", "append", 4, 8000, 3000, False, 0, 8, 128, page=64),
        # Quantised sequences handed to something that wants them dense.
        _case("read 16 x 8000, e4m3", "read", 16, 8000, 9000, True, 0, 8, 128, cache="e4m3",
              page=64),
        # One short sequence read back.
        _case("read 1 x 700, fp16", "read", 1, 700, 1000, False, 0, 4, 64, dtype="fp16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["attention", "attention", "attention", "append", "read"])
        hkv = rng.choice([1, 2, 4, 5, 8, 8, 16])
        c = _case(None, op, _log_int(rng, 1, 512), 1, _log_int(rng, 1, 131000),
                  rng.random() < 0.7, 0, hkv, rng.choice([64, 128, 128, 80]),
                  rng.choice(["bf16", "bf16", "fp16"]), rng.choice(["16", "e4m3"]),
                  rng.choice([16, 32, 64, 128]), rng.random() < 0.4, 0)
        if op == "attention":
            c["hq"] = hkv * rng.choice([1, 3, 4, 4, 7, 8])
            kind = rng.choice(["single", "draft", "draft", "piece"])
            c["chunk"] = {"single": 1, "draft": rng.randint(2, 17)}.get(kind) or \
                _log_int(rng, 18, 2048)
            if rng.random() < 0.2:
                c["window"] = _log_int(rng, 64, 4096)
        else:
            c["chunk"] = _log_int(rng, 1, 8000)
            c["context"] = min(c["context"], 9000)
            if op == "read":
                c["context"] = max(c["context"], c["chunk"])
        w = work(c)
        longest = c["context"] + (c["chunk"] if op != "read" else 0)
        if w["bytes"] <= 2.5e9 and w["flops"] <= 2.5e11 \
                and c["B"] * longest * hkv * c["d"] <= 1.5e9 \
                and c["B"] * c["hq"] * c["chunk"] * longest <= 1.0e9 \
                and (op == "attention" or c["B"] * c["chunk"] * hkv * c["d"] <= 1.4e8):
            return c


def _lengths(c):
    """(cached, chunk) of every sequence, the same for every seed but for their order. For a read:
    (first token, tokens read)."""
    B, out = c["B"], []
    for b in range(B):
        f = b / (B - 1) if c["ragged"] and B > 1 else 1.0
        g = (b * 7 % B) / (B - 1) if c["ragged"] and B > 1 else 1.0
        chunk = 1 + round((c["chunk"] - 1) * g)
        cached = c["context"] - round(0.75 * c["context"] * (1 - f))
        out.append((max(0, cached - chunk), min(chunk, cached)) if c["op"] == "read"
                   else (cached, chunk))
    return out


def _keys(c, cached, t):
    """How many keys query t sees."""
    n = cached + t + 1
    return min(n, c["window"]) if c["window"] else n


def work(case):
    c = case
    es = 2 if c["cache"] == "16" else 1
    vec = 2 * c["hkv"] * (c["d"] * es + (0 if c["cache"] == "16" else 1))  # K and V of one token
    dense = 2 * c["hkv"] * c["d"] * 2
    total, flops = 0, 0.0
    for cached, chunk in _lengths(c):
        pages = -(-(cached + chunk) // c["page"]) * 4
        if c["op"] == "attention":
            first = max(0, cached - c["window"] + 1) if c["window"] else 0
            total += (cached + chunk - first) * vec + pages
            total += chunk * c["hq"] * (c["d"] * 4 + 4)  # query in, output and lse out
            keys = _keys(c, cached, 0) + _keys(c, cached, chunk - 1)
            flops += 4.0 * c["hq"] * c["d"] * chunk * keys / 2
        elif c["op"] == "append":
            total += chunk * (dense + vec)
            if c["cache"] != "16":
                total += chunk * (dense + vec)  # and read back
        else:
            total += chunk * (dense + vec)
    return {"bytes": total, "flops": flops}


def _quantise(x):
    """e4m3 codes (as uint8) and exponent bytes of the vectors along the last axis: the smallest
    power of two that brings the largest magnitude to 448 or below."""
    f = x.float()
    top = f.abs().amax(-1)
    mantissa, e = torch.frexp(top)  # top = mantissa 2^e, mantissa in [0.5, 1)
    e = torch.where(mantissa <= 0.875, e - 9, e - 8)
    e = torch.where(top > 0, e.clamp(min=-117), torch.full_like(e, -117))
    code = torch.ldexp(f, -e.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
    return code, (e + 127).to(torch.uint8)


def _powers(b):
    """2^(b - 127) of exponent bytes, in 32 bits."""
    return torch.ldexp(torch.ones((), device=b.device), b.to(torch.int32) - 127)


def _random(c, shape, g):
    """Keys and values as a model makes them: normal, some channels much larger than others."""
    x = torch.empty(shape, dtype=DTYPES[c["dtype"]], device="cuda").normal_(generator=g)
    return x.mul_(1.0 + 3.0 * (torch.arange(c["d"], device="cuda") % 37 == 5).to(x.dtype))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    B, P = c["B"], c["page"]
    pairs = _lengths(c)
    pairs = [pairs[i] for i in torch.randperm(B, generator=h).tolist()]
    ends = [a + t for a, t in pairs]
    need = [-(-n // P) for n in ends]
    max_pages = max(need)
    pool = sum(need) + 8
    order = torch.randperm(pool, generator=h).to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    row = torch.repeat_interleave(torch.arange(B), torch.tensor(need))
    first = torch.cumsum(torch.tensor(need), 0) - torch.tensor(need)
    table[row, torch.arange(sum(need)) - first[row]] = order[:sum(need)]
    starts = torch.zeros(B + 1, dtype=torch.int32)
    starts[1:] = torch.cumsum(torch.tensor([t for _, t in pairs]), 0)
    N = int(starts[-1])
    s = {"case": c, "N": N, "max_len": max(ends), "max_chunk": max(t for _, t in pairs),
         "page_table": table.cuda(), "chunk_starts": starts.cuda(),
         "cached_lens": torch.tensor([a for a, _ in pairs], dtype=torch.int32).cuda(),
         "k_exps": None, "v_exps": None}
    shape = (pool, c["hkv"], P, c["d"]) if c["heads_first"] else (pool, P, c["hkv"], c["d"])

    def pages(x):
        return x.transpose(1, 2) if c["heads_first"] else x

    for kv in ("k", "v"):
        # What the unused slots hold is left from other sequences.
        x = _random(c, shape, g)
        if c["cache"] == "e4m3":
            x, e = _quantise(x)
            x = x.view(torch.float8_e4m3fn)
            s[kv + "_exps"] = pages(e)
        s[kv + "_pages"] = pages(x)
    if c["op"] == "append":
        s["key"] = _random(c, (N, c["hkv"], c["d"]), g)
        s["value"] = _random(c, (N, c["hkv"], c["d"]), g)
    if c["op"] == "attention":
        s["query"] = _random(c, (N, c["hq"], c["d"]), g).mul_(1.5)
        s["scale"] = c["d"] ** -0.5
    return s


def _rows(s):
    """Sequence and place in its chunk of every packed token."""
    starts = s["chunk_starts"].long()
    b = torch.repeat_interleave(torch.arange(starts.numel() - 1, device=starts.device),
                                starts.diff(), output_size=s["N"])
    return b, torch.arange(s["N"], device=starts.device) - starts[b]


def _where(s, b, position):
    """Page and slot of a position of sequence b."""
    P = s["case"]["page"]
    return s["page_table"][b, position // P].long().clamp(min=0), position % P


def _gather(s, kv, page, slot):
    """The cached vectors at (page, slot), in 32 bits."""
    x = s[kv + "_pages"]
    if s["case"]["cache"] == "16":
        return x[page, slot].float()
    codes = x.view(torch.uint8)[page, slot].view(torch.float8_e4m3fn).float()
    return codes * _powers(s[kv + "_exps"][page, slot]).unsqueeze(-1)


def _plain_append(s):
    b, t = _rows(s)
    at = _where(s, b, s["cached_lens"].long()[b] + t)

    def put(kv, x):
        if s["case"]["cache"] == "16":
            s[kv + "_pages"][at] = x
            return s[kv + "_pages"]
        code, e = _quantise(x)
        s[kv + "_pages"].view(torch.uint8)[at] = code
        s[kv + "_exps"][at] = e
        return _gather(s, kv, *at).to(x.dtype)

    return {"k": put("k", s["key"]), "v": put("v", s["value"])}


def _plain_read(s):
    b, t = _rows(s)
    at = _where(s, b, s["cached_lens"].long()[b] + t)
    dt = DTYPES[s["case"]["dtype"]]
    return {"k": _gather(s, "k", *at).to(dt), "v": _gather(s, "v", *at).to(dt)}


def _plain_attention(s):
    c = s["case"]
    B, G, T, L = c["B"], c["hq"] // c["hkv"], s["max_chunk"], s["max_len"]
    dev = s["query"].device
    j = torch.arange(L, device=dev)
    at = _where(s, torch.arange(B, device=dev)[:, None], j[None, :])
    k = _gather(s, "k", *at).permute(0, 2, 3, 1)  # [B, hkv, d, L]
    t = torch.arange(T, device=dev)
    rows = (s["chunk_starts"].long()[:-1, None] + t).clamp(max=s["N"] - 1)
    q = s["query"][rows].float().view(B, T, c["hkv"], G, c["d"])
    q = q.permute(0, 2, 1, 3, 4).reshape(B, c["hkv"], T * G, c["d"])
    x = torch.matmul(q, k).mul_(s["scale"]).view(B, c["hkv"], T, G, L)
    del k
    last = s["cached_lens"].long()[:, None] + t  # position of query (b, t)
    seen = j <= last[..., None]
    if c["window"]:
        seen &= j > (last - c["window"])[..., None]
    x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    v = _gather(s, "v", *at).permute(0, 2, 1, 3)  # [B, hkv, L, d]
    o = torch.matmul(x.view(B, c["hkv"], T * G, L), v).view(B, c["hkv"], T, G, c["d"]) / total
    lse = (top + total.log()).squeeze(-1)
    b, i = _rows(s)
    return {"out": o[b, :, i].reshape(s["N"], c["hq"], c["d"]).to(s["query"].dtype),
            "lse": lse[b, :, i].reshape(s["N"], c["hq"])}


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"append": _plain_append, "read": _plain_read, "attention": _plain_attention}[op](s)
    import speculative_decoding_verification_66_gb300 as sv
    cache = (s["k_pages"], s["v_pages"], s["page_table"], s["cached_lens"], s["chunk_starts"])
    exps = dict(k_exps=s["k_exps"], v_exps=s["v_exps"])
    if op == "attention":
        out, lse = sv.sv_chunk_attention(s["query"], *cache, **exps, scale=s["scale"],
                                         window=s["case"]["window"], max_chunk=s["max_chunk"],
                                         return_lse=True)
        return {"out": out, "lse": lse}
    if op == "append":
        sv.sv_kv_append(s["key"], s["value"], *cache, **exps)
        if s["case"]["cache"] == "16":
            return {"k": s["k_pages"], "v": s["v_pages"]}
    k, v = sv.sv_kv_read(*cache, s["N"], **exps, dtype=DTYPES[s["case"]["dtype"]])
    return {"k": k, "v": v}


def _values64(pages, exps, at):
    """The cached vectors at `at` (page, slot), in 64 bits."""
    if exps is None:
        return pages[at].double()
    e = exps[at].double() - 127.0
    return pages.view(torch.uint8)[at].view(torch.float8_e4m3fn).double() * torch.exp2(e)[..., None]


def _rounded64(x):
    """e4m3 with a shared power of two, in 64 bits: the exponent from logarithms, the codes as
    multiples of their step (three mantissa bits; the least step is 2^-9)."""
    x = x.double()
    e = torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -109) / 448.0))
    e = e.clamp(min=-117)
    y = x / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * torch.exp2(e)


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    cached, starts = s["cached_lens"].tolist(), s["chunk_starts"].tolist()
    P, G = c["page"], max(1, c["hq"] // c["hkv"])

    def at(b, lo, hi):
        p = torch.arange(lo, hi, device="cuda")
        return s["page_table"][b].long()[p // P], p % P

    if c["op"] == "append" and c["cache"] != "16":
        return {"k": _rounded64(s["key"]), "v": _rounded64(s["value"])}
    if c["op"] == "append":
        if s["k_pages"].numel() > 3e8:
            return None
        out = {"k": s["k_pages"].double(), "v": s["v_pages"].double()}
        for b in range(c["B"]):
            w = at(b, cached[b], cached[b] + starts[b + 1] - starts[b])
            out["k"][w] = s["key"][starts[b]:starts[b + 1]].double()
            out["v"][w] = s["value"][starts[b]:starts[b + 1]].double()
        return out
    if c["op"] == "read":
        w = [at(b, cached[b], cached[b] + starts[b + 1] - starts[b]) for b in range(c["B"])]
        w = tuple(torch.cat(x) for x in zip(*w))
        return {"k": _values64(s["k_pages"], s["k_exps"], w),
                "v": _values64(s["v_pages"], s["v_exps"], w)}
    out = torch.empty(s["query"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["query"].shape[:2], dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        n = starts[b + 1] - starts[b]
        w = at(b, 0, cached[b] + n)
        k = _values64(s["k_pages"], s["k_exps"], w)
        v = _values64(s["v_pages"], s["v_exps"], w)
        key = torch.arange(cached[b] + n, device="cuda")
        query = torch.arange(cached[b], cached[b] + n, device="cuda")[:, None]
        hidden = key > query
        if c["window"]:
            hidden |= key <= query - c["window"]
        for h in range(c["hq"]):
            x = s["query"][starts[b]:starts[b + 1], h].double() @ k[:, h // G].T * s["scale"]
            x[hidden] = -math.inf
            z = torch.logsumexp(x, -1)
            out[starts[b]:starts[b + 1], h] = torch.exp(x - z[:, None]) @ v[:, h // G]
            lse[starts[b]:starts[b + 1], h] = z
    return {"out": out, "lse": lse}
