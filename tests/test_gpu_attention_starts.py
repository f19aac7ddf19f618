"""Starts that are out of order or leave the packed arrays: no row has two owners, what has no good
owner is NaN and is not written, and the good sequences are as if they were alone."""
import random

import pytest
import torch

import speculative_decoding_verification_66_gb300 as sv
from attention_util import Cache

pytestmark = pytest.mark.gpu
N = 20  # rows of the packed arrays


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_attention()
    torch.cuda.set_device(0)


def shuffled(B, n, seed):
    """Mostly rising starts in [0, n], some of them out of their place."""
    r = random.Random(seed)
    s = sorted(r.randint(0, n) for _ in range(B + 1))
    for _ in range(max(1, B // 8)):
        s[r.randrange(B + 1)] = r.randint(0, n)
    return s


STARTS = [[0, 5, 3, 20], [0, 12, 4, 8, 20], [3, 8, 0, 20], [0, 20, 0, 20], [5, 5, 2, 2, 9]] \
    + [shuffled(B, N, B) for B in (6, 9, 33, 70)] + [shuffled(1100, N, 3)]


def call(starts, tokens=N):
    """A cache whose sequences could each take all rows, and the call's arrays."""
    B = len(starts) - 1
    c = Cache([8] * B, [tokens] * B, 2, 64, 8, "bf16", False, seed=B)
    c.starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(B)
    q, k, v = ((torch.randn(tokens, h, 64, generator=g)).bfloat16().cuda() for h in (8, 2, 2))
    return c, q, k, v


def owners(status, starts, tokens):
    """The good sequence of every row, or None; the good ones share none."""
    own = [None] * tokens
    for b, s in enumerate(status):
        if s == 0:
            assert 0 <= starts[b] <= starts[b + 1] <= tokens
            for t in range(starts[b], starts[b + 1]):
                assert own[t] is None
                own[t] = b
    return own


def expected_status(starts, tokens, capacity):
    """Falls and lengths are each sequence's own matter; of the others, the ones that share no row
    with another have to be good."""
    B = len(starts) - 1
    bad = [not (0 <= starts[b] <= starts[b + 1] <= tokens)
           or 8 + starts[b + 1] - starts[b] > capacity for b in range(B)]
    alone = []
    for b in range(B):
        mine = set(range(starts[b], starts[b + 1]))
        alone.append(all(starts[j] <= starts[b] for j in range(b)) and
                     all(starts[j] >= starts[b + 1] for j in range(b + 1, B)) or not mine)
    return bad, alone


@pytest.mark.parametrize("starts", STARTS, ids=lambda s: f"{len(s) - 1}-{s[0]}-{s[1]}-{s[2]}")
@pytest.mark.parametrize("max_chunk", [0, 4])
def test_attention(starts, max_chunk):
    c, q, _, _ = call(starts)
    B = len(starts) - 1
    status = torch.full((B,), 99, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    sv.sv_chunk_attention(q, *c.args(), out=out, lse=lse, seq_status=status, max_chunk=max_chunk)
    status = status.tolist()
    bad, alone = expected_status(starts, N, c.table.shape[1] * 8)
    if max_chunk:
        bad = [x or starts[b + 1] - starts[b] > max_chunk for b, x in enumerate(bad)]
    for b in range(B):
        assert bool(status[b] & sv.SV_SEQ_BAD_LENGTH) == bad[b]
        assert status[b] in (0, sv.SV_SEQ_BAD_LENGTH, sv.SV_SEQ_OVERLAP)
        if alone[b] and not bad[b]:
            assert status[b] == 0
    own = owners(status, starts, N)
    claimed = [any(min(max(starts[b], 0), N) <= t < min(max(starts[b + 1], 0), N) for b in range(B))
               for t in range(N)]
    for t in range(N):
        if own[t] is None:
            assert out[t].isnan().all() and lse[t].isnan().all() if claimed[t] else \
                (out[t] == 7.0).all() and (lse[t] == 7.0).all()
    for b in set(own) - {None}:
        s, e = starts[b], starts[b + 1]
        one = torch.tensor([0, e - s], dtype=torch.int32, device="cuda")
        want = sv.sv_chunk_attention(q[s:e], *c.parts, c.table[b:b + 1], c.cached[b:b + 1], one)
        assert torch.allclose(out[s:e].float(), want.float(), atol=2e-2, rtol=2e-2)


@pytest.mark.parametrize("starts", STARTS, ids=lambda s: f"{len(s) - 1}-{s[0]}-{s[1]}-{s[2]}")
def test_append_and_read(starts):
    c, _, k, v = call(starts)
    B = len(starts) - 1
    before = [x.clone() for x in c.parts]
    status = torch.full((B,), 99, dtype=torch.int32, device="cuda")
    sv.sv_kv_append(k, v, *c.args(), seq_status=status)
    first = status.tolist()
    bad, alone = expected_status(starts, N, c.table.shape[1] * 8)
    for b in range(B):
        assert bool(first[b] & sv.SV_SEQ_BAD_LENGTH) == bad[b]
        if alone[b] and not bad[b]:
            assert first[b] == 0
    own = owners(first, starts, N)
    for t, b in enumerate(own):
        if b is not None:
            p = 8 + t - starts[b]
            for i, x in enumerate((k, v)):
                before[i][c.pages_of[b][p // 8], p % 8] = x[t]
    for i in range(2):
        assert torch.equal(c.parts[i], before[i])
    key, value = sv.sv_kv_read(*c.args(), N, seq_status=status)
    assert status.tolist() == first
    for t, b in enumerate(own):
        for x, y in ((key, k), (value, v)):
            assert torch.equal(x[t], y[t]) if b is not None else x[t].isnan().all()


@pytest.mark.parametrize("starts", [[2, 5, 9, 99], [-4, 5, 9, 20], [0, 99, 4, 20], [0, 5, 21, 30],
                                    [-9, -2, 4, 20], [0, 5, 10, -3]])
@pytest.mark.parametrize("d,max_chunk", [(64, 0), (64, 1), (256, 0)])
def test_rows_of_sequences_that_leave_the_arrays_are_nan(starts, d, max_chunk):
    c = Cache([8, 8, 8], [N] * 3, 2, d, 32, "bf16", False, seed=9)
    c.starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
    q = torch.randn(N, 8, d, device="cuda").bfloat16()
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    status = torch.empty(3, dtype=torch.int32, device="cuda")
    sv.sv_chunk_attention(q, *c.args(), out=out, lse=lse, max_chunk=max_chunk, seq_status=status)
    kind = [7.0] * N
    for b in range(3):
        for t in range(max(0, starts[b]), min(N, starts[b + 1])):
            kind[t] = "nan"
    for b, s in enumerate(status.tolist()):
        if s == 0:
            kind[starts[b]:starts[b + 1]] = ["good"] * (starts[b + 1] - starts[b])
    for t in range(N):
        if kind[t] == "good":
            assert out[t].isfinite().all() and lse[t].isfinite().all()
        elif kind[t] == "nan":
            assert out[t].isnan().all() and lse[t].isnan().all()
        else:
            assert (out[t] == 7.0).all() and (lse[t] == 7.0).all()
    # Nothing of the bad ones is written to the cache.
    before = [x.clone() for x in c.parts]
    k = torch.randn(N, 2, d, device="cuda").bfloat16()
    sv.sv_kv_append(k, k, *c.args(), seq_status=status)
    for b, s in enumerate(status.tolist()):
        if s == 0:
            for t in range(starts[b], starts[b + 1]):
                p = 8 + t - starts[b]
                for x in before:
                    x[c.pages_of[b][p // 32], p % 32] = k[t]
    assert all(torch.equal(x, y) for x, y in zip(before, c.parts))


def test_statuses_of_calls_without_rows():
    """No rows in the packed arrays: starts other than 0 and negative lengths are still bad."""
    c, q, k, v = call([0, 0, 0, 0, 5])
    c.cached[1] = -3
    want = [0, sv.SV_SEQ_BAD_LENGTH, 0, sv.SV_SEQ_BAD_LENGTH]
    status = torch.full((4,), 99, dtype=torch.int32, device="cuda")
    sv.sv_chunk_attention(q[:0], *c.args(), seq_status=status)
    assert status.tolist() == want
    status.fill_(99)
    sv.sv_kv_append(k[:0], v[:0], *c.args(), seq_status=status)
    assert status.tolist() == want
    status.fill_(99)
    sv.sv_kv_read(*c.args(), 0, seq_status=status)
    assert status.tolist() == want
