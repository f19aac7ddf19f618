"""sv_chunk_attention against the definition in 64 bits (attention_util), with
error bounds derived there from the types and lengths alone."""
import math

import pytest
import torch

import speculative_decoding_verification_66_gb300 as sv
from attention_util import Cache, check, quantise, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_attention()
    torch.cuda.set_device(0)


def make_query(c, G, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed + 1000)
    return (torch.randn(c.tokens, c.heads * G, c.d, generator=g) * spread).to(c.dtype).cuda()


def attend(c, q, window=0, scale=None, **kw):
    return sv.sv_chunk_attention(q, *c.args(), **c.exp_args(), window=window, scale=scale,
                                 return_lse=True, **kw)


def run(lens, chunks, heads, G, d, page, dtype, e4m3, hf=False, window=0, seed=0, fill=None,
        scale=None, max_chunk=0, spread=1.0):
    c = Cache(lens, chunks, heads, d, page, dtype, e4m3, hf, seed=seed, fill=fill, spread=spread)
    q = make_query(c, G, seed)
    status = torch.full((len(lens),), 99, dtype=torch.int32, device="cuda")
    out, lse = attend(c, q, window, scale, seq_status=status, max_chunk=max_chunk)
    assert not status.any()
    check(out, lse, c, q, scale or d ** -0.5, window)
    return c, q, out, lse


TYPES = [("bf16", False), ("fp16", False), ("bf16", True), ("fp16", True)]
LENGTHS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 700]


@pytest.mark.parametrize("dtype,e4m3", TYPES)
@pytest.mark.parametrize("heads,G", [(1, 1), (2, 4), (1, 7), (2, 8), (1, 16)])
def test_single_tokens(dtype, e4m3, heads, G):
    """One new token a sequence, at every length near a tile's or page's edge."""
    run(LENGTHS, [1] * len(LENGTHS), heads, G, 128, 16, dtype, e4m3, max_chunk=1)


@pytest.mark.parametrize("dtype,e4m3", TYPES)
@pytest.mark.parametrize("G,T", [(1, 5), (4, 5), (4, 8), (4, 9), (7, 5), (8, 4), (8, 9), (8, 17),
                                 (3, 43), (1, 130)])
def test_drafts(dtype, e4m3, G, T):
    """T new tokens a sequence: rows of one tile, one more than a tile, several tiles."""
    run([0, 1, 60, 64, 200, 513], [T] * 6, 2, G, 128, 32, dtype, e4m3, max_chunk=T, seed=T)


@pytest.mark.parametrize("dtype,e4m3", TYPES)
@pytest.mark.parametrize("d", [16, 48, 64, 80, 96, 112, 192, 256])
def test_head_sizes(dtype, e4m3, d):
    run([0, 33, 300], [1, 9, 40], 2, 3, d, 16, dtype, e4m3, seed=d)
    run([130, 64], [1, 1], 2, 4, d, 16, dtype, e4m3, seed=d, max_chunk=1)


@pytest.mark.parametrize("dtype,e4m3", TYPES)
@pytest.mark.parametrize("page", [8, 16, 64, 128, 256, 1024])
@pytest.mark.parametrize("hf", [False, True])
def test_pages(dtype, e4m3, page, hf):
    run([0, 7, 250, 1025], [5, 1, 70, 4], 2, 2, 64, page, dtype, e4m3, hf, seed=page)
    run([3, 500], [9, 60], 1, 4, 128, page, dtype, e4m3, hf, seed=page)


@pytest.mark.parametrize("dtype,e4m3", TYPES)
@pytest.mark.parametrize("window", [1, 2, 17, 64, 100, 129, 5000])
def test_windows(dtype, e4m3, window):
    run([0, 40, 128, 700], [1, 9, 150, 30], 1, 4, 128, 16, dtype, e4m3, window=window, seed=window)
    run([0, 40, 128, 700], [1, 5, 5, 5], 2, 4, 64, 16, dtype, e4m3, window=window, max_chunk=5)


@pytest.mark.parametrize("dtype,e4m3", TYPES)
def test_ragged_with_empty_sequences(dtype, e4m3):
    run([10, 0, 500, 3, 0, 90], [0, 3, 0, 200, 0, 1], 2, 4, 128, 16, dtype, e4m3)
    run([10, 900], [0, 0], 2, 4, 128, 16, dtype, e4m3)


@pytest.mark.parametrize("dtype,e4m3", TYPES)
@pytest.mark.parametrize("T", [1, 5, 60])
def test_long_context(dtype, e4m3, T):
    """Work split over the keys and joined."""
    run([9000, 20011], [T, T], 1, 4, 128, 64, dtype, e4m3, seed=3, max_chunk=T)


@pytest.mark.parametrize("dtype,e4m3", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 5, 40])
def test_many_tiles_a_block(dtype, e4m3, d, T):
    """More tiles of several items to a thread block than its shared memory holds at one time."""
    run([6000, 4100, 5003, 777], [T] * 4, 16, 4, d, 64, dtype, e4m3, seed=4, max_chunk=T)


@pytest.mark.parametrize("dtype,e4m3", TYPES)
def test_long_piece(dtype, e4m3):
    run([257], [600], 2, 2, 128, 64, dtype, e4m3, seed=5)


@pytest.mark.parametrize("B,T", [(1300, 1), (1300, 4), (300, 40)])
def test_many_sequences(B, T):
    g = torch.Generator().manual_seed(T)
    lens = torch.randint(0, 90, (B,), generator=g).tolist()
    chunks = torch.randint(0, T + 1, (B,), generator=g).tolist()
    run(lens, chunks, 1, 2, 32, 8, "bf16", False, max_chunk=T)


@pytest.mark.parametrize("dtype,e4m3", TYPES)
@pytest.mark.parametrize("fill", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("T", [1, 5, 70])
def test_unused_slots_have_no_influence(dtype, e4m3, fill, T):
    """NaN and infinities in the spare pages and behind the last token."""
    run([0, 7, 100, 513], [T] * 4, 2, 4, 128, 64, dtype, e4m3, fill=fill, max_chunk=T)


@pytest.mark.parametrize("dtype,e4m3", TYPES)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("lens,T,at,window", [(50, 6, 53, 0), (200, 90, 240, 0), (300, 5, 283, 20),
                                              (300, 80, 290, 64), (6000, 5, 6001, 0)])
def test_masked_values_have_no_influence(dtype, e4m3, bad, lens, T, at, window):
    """A key and a value that are NaN or infinite at a position that some rows see and others
    (earlier ones, or ones whose window has passed it) do not."""
    c = Cache([lens, 40], [T, T], 2, 128, 16, dtype, False, seed=8)
    c.parts[0][c.pages_of[0][at // 16], at % 16, :, 3] = bad
    c.parts[1][c.pages_of[0][at // 16], at % 16, 1, 7] = bad
    if e4m3:
        c.e4m3 = True
        for i in range(2):
            code, c.exps[i] = quantise(c.parts[i])
            c.parts[i] = code.view(torch.float8_e4m3fn)
    q = make_query(c, 4, 9)
    out, lse = attend(c, q, window, max_chunk=T)
    seen = torch.zeros(2 * T, dtype=torch.bool)
    for t in range(T):
        p = lens + t
        seen[t] = at <= p and (window == 0 or at > p - window)
    assert seen.any() and not seen.all()
    check(out, lse, c, q, 128 ** -0.5, window, rows=(~seen).nonzero().squeeze(1).cuda())
    # Rows that see a NaN key are NaN throughout.
    if math.isnan(bad) or e4m3:
        assert out[seen.cuda()].isnan().all()


@pytest.mark.parametrize("T", [1, 6, 70])
def test_visible_bad_values_reach_only_their_elements(T):
    """A NaN in one element of a value that every row sees: that element of the output alone."""
    c = Cache([300], [T], 1, 128, 16, "bf16", False, seed=8)
    c.parts[1][c.pages_of[0][2], 5, 0, 7] = math.nan
    q = make_query(c, 4, 9)
    out, lse = attend(c, q, max_chunk=T)
    assert out[:, :, 7].isnan().all() and lse.isfinite().all()
    keep = torch.arange(128, device="cuda") != 7
    assert out[:, :, keep].isfinite().all()
    ref, _, tol, _ = reference(c, q, 128 ** -0.5)
    assert ((out.double() - ref).abs() <= tol)[:, :, keep].all()


@pytest.mark.parametrize("dtype,e4m3", TYPES)
@pytest.mark.parametrize("T", [1, 40])
def test_extreme_scores(dtype, e4m3, T):
    """Scores of thousands of either sign (one key takes all the weight), all scores equal, and
    values near the type's ends."""
    run([200, 3], [T, T], 2, 4, 128, 16, dtype, e4m3, scale=40.0, max_chunk=T)
    run([200, 3], [T, T], 2, 4, 128, 16, dtype, e4m3, scale=1e-9, max_chunk=T)
    c = Cache([300], [T], 1, 64, 16, dtype, e4m3, seed=2, spread=3000.0)
    q = make_query(c, 4, 3, spread=1e-3)
    out, lse = attend(c, q, max_chunk=T)
    check(out, lse, c, q, 0.125)
    # Scores falling and rising along the keys: the running maximum moves at every tile or never.
    for sign in (1.0, -1.0):
        c = Cache([2000], [T], 1, 64, 16, dtype, False, seed=2)
        ramp = torch.linspace(-8, 8, 2000 + T, device="cuda") * sign
        p = torch.arange(2000 + T, device="cuda")
        c.parts[0][c.table[0].long()[p // 16], p % 16] = ramp[:, None, None].to(c.dtype)
        q = torch.full((T, 4, 64), 1.5, dtype=c.dtype, device="cuda")
        out, lse = attend(c, q, max_chunk=T)
        check(out, lse, c, q, 0.125)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 5, 60])
@pytest.mark.parametrize("kind", ["drift", "steps", "apart", "zeros"])
def test_e4m3_exponents(dtype, T, kind):
    """Keys and values whose sizes drift along the sequence, change between tiles, lie far apart
    within a tile, or are all zero for long stretches."""
    n = 900 + T
    c = Cache([900, 40], [T, T], 2, 128, 16, dtype, False, seed=4)
    p = torch.arange(n, device="cuda")
    size = {"drift": torch.exp2(p / 60.0 - 8.0),
            "steps": torch.exp2(((p // 150) % 3 - 1) * 5.0),
            "apart": torch.exp2(-(p % 3) * 8.0),
            "zeros": ((p // 200) % 2).double()}[kind]
    page, slot = c.table[0].long()[p // 16], p % 16
    for i in range(2):
        x = c.parts[i][page, slot].double() * size[:, None, None]
        c.parts[i][page, slot] = x.to(c.dtype)
        c.parts[i], c.exps[i] = (lambda q: (q[0].view(torch.float8_e4m3fn), q[1]))(
            quantise(c.parts[i]))
    c.e4m3 = True
    q = make_query(c, 4, 9, spread=0.02 if kind == "drift" else 1.0)
    out, lse = attend(c, q, max_chunk=T)
    check(out, lse, c, q, 128 ** -0.5)


@pytest.mark.parametrize("T", [1, 5, 80])
def test_strided_queries(T):
    """Queries as a slice of a fused projection, heads not adjacent."""
    c = Cache([100, 17], [T, T], 2, 64, 16, "bf16", False, seed=6)
    fused = torch.randn(2 * T, 24 * 64, device="cuda").bfloat16()
    q = fused.as_strided((2 * T, 8, 64), (24 * 64, 128, 1), 256)
    out, lse = attend(c, q, max_chunk=T)
    check(out, lse, c, q, 0.125)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T", [1, 5, 70])
def test_bad_sequences_and_pages(e4m3, T):
    c = Cache([40, 40, 40, 40, 0], [T] * 5, 2, 64, 8, "bf16", e4m3, seed=7)
    q = make_query(c, 4, 8)
    ref_out, _ = attend(c, q, max_chunk=T)
    c.cached[1] = -7
    c.table[2, 3] = c.parts[0].shape[0] + 5
    c.cached[3] = c.table.shape[1] * 8 - T + 1
    status = torch.zeros(5, dtype=torch.int32, device="cuda")
    out, lse = attend(c, q, max_chunk=T, seq_status=status)
    assert status.tolist() == [0, sv.SV_SEQ_BAD_LENGTH, sv.SV_SEQ_BAD_PAGE, sv.SV_SEQ_BAD_LENGTH, 0]
    assert out[T:4 * T].isnan().all() and lse[T:4 * T].isnan().all()
    for s in (slice(0, T), slice(4 * T, 5 * T)):
        # (the split of the work follows all lengths: equal to rounding, not bit for bit)
        assert torch.allclose(out[s].float(), ref_out[s].float(), atol=2e-2, rtol=2e-2)
    # A sequence with more new tokens than max_chunk.
    if T > 1:
        out, lse = attend(c, q, max_chunk=T - 1, seq_status=status)
        assert all(s & sv.SV_SEQ_BAD_LENGTH for s in status.tolist()) and out.isnan().all()
    # Page 0 table entries before a window are not needed.
    c = Cache([400], [T], 2, 64, 8, "bf16", e4m3, seed=7)
    q = make_query(c, 4, 8)
    first = (400 - 50 + 1) // 8
    want = attend(c, q, window=50, max_chunk=T)
    c.table[0, :first] = -3
    out, lse = attend(c, q, window=50, max_chunk=T, seq_status=status[:1])
    assert status[0] == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("starts", [[0, 5, 3, 20], [2, 5, 9, 99], [-4, 5, 9, 20], [0, 99, 4, 20]])
def test_bad_starts(starts):
    c = Cache([8, 8, 8], [5, 5, 10], 2, 64, 32, "bf16", False, seed=9)
    q = make_query(c, 4, 8)
    c.starts.copy_(torch.tensor(starts, dtype=torch.int32))
    status = torch.zeros(3, dtype=torch.int32, device="cuda")
    attend(c, q, seq_status=status)
    torch.cuda.synchronize()
    bad = [not (0 <= starts[b] <= starts[b + 1] <= c.tokens) for b in range(3)]
    assert [bool(s & sv.SV_SEQ_BAD_LENGTH) for s in status.tolist()] == bad


def test_offsets_past_32_bits():
    """Pages 2^31 elements apart, in a 16-bit and in an e4m3 cache."""
    step = 1 << 31
    i32 = dict(dtype=torch.int32, device="cuda")
    for T in (1, 60):
        x = torch.randn(128, 1, 64, device="cuda").bfloat16()
        table = torch.tensor([[2, 0, 3, 1]], **i32)
        args = (table, torch.tensor([128 - T], **i32), torch.tensor([0, T], **i32))
        q = torch.randn(T, 4, 64, device="cuda").bfloat16()
        near = torch.empty(4, 32, 1, 64, dtype=torch.bfloat16, device="cuda")
        near[[2, 0, 3, 1]] = x.view(4, 32, 1, 64)
        want = sv.sv_chunk_attention(q, near, near, *args, max_chunk=T)
        store = torch.empty(3 * step + 4096, dtype=torch.bfloat16, device="cuda")
        far = store.as_strided((4, 32, 1, 64), (step, 64, 64, 1))
        far.copy_(near)
        out = sv.sv_chunk_attention(q, far, far, *args, max_chunk=T)
        assert torch.equal(out, want)
        del store, far


@pytest.mark.parametrize("T", [1, 5, 70])
def test_the_same_call_gives_the_same_bits(T):
    c = Cache([3000, 70, 900], [T] * 3, 2, 128, 16, "bf16", True, seed=1)
    q = make_query(c, 4, 2)
    out, lse = attend(c, q, max_chunk=T)
    for _ in range(5):
        o, z = attend(c, q, max_chunk=T)
        assert torch.equal(o, out) and torch.equal(z, lse)


@pytest.mark.parametrize("T", [1, 5, 70])
@pytest.mark.parametrize("e4m3", [False, True])
def test_captured_and_replayed_with_other_lengths(T, e4m3):
    """One graph of append and attention, replayed with new rows, lengths and pages."""
    a = Cache([600, 30, 0], [T] * 3, 2, 128, 16, "bf16", e4m3, seed=1)
    b = Cache([31, 590, 200], [T] * 3, 2, 128, 16, "bf16", e4m3, seed=2)
    for c in (a, b):  # one shape for both
        wide = torch.full((3, 64), -1, dtype=torch.int32, device="cuda")
        wide[:, :c.table.shape[1]] = c.table
        c.table = wide
    pool = max(a.parts[0].shape[0], b.parts[0].shape[0])
    pages = [torch.zeros((pool,) + a.parts[0].shape[1:], dtype=a.parts[0].dtype, device="cuda")
             for _ in range(2)]
    exps = [torch.zeros(pages[0].shape[:3], dtype=torch.uint8, device="cuda") if e4m3 else None
            for _ in range(2)]
    table, cached, starts = (torch.empty_like(x) for x in (a.table, a.cached, a.starts))
    q, k, v = (torch.empty(3 * T, h, 128, dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2))

    def load(c, seed):
        for x, y in ((table, c.table), (cached, c.cached), (starts, c.starts)):
            x.copy_(y)
        for i in range(2):
            n = c.parts[i].shape[0]
            pages[i].view(torch.int8 if e4m3 else torch.int16)[:n] = \
                c.parts[i].view(torch.int8 if e4m3 else torch.int16)
            if e4m3:
                exps[i][:n] = c.exps[i]
        g = torch.Generator(device="cuda").manual_seed(seed)
        for x in (q, k, v):
            x.normal_(generator=g)

    def step():
        kw = dict(k_exps=exps[0], v_exps=exps[1])
        sv.sv_kv_append(k, v, *pages, table, cached, starts, **kw)
        return sv.sv_chunk_attention(q, *pages, table, cached, starts, **kw, max_chunk=T,
                                     return_lse=True)

    load(a, 1)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        out, lse = step()
    for c, seed in ((a, 3), (b, 4), (a, 5)):
        load(c, seed)
        graph.replay()
        got = out.clone(), lse.clone()
        load(c, seed)
        want = step()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        c.parts, c.exps = pages, exps
        check(want[0], want[1], c, q, 128 ** -0.5)


def test_another_stream():
    c = Cache([2000, 3], [6, 2], 4, 128, 16, "bf16", False, seed=11)
    q = make_query(c, 4, 12)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = attend(c, q, stream=s)
    s.synchronize()
    check(out, lse, c, q, 128 ** -0.5)


def test_given_outputs_and_workspace():
    c = Cache([900, 3], [6, 2], 2, 128, 16, "bf16", False, seed=11)
    q = make_query(c, 4, 12)
    out = torch.full_like(q, 7.0)
    lse = torch.empty(8, 8, dtype=torch.float32, device="cuda")
    ws = torch.empty(sv.sv_chunk_attention_workspace_bytes(2, 8, 8, 2, 128, 6) + 512,
                     dtype=torch.uint8, device="cuda").fill_(0xFF)
    o, z = attend(c, q, out=out, lse=lse, workspace=ws, max_chunk=6)
    assert o is out and z is lse
    check(out, lse, c, q, 128 ** -0.5)
    alone = sv.sv_chunk_attention(q, *c.args(), max_chunk=6)  # without lse: the same bits
    assert torch.equal(alone, out)


def test_kept_workspaces_grow_and_keep_apart():
    """Calls of growing sizes, on two streams and from two threads at a time."""
    import threading
    cases = []
    for i, (lens, T) in enumerate([([30], 1), ([3000, 70], 4), ([900, 5000], 40), ([200], 2)]):
        c = Cache(lens, [T] * len(lens), 2, 128, 16, "bf16", i % 2 == 1, seed=i)
        q = make_query(c, 4, i)
        cases.append((c, q, T, attend(c, q, max_chunk=T)))
    torch.cuda.synchronize()
    bad = []

    def work(stream):
        with torch.cuda.stream(stream):
            got = [attend(c, q, max_chunk=T) for _ in range(8) for c, q, T, _ in cases]
            stream.synchronize()
            for i, (o, z) in enumerate(got):
                want = cases[i % len(cases)][3]
                if not (torch.equal(o, want[0]) and torch.equal(z, want[1])):
                    bad.append(i)

    same, other = torch.cuda.Stream(), torch.cuda.Stream()
    threads = [threading.Thread(target=work, args=(s,)) for s in (same, same, other)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_rows_of_no_sequence_are_left_alone():
    """Packed arrays longer than the chunks (a graph's padded batch)."""
    c = Cache([100, 3], [4, 2], 2, 128, 16, "bf16", False, seed=11)
    q = torch.randn(40, 8, 128, device="cuda").bfloat16()
    out = torch.full_like(q, 7.0)
    attend(c, q, out=out, max_chunk=4)
    assert (out[6:] == 7.0).all()
    check(out[:6], None, c, q[:6], 128 ** -0.5)


def test_refusals():
    c = Cache([4], [2], 2, 64, 8)
    q = make_query(c, 4, 1)
    for bad in (q[:, :3], q.float(), q.half(), q[:, :, :32], q.cpu(), q[0]):
        with pytest.raises((ValueError, TypeError)):
            sv.sv_chunk_attention(bad, *c.args())
    with pytest.raises(ValueError):
        sv.sv_chunk_attention(q, *c.args(), out=torch.empty_like(q).float())
    with pytest.raises(ValueError):
        sv.sv_chunk_attention(q, *c.args(), lse=torch.empty(2, 8, device="cuda").half())
    for kw in (dict(scale=0.0), dict(scale=math.nan), dict(window=-1), dict(max_chunk=-1),
               dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(sv.SpecVerifyError):
            sv.sv_chunk_attention(q, *c.args(), **kw)


@pytest.mark.parametrize("dtype,e4m3", TYPES)
@pytest.mark.parametrize("T", [1, 8, 40])
def test_many_small_weights_add_up(dtype, e4m3, T):
    """One key takes most of the weight, 60000 others 2^-18.75 of it each and a seventh of the sum
    together, the first tile's values 2^6 times the others'. 160 sequences on the same pages, so
    that blocks work through whole ones."""
    n, B = 60000, 160
    c = Cache([n], [T], 1, 64, 64, dtype, False)
    k = torch.zeros(c.parts[0].shape, dtype=c.dtype, device="cuda")
    v = torch.ones_like(k)
    p = torch.arange(128, device="cuda")
    page, slot = c.table[0].long()[p // 64], p % 64
    v[page, slot] = 64.0
    k[page[0], 0], v[page[0], 0] = 1.625, 0.0  # scores 0.125 * 64 * 1.625 = 13, and 0
    c.parts = [k, v]
    if e4m3:
        (kc, ke), (vc, ve) = quantise(k), quantise(v)
        c.parts = [kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn)]
        c.exps, c.e4m3 = [ke, ve], True
    q = torch.ones(T, 4, 64, dtype=c.dtype, device="cuda")
    ref, z, tol, tol_z = reference(c, q, 0.125)
    out, lse = sv.sv_chunk_attention(
        q.repeat(B, 1, 1), *c.parts, c.table.repeat(B, 1), c.cached.repeat(B),
        torch.arange(0, B * T + 1, T, dtype=torch.int32, device="cuda"), **c.exp_args(),
        scale=0.125, max_chunk=T, return_lse=True)
    # (float16 weights keep 2^-27 of the largest at least, whatever the tile's values)
    tol = tol - 2.0 ** -24 * (n + T + 127 * 64) + 2.0 ** -27 * (n + T + 127 * 64)
    err = (out.view(B, T, 4, 64).double() - ref).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert ((lse.view(B, T, 4).double() - z).abs() <= tol_z).all()


def test_page_tables_that_overlap_are_refused():
    c = Cache([4, 4], [2, 2], 2, 64, 8)
    q = make_query(c, 4, 1)
    k, v, table, cached, starts = c.args()
    with pytest.raises(ValueError):
        sv.sv_chunk_attention(q, k, v, table[:1].expand(2, -1), cached, starts)
    # (one row has no distance to a next)
    out = sv.sv_chunk_attention(q[:2], k, v, table[:1].expand(1, -1), cached[:1], starts[:2])
    assert out.isfinite().all()


@pytest.mark.parametrize("dtype,e4m3", TYPES)
@pytest.mark.parametrize("d", [144, 192, 208, 256])
def test_large_heads(dtype, e4m3, d):
    """Head sizes past 128: 16 rows at a time, whatever the chunk is."""
    run([0, 7, 250, 1025], [5, 1, 70, 4], 2, 4, d, 16, dtype, e4m3, seed=d)
    run([3, 500], [1, 1], 1, 16, d, 128, dtype, e4m3, True, seed=d, max_chunk=1)
    run([40, 700, 129], [9, 33, 4], 2, 3, d, 64, dtype, e4m3, window=100, seed=d)
    run([9000, 20011], [3, 6], 1, 8, d, 64, dtype, e4m3, seed=d, max_chunk=6)
    run([6000, 4100, 777], [17] * 3, 8, 4, d, 64, dtype, e4m3, seed=d, max_chunk=17)


@pytest.mark.parametrize("dtype,e4m3", TYPES)
@pytest.mark.parametrize("fill", [math.nan, math.inf])
def test_large_heads_unused_slots_have_no_influence(dtype, e4m3, fill):
    run([3, 100, 130, 517], [1, 9, 6, 40], 2, 4, 256, 16, dtype, e4m3, fill=fill)


@pytest.mark.parametrize("dtype,e4m3", TYPES)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_large_heads_masked_values_have_no_influence(dtype, e4m3, bad):
    """A bad value of a late position: rows before it do not see it, those from it on do."""
    lens, T, at = 300, 12, 305
    c = Cache([lens], [T], 2, 256, 16, dtype, False)
    c.parts[1][c.table[0, at // 16], at % 16, :, 3] = bad
    if e4m3:
        for i in range(2):
            code, c.exps[i] = quantise(c.parts[i])
            c.parts[i] = code.view(torch.float8_e4m3fn)
        c.e4m3 = True
    q = make_query(c, 4, 2)
    out, lse = attend(c, q, max_chunk=T)
    check(out, lse, c, q, 256 ** -0.5, rows=slice(0, at - lens))
    assert not out[at - lens:, :, 3].isfinite().any()


def test_large_heads_bad_pages():
    c = Cache([300, 200], [20, 20], 2, 256, 16)
    q = make_query(c, 4, 2)
    c.table[0, 3] = 10 ** 6
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = sv.sv_chunk_attention(q, *c.args(), seq_status=status, max_chunk=20)
    assert status.tolist() == [sv.SV_SEQ_BAD_PAGE, 0]
    assert out[:20].isnan().all() and out[20:].isfinite().all()


@pytest.mark.parametrize("T", [1, 30])
def test_strides_of_single_elements_are_not_looked_at(T):
    """One head, one page and one token with whatever stride torch may have left there."""
    c = Cache([40 - T], [T], 1, 64, 64, "bf16", False, spare=0)
    q, x = make_query(c, 1, 1), make_query(c, 1, 2)
    want = sv.sv_chunk_attention(q, *c.args(), max_chunk=T)

    def odd(t):
        st = list(t.stride())
        for i, n in enumerate(t.shape):
            if n == 1:
                st[i] = (1 << 39) + 3
        return t.as_strided(t.shape, st)

    k, v = (odd(t) for t in c.parts)
    assert k.stride(0) == k.stride(2) == (1 << 39) + 3
    out = sv.sv_chunk_attention(odd(q), k, v, *c.args()[2:], max_chunk=T)
    assert torch.equal(out, want)
    sv.sv_kv_append(odd(x), odd(q), k, v, *c.args()[2:])
    key, value = sv.sv_kv_read(k, v, *c.args()[2:], T)
    assert torch.equal(key, x) and torch.equal(value, q)


@pytest.mark.parametrize("dtype,e4m3", TYPES)
@pytest.mark.parametrize("T", [1, 30])
def test_a_cache_without_pages(dtype, e4m3, T):
    c = Cache([8, 8, 0, 0], [T, 0, T, T], 2, 64, 8, dtype, e4m3, seed=9)
    q = make_query(c, 4, 8)
    for i in range(2):
        c.parts[i] = c.parts[i][:0]
        c.exps[i] = c.exps[i][:0] if e4m3 else None
    c.cached[3] = -1
    status = torch.full((4,), 99, dtype=torch.int32, device="cuda")
    out, lse = attend(c, q, seq_status=status)
    assert status.tolist() == [sv.SV_SEQ_BAD_PAGE, 0, sv.SV_SEQ_BAD_PAGE, sv.SV_SEQ_BAD_LENGTH]
    assert out.isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("T", [1, 30])
def test_pages_and_heads_that_share_memory(T):
    """Strides of zero: every page, or every head, is the same."""
    c = Cache([200], [T], 2, 64, 16, "bf16", False, seed=9)
    q = make_query(c, 4, 8)
    for kind in ("pages", "heads"):
        k, v = ((x[:1].expand(x.shape) if kind == "pages" else x[:, :, :1].expand(x.shape))
                for x in c.parts)
        out = sv.sv_chunk_attention(q, k, v, *c.args()[2:], max_chunk=T)
        want = sv.sv_chunk_attention(q, k.contiguous(), v.contiguous(), *c.args()[2:], max_chunk=T)
        assert torch.equal(out, want)


def with_page_0_unused(*args, **kw):
    """A cache whose page 0, which takes the place of pages out of range, is a spare one."""
    for seed in range(100):
        c = Cache(*args, seed=seed, spare=20, **kw)
        if 0 in c.unused:
            return c


@pytest.mark.parametrize("dtype,e4m3", TYPES)
@pytest.mark.parametrize("T,d", [(4, 64), (4, 128), (20, 128), (75, 64), (75, 128), (12, 256)])
@pytest.mark.parametrize("at,window", [(304, 0), (288, 10), (256, 40), (307, 3)])
def test_a_bad_page_reaches_only_the_rows_that_see_it(dtype, e4m3, T, d, at, window):
    """A page out of range among the new tokens' own, or one that the window passes."""
    c = with_page_0_unused([300, 4000], [T, T], 2, d, 16, dtype, e4m3, fill=math.inf)
    q = make_query(c, 4, 1)
    for b, shift in ((0, 0), (1, 3696)):
        c.table[b, (at + shift) // 16] = 10 ** 6
    status = torch.empty(2, dtype=torch.int32, device="cuda")
    out, lse = attend(c, q, window, max_chunk=T, seq_status=status)
    lo, hi = at // 16 * 16, at // 16 * 16 + 15  # the page's positions (of sequence 0)
    seen = torch.tensor([p >= lo and (window == 0 or p - window + 1 <= hi)
                         for p in range(300, 300 + T)]).repeat(2)
    # (sequence 1's positions are 3700 on, and its page's 3696 further: 3996 and so on)
    first = 4000 - 300 - 3696
    for t in range(T):
        p = 4000 + t - 3696
        seen[T + t] = p >= lo and (window == 0 or p - window + 1 <= hi)
    assert first == 4
    assert status.tolist() == [sv.SV_SEQ_BAD_PAGE if seen[b * T:b * T + T].any() else 0
                               for b in range(2)]
    assert out[seen.cuda()].isnan().all() and lse[seen.cuda()].isnan().all()
    good = (~seen).nonzero().squeeze(1).cuda()
    if len(good):
        for b in range(2):  # (never read by the good rows: any page will do for the reference)
            c.table[b, (at + (0, 3696)[b]) // 16] = c.unused[0]
        check(out, lse, c, q, d ** -0.5, window, rows=good)


@pytest.mark.parametrize("T", [1, 20])
def test_windows_longer_than_30_bits(T):
    """A window of 2^30 + 2^29 positions on two pages, one of which is nearly all of them; weights are
    all alike but for a key right before the first row's window and one that the first rows see."""
    window, P = (1 << 30) + (1 << 29), 1024
    low = (1 << 28) + 500
    cached = low + window - 1
    assert low % P == 500 and 500 % 128 < 124 and cached + T < 1 << 31
    pages = torch.zeros(2, P, 1, 16, device="cuda").bfloat16()
    values = torch.ones_like(pages)
    pages[1, 499], pages[1, 503] = 8.0, 8.0  # scores of 32 under queries of ones
    values[1, 499], values[1, 503] = 100.0, 5.0
    table = torch.zeros(1, 1 << 21, dtype=torch.int32, device="cuda")
    table[0, low // P] = 1
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.ones(T, 1, 16, device="cuda").bfloat16()
    out, lse = sv.sv_chunk_attention(q, pages, values, table, torch.tensor([cached], **i32),
                                     torch.tensor([0, T], **i32), window=window, max_chunk=T,
                                     return_lse=True)
    # Row t sees position low + t on: the key of 32 at low + 3 weighs e^32 = 8e13 against 1.6e9.
    for t in range(T):
        want = 5.0 if t <= 3 else 1.0
        assert (out[t].float() - want).abs().max() <= 2.0 ** -8 * want + 4.0 * window / math.exp(32)
        assert abs(float(lse[t, 0]) - (32.0 if t <= 3 else math.log(window))) < 1e-3
