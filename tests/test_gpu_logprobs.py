"""Log probabilities of given tokens, entropy, ranks and top alternatives, and their gradient,
against the plain form in 64 bits."""
import math

import pytest
import torch

import logprobs_util as u
import speculative_decoding_verification_66_gb300 as sv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_logprobs()
    torch.cuda.set_device(0)


def draw(shape, dtype, seed=0, spread=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * spread).to(u.DTYPES[dtype])


def draw_tokens(shape, V, seed=1, skip=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randint(0, V, shape, generator=g, device="cuda", dtype=torch.int32)
    return torch.where(torch.rand(shape, generator=g, device="cuda") < skip, -1, t)


def call(x, tokens, temperature=1.0, k=0):
    status = torch.full(x.shape[:-1], 77, dtype=torch.int32, device="cuda")
    r = sv.sv_token_logprobs(x, tokens, temperature=temperature, top_k=k, row_status=status)
    return u.check_logprobs(x, tokens, temperature, k, r, status), r


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 5, 8, 31, 255, 256, 257, 1000, 2049, 4099, 12345, 32003, 50001])
def test_vocabularies(dtype, V):
    for rows, k in ((1, 1), (3, 20), (40, 0), (17, 128)):
        x = draw((rows, V), dtype, V + rows)
        call(x, draw_tokens((rows,), V), 0.7, min(k, V))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 2, 75, 152, 153, 400])
def test_rows_of_large_vocabularies(dtype, rows):
    x = draw((rows, 128256), dtype, rows)
    call(x, draw_tokens((rows,), 128256), 1.0, 20)


def test_the_largest_vocabulary_with_alternatives():
    for dtype in ("bf16", "f32"):
        x = draw((2, 1 << 20), dtype)
        call(x, draw_tokens((2,), 1 << 20, skip=0), 1.0, 128)


def test_a_vocabulary_beyond_that_without():
    x = draw((2, (1 << 20) + 77), "bf16")
    call(x, draw_tokens((2,), x.shape[1], skip=0))
    with pytest.raises(sv.SpecVerifyError) as e:
        sv.sv_token_logprobs(x, top_k=1)
    assert e.value.code == -6


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "f32"])
def test_ties_go_to_the_lowest_index(dtype):
    V = 9001
    rows = [torch.zeros(V), torch.arange(V) % 3, -(torch.arange(V) % 700).float(),
            torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0), torch.arange(V) // 64]
    x = torch.stack([r.float() for r in rows]).to(u.DTYPES[dtype]).cuda()
    for t in (0, 1, 4500, V - 1):
        call(x, torch.full((len(rows),), t, dtype=torch.int32, device="cuda"), 1.0, 128)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "f32"])
@pytest.mark.parametrize("V", [300, 40000])
def test_orders_and_crowds(dtype, V):
    """Rows in order either way, the largest all in one place, and few distinct values."""
    base = draw((V,), dtype, 3).float().sort().values
    crowd = draw((V,), dtype, 4).float()
    crowd[V // 2:V // 2 + 200] += 30.0
    late = torch.full((V,), -5.0, device="cuda")
    late[-130:] = torch.arange(130, device="cuda").float() / 16
    x = torch.stack([base, base.flip(0), crowd, late, (base * 2).round() / 2]).to(u.DTYPES[dtype])
    for k in (1, 7, 128):
        call(x, draw_tokens((5,), V, skip=0), 1.0, k)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "f32"])
def test_masked_and_extreme_logits(dtype):
    V, big = 5003, float(torch.finfo(u.DTYPES[dtype]).max)
    x = draw((12, V), dtype, 5)
    x[0, 100:] = -math.inf                      # most of the vocabulary masked
    x[1] = -math.inf
    x[1, 4000] = 3.0                            # all but one
    x[2, ::2] = -big                            # masked by the type's lowest value
    x[3] = -big
    x[3, 7] = big                               # both ends
    x[4] = -big                                 # nothing but the lowest value
    x[5, 17] = math.nan
    x[6, 5002] = math.inf
    x[7] = -math.inf                            # nothing left
    x[8, 0] = -math.nan
    x[9] += 1000.0                              # far from zero
    x[10] *= 1000.0
    x[11, :] = 0.0
    x[11, 2500] = 80.0                          # certain
    tokens = torch.tensor([50, 4000, 1, 7, 0, 17, 3, 5, 1, 2, 3, 2500], dtype=torch.int32,
                          device="cuda")
    w, _ = call(x, tokens, 1.0, 128)
    assert w["status"].tolist() == [0, 0, 0, 0, 0, 2, 2, 2, 2, 0, 0, 0]
    tokens[0], tokens[1] = 200, 0               # masked tokens: log probability -inf
    w, r = call(x, tokens, 0.5, 20)
    assert r.logprobs[0] == -math.inf and r.logprobs[1] == -math.inf
    call(x, torch.full_like(tokens, -1), 1.0, 5)
    call(x, None, 30.0, 5)


def test_tokens_out_of_range():
    x = draw((6, 700), "bf16")
    tokens = torch.tensor([-2, 700, 699, 0, -1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    w, r = call(x, tokens, 1.0, 3)
    assert w["status"].tolist() == [1, 1, 0, 0, 0, 1]


def test_sizes_of_nothing():
    for shape in ((0, 50), (3, 0, 50), (0, 4, 50)):
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        r = sv.sv_token_logprobs(x, torch.empty(shape[:-1], dtype=torch.int32, device="cuda"),
                                 top_k=3)
        assert r.logprobs.shape == shape[:-1] and r.top_tokens.shape == (*shape[:-1], 3)
    r = sv.sv_token_logprobs(draw((50,), "f32"), top_k=2)
    assert r.entropy.shape == () and r.top_tokens.shape == (2,) and r.logprobs is None


def layouts(dtype, V):
    """Tensors of rows that begin anywhere."""
    base = draw((5, 6, V + 40), dtype, 9)
    yield base[..., :V]                              # a padded vocabulary
    yield base[:, :4, :V]                            # some positions
    yield base[..., 1:V + 1]                         # off by one element
    yield base[..., 7:V + 7].transpose(0, 1)         # rows in another order
    yield base[2, :, 3:V + 3]
    yield base[1:2, 1:2, 5:V + 5]
    yield base[0, 0, 2:V + 2]
    yield base[0, :1, :V].expand(7, V)               # one row, many times
    yield draw((5, 3, V), dtype, 10)
    yield draw((64 * 1024 + V,), dtype, 11).as_strided((9, V), (V // 2 + 1, 1))  # overlapping rows


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "f32"])
@pytest.mark.parametrize("V", [33, 2048, 10007])
def test_strides_and_alignments(dtype, V):
    for x in layouts(dtype, V):
        tokens = draw_tokens(x.shape[:-1], V)
        call(x, tokens, 1.3, 10)
        y = x.detach().requires_grad_()
        r = sv.sv_token_logprobs(y, tokens, temperature=1.3)
        a, b, c = (torch.randn(x.shape[:-1], device="cuda") for _ in range(3))
        g, = torch.autograd.grad((r.logprobs, r.entropy, r.lse), y, (a, b, c))
        check_gradient(g, x, tokens, a, b, c, 1.3)


def check_gradient(g, x, tokens, a, b, c, temperature):
    V = x.shape[-1]
    flat = x.detach().reshape(-1, V)
    f = [None if t is None else t.reshape(-1) for t in (tokens, a, b, c)]
    want = u.logprobs_grad(flat, *f, temperature)
    w = u.logprobs(flat, f[0], temperature)
    H = torch.where(w["entropy"].isfinite(), w["entropy"], 0.0)

    def size(t):
        return 0.0 if t is None else t.double().abs()[:, None]

    far = torch.where(w["p"] > 0, w["logp"].abs(), 0.0) + H[:, None] + 1
    p = torch.where(w["p"].isfinite(), w["p"], 0.0)
    scale = (p * (size(f[1]) + size(f[3]) + size(f[2]) * far) * far + size(f[1]) * 1e-3) / temperature
    u.check_grad(g, want, scale, V, 8.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "f32"])
@pytest.mark.parametrize("V", [1, 3, 1000, 32003])
@pytest.mark.parametrize("which", ["a", "b", "c", "abc"])
def test_gradients(dtype, V, which):
    x = draw((37, V), dtype, V).requires_grad_()
    tokens = draw_tokens((37,), V)
    up = {n: torch.randn(37, device="cuda") if n in which else None for n in "abc"}
    r = sv.sv_token_logprobs(x, tokens, temperature=0.8)
    pairs = [(o, up[n]) for o, n in ((r.logprobs, "a"), (r.entropy, "b"), (r.lse, "c"))
             if up[n] is not None]
    g, = torch.autograd.grad([o for o, _ in pairs], x, [w for _, w in pairs])
    assert g.dtype == x.dtype and g.shape == x.shape
    check_gradient(g, x, tokens, up["a"], up["b"], up["c"], 0.8)


def test_gradients_of_masked_rows_and_bad_rows():
    x = draw((6, 3001), "f32")
    x[0, 40:] = -math.inf
    x[1, ::3] = -torch.finfo(torch.float32).max
    x[2, 5] = math.nan
    x[3] = -math.inf
    x[4, 1000] = 90.0
    tokens = torch.tensor([3, 1, 1, 1, 1000, 3001], dtype=torch.int32, device="cuda")
    x.requires_grad_()
    r = sv.sv_token_logprobs(x, tokens)
    a, b, c = (torch.randn(6, device="cuda") for _ in range(3))
    g, = torch.autograd.grad((r.logprobs, r.entropy, r.lse), x, (a, b, c))
    check_gradient(g, x, tokens, a, b, c, 1.0)
    assert g[2].isnan().all() and g[3].isnan().all() and g[5].isnan().all()
    assert (g[0, 40:] == 0).all()


def test_gradients_by_differences():
    """Central differences of the plain form: 64 bits, step 1e-4, third derivatives below 10 T^-3."""
    x = draw((4, 50), "f32", 3).requires_grad_()
    tokens = torch.tensor([3, -1, 49, 0], dtype=torch.int32, device="cuda")
    r = sv.sv_token_logprobs(x, tokens, temperature=0.9)
    (r.logprobs.sum() + 0.3 * r.entropy.sum()).backward()

    def value(y):
        w = u.logprobs(y, tokens, 0.9)
        return w["logprobs"] + 0.3 * w["entropy"]

    h, y = 1e-4, x.detach().double()
    for v in range(50):
        d = torch.zeros_like(y)
        d[:, v] = h
        slope = (value(y + d) - value(y - d)) / (2 * h)
        u.close(x.grad[:, v], slope, 1e-6, "slope")


def test_sums_and_means_and_unused_outputs():
    """Upstream gradients that are broadcast scalars, strided, or missing; no grad mode."""
    x = draw((3, 5, 700), "f32").requires_grad_()
    tokens = draw_tokens((3, 5), 700)
    r = sv.sv_token_logprobs(x, tokens)
    r.logprobs.sum().backward()
    ones = torch.ones(3, 5, device="cuda")
    check_gradient(x.grad, x, tokens, ones, None, None, 1.0)
    x.grad = None
    up = torch.randn(5, 3, device="cuda")
    r = sv.sv_token_logprobs(x, tokens, top_k=4)
    (r.entropy.t() * up).mean().backward()
    check_gradient(x.grad, x, tokens, None, up.t() / 15, None, 1.0)
    assert not r.top_logprobs.requires_grad and not r.rank.requires_grad
    with torch.no_grad():
        assert not sv.sv_token_logprobs(x, tokens).logprobs.requires_grad
    assert not sv.sv_token_logprobs(x.detach(), tokens).logprobs.requires_grad


def test_the_same_gradient_twice_and_second_derivatives_refused():
    x = draw((3, 500), "f32").requires_grad_()
    r = sv.sv_token_logprobs(x, draw_tokens((3,), 500, skip=0))
    g, = torch.autograd.grad(r.logprobs.sum(), x, retain_graph=True)
    h, = torch.autograd.grad(r.logprobs.sum(), x, retain_graph=True)
    assert torch.equal(g, h)
    g, = torch.autograd.grad(r.logprobs.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.sum(), x)


def test_backward_into_the_logits_themselves():
    x = draw((9, 3001), "bf16")
    tokens = draw_tokens((9,), 3001)
    stats = torch.empty(9, sv.SV_ROW_STATS, device="cuda")
    sv.sv_token_logprobs(x, tokens, row_stats=stats)
    a = torch.randn(9, device="cuda")
    want = sv.sv_token_logprobs_backward(x, stats, tokens=tokens, grad_logprobs=a)
    got = sv.sv_token_logprobs_backward(x, stats, tokens=tokens, grad_logprobs=a, grad=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(want, got)


def test_logits_changed_before_the_backward_pass_are_noticed():
    x = draw((3, 500), "f32").requires_grad_()
    y = x * 1.0
    r = sv.sv_token_logprobs(y, draw_tokens((3,), 500))
    y.mul_(2.0)
    with pytest.raises(RuntimeError):
        r.logprobs.sum().backward()


def test_the_same_bits_every_time():
    x = draw((60, 128256), "bf16")
    tokens = draw_tokens((60,), 128256)
    first = sv.sv_token_logprobs(x, tokens, top_k=50)
    for _ in range(3):
        for p, q in zip(first, sv.sv_token_logprobs(x, tokens, top_k=50)):
            assert torch.equal(p, q)


def test_streams():
    x = draw((30, 32003), "f32")
    tokens = draw_tokens((30,), 32003)
    want = sv.sv_token_logprobs(x, tokens, top_k=5)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sv.sv_token_logprobs(x, tokens, top_k=5, stream=side)
    y = x.detach().requires_grad_()
    r = sv.sv_token_logprobs(y, tokens, stream=side)
    side.synchronize()
    for p, q in zip(want, got):
        assert torch.equal(p, q)
    r.logprobs.sum().backward()
    z = x.detach().requires_grad_()
    sv.sv_token_logprobs(z, tokens).logprobs.sum().backward()
    torch.cuda.synchronize()
    assert torch.equal(y.grad, z.grad)


def test_captured_and_replayed():
    """Forward and backward in a graph, replayed with other logits and tokens."""
    x = draw((20, 9001), "bf16").requires_grad_()
    tokens = draw_tokens((20,), 9001)
    a = torch.randn(20, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        r = sv.sv_token_logprobs(x, tokens, top_k=7)
        torch.autograd.grad(r.logprobs, x, a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = sv.sv_token_logprobs(x, tokens, top_k=7)
        g, = torch.autograd.grad(r.logprobs, x, a)
    for seed in (5, 6):
        with torch.no_grad():
            x.copy_(draw((20, 9001), "bf16", seed))
        tokens.copy_(draw_tokens((20,), 9001, seed))
        graph.replay()
        u.check_logprobs(x.detach(), tokens, 1.0, 7, r)
        check_gradient(g, x, tokens, a, None, None, 1.0)


def test_refusals():
    x = draw((4, 100), "bf16")
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    bad = [dict(tokens=t.long()), dict(tokens=t[:3]), dict(tokens=t.cpu()), dict(top_k=101),
           dict(top_k=-1), dict(row_status=t.float()), dict(row_stats=t)]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            sv.sv_token_logprobs(x, **kw)
    for T in (0.0, -1.0, math.inf, math.nan, 1e-39):
        with pytest.raises((sv.SpecVerifyError, OverflowError)):
            sv.sv_token_logprobs(x, temperature=T)
    for y in (x.t(), x.double(), x.int(), x[None, None], x[:, :0], x.cpu()):
        with pytest.raises((ValueError, TypeError)):
            sv.sv_token_logprobs(y)
    stats = torch.zeros(4, sv.SV_ROW_STATS, device="cuda")
    with pytest.raises(ValueError):
        sv.sv_token_logprobs_backward(x, stats, grad=x[:, 1:])
    big = draw((5, 100), "bf16")
    with pytest.raises(ValueError):  # overlaps the logits in part
        sv.sv_token_logprobs_backward(big[:4], stats, grad=big[1:])
    with pytest.raises(sv.SpecVerifyError):  # rows of the gradient overlap
        sv.sv_token_logprobs_backward(x, stats, grad=torch.empty(1, 100, device="cuda",
                                                                 dtype=x.dtype).expand(4, 100))
    with pytest.raises(sv.SpecVerifyError):  # a gradient of log probabilities of no tokens
        sv.sv_token_logprobs_backward(x, stats, grad_logprobs=stats[:, 0].contiguous())


@pytest.mark.parametrize("dtype,rows,V", [("bf16", 70000, 300), ("f32", 66000, 130), ("bf16", 5000, 40000),
                                          ("fp16", 700, 70001), ("f32", 1300, 33001),
                                          ("bf16", 2500, 66000)])
def test_many_rows(dtype, rows, V):
    """More rows than are cut into pieces, rows of more turns than one piece has, and rows in two."""
    x = draw((rows, V), dtype, V)
    tokens = draw_tokens((rows,), V)
    status = torch.full((rows,), 77, dtype=torch.int32, device="cuda")
    r = sv.sv_token_logprobs(x, tokens, temperature=0.9, top_k=11, row_status=status)
    step = max(1, 20_000_000 // V)
    for i in list(range(0, rows, step))[::4] + [rows - step]:
        s = slice(max(i, 0), max(i, 0) + step)
        part = sv.TokenLogprobs(*(t[s] for t in r))
        u.check_logprobs(x[s], tokens[s], 0.9, 11, part, status[s])


def test_tokens_around_turns_and_pieces():
    """Tokens on both sides of every boundary of a turn of 1024 elements, tied with their
    neighbours."""
    V = 20 * 1024 + 5
    row = (torch.arange(V) // 3 % 50).float()
    tokens = torch.tensor([t + d for t in range(0, V, 1024) for d in (-1, 0, 1)][1:],
                          dtype=torch.int32, device="cuda")
    for offset in (0, 3):
        base = torch.zeros(V + 8, device="cuda", dtype=torch.bfloat16)
        base[offset:offset + V] = row
        x = base[offset:offset + V].expand(len(tokens), V)
        call(x, tokens, 1.0, 3)


def test_a_given_workspace():
    """Calls of different sizes share one; its counters are zeros between them."""
    big, small = draw((40, 128256), "bf16"), draw((9, 20000), "f32")
    n = max(sv.sv_logprobs_workspace_bytes(40, 128256, torch.bfloat16, 20),
            sv.sv_logprobs_workspace_bytes(9, 20000, torch.float32, 20))
    w = torch.full((n,), 123, dtype=torch.uint8, device="cuda")
    w[:sv.SV_LOGPROBS_COUNTER_BYTES] = 0
    for x in (big, small, big, small):
        tokens = draw_tokens(x.shape[:1], x.shape[1])
        r = sv.sv_token_logprobs(x, tokens, top_k=20, workspace=w)
        u.check_logprobs(x, tokens, 1.0, 20, r)
        assert (w[:sv.SV_LOGPROBS_COUNTER_BYTES] == 0).all()
        ids = r.top_tokens.clone()
        loss, grad = sv.sv_distill(x, ids, r.top_logprobs, tail="bucket", workspace=w)
        assert loss.abs().max() < 1e-4
        assert (w[:sv.SV_LOGPROBS_COUNTER_BYTES] == 0).all()
    for bad in (w.float(), w.cpu(), w[::2]):
        with pytest.raises(ValueError):
            sv.sv_token_logprobs(big, workspace=bad)
    with pytest.raises(sv.SpecVerifyError) as e:
        sv.sv_token_logprobs(big, top_k=20, workspace=w[:1024])
    assert e.value.code == -4


def test_two_streams_and_two_graphs_at_once():
    """Calls on two streams and replays of two graphs run beside one another; each has its own
    workspace."""
    xs = [draw((60, 128256), "bf16", s) for s in (1, 2)]
    tokens = [draw_tokens((60,), 128256, s) for s in (3, 4)]
    want = [sv.sv_token_logprobs(x, t, top_k=20) for x, t in zip(xs, tokens)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append(sv.sv_token_logprobs(xs[i], tokens[i], top_k=20, stream=streams[i]))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(sv.sv_token_logprobs(xs[i], tokens[i], top_k=20))
        graphs.append(graph)
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i] + [outs[i]]:
            for p, q in zip(want[i], r):
                assert torch.equal(p, q)


def test_a_captured_gradient_beside_an_eager_graph_of_the_same_leaf():
    x = draw((20, 9001), "f32").requires_grad_()
    tokens = draw_tokens((20,), 9001)
    a = torch.randn(20, device="cuda")
    alive = sv.sv_token_logprobs(x, tokens)
    want, = torch.autograd.grad(alive.logprobs, x, a, retain_graph=True)
    stats = torch.empty(20, sv.SV_ROW_STATS, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with torch.no_grad():
            sv.sv_token_logprobs(x, tokens, row_stats=stats)
            got = sv.sv_token_logprobs_backward(x.detach(), stats, tokens=tokens, grad_logprobs=a)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    again, = torch.autograd.grad(alive.logprobs, x, a)
    assert torch.equal(again, want)


def test_inputs_changed_before_the_backward_pass_are_noticed():
    x = draw((3, 500), "f32").requires_grad_()
    tokens = draw_tokens((3,), 500)
    r = sv.sv_token_logprobs(x, tokens)
    tokens.add_(0)
    with pytest.raises(RuntimeError):
        r.logprobs.sum().backward()


def test_what_a_call_overwrites_is_noticed():
    x = draw((3, 500), "f32").requires_grad_()
    tokens = draw_tokens((3,), 500)
    stats = torch.empty(3, sv.SV_ROW_STATS, device="cuda")
    r = sv.sv_token_logprobs(x, tokens, row_stats=stats)
    sv.sv_token_logprobs(x.detach() * 2.0, tokens, row_stats=stats)
    with pytest.raises(RuntimeError):
        r.logprobs.sum().backward()
    y = x * 1.0
    r = sv.sv_token_logprobs(y, tokens, row_stats=stats)
    sv.sv_token_logprobs_backward(y, stats, tokens=tokens, grad_lse=torch.ones(3, device="cuda"), grad=y)
    with pytest.raises(RuntimeError):
        r.logprobs.sum().backward()


def test_tokens_made_in_inference_mode():
    x = draw((3, 500), "f32").requires_grad_()
    with torch.inference_mode():
        tokens = draw_tokens((3,), 500, skip=0.0)
        stats = torch.empty(3, sv.SV_ROW_STATS, device="cuda")
        sv.sv_token_logprobs(x, tokens, row_stats=stats)
    grads = []
    for t, s in ((tokens, stats), (tokens.clone(), None)):
        x.grad = None
        sv.sv_token_logprobs(x, t, row_stats=s).logprobs.sum().backward()
        grads.append(x.grad)
    assert torch.equal(*grads)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [21, 304, 305, 608, 609])
def test_alternatives_by_blocks_of_any_size(dtype, rows):
    """Many and few alternatives by blocks of 4 to 16 warps; rows of ties among the others."""
    V = 50001
    x = draw((rows, V), dtype, rows)
    x[::7] = (x[::7] * 2).round()
    x[5::50, 100:] = -math.inf
    tokens = draw_tokens((rows,), V)
    for k in (3, 128):
        call(x, tokens, 0.9, k)
