"""Distillation from a teacher's top logits, loss and gradient, against the plain form in 64 bits."""
import math

import pytest
import torch

import logprobs_util as u
import speculative_decoding_verification_66_gb300 as sv
from test_gpu_logprobs import layouts

pytestmark = pytest.mark.gpu

TAILS = ["renormalise", "bucket"]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_logprobs()
    torch.cuda.set_device(0)


def teacher(shape, V, k, seed=0, missing=0.1, none=0.15, temperature=1.0):
    """Top alternatives of rows that the student's are near to, entries and rows missing here and
    there. The student's logits, and (ids, log probabilities)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((*shape, V), generator=g, device="cuda") * 2.5
    lp, ids = torch.log_softmax(x.double() / temperature, -1).topk(k, -1)
    lp, ids = lp.float(), ids.int()
    gone = torch.rand(ids.shape, generator=g, device="cuda") < missing
    gone |= (torch.rand(shape, generator=g, device="cuda") < none)[..., None]
    ids[gone], lp[gone] = -1, -math.inf
    return 0.8 * x + torch.randn(x.shape, generator=g, device="cuda"), ids, lp


def check(x, ids, lp, temperature, tail, loss, grad, weights=None, status=None):
    V, k = x.shape[-1], ids.shape[-1]
    flat = x.detach().reshape(-1, V)
    want, g, st = u.distill(flat, ids.reshape(-1, k), lp.reshape(-1, k), temperature, tail)
    if status is not None:
        assert torch.equal(status.reshape(-1), st)
    if loss is not None:
        assert loss.dtype == torch.float32 and loss.shape == x.shape[:-1]
        # The entries' probabilities are off by 2 u, their logarithms by u and the sums' tolerance;
        # log q by its distance from the row's mean, of some 20; the sum of the others' too.
        P = torch.where(ids >= 0, lp.double(), -math.inf).reshape(-1, k)
        mean = torch.where(P.isfinite(), P.abs(), 0.0).amax(-1).clamp(max=200.0)
        tol = u.sum_tol(V, 8.0) + 4 * u.U * (mean + 20 + torch.where(want.isfinite(), want.abs(), 0.0))
        u.close(loss.detach().reshape(-1), want, tol, "loss")
    if grad is not None:
        assert grad.dtype == x.dtype and grad.shape == x.shape
        w = torch.ones(flat.shape[0], device="cuda") if weights is None else weights.reshape(-1)
        bad = (st != 0)[:, None]
        g = torch.where(bad, math.nan, g * w.double()[:, None])
        q = torch.log_softmax(flat.double() / temperature, -1).exp()
        scale = (torch.where(q.isfinite(), q, 0.0) * 20 + torch.where(g.isfinite(), g.abs(), 0.0)) \
            * w.double().abs()[:, None].clamp(min=1.0) / min(1.0, temperature)
        u.check_grad(grad, g, scale, V, 8.0)


def both(x, ids, lp, temperature=1.0, tail="renormalise", weights=None):
    """In one call, and through autograd."""
    status = torch.full(x.shape[:-1], 55, dtype=torch.int32, device="cuda")
    loss, grad = sv.sv_distill(x, ids, lp, weights=weights, temperature=temperature, tail=tail,
                               row_status=status)
    check(x, ids, lp, temperature, tail, loss, grad, weights, status)
    y = x.detach().requires_grad_()
    status.fill_(55)
    loss = sv.sv_distill_loss(y, ids, lp, temperature=temperature, tail=tail, row_status=status)
    up = torch.ones(x.shape[:-1], device="cuda") if weights is None else weights
    g, = torch.autograd.grad(loss, y, up)
    check(x, ids, lp, temperature, tail, loss, g, up, status)
    return loss, g


@pytest.mark.parametrize("tail", TAILS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 257, 1000, 4099, 32003, 50001])
def test_vocabularies(dtype, V, tail):
    for rows, k in ((1, 1), (33, 20), (5, 128)):
        x, ids, lp = teacher((rows,), V, min(k, V), V + rows)
        both(x.to(u.DTYPES[dtype]), ids, lp, 0.8, tail,
             torch.rand(rows, device="cuda") if rows > 1 else None)


@pytest.mark.parametrize("tail", TAILS)
@pytest.mark.parametrize("dtype,rows,V", [("bf16", 1, 128256), ("bf16", 200, 128256),
                                          ("f32", 40, 152064), ("f32", 3, 300001),
                                          ("fp16", 2, 1 << 20), ("f32", 1, 1 << 20)])
def test_large_vocabularies(dtype, rows, V, tail):
    x, ids, lp = teacher((rows,), V, 64, rows)
    both(x.to(u.DTYPES[dtype]), ids, lp, 1.0, tail)


@pytest.mark.parametrize("tail", TAILS)
def test_tokens_given_twice_add_up(tail):
    V = 5003
    x, ids, lp = teacher((6,), V, 40, 3, none=0.0)
    ids[0] = ids[0, 0].clone()               # one token forty times
    ids[1, 20:] = ids[1, :20]                # each twice
    ids[2, 39] = ids[2, 0]
    ids[3, 1:] = -1                          # one entry
    ids[4, :39] = -1
    ids[5] = torch.tensor([V - 1, 0] * 20, dtype=torch.int32)
    lp[:] = lp.clamp(min=-30.0)              # (no missing entry's -inf beside a token)
    both(x, ids, lp, 1.0, tail)
    both(x.bfloat16(), ids, lp, 2.0, tail)


@pytest.mark.parametrize("tail", TAILS)
@pytest.mark.parametrize("V", [1, 3, 100, 128])
def test_all_tokens_have_entries(V, tail):
    x, ids, lp = teacher((20,), V, V, V, missing=0.0, none=0.0)
    loss, g = both(x, ids, lp, 1.0, tail)
    both(x, ids.flip(-1).contiguous(), lp.flip(-1).contiguous(), 1.0, tail)
    # A teacher that is the student: nothing to learn.
    y = torch.log_softmax(x.double(), -1).gather(-1, ids.long()).float()
    loss, g = both(x, ids, y, 1.0, tail)
    assert loss.abs().max() < 1e-5 and g.abs().max() < 1e-5


@pytest.mark.parametrize("tail", TAILS)
def test_probabilities_at_their_ends(tail):
    V = 3001
    x, ids, lp = teacher((9,), V, 5, 8, missing=0.0, none=0.0)
    lp[0] = torch.tensor([0.0, -math.inf, -math.inf, -math.inf, -math.inf])   # certain
    lp[1] = -math.inf                                                         # of nothing
    lp[2] = torch.tensor([-300.0, -301.0, -1e30, -math.inf, -302.0])          # next to nothing
    lp[3] = torch.tensor([-1e-7, -20.0, -21.0, -22.0, -23.0])                 # nearly certain
    lp[4] = torch.log(torch.tensor([0.5, 0.5, 0.25, 0.25, 0.1]))              # more than 1
    lp[5] = torch.tensor([5.0, 4.0, 30.0, 2.0, 1.0])                          # logits
    x[6, ids[6, 0].long()] = 60.0                                             # a certain student
    x[7] -= 500.0
    x[8, ids[8, 1].long()] = -80.0
    if tail == "bucket":
        lp[5] = -1.0
    both(x, ids, lp, 1.0, tail)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "f32"])
@pytest.mark.parametrize("tail", TAILS)
def test_masked_students(dtype, tail):
    V = 5003
    x, ids, lp = teacher((8,), V, 20, 8, missing=0.0, none=0.0)
    x = x.to(u.DTYPES[dtype])
    low = -float(torch.finfo(u.DTYPES[dtype]).max)
    x[0, 3000:] = -math.inf
    x[1, ids[1].long()] = -math.inf          # what the teacher wants is impossible: infinite
    x[2] = -math.inf
    x[3, 11] = math.nan
    x[4, 12] = math.inf
    x[5, :2000] = low
    x[6] = low
    keep = x[7, ids[7].long()].clone()       # nothing but the entries left
    x[7] = -math.inf
    x[7, ids[7].long()] = keep
    lp[7] -= torch.logsumexp(lp[7].double(), -1).float() + 1e-3
    ids[0] = torch.where(ids[0] < 3000, ids[0], -1)
    n = 8 if tail == "renormalise" else 7
    both(x[:n], ids[:n], lp[:n], 1.0, tail)
    if tail == "bucket":
        # The others' probability is 0 and should not be: infinite, and no gradient through it.
        loss, grad = sv.sv_distill(x[7:], ids[7:], lp[7:], tail=tail)
        assert loss.item() == math.inf and grad.isfinite().all()


def test_bad_teachers():
    V = 4001
    x, ids, lp = teacher((8,), V, 6, 4, missing=0.0, none=0.0)
    ids[0, 3] = V
    ids[1, 0] = -2
    ids[2, 5] = 2 ** 31 - 1
    lp[3, 2] = math.nan
    lp[4, 2] = math.inf
    lp[5, 1], ids[5, 1] = math.nan, -1
    ids[6], lp[6] = -1, math.nan             # what log probabilities of a bad row give
    for tail in TAILS:
        loss, g = both(x, ids, lp, 1.0, tail)
        assert loss[:7].isnan().all() and loss[7].isfinite() and g[6].isnan().all()


def test_rows_without_a_teacher_are_not_read():
    x, ids, lp = teacher((4,), 2000, 6, 4, missing=0.0, none=0.0)
    ids[1], lp[1] = -1, -math.inf
    x[1] = math.nan
    loss, g = both(x, ids, lp)
    assert loss[1] == 0 and (g[1] == 0).all()


@pytest.mark.parametrize("tail", TAILS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "f32"])
@pytest.mark.parametrize("V", [33, 2048, 10007])
def test_strides_and_alignments(dtype, V, tail):
    for x in layouts(dtype, V):
        _, ids, lp = teacher(x.shape[:-1], V, 10, 5)
        both(x, ids, lp, 1.3, tail, torch.rand(x.shape[:-1], device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [2048, 10007])
def test_gradients_of_any_layout(dtype, V):
    x, ids, lp = teacher((4, 3), V, 10, 5)
    x = x.to(u.DTYPES[dtype])
    room = torch.full((4, 3, V + 40), 7.0, dtype=x.dtype, device="cuda")
    outs = [room[..., 3:V + 3], room[..., 8:V + 8],
            torch.full((3, 4, V), 7.0, dtype=x.dtype, device="cuda").transpose(0, 1)]
    for grad in outs:
        loss, g = sv.sv_distill(x, ids, lp, grad=grad)
        assert g is grad
        check(x, ids, lp, 1.0, "renormalise", loss, g)
        stats = torch.empty(4, 3, sv.SV_ROW_STATS, device="cuda")
        w = torch.rand(4, 3, device="cuda")
        sv.sv_distill(x, ids, lp, row_stats=stats)
        g = sv.sv_distill_backward(x, ids, lp, stats, w, grad=grad)
        check(x, ids, lp, 1.0, "renormalise", None, g, w)
    # What lies between the rows is left as it was.
    room.fill_(7.0)
    sv.sv_distill(x, ids, lp, grad=room[..., 3:V + 3])
    assert (room[..., :3] == 7).all() and (room[..., V + 3:] == 7).all()


@pytest.mark.parametrize("dtype,V", [("bf16", 3001), ("bf16", 128256), ("f32", 300001)])
@pytest.mark.parametrize("tail", TAILS)
def test_into_the_logits_themselves(dtype, V, tail):
    x, ids, lp = teacher((5,), V, 30, 2)
    x = x.to(u.DTYPES[dtype])
    y = x.clone()
    loss, grad = sv.sv_distill(y, ids, lp, tail=tail, grad=y)
    assert grad.data_ptr() == y.data_ptr()
    check(x, ids, lp, 1.0, tail, loss, grad)
    l2, g2 = sv.sv_distill(x, ids, lp, tail=tail)
    assert torch.equal(l2, loss) and torch.equal(g2, grad)


@pytest.mark.parametrize("tail", TAILS)
def test_gradients_by_differences(tail):
    """Central differences of the plain form, as for the log probabilities."""
    x, ids, lp = teacher((4,), 60, 9, 3, none=0.0)
    ids[1, 3] = ids[1, 0]
    lp[1, 3] = -2.0
    loss, g = sv.sv_distill(x, ids, lp, temperature=0.9, tail=tail)
    y, h = x.double(), 1e-4
    for v in range(60):
        d = torch.zeros_like(y)
        d[:, v] = h
        slope = (u.distill(y + d, ids, lp, 0.9, tail)[0] - u.distill(y - d, ids, lp, 0.9, tail)[0]) \
            / (2 * h)
        u.close(g[:, v], slope, 1e-6, "slope")


def test_sums_and_strided_upstream_gradients():
    x, ids, lp = teacher((3, 4), 700, 5, 1)
    x.requires_grad_()
    sv.sv_distill_loss(x, ids, lp).mean().backward()
    check(x, ids, lp, 1.0, "renormalise", None, x.grad, torch.full((3, 4), 1 / 12, device="cuda"))
    x.grad = None
    w = torch.rand(4, 3, device="cuda")
    (sv.sv_distill_loss(x, ids, lp).t() * w).sum().backward()
    check(x, ids, lp, 1.0, "renormalise", None, x.grad, w.t().contiguous())
    with torch.no_grad():
        assert not sv.sv_distill_loss(x, ids, lp).requires_grad


def test_small_divergences_keep_their_digits():
    """A warm student next to the teacher, one entry, the rest one outcome: losses of 10^-5 from
    numbers near 10. Off by the probabilities' roundings and the sums', at most."""
    V = 32003
    x, ids, lp = teacher((200,), V, 1, 6, missing=0.0, none=0.0, temperature=3.0)
    loss, _ = sv.sv_distill(x, ids, lp, temperature=3.0, tail="bucket")
    want, _, _ = u.distill(x, ids, lp, 3.0, "bucket")
    P = lp.double().exp().amax()
    assert want.median() < 1e-2
    u.close(loss, want, 64 * u.sum_tol(V, 8.0) * float(P), "loss")


def test_streams():
    x, ids, lp = teacher((30,), 32003, 20, 1)
    loss, grad = sv.sv_distill(x, ids, lp)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    l2, g2 = sv.sv_distill(x, ids, lp, stream=side)
    y = x.detach().requires_grad_()
    l3 = sv.sv_distill_loss(y, ids, lp, stream=side)
    side.synchronize()
    l3.sum().backward()
    torch.cuda.synchronize()
    assert torch.equal(loss, l2) and torch.equal(grad, g2) and torch.equal(loss, l3)
    check(x, ids, lp, 1.0, "renormalise", l3, y.grad)


def test_captured_and_replayed():
    x, ids, lp = teacher((20,), 9001, 12, 1)
    x.requires_grad_()
    w = torch.rand(20, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        sv.sv_distill(x, ids, lp)
        torch.autograd.grad(sv.sv_distill_loss(x, ids, lp), x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, grad = sv.sv_distill(x, ids, lp, weights=w)
        l2 = sv.sv_distill_loss(x, ids, lp)
        g2, = torch.autograd.grad(l2, x, w)
    for seed in (5, 6):
        y, i2, p2 = teacher((20,), 9001, 12, seed)
        with torch.no_grad():
            x.copy_(y)
        ids.copy_(i2), lp.copy_(p2), w.copy_(torch.rand(20, device="cuda"))
        graph.replay()
        check(x, ids, lp, 1.0, "renormalise", loss, grad, w)
        check(x, ids, lp, 1.0, "renormalise", l2, g2, w)


def test_sizes_of_nothing():
    x = torch.empty(0, 50, device="cuda")
    loss, grad = sv.sv_distill(x, torch.empty(0, 3, dtype=torch.int32, device="cuda"),
                               torch.empty(0, 3, device="cuda"))
    assert loss.shape == (0,) and grad.shape == (0, 50)
    x, ids, lp = teacher((), 50, 3, 1, none=0.0)
    loss, grad = sv.sv_distill(x, ids, lp)
    check(x, ids, lp, 1.0, "renormalise", loss, grad)


def test_refusals():
    x, ids, lp = teacher((4,), 100, 5, 1)
    for args, kw in (((x, ids.long(), lp), {}), ((x, ids, lp.double()), {}), ((x, ids[:3], lp[:3]), {}),
                     ((x, ids[:, :0], lp[:, :0]), {}), ((x, ids, lp[:, :4]), {}),
                     ((x, ids.cpu(), lp), {}), ((x.cpu(), ids, lp), {}), ((x, ids, lp), dict(tail="x")),
                     ((x, ids[:, 0], lp[:, 0]), {}), ((x.double(), ids, lp), {}),
                     ((x, ids.t().contiguous().t(), lp), {}),
                     ((x, ids.repeat(1, 30), lp.repeat(1, 30)), {})):
        with pytest.raises((ValueError, TypeError)):
            sv.sv_distill_loss(*args, **kw)
        with pytest.raises((ValueError, TypeError)):
            sv.sv_distill(*args, **kw)
    for kw in (dict(weights=lp), dict(weights=lp[:, 0]), dict(loss=ids[:, 0].contiguous()),
               dict(grad=x[:3]), dict(grad=x.bfloat16()), dict(row_stats=lp)):
        with pytest.raises(ValueError):
            sv.sv_distill(x, ids, lp, **kw)
    big = torch.zeros(5, 100, device="cuda")
    with pytest.raises(ValueError):
        sv.sv_distill(big[:4], ids, lp, grad=big[1:])
    with pytest.raises(sv.SpecVerifyError):
        sv.sv_distill(x, ids, lp, temperature=0.0)


@pytest.mark.parametrize("tail", TAILS)
def test_certain_students_keep_finite_losses_and_gradients(tail):
    """A logit 200 above all others: the others' probabilities are below float32's least, their
    logarithms and (as one outcome) their shares of one another are not."""
    V = 3001
    x, ids, lp = teacher((3,), V, 5, 8, missing=0.0, none=0.0)
    x[0, ids[0, 0].long()] = 200.0
    x[1, ids[1, 4].long()] = 500.0
    x[2, (ids[2, 0].long() + 1) % V] = 300.0     # (certain of a token that is not listed)
    loss, g = both(x, ids, lp, 1.0, tail)
    assert loss.isfinite().all() and (loss > 20).all()


@pytest.mark.parametrize("tail", TAILS)
@pytest.mark.parametrize("dtype,rows,V", [("bf16", 70000, 300), ("bf16", 5000, 40000),
                                          ("fp16", 700, 70001), ("f32", 1300, 33001)])
def test_many_rows(dtype, rows, V, tail):
    x = torch.empty((rows, V), dtype=u.DTYPES[dtype], device="cuda")
    ids = torch.empty((rows, 7), dtype=torch.int32, device="cuda")
    lp = torch.empty((rows, 7), device="cuda")
    step = max(1, 20_000_000 // V)
    for n, i in enumerate(range(0, rows, step)):
        s = slice(i, min(i + step, rows))
        x[s], ids[s], lp[s] = teacher((s.stop - s.start,), V, 7, n)
    loss, grad = sv.sv_distill(x, ids, lp, tail=tail)
    y = x.detach().requires_grad_()
    l2 = sv.sv_distill_loss(y, ids, lp, tail=tail)
    g2, = torch.autograd.grad(l2.sum(), y)
    for i in list(range(0, rows, step))[::4] + [max(0, rows - step)]:
        s = slice(i, i + step)
        check(x[s], ids[s], lp[s], 1.0, tail, loss[s], grad[s])
        check(x[s], ids[s], lp[s], 1.0, tail, l2[s], g2[s])


def test_entries_in_every_turn_and_twice_across_them():
    """Entries at the ends of turns of 1024 elements, some tokens twice, at odd alignments."""
    V = 70 * 1024 + 3
    x, _, _ = teacher((4,), V, 1, 3)
    at = torch.tensor([t + d for t in range(0, V - 1, 1200) for d in (0, 1)])[:110]
    ids = at.repeat(4, 1).to(torch.int32).cuda()
    ids[1, :55] = ids[1, 55:]
    ids[2, 1::2] = ids[2, ::2]
    lp = torch.full(ids.shape, -6.0, device="cuda") - torch.rand(ids.shape, device="cuda")
    for dtype in ("bf16", "f32"):
        room = torch.zeros(4, V + 9, dtype=u.DTYPES[dtype], device="cuda")
        room[:, 3:V + 3] = x
        for tail in TAILS:
            both(room[:, 3:V + 3], ids, lp, 1.0, tail)


def test_inputs_changed_before_the_backward_pass_are_noticed():
    x, ids, lp = teacher((4,), 500, 5, 1)
    x.requires_grad_()
    loss = sv.sv_distill_loss(x, ids, lp)
    lp.mul_(1.0)
    with pytest.raises(RuntimeError):
        loss.sum().backward()


def test_what_a_call_overwrites_is_noticed():
    x, ids, lp = teacher((4,), 500, 5, 1)
    y = x.requires_grad_() * 1.0
    loss = sv.sv_distill_loss(y, ids, lp)
    sv.sv_distill(y, ids, lp, grad=y)
    with pytest.raises(RuntimeError):
        loss.sum().backward()


def test_a_teacher_made_in_inference_mode():
    x, ids, lp = teacher((4,), 500, 5, 1)
    x.requires_grad_()
    with torch.inference_mode():
        there = ids.clone(), lp.clone()
    grads = []
    for t in (there, (ids, lp)):
        x.grad = None
        sv.sv_distill_loss(x, *t).sum().backward()
        grads.append(x.grad)
    assert torch.equal(*grads)


@pytest.mark.parametrize("tail", TAILS)
def test_long_rows_captured_and_replayed_without_a_pause(tail):
    # (their gradient is a launch of its own, which begins before the sums' ends)
    shape, V, k = (9,), 70001, 12
    x, ids, lp = teacher(shape, V, k, 1)
    graph = torch.cuda.CUDAGraph()
    sv.sv_distill(x, ids, lp, tail=tail)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        loss, grad = sv.sv_distill(x, ids, lp, tail=tail)
        l2, g2 = sv.sv_distill(grad, ids, lp, tail=tail)
    inputs = [teacher(shape, V, k, seed) for seed in (5, 6, 7)]
    torch.cuda.synchronize()
    results = []
    for y, i, p in inputs:
        x.copy_(y), ids.copy_(i), lp.copy_(p)
        graph.replay()
        results.append([t.clone() for t in (loss, grad, l2, g2)])
    for (y, i, p), (loss, grad, l2, g2) in zip(inputs, results):
        check(y, i, p, 1.0, tail, loss, grad)
        check(grad, i, p, 1.0, tail, l2, g2)


@pytest.mark.parametrize("tail", TAILS)
@pytest.mark.parametrize("dtype,rows,V", [("bf16", 40, 50257), ("bf16", 153, 33000), ("bf16", 300, 100003),
                                          ("fp16", 305, 131001), ("f32", 608, 66001), ("f32", 609, 60001)])
def test_a_row_to_a_block_of_any_size(dtype, rows, V, tail):
    """Loss and gradient by blocks of 4 to 16 warps, whose bitmaps are filled several times; rows at
    odd alignments, tokens twice."""
    room = torch.zeros((rows, V + 5), dtype=u.DTYPES[dtype], device="cuda")
    x, out = room[:, 1:V + 1], torch.full_like(room, 7.0)
    ids = torch.empty((rows, 40), dtype=torch.int32, device="cuda")
    lp = torch.empty((rows, 40), device="cuda")
    step = max(1, 20_000_000 // V)
    for n, i in enumerate(range(0, rows, step)):
        s = slice(i, min(i + step, rows))
        x[s], ids[s], lp[s] = teacher((s.stop - s.start,), V, 40, n)
    ids[::5, 20:] = ids[::5, :20]
    ids[3::50, 0] = V
    status = torch.full((rows,), 55, dtype=torch.int32, device="cuda")
    w = torch.rand(rows, device="cuda")
    loss, grad = sv.sv_distill(x, ids, lp, weights=w, tail=tail, row_status=status, grad=out[:, 1:V + 1])
    for i in range(0, rows, step):
        s = slice(i, min(i + step, rows))
        check(x[s], ids[s], lp[s], 1.0, tail, loss[s], grad[s], w[s], status[s])
    assert (out[:, 0] == 7.0).all() and (out[:, V + 1:] == 7.0).all()
