"""Writing to the paged cache and reading it back, against the definition: what
is written is compared bit for bit, and nothing else may change."""
import math

import pytest
import torch

import speculative_decoding_verification_66_gb300 as sv
from attention_util import DTYPES, Cache, quantise, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_attention()
    torch.cuda.set_device(0)


def bits(x):
    return x.contiguous().view(torch.uint8 if x.element_size() == 1 else torch.int16)


def new_rows(c, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    shape = (c.tokens, c.heads, c.d)
    return [(torch.randn(shape, generator=g) * spread).to(c.dtype).cuda() for _ in range(2)]


def expected_append(c, rows):
    """The cache's tensors after the append, by plain indexing."""
    want = [x.clone() for x in c.parts]
    exps = [None if e is None else e.clone() for e in c.exps]
    r = 0
    for b, (n, t) in enumerate(zip(c.lens, c.chunks)):
        for i in range(t):
            page, slot = c.pages_of[b][(n + i) // c.page], (n + i) % c.page
            for kv in range(2):
                if c.e4m3:
                    code, e = quantise(rows[kv][r])
                    want[kv].view(torch.uint8)[page, slot] = code
                    exps[kv][page, slot] = e
                else:
                    want[kv][page, slot] = rows[kv][r]
            r += 1
    return want, exps


CASES = [
    # lens, chunks, heads, d, page, dtype, e4m3, heads first
    ([0], [1], 1, 16, 8, "bf16", False, False),
    ([700], [1], 8, 128, 16, "bf16", False, False),
    ([15, 16, 17, 0], [1, 1, 3, 40], 8, 128, 16, "bf16", True, False),
    ([3, 0, 100], [5, 0, 33], 3, 64, 32, "fp16", True, True),
    ([3, 0, 100], [5, 0, 33], 3, 80, 32, "fp16", False, True),
    ([60, 64, 1], [9, 9, 9], 5, 256, 64, "bf16", True, False),
    ([250, 1], [300, 7], 2, 48, 8, "bf16", True, True),
    ([0] * 40, [2] * 40, 4, 112, 16, "fp16", True, False),
    ([5] * 1100, [1] * 1100, 1, 32, 8, "bf16", True, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[2:]))
def test_append_and_read(case):
    lens, chunks, heads, d, page, dtype, e4m3, hf = case
    c = Cache(lens, chunks, heads, d, page, dtype, e4m3, hf, seed=1)
    rows = new_rows(c, 2, spread=3.0)
    want, exps = expected_append(c, rows)
    status = torch.full((len(lens),), 77, dtype=torch.int32, device="cuda")
    sv.sv_kv_append(*rows, *c.args(), **c.exp_args(), seq_status=status)
    for kv in range(2):
        assert torch.equal(bits(c.parts[kv]), bits(want[kv]))
        if e4m3:
            assert torch.equal(c.exps[kv], exps[kv])
    assert not status.any()
    status.fill_(77)
    out = sv.sv_kv_read(*c.args(), c.tokens, **c.exp_args(), dtype=c.dtype, seq_status=status)
    assert not status.any()
    for kv in range(2):
        if not e4m3:
            assert torch.equal(bits(out[kv]), bits(rows[kv]))
            continue
        v = values(*quantise(rows[kv]))
        assert torch.equal(out[kv].double(), v.to(c.dtype).double())  # one rounding; exact in bf16
        if c.dtype == torch.bfloat16:
            assert torch.equal(out[kv].double(), v)
        # Half an e4m3 step of each value, or of the least normal code of its vector.
        top = rows[kv].double().abs().amax(-1, keepdim=True)
        assert ((v - rows[kv].double()).abs()
                <= 2.0 ** -4 * rows[kv].double().abs() + top / 224 * 2.0 ** -10).all()


def test_read_elsewhere_and_other_type():
    """A range in the middle, into given buffers, e4m3 into the other 16-bit type."""
    c = Cache([100, 40, 0], [30, 1, 7], 4, 64, 16, "bf16", True, seed=4)
    first = torch.tensor([50, 17, 0], dtype=torch.int32, device="cuda")
    key = torch.empty(38, 4, 64, dtype=torch.float16, device="cuda")
    value = torch.empty_like(key)
    k, v = sv.sv_kv_read(*c.args()[:3], first, c.starts, 38, **c.exp_args(), key=key, value=value)
    assert k is key and v is value
    for i, x in enumerate((k, v)):
        want = torch.cat([c.dense(i, 0, 80)[50:], c.dense(i, 1, 18)[17:], c.dense(i, 2, 7)])
        assert torch.equal(x, want.to(torch.float16))


SPECIAL = [0.0, -0.0, 448.0, 449.0, 447.9, 1.75 * 2 ** 100, 2.0 ** 101, 2.0 ** -120, 2.0 ** -126,
           2.0 ** -133, 3.0e38, 1.0, 1.7500001, 61440.0, 65504.0, 2.0 ** -24, 2.0 ** -14]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("special", SPECIAL + [math.nan, math.inf, -math.inf])
def test_exponents_of_special_vectors(dtype, special):
    c = Cache([0], [3], 2, 32, 8, dtype, True, seed=3)
    rows = new_rows(c, 5)
    scale = special if math.isfinite(special) and special else 1.0
    x = (rows[0].double() * scale * 0.3).clamp(-abs(scale), abs(scale)).to(c.dtype)
    x = torch.where(x.isfinite(), x, torch.zeros_like(x))
    x[1, 1, 7] = special
    if special == 0.0:
        x[1, 1] = special
    rows[0] = x
    want, exps = expected_append(c, rows)
    sv.sv_kv_append(*rows, *c.args(), **c.exp_args())
    assert torch.equal(c.exps[0], exps[0])
    assert torch.equal(bits(c.parts[0]), bits(want[0]))
    k, _ = sv.sv_kv_read(*c.args(), 3, **c.exp_args(), dtype=c.dtype)
    ref = values(*quantise(x)).to(c.dtype)
    assert torch.equal(k.isnan(), ref.isnan())
    assert torch.equal(torch.nan_to_num(k.double()), torch.nan_to_num(ref.double()))
    if dtype == "fp16":
        assert not k.isinf().any()


def test_strided_rows():
    """Keys and values as slices of one fused projection."""
    c = Cache([9, 30], [4, 11], 4, 64, 16, "bf16", True, seed=6)
    fused = torch.randn(15, 12 * 64 + 16, device="cuda").bfloat16()
    k = fused.as_strided((15, 4, 64), (784, 64, 1), 0)
    v = fused.as_strided((15, 4, 64), (784, 128, 1), 256)
    want, exps = expected_append(c, [k, v])
    sv.sv_kv_append(k, v, *c.args(), **c.exp_args())
    for kv in range(2):
        assert torch.equal(bits(c.parts[kv]), bits(want[kv])) and torch.equal(c.exps[kv], exps[kv])


@pytest.mark.parametrize("e4m3", [False, True])
def test_bad_sequences_and_pages(e4m3):
    """Bad lengths and pages are reported, nothing of theirs is written, the rest is."""
    c = Cache([20, 20, 20, 20], [5, 5, 5, 5], 2, 64, 8, "bf16", e4m3, seed=7)
    rows = new_rows(c, 8)
    want, exps = expected_append(c, rows)
    before = [x.clone() for x in c.parts]
    # Sequence 1: negative length. 2: the page of its positions 24 .. out of range. 3: too long.
    c.cached[1] = -1
    c.table[2, 3] = c.parts[0].shape[0]
    c.cached[3] = c.table.shape[1] * 8 - 4
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    sv.sv_kv_append(*rows, *c.args(), **c.exp_args(), seq_status=status)
    assert status.tolist() == [0, sv.SV_SEQ_BAD_LENGTH, sv.SV_SEQ_BAD_PAGE, sv.SV_SEQ_BAD_LENGTH]
    for kv in range(2):
        expect = before[kv].clone()
        for p in c.pages_of[0]:
            expect.view(torch.uint8 if e4m3 else torch.int16)[p] = \
                want[kv].view(torch.uint8 if e4m3 else torch.int16)[p]
        p = c.pages_of[2][2]  # positions 16 .. 23 of sequence 2 have a good page
        expect.view(torch.uint8 if e4m3 else torch.int16)[p] = \
            want[kv].view(torch.uint8 if e4m3 else torch.int16)[p]
        assert torch.equal(bits(c.parts[kv]), bits(expect))
    k, v = sv.sv_kv_read(*c.args(), 20, **c.exp_args(), seq_status=status)
    assert status.tolist() == [0, sv.SV_SEQ_BAD_LENGTH, sv.SV_SEQ_BAD_PAGE, sv.SV_SEQ_BAD_LENGTH]
    for x in (k, v):
        assert x[:5].isfinite().all() and x[5:10].isnan().all() and x[15:].isnan().all()
        assert x[10:14].isfinite().all() and x[14].isnan().all()


@pytest.mark.parametrize("starts", [[0, 5, 3, 20], [2, 5, 9, 99], [-4, 5, 9, 20], [0, 99, 4, 20]])
def test_bad_starts(starts):
    c = Cache([8, 8, 8], [5, 5, 10], 2, 64, 8, "bf16", False, seed=9)
    rows = new_rows(c, 10)
    c.starts.copy_(torch.tensor(starts, dtype=torch.int32))
    status = torch.zeros(3, dtype=torch.int32, device="cuda")
    sv.sv_kv_append(*rows, *c.args(), seq_status=status)
    k, v = sv.sv_kv_read(*c.args(), c.tokens, seq_status=status)
    torch.cuda.synchronize()
    bad = [not (0 <= starts[b] <= starts[b + 1] <= c.tokens) or
           8 + starts[b + 1] - starts[b] > c.table.shape[1] * 8 for b in range(3)]
    assert [s == sv.SV_SEQ_BAD_LENGTH for s in status.tolist()] == bad


def test_empty_calls():
    c = Cache([4, 9], [0, 0], 2, 64, 8)
    rows = new_rows(c, 1)
    before = [x.clone() for x in c.parts]
    sv.sv_kv_append(*rows, *c.args())
    k, v = sv.sv_kv_read(*c.args(), 0)
    assert k.shape == (0, 2, 64) and all(torch.equal(a, b) for a, b in zip(before, c.parts))


def test_offsets_past_32_bits():
    """Pages 2^31 elements apart: byte offsets of 2^32 and more."""
    step = 1 << 31
    store = torch.zeros(2 * step + 4096, dtype=torch.bfloat16, device="cuda")
    pages = store.as_strided((3, 8, 1, 64), (step, 64, 64, 1))
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    x = torch.randn(24, 1, 64, device="cuda").bfloat16()
    args = (pages, pages, table, torch.tensor([0], **i32), torch.tensor([0, 24], **i32))
    sv.sv_kv_append(x, x, *args)
    assert torch.equal(pages[[2, 0, 1]].reshape(24, 1, 64), x)
    k, v = sv.sv_kv_read(*args, 24)
    assert torch.equal(k, x) and torch.equal(v, x)


def test_another_stream():
    c = Cache([100, 3], [6, 2], 4, 128, 16, "bf16", True, seed=11)
    rows = new_rows(c, 12)
    want, exps = expected_append(c, rows)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sv.sv_kv_append(*rows, *c.args(), **c.exp_args(), stream=s)
    k, v = sv.sv_kv_read(*c.args(), 8, **c.exp_args(), stream=s)
    s.synchronize()
    assert torch.equal(c.exps[0], exps[0]) and torch.equal(bits(c.parts[1]), bits(want[1]))
    assert torch.equal(k.double(), values(*quantise(rows[0])))


def test_refusals():
    c = Cache([4], [2], 2, 64, 8)
    k, v = new_rows(c, 1)
    for bad in (k[:, :1], k.float(), k.half(), k[:, :, :32], k.cpu()):
        with pytest.raises((ValueError, TypeError)):
            sv.sv_kv_append(bad, v, *c.args())
    with pytest.raises(ValueError):
        sv.sv_kv_append(k, v, c.parts[0], c.parts[1][:1], c.table, c.cached, c.starts)
    with pytest.raises(ValueError):
        sv.sv_kv_append(k, v, *c.args(), k_exps=torch.zeros(1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        sv.sv_kv_append(k, v, c.parts[0], c.parts[1], c.table.long(), c.cached, c.starts)
    with pytest.raises(ValueError):
        sv.sv_kv_append(k, v, c.parts[0], c.parts[1], c.table, c.cached, c.starts[:1])
    with pytest.raises(ValueError):
        sv.sv_kv_read(*c.args(), -1)
    with pytest.raises(sv.SpecVerifyError):  # rows that are not 16-byte aligned
        flat = torch.zeros(2 * 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")
        x = flat[4:].view(2, 2, 64)
        sv.sv_kv_append(x, x, *c.args())


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_read_of_no_sequences_is_nan(e4m3):
    c = Cache([4], [2], 2, 64, 8, "bf16", e4m3)
    i32 = dict(dtype=torch.int32, device="cuda")
    key, value = (torch.full((5, 2, 64), 7.0, device="cuda").bfloat16() for _ in range(2))
    args = (c.parts[0], c.parts[1], torch.empty((0, 4), **i32), torch.empty(0, **i32),
            torch.zeros(1, **i32))
    sv.sv_kv_read(*args, 5, **c.exp_args(), key=key, value=value)
    assert key.isnan().all() and value.isnan().all()
    before = [x.clone() for x in c.parts]
    sv.sv_kv_append(key, value, *args, **c.exp_args())
    assert all(torch.equal(bits(x), bits(y)) for x, y in zip(before, c.parts))
