"""The attention kernels' bounded waits, without a fault: the values' loads of one thread block, or of
all, wait on a device flag that nothing sets. The wait runs out (about 2 s), the block gives up with
its other loads landed and returns, and the call is reported as timed out."""
import functools

import pytest
import torch

import speculative_decoding_verification_66_gb300 as sv
from attention_util import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_attention()
    torch.cuda.set_device(0)


# New tokens, head size: the few-row kernel, the tile kernel with items of 128 and of 256 rows, and
# large heads. More tiles a block than its shared memory holds, so that loads are under way.
SHAPES = [(1, 64), (4, 128), (9, 128), (70, 128), (70, 64), (5, 256)]
LENS = [2000, 1300, 1703, 277]


@functools.lru_cache(maxsize=None)
def case(T, d, e4m3):
    c = Cache(LENS, [T] * 4, 16, d, 64, "bf16", e4m3, seed=T)
    g = torch.Generator(device="cuda").manual_seed(d)
    q = torch.randn(c.tokens, 64, d, device="cuda", generator=g).bfloat16()
    return c, q, dict(c.exp_args(), max_chunk=T)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("block", [-1, 70])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(T, d, e4m3, block):
    c, q, kw = case(T, d, e4m3)
    want = sv.sv_chunk_attention(q, *c.args(), **kw, return_lse=True)
    gate = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = sv.sv_chunk_attention_gated(q, *c.args(), gate, block=block, **kw)
    torch.cuda.synchronize()
    assert r["seq_status"].tolist() == [sv.SV_SEQ_TIMEOUT] * 4
    again = sv.sv_chunk_attention(q, *c.args(), **kw, return_lse=True)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    gate.fill_(1)
    r = sv.sv_chunk_attention_gated(q, *c.args(), gate, block=block, **kw)
    assert not r["seq_status"].any()
    assert torch.equal(r["out"], want[0]) and torch.equal(r["lse"], want[1])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,d", SHAPES)
def test_no_ordinary_call_waits_for_its_limit(T, d, e4m3):
    c, q, kw = case(T, d, e4m3)
    sv.sv_chunk_attention(q, *c.args(), **kw)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(3):
        sv.sv_chunk_attention(q, *c.args(), **kw)
    end.record()
    torch.cuda.synchronize()
    assert begin.elapsed_time(end) < 1000.0  # a wait's limit is about 2000


@pytest.mark.parametrize("T,d", SHAPES)
def test_one_block_that_gives_up_makes_every_output_nan(T, d):
    """Also the rows that other blocks finished or join from that block's unwritten share, which the
    call before left there."""
    c, q, kw = case(T, d, False)
    for block in (0, 33, 150):
        sv.sv_chunk_attention(q, *c.args(), **kw)
        gate = torch.zeros(1, dtype=torch.int32, device="cuda")
        r = sv.sv_chunk_attention_gated(q, *c.args(), gate, block=block, **kw)
        assert r["out"].isnan().all() and r["lse"].isnan().all()


def test_refusals():
    c, q, kw = case(1, 64, False)
    with pytest.raises(ValueError):
        sv.sv_chunk_attention_gated(q, *c.args(), torch.zeros(1, device="cuda"), **kw)
    with pytest.raises(ValueError):
        sv.sv_chunk_attention_gated(q, *c.args(), torch.zeros(1, dtype=torch.int32), **kw)
