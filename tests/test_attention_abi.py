"""libsvattention without a GPU: it exports what include/sv_attention.h
declares, and its calls refuse bad arguments on the host before any CUDA call."""
import ctypes
import os
import re
import shutil
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sv_attention.h")
SV_OK, ARG, DTYPE, ALIGN, WORKSPACE, CUDA, SIZE = 0, -1, -2, -3, -4, -5, -6
F32, BF16, F16, E4M3 = 0, 1, 2, 3


def declared_functions():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*int\s+(\w+)\s*\(", text, flags=re.M)))


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from speculative_decoding_verification_66_gb300 import _build, _lib
    _build.build_attention()
    return _lib.load_attention()


def test_exports_match_the_header_and_the_binding(lib):
    import speculative_decoding_verification_66_gb300 as sv
    from speculative_decoding_verification_66_gb300 import _lib
    assert sorted(_lib.ATTENTION_SIGNATURES) == declared_functions()
    for name in declared_functions():
        assert callable(getattr(sv, name)), name
    nm = shutil.which("nm")
    if nm is None:
        pytest.skip("nm not available")
    out = subprocess.run([nm, "-D", "--defined-only", _lib.ATTENTION_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert sorted(x.split()[-1] for x in out.splitlines() if " T " in x) == declared_functions()


def test_a_missing_library_says_so(monkeypatch, tmp_path):
    from speculative_decoding_verification_66_gb300 import _lib
    monkeypatch.setattr(_lib, "_attention", None)
    monkeypatch.setattr(_lib, "ATTENTION_PATH", str(tmp_path / "absent.so"))
    with pytest.raises(_lib.LibraryMissing):
        _lib.load_attention()


# Addresses that are never followed: every call below is refused first, or has
# nothing to do (no tokens, no sequences).
P = 1 << 20
FIELDS = ["k", "v", "ke", "ve", "kps", "vps", "kss", "vss", "khs", "vhs", "keps", "veps", "kess",
          "vess", "kehs", "vehs", "num_pages", "page_size", "kv_heads", "head_dim", "dtype",
          "table", "table_stride", "max_pages", "cached", "starts", "batch"]
GOOD = dict(k=P, v=P, ke=0, ve=0, kps=16 * 8 * 128, vps=16 * 8 * 128, kss=8 * 128, vss=8 * 128,
            khs=128, vhs=128, keps=0, veps=0, kess=0, vess=0, kehs=0, vehs=0, num_pages=10,
            page_size=16, kv_heads=8, head_dim=128, dtype=BF16, table=P, table_stride=4,
            max_pages=4, cached=P, starts=P, batch=3)


def cache(**kw):
    d = dict(GOOD, **kw)
    if d["dtype"] == E4M3 and "ke" not in kw:
        d.update(ke=P, ve=P)
    return struct.pack("@4P12qq4iP2q2Pq", *[d[f] for f in FIELDS])


def append(lib, c, key=P, value=P, dtype=BF16, tokens=5, strides=(1024, 128, 1024, 128), status=0):
    return lib.sv_kv_append(c, key, value, dtype, tokens, *strides, status, 0)


def read(lib, c, key=P, value=P, dtype=BF16, tokens=5, status=0):
    return lib.sv_kv_read(c, key, value, dtype, tokens, status, 0)


def attend(lib, c, query=P, dtype=BF16, tokens=5, q_heads=32, ts=4096, hs=128, scale=0.1, window=0,
           max_chunk=0, out=P, lse=0, status=0, ws=P, ws_bytes=1 << 40):
    return lib.sv_chunk_attention(c, query, dtype, tokens, q_heads, ts, hs, scale, window,
                                  max_chunk, out, lse, status, ws, ws_bytes, 0)


BAD_CACHES = [
    (dict(dtype=F32), DTYPE), (dict(dtype=9), DTYPE), (dict(batch=-1), ARG),
    (dict(kv_heads=0), ARG), (dict(num_pages=-1), ARG), (dict(max_pages=-1), ARG),
    (dict(table_stride=3), ARG), (dict(head_dim=8), SIZE), (dict(head_dim=72), SIZE),
    (dict(head_dim=272), SIZE), (dict(page_size=0), SIZE), (dict(page_size=4), SIZE),
    (dict(page_size=24), SIZE), (dict(page_size=2048), SIZE), (dict(num_pages=1 << 31), SIZE),
    (dict(batch=1 << 31), SIZE), (dict(k=0), ARG), (dict(v=0), ARG), (dict(k=P + 8), ALIGN),
    (dict(kps=-128), ARG), (dict(kss=1028), ALIGN), (dict(vhs=132), ALIGN), (dict(ke=P), ARG),
    (dict(dtype=E4M3, ke=0, ve=0), ARG), (dict(dtype=E4M3, vess=-1), ARG),
    (dict(dtype=E4M3, khs=136), ALIGN), (dict(table=0), ARG), (dict(cached=0), ARG),
    (dict(starts=0), ARG), (dict(cached=P + 2), ALIGN),
]


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_bad_caches(lib, change, code):
    c = cache(**change)
    dtype = BF16
    assert append(lib, c, dtype=dtype) == code
    assert read(lib, c, dtype=dtype) == code
    assert attend(lib, c, dtype=dtype) == code


def test_no_cache(lib):
    assert append(lib, None) == ARG and read(lib, None) == ARG and attend(lib, None) == ARG


@pytest.mark.parametrize("kw,code", [
    (dict(key=0), ARG), (dict(value=0), ARG), (dict(key=P + 4), ALIGN), (dict(dtype=F32), DTYPE),
    (dict(dtype=F16), DTYPE), (dict(dtype=E4M3), DTYPE), (dict(tokens=-1), ARG),
    (dict(tokens=1 << 31), SIZE), (dict(strides=(1024, 128, 1024, 132)), ALIGN),
    (dict(strides=(-1024, 128, 1024, 128)), ARG), (dict(status=P + 1), ALIGN)])
def test_bad_appends(lib, kw, code):
    assert append(lib, cache(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(key=0), ARG), (dict(value=0), ARG), (dict(value=P + 4), ALIGN), (dict(dtype=F32), DTYPE),
    (dict(dtype=F16), DTYPE), (dict(tokens=-1), ARG), (dict(tokens=1 << 31), SIZE),
    (dict(status=P + 1), ALIGN)])
def test_bad_reads(lib, kw, code):
    assert read(lib, cache(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(query=0), ARG), (dict(query=P + 8), ALIGN), (dict(out=0), ARG), (dict(out=P + 8), ALIGN),
    (dict(lse=P + 2), ALIGN), (dict(status=P + 2), ALIGN), (dict(dtype=F32), DTYPE),
    (dict(dtype=F16), DTYPE), (dict(tokens=-1), ARG), (dict(tokens=1 << 31), SIZE),
    (dict(q_heads=0), ARG), (dict(q_heads=12), ARG), (dict(ts=4100), ALIGN), (dict(hs=-128), ARG),
    (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG),
    (dict(scale=float("inf")), ARG), (dict(scale=3e38), ARG), (dict(window=-1), ARG),
    (dict(window=1 << 31), ARG), (dict(max_chunk=-1), ARG), (dict(ws=0), WORKSPACE),
    (dict(ws=P + 16), WORKSPACE), (dict(ws_bytes=0), WORKSPACE)])
def test_bad_attentions(lib, kw, code):
    assert attend(lib, cache(), **kw) == code


def test_nothing_to_do_makes_no_cuda_call(lib):
    for c in (cache(), cache(batch=0, table=0, cached=0, starts=0, k=0, v=0)):
        kw = dict(tokens=0)
        assert append(lib, c, key=0, value=0, **kw) == SV_OK
        assert read(lib, c, key=0, value=0, **kw) == SV_OK
        assert attend(lib, c, query=0, out=0, **kw) == SV_OK


def test_workspace_sizes(lib):
    n = ctypes.c_size_t(0)
    f = lib.sv_chunk_attention_workspace_bytes
    assert f(3, 5, 32, 8, 128, 0, None) == ARG
    assert f(3, 5, 30, 8, 128, 0, ctypes.byref(n)) == ARG
    assert f(3, 5, 32, 8, 24, 0, ctypes.byref(n)) == SIZE
    assert f(-1, 5, 32, 8, 128, 0, ctypes.byref(n)) == ARG
    assert f(3, 5, 32, 8, 128, 0, ctypes.byref(n)) == SV_OK and n.value >= 256


def test_the_binding_refuses_host_tensors():
    import torch
    import speculative_decoding_verification_66_gb300 as sv
    pages = torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16)
    i32 = torch.zeros(1, 1, dtype=torch.int32)
    starts = torch.tensor([0, 1], dtype=torch.int32)
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sv.sv_chunk_attention(q, pages, pages, i32, i32[0], starts)
    with pytest.raises(ValueError):
        sv.sv_kv_append(q, q, pages, pages, i32, i32[0], starts)


def test_the_gated_call_needs_its_gate(lib):
    def gated(gate):
        return lib.sv_chunk_attention_gated(cache(), P, BF16, 5, 32, 4096, 128, 0.1, 0, 0, P, 0, 0,
                                            P, 1 << 40, 0, -1, gate)
    assert gated(0) == ARG and gated(P + 2) == ALIGN


def test_strides_of_single_elements_are_not_looked_at(lib):
    one = dict(kv_heads=1, khs=3, vhs=-5, num_pages=1, kps=1 << 60, vps=7)
    for c in (cache(**one), cache(dtype=E4M3, kehs=-1, veps=-2, **one)):
        assert append(lib, c, tokens=0, strides=(3, 5, -7, 1)) == SV_OK
        assert read(lib, c, tokens=0) == SV_OK
        assert attend(lib, c, tokens=0, q_heads=1, ts=3, hs=-1) == SV_OK
    assert append(lib, cache(kv_heads=1, khs=3, vhs=3, kss=1028), tokens=0) == ALIGN
    assert append(lib, cache(kps=1 << 39), tokens=0) == ARG  # 2^40 bytes
