"""libsvlogprobs without a GPU: it exports what include/sv_logprobs.h declares, its calls refuse bad
arguments on the host before any CUDA call, and the plain forms that the GPU tests use are right."""
import ctypes
import math
import os
import re
import shutil
import struct
import subprocess

import pytest
import torch

import logprobs_util as u

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sv_logprobs.h")
SV_OK, ARG, DTYPE, ALIGN, WORKSPACE, SIZE = 0, -1, -2, -3, -4, -6
F32, BF16, F16, E4M3 = 0, 1, 2, 3


def declared_functions():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*int\s+(\w+)\s*\(", text, flags=re.M)))


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from speculative_decoding_verification_66_gb300 import _build, _lib
    _build.build_logprobs()
    return _lib.load_logprobs()


def test_exports_match_the_header_and_the_binding(lib):
    import speculative_decoding_verification_66_gb300 as sv
    from speculative_decoding_verification_66_gb300 import _lib
    assert sorted(_lib.LOGPROBS_SIGNATURES) == declared_functions()
    for name in declared_functions():
        assert callable(getattr(sv, name)), name
    nm = shutil.which("nm")
    if nm is None:
        pytest.skip("nm not available")
    out = subprocess.run([nm, "-D", "--defined-only", _lib.LOGPROBS_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert sorted(x.split()[-1] for x in out.splitlines() if " T " in x) == declared_functions()


def test_the_header_goes_with_the_others(tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("gcc not available")
    for i, order in enumerate((("spec_verify", "sv_attention", "sv_logprobs"),
                               ("sv_logprobs", "sv_attention"))):
        src = tmp_path / f"t{i}.c"
        src.write_text("".join(f'#include "{h}.h"\n' for h in order) + "int x = SV_F16;\n")
        subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                        "-c", str(src), "-o", str(tmp_path / "t.o")], check=True)


def test_a_missing_library_says_so(monkeypatch, tmp_path):
    from speculative_decoding_verification_66_gb300 import _lib
    monkeypatch.setattr(_lib, "_logprobs", None)
    monkeypatch.setattr(_lib, "LOGPROBS_PATH", str(tmp_path / "absent.so"))
    with pytest.raises(_lib.LibraryMissing):
        _lib.load_logprobs()


# An address that is never followed: every call below is refused first, or has nothing to do.
P = 1 << 20
GOOD = dict(logits=P, outer=2, inner=3, so=300, si=100, vocab=100, dtype=BF16, T=1.0)


def rows(**kw):
    d = dict(GOOD, **kw)
    return struct.pack("@P5qif", d["logits"], d["outer"], d["inner"], d["so"], d["si"], d["vocab"],
                       d["dtype"], d["T"])


def logprobs(lib, r, tokens=P, k=5, logprobs=P, entropy=P, lse=P, rank=P, top=P, top_lp=P, stats=P,
             status=P, ws=P, ws_bytes=1 << 40):
    return lib.sv_token_logprobs(r, tokens, k, logprobs, entropy, lse, rank, top, top_lp, stats,
                                 status, ws, ws_bytes, 0)


def logprobs_grad(lib, r, tokens=P, stats=P, a=P, b=P, c=P, grad=P, so=300, si=100):
    return lib.sv_token_logprobs_backward(r, tokens, stats, a, b, c, grad, so, si, 0)


def distill(lib, r, ids=P, lp=P, k=5, tail=0, weights=P, loss=P, grad=P, so=300, si=100, stats=P,
            status=P, ws=P, ws_bytes=1 << 40):
    return lib.sv_distill(r, ids, lp, k, tail, weights, loss, grad, so, si, stats, status, ws,
                          ws_bytes, 0)


def distill_grad(lib, r, ids=P, lp=P, k=5, tail=0, stats=P, up=P, grad=P, so=300, si=100):
    return lib.sv_distill_backward(r, ids, lp, k, tail, stats, up, grad, so, si, 0)


CALLS = [logprobs, logprobs_grad, distill, distill_grad]


@pytest.mark.parametrize("change,code", [
    (dict(dtype=E4M3), DTYPE), (dict(dtype=-1), DTYPE), (dict(outer=-1), ARG), (dict(inner=-1), ARG),
    (dict(vocab=0), ARG), (dict(vocab=1 << 31), SIZE), (dict(outer=1 << 31), SIZE),
    (dict(outer=1 << 16, inner=1 << 15), SIZE), (dict(so=-1), ARG), (dict(si=-100), ARG),
    (dict(so=(1 << 40) + 1), ARG), (dict(logits=0), ARG), (dict(logits=P + 1), ALIGN),
    (dict(logits=P + 2, dtype=F32), ALIGN), (dict(T=0.0), ARG), (dict(T=-1.0), ARG),
    (dict(T=math.inf), ARG), (dict(T=math.nan), ARG), (dict(T=1e-39), ARG)])
def test_bad_rows(lib, change, code):
    for call in CALLS:
        assert call(lib, rows(**change)) == code, call.__name__


def test_no_rows(lib):
    for call in CALLS:
        assert call(lib, None) == ARG
    for kw in (dict(outer=0), dict(inner=0), dict(outer=0, inner=0, logits=0)):
        assert logprobs(lib, rows(**kw), 0, 5, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0) == SV_OK
        assert logprobs_grad(lib, rows(**kw), 0, 0, 0, 0, 0, 0) == SV_OK
        assert distill(lib, rows(**kw), 0, 0, 1, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0) == SV_OK
        assert distill_grad(lib, rows(**kw), 0, 0, 1, 0, 0, 0, 0) == SV_OK


@pytest.mark.parametrize("kw,code", [
    (dict(k=-1), ARG), (dict(k=101), ARG), (dict(tokens=0), ARG), (dict(top=0), ARG),
    (dict(top=0, top_lp=0), ARG), (dict(tokens=P + 2), ALIGN), (dict(logprobs=P + 1), ALIGN),
    (dict(entropy=P + 2), ALIGN), (dict(lse=P + 2), ALIGN), (dict(rank=P + 3), ALIGN),
    (dict(top=P + 2), ALIGN), (dict(top_lp=P + 2), ALIGN), (dict(stats=P + 8), ALIGN),
    (dict(status=P + 2), ALIGN)])
def test_bad_logprobs(lib, kw, code):
    assert logprobs(lib, rows(), **kw) == code


def test_too_many_alternatives(lib):
    assert logprobs(lib, rows(vocab=1000), k=129) == SIZE
    assert logprobs(lib, rows(vocab=(1 << 20) + 1), k=1) == SIZE


GRADS = [(dict(grad=0), ARG), (dict(grad=P + 1), ALIGN), (dict(so=-1), ARG), (dict(si=99), ARG),
         (dict(so=299), ARG), (dict(so=99, si=300), ARG), (dict(so=1 << 41), ARG), (dict(stats=0), ARG),
         (dict(stats=P + 4), ALIGN)]


@pytest.mark.parametrize("kw,code", GRADS + [
    (dict(tokens=0), ARG), (dict(tokens=P + 2), ALIGN), (dict(a=P + 2), ALIGN),
    (dict(b=P + 2), ALIGN), (dict(c=P + 2), ALIGN)])
def test_bad_logprobs_gradients(lib, kw, code):
    assert logprobs_grad(lib, rows(), **kw) == code


TEACHERS = [(dict(k=0), ARG), (dict(k=129), SIZE), (dict(tail=2), ARG), (dict(tail=-1), ARG),
            (dict(ids=0), ARG), (dict(lp=0), ARG), (dict(ids=P + 2), ALIGN), (dict(lp=P + 2), ALIGN)]


@pytest.mark.parametrize("kw,code", TEACHERS + GRADS[1:7] + [
    (dict(weights=P + 2), ALIGN), (dict(loss=P + 2), ALIGN), (dict(stats=P + 4), ALIGN),
    (dict(status=P + 2), ALIGN)])
def test_bad_distillations(lib, kw, code):
    assert distill(lib, rows(), **kw) == code


@pytest.mark.parametrize("kw,code", TEACHERS + GRADS + [(dict(up=0), ARG), (dict(up=P + 2), ALIGN)])
def test_bad_distillation_gradients(lib, kw, code):
    assert distill_grad(lib, rows(), **kw) == code


def workspace_bytes(lib, r, k=0):
    n = ctypes.c_size_t(77)
    rc = lib.sv_logprobs_workspace_bytes(r, k, ctypes.byref(n))
    return n.value if rc == SV_OK else rc


def test_workspaces(lib):
    big = dict(vocab=128256, so=3 * 128256, si=128256, dtype=BF16)
    need = workspace_bytes(lib, rows(**big), 20)
    assert need > 262144  # (the counters)
    assert workspace_bytes(lib, rows(logits=0, so=-5, si=-5, vocab=128256), 20) == need
    assert 262144 <= workspace_bytes(lib, rows(vocab=5)) <= 262144 + 4096
    assert lib.sv_logprobs_workspace_bytes(rows(), 0, None) == ARG
    assert workspace_bytes(lib, None) == ARG and workspace_bytes(lib, rows(), -1) == ARG
    assert workspace_bytes(lib, rows(), 101) == ARG and workspace_bytes(lib, rows(vocab=500), 129) == SIZE
    for kw in (dict(ws=0), dict(ws=P + 16), dict(ws_bytes=1000), dict(ws_bytes=0)):
        assert logprobs(lib, rows(**big), k=20, **kw) == WORKSPACE
        assert distill(lib, rows(**big), so=3 * 128256, si=128256, **kw) == WORKSPACE
    import speculative_decoding_verification_66_gb300 as sv
    assert sv.sv_logprobs_workspace_bytes(6, 128256, torch.bfloat16, 20) == need
    with pytest.raises(TypeError):
        sv.sv_logprobs_workspace_bytes(6, 128256, torch.float64)


def test_the_binding_refuses_host_tensors():
    import speculative_decoding_verification_66_gb300 as sv
    x, t = torch.zeros(2, 50), torch.zeros(2, dtype=torch.int32)
    ids, lp = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    for call in (lambda: sv.sv_token_logprobs(x, t), lambda: sv.sv_distill(x, ids, lp),
                 lambda: sv.sv_distill_loss(x, ids, lp),
                 lambda: sv.sv_token_logprobs_backward(x, torch.zeros(2, 4)),
                 lambda: sv.sv_distill_backward(x, ids, lp, torch.zeros(2, 4), lp[:, 0])):
        with pytest.raises(ValueError):
            call()


def slopes(f, x, h=1e-5):
    out = torch.zeros_like(x)
    for v in range(x.shape[1]):
        d = torch.zeros_like(x)
        d[:, v] = h
        out[:, v] = (f(x + d) - f(x - d)) / (2 * h)
    return out


def test_the_plain_forms_gradients_are_their_slopes():
    g = torch.Generator().manual_seed(1)
    x = 2 * torch.randn(5, 30, generator=g, dtype=torch.float64)
    x[0, 3] = -40.0
    tokens = torch.tensor([3, 0, -1, 29, 7], dtype=torch.int32)
    a, b, c = (torch.randn(5, generator=g, dtype=torch.float64) for _ in range(3))

    def value(y):
        r = u.logprobs(y, tokens, 0.7)
        return a * r["logprobs"] + b * r["entropy"] + c * r["lse"]

    assert torch.allclose(slopes(value, x), u.logprobs_grad(x, tokens, a, b, c, 0.7), atol=1e-8)
    ids = torch.tensor([[1, 2, 3], [4, 4, 0], [-1, -1, -1], [9, -1, 8], [29, 0, 29]])
    lp = torch.log(torch.rand(5, 3, generator=g, dtype=torch.float64) / 3)
    for tail in ("renormalise", "bucket"):
        loss, grad, status = u.distill(x, ids, lp, 1.4, tail)
        assert torch.allclose(slopes(lambda y: u.distill(y, ids, lp, 1.4, tail)[0], x), grad,
                              atol=1e-8)
        assert status.eq(0).all() and loss[2] == 0 and (loss[[0, 1, 3, 4]] > 0).all()


def test_the_plain_divergence_is_the_closed_form():
    """Two tokens of three listed, by hand."""
    x = torch.log(torch.tensor([[0.5, 0.3, 0.2]], dtype=torch.float64))
    ids, lp = torch.tensor([[0, 1]]), torch.log(torch.tensor([[0.6, 0.2]], dtype=torch.float64))
    loss = u.distill(x, ids, lp, 1.0, "bucket")[0].item()
    assert math.isclose(loss, 0.6 * math.log(1.2) + 0.2 * math.log(2 / 3) + 0.2 * math.log(1.0),
                        rel_tol=1e-12)
    loss = u.distill(x, ids, lp, 1.0, "renormalise")[0].item()
    assert math.isclose(loss, 0.75 * math.log(1.5) + 0.25 * math.log(0.25 / 0.3), rel_tol=1e-12)
