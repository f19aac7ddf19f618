"""Python binding of the log probabilities of given tokens and of distillation
(include/sv_logprobs.h): the same names, torch tensors in, and autograd.

Argument marshalling only, as in api.py. Logits are [V], [rows, V] or
[B, rows, V], bfloat16, float16 or float32, with any strides but the last (a
slice of positions or of a padded vocabulary is read where it lies). What is
given or returned for each row has the logits' shape without V.

``sv_token_logprobs`` and ``sv_distill_loss`` are differentiable in the logits, once
and in reverse mode; tokens, teachers and weights are constants to them.
``sv_distill`` gives loss and gradient at once, for training that calls
``logits.backward(grad)`` itself; the ``_backward`` calls are the gradients alone.
All of these can be captured into a CUDA graph. Of a backward
pass through autograd torch asks that no eager graph of the same leaf is alive when
it is captured: that graph has bound the leaf to its own stream, and the capture ends
in an error (``torch.autograd.grad`` included). ``sv_distill`` and the ``_backward``
calls go without autograd, and are captured beside anything.
"""
from __future__ import annotations

import ctypes
import struct
import threading
from functools import lru_cache
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad

from . import _lib
from .api import SV_BF16, SV_F32, _check
from .attention import SV_F16, _on

SV_MAX_TOP, SV_MAX_TOP_VOCAB, SV_ROW_STATS = 128, 1 << 20, 8
SV_LOGPROBS_COUNTER_BYTES = 262144
SV_TAIL_RENORMALISE, SV_TAIL_BUCKET = 0, 1

_CODES = {torch.float32: SV_F32, torch.bfloat16: SV_BF16, torch.float16: SV_F16}
_TAILS = {"renormalise": SV_TAIL_RENORMALISE, "bucket": SV_TAIL_BUCKET}
# struct sv_logit_rows
_ROWS = struct.Struct("@P5qif")


class TokenLogprobs(NamedTuple):
    """What ``sv_token_logprobs`` returns; None where it was not asked for."""
    logprobs: Optional[torch.Tensor]
    rank: Optional[torch.Tensor]
    entropy: torch.Tensor
    lse: torch.Tensor
    top_tokens: Optional[torch.Tensor]
    top_logprobs: Optional[torch.Tensor]


def _strides(x):
    """(outer, inner, outer stride, inner stride) of the rows of x."""
    shape, st = x.shape, x.stride()
    if len(shape) == 3:
        return shape[0], shape[1], st[0], st[1]
    if len(shape) == 2:
        return 1, shape[0], 0, st[0]
    return 1, 1, 0, 0


def _steps(x):
    """The same, with stride 0 where there is one of a kind: equal wherever the rows are."""
    outer, inner, s, t = _strides(x)
    return outer, inner, s if outer > 1 else 0, t if inner > 1 else 0


def _describe(logits, temperature):
    """(packed struct sv_logit_rows, device, shape of the rows)."""
    shape = logits.shape
    if not logits.is_cuda or not 1 <= len(shape) <= 3:
        raise ValueError("logits must be a CUDA tensor [V], [rows, V] or [B, rows, V]")
    code = _CODES.get(logits.dtype)
    if code is None:
        raise TypeError(f"logits must be float32, bfloat16 or float16, got {logits.dtype}")
    if shape[-1] < 1 or (shape[-1] > 1 and logits.stride(-1) != 1):
        raise ValueError("logits must be contiguous along a vocabulary of at least one token")
    packed = _ROWS.pack(logits.data_ptr(), *_strides(logits), shape[-1], code, temperature)
    return packed, logits.device, shape[:-1]


@lru_cache(maxsize=256)
def _workspace_bytes(rows, V, code, top_k):
    n = ctypes.c_size_t(0)
    _check(_lib.load_logprobs().sv_logprobs_workspace_bytes(
        _ROWS.pack(0, 1, rows, 0, 0, V, code, 1.0), top_k, ctypes.byref(n)),
        "sv_logprobs_workspace_bytes")
    return n.value


def sv_logprobs_workspace_bytes(rows: int, V: int, dtype, top_k: int = 0) -> int:
    """Workspace that ``sv_token_logprobs``, ``sv_distill`` and ``sv_distill_loss`` need for so many
    rows, with up to ``top_k`` alternatives."""
    if dtype not in _CODES:
        raise TypeError(f"logits must be float32, bfloat16 or float16, got {dtype}")
    return _workspace_bytes(rows, V, _CODES[dtype], top_k)


_kept = threading.local()


def _workspace(given, logits, rows, top_k, stream):
    """(address, bytes) of a workspace: the one given, or one that is kept for this thread's calls on
    this stream, which the stream puts in order. A call that is being captured gets one of its own,
    from the graph's pool: its replays may run beside anything."""
    dev = logits.device
    if given is not None:
        if given.device != dev or given.dtype != torch.uint8 or not given.is_contiguous():
            raise ValueError("workspace must be contiguous uint8 on the logits' device")
        return given.data_ptr(), given.numel()
    need = _workspace_bytes(rows, logits.shape[-1], _CODES[logits.dtype], top_k)
    if need == 0:
        return None, 0
    if torch.cuda.is_current_stream_capturing():
        w = _zeroed(need, dev)
    else:
        kept = _kept.__dict__
        w = kept.get((dev.index, stream))
        if w is None or w.numel() < need:
            w = kept[(dev.index, stream)] = _zeroed(need, dev)
    return w.data_ptr(), w.numel()


def _zeroed(nbytes, dev):
    w = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    w[:SV_LOGPROBS_COUNTER_BYTES].zero_()
    return w


def _per_row(x, name, shape, dtype, dev, last=()):
    """Address of a contiguous array for each row, or None."""
    if x is None:
        return None
    if x.dtype != dtype or x.shape != (*shape, *last) or not x.is_contiguous() or x.device != dev:
        kind = str(dtype).replace("torch.", "")
        raise ValueError(f"{name} must be contiguous {kind} {list((*shape, *last))} on the logits' "
                         "device")
    return x.data_ptr()


def _grad_like(logits):
    """An uninitialised gradient. Its rows begin as far from 16-byte boundaries as the logits' do,
    which lets both be moved by whole vectors; so rows that are padded stay padded."""
    shape, V = logits.shape, logits.shape[-1]
    vector = 16 // logits.element_size()
    if V % vector == 0 or logits.is_contiguous() or \
            any(s % vector for s, n in zip(logits.stride()[:-1], shape[:-1]) if n > 1):
        return torch.empty(shape, dtype=logits.dtype, device=logits.device)
    padded = torch.empty((*shape[:-1], V + -V % vector), dtype=logits.dtype, device=logits.device)
    return padded[..., :V]


def _span(x):
    """Bytes [first, end) that the elements of x lie in."""
    last = sum((n - 1) * s for n, s in zip(x.shape, x.stride()))
    return x.data_ptr(), x.data_ptr() + (last + 1) * x.element_size()


def _apart(grad, logits):
    """Whether the rows of grad, which have no element in common with one another, have none in common
    with those of logits, whose spans they share. Known of equal strides alone: then a row of the one
    lies d + i s + j t elements from a row of the other, with s and t the strides and i and j the
    distances along the dimensions, the rows' own lengths apart along the larger stride."""
    outer, inner, s, t = _steps(grad)
    if (outer, inner, s, t) != _steps(logits):
        return False
    d, V = (grad.data_ptr() - logits.data_ptr()) // grad.element_size(), grad.shape[-1]
    if s < t:
        outer, inner, s, t = inner, outer, t, s
    if s < (inner - 1) * t + V and outer > 1 and inner > 1:
        return False
    s, t = max(s, 1), max(t, 1)
    near = range(max(1 - outer, (-d - inner * t - V) // s), min(outer - 1, (-d + inner * t + V) // s + 1) + 1)
    for i in near:
        left = d + i * s
        for j in (-left // t, -left // t + 1):
            if abs(left + min(max(j, 1 - inner), inner - 1) * t) < V:
                return False
    return True


def _check_grad(grad, logits):
    if grad.shape != logits.shape or grad.dtype != logits.dtype or grad.device != logits.device \
            or (grad.shape[-1] > 1 and grad.stride(-1) != 1):
        raise ValueError("grad must have the logits' shape, dtype and device, and be contiguous "
                         "along the vocabulary")
    if grad.numel() == 0:
        return
    a, b = _span(grad), _span(logits)
    if a[0] < b[1] and b[0] < a[1] and (a[0] != b[0] or _steps(grad) != _steps(logits)) \
            and not _apart(grad, logits):
        raise ValueError("grad must be the logits themselves or lie apart from them (between their rows: "
                         "with their strides)")


def _logprobs(described, logits, tokens, top_k, row_status, workspace, row_stats):
    rows, dev, shape = described
    stream = torch._C._cuda_getCurrentRawStream(dev.index)
    i32, f32 = torch.int32, torch.float32
    token_ptr = _per_row(tokens, "tokens", shape, i32, dev)
    stats_ptr = _per_row(row_stats, "row_stats", shape, f32, dev, (SV_ROW_STATS,))
    status_ptr = _per_row(row_status, "row_status", shape, i32, dev)
    if not 0 <= top_k <= min(SV_MAX_TOP, logits.shape[-1]):
        raise ValueError(f"top_k must be from 0 to {SV_MAX_TOP} and at most the vocabulary")
    entropy = torch.empty(shape, dtype=f32, device=dev)
    lse = torch.empty_like(entropy)
    logprobs = rank = top_tokens = top_logprobs = None
    if tokens is not None:
        logprobs = torch.empty_like(entropy)
        rank = torch.empty(shape, dtype=i32, device=dev)
    if top_k:
        top_tokens = torch.empty((*shape, top_k), dtype=i32, device=dev)
        top_logprobs = torch.empty((*shape, top_k), dtype=f32, device=dev)

    def ptr(x):
        return None if x is None else x.data_ptr()

    _check(_lib.load_logprobs().sv_token_logprobs(
        rows, token_ptr, top_k, ptr(logprobs), entropy.data_ptr(), lse.data_ptr(), ptr(rank),
        ptr(top_tokens), ptr(top_logprobs), stats_ptr, status_ptr,
        *_workspace(workspace, logits, shape.numel(), top_k, stream), stream), "sv_token_logprobs")
    _wrote(row_stats, row_status)
    return TokenLogprobs(logprobs, rank, entropy, lse, top_tokens, top_logprobs)


def _version(x):
    """How often a tensor was changed in place (inference tensors do not tell)."""
    return None if x.is_inference() else x._version


def _wrote(*tensors):
    """Tells autograd of a caller's tensors that a call has written, as torch's own calls do: a graph
    that has saved one of them refuses its backward pass."""
    for x in tensors:
        if x is not None:
            torch.autograd.graph.increment_version(x)


class _Call:
    """What a differentiable call's backward pass needs beside the logits. (One object in place of
    arguments and saved tensors: autograd takes its time for each of those. Inputs that were
    changed in between are noticed here, as autograd notices it of the logits.) ``described`` is
    for the forward call alone: the logits that autograd hands back may be others in another place
    (recomputed under a checkpoint, or copied by a hook for saved tensors)."""
    __slots__ = ("described", "temperature", "inputs", "versions", "row_stats", "results", "args")

    def __init__(self, described, temperature, inputs, row_stats, args):
        # (a number: a tensor given for it may change before the backward pass)
        self.described, self.temperature, self.inputs = described, float(temperature), inputs
        self.row_stats, self.args, self.results = row_stats, args, None

    def begun(self):
        """To be called when the forward call has written its results."""
        self.versions = [_version(x) for x in (*self.inputs, self.row_stats)]

    def check(self):
        if [_version(x) for x in (*self.inputs, self.row_stats)] != self.versions:
            raise RuntimeError("an input or the row_stats of the forward call has been changed in "
                               "place since")


def _refuse_tangents(logits):
    # (nobody's outside of a dual level, which is known at once)
    if forward_ad._current_level >= 0 and forward_ad.unpack_dual(logits).tangent is not None:
        raise NotImplementedError("log probabilities and divergences have no forward-mode derivatives")


def _saved(ctx):
    """(logits, packed struct sv_logit_rows of where they are now, call) of a backward pass."""
    (logits,), call = ctx.saved_tensors, ctx.call
    call.check()
    if logits.stride(-1) != 1:
        logits = logits.contiguous()
    return logits, _describe(logits, call.temperature)[0], call


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, call):
        """The differentiable results; the others are in call.results."""
        if call.row_stats is None:
            call.row_stats = torch.empty((*call.described[2], SV_ROW_STATS), dtype=torch.float32,
                                         device=logits.device)
        call.results = out = _logprobs(call.described, logits, *call.args, call.row_stats)
        call.begun()
        call.described = None
        ctx.save_for_backward(logits)
        ctx.call = call
        ctx.set_materialize_grads(False)
        return out.logprobs, out.entropy, out.lse

    @staticmethod
    def backward(ctx, *grads):
        return (_logprobs_backward_once if torch.is_grad_enabled() else _logprobs_backward)(
            ctx, *grads)


def _logprobs_backward(ctx, grad_logprobs, grad_entropy, grad_lse):
    logits, rows, call = _saved(ctx)
    grads = [None if g is None else g.contiguous() for g in (grad_logprobs, grad_entropy, grad_lse)]
    out = _grad_like(logits)
    _check(_lib.load_logprobs().sv_token_logprobs_backward(
        rows, call.inputs[0].data_ptr() if call.inputs else None, call.row_stats.data_ptr(),
        *[None if g is None else g.data_ptr() for g in grads], out.data_ptr(), *_strides(out)[2:],
        torch._C._cuda_getCurrentRawStream(logits.device.index)), "sv_token_logprobs_backward")
    return out, None


# (refuses second derivatives; only where a graph of the backward pass is asked for, since it takes
# its time)
_logprobs_backward_once = torch.autograd.function.once_differentiable(_logprobs_backward)


def sv_token_logprobs(logits, tokens=None, *, temperature: float = 1.0, top_k: int = 0,
                      row_stats=None, row_status=None, workspace=None,
                      stream=None) -> TokenLogprobs:
    """Log probabilities of ``tokens`` (int32, one for each row) under softmax(logits / temperature),
    their ranks (how many tokens are ahead; ties go to the lower index), the rows' entropies and
    log-sum-exps, and with ``top_k`` the first tokens in order with their log probabilities.

    A token of -1, as ``spec_verify`` leaves behind a sequence's last one, asks nothing of its row:
    the row is not read and gets zeros, rank and top tokens -1, top log probabilities -inf. Without
    ``tokens`` there are no log probabilities and ranks. ``row_status``: int32, receives SV_SEQ_BAD_TOKEN
    and SV_SEQ_NONFINITE for rows whose results are NaN. ``row_stats``: float32 [..., SV_ROW_STATS], receives
    what ``sv_token_logprobs_backward`` needs. Differentiable in the logits (logprobs, entropy and
    lse). A workspace is kept for the thread and stream unless one is given
    (``sv_logprobs_workspace_bytes``, its first SV_LOGPROBS_COUNTER_BYTES zeros when it is new).
    Asynchronous on ``stream`` (default: the current stream of the logits' device)."""
    described = _describe(logits, temperature)
    _refuse_tangents(logits)

    def call(_):
        if logits.requires_grad and torch.is_grad_enabled():
            c = _Call(described, temperature, () if tokens is None else (tokens,), row_stats,
                      (tokens, top_k, row_status, workspace))
            logprobs, entropy, lse = _TokenLogprobs.apply(logits, c)
            _, rank, _, _, top_tokens, top_logprobs = c.results
            c.results = None
            return TokenLogprobs(logprobs, rank, entropy, lse, top_tokens, top_logprobs)
        return _logprobs(described, logits, tokens, top_k, row_status, workspace, row_stats)

    return _on(logits.device, stream, call, (logits, tokens, row_stats, row_status, workspace))


def sv_token_logprobs_backward(logits, row_stats, *, tokens=None, grad_logprobs=None,
                               grad_entropy=None, grad_lse=None, temperature: float = 1.0,
                               grad=None, stream=None):
    """The logits' gradient from those of ``sv_token_logprobs``' log probabilities, entropies and
    log-sum-exps (float32, one for each row; None: zeros), with the ``row_stats`` that it filled.
    ``tokens`` may be others than the forward call's, or given here alone; rows whose token is out of
    range get NaN, rows of token -1 zeros. ``grad`` may be the logits themselves, whose values are
    then gone."""
    rows, dev, shape = _describe(logits, temperature)
    f32 = torch.float32
    ptrs = [_per_row(tokens, "tokens", shape, torch.int32, dev),
            _per_row(row_stats, "row_stats", shape, f32, dev, (SV_ROW_STATS,)),
            _per_row(grad_logprobs, "grad_logprobs", shape, f32, dev),
            _per_row(grad_entropy, "grad_entropy", shape, f32, dev),
            _per_row(grad_lse, "grad_lse", shape, f32, dev)]
    if grad is not None:
        _check_grad(grad, logits)

    def call(s):
        g = _grad_like(logits) if grad is None else grad
        _check(_lib.load_logprobs().sv_token_logprobs_backward(
            rows, *ptrs, g.data_ptr(), *_strides(g)[2:], s), "sv_token_logprobs_backward")
        _wrote(grad)
        return g

    return _on(dev, stream, call, (logits, row_stats, tokens, grad_logprobs, grad_entropy, grad_lse,
                                   grad))


def _teacher(teacher_tokens, teacher_logprobs, shape, dev, tail):
    """(address of tokens, of log probabilities, entries a row, code of tail)."""
    if teacher_tokens.dim() != len(shape) + 1:
        raise ValueError("teacher_tokens must be [..., k], beside logits [..., V]")
    k = teacher_tokens.shape[-1]
    if not 1 <= k <= SV_MAX_TOP:
        raise ValueError(f"a teacher has from 1 to {SV_MAX_TOP} entries a row")
    if tail not in _TAILS:
        raise ValueError(f"tail must be one of {sorted(_TAILS)}, got {tail!r}")
    return (_per_row(teacher_tokens, "teacher_tokens", shape, torch.int32, dev, (k,)),
            _per_row(teacher_logprobs, "teacher_logprobs", shape, torch.float32, dev, (k,)), k,
            _TAILS[tail])


def _distill(described, logits, teacher_tokens, teacher_logprobs, weights, tail, loss, grad,
             row_stats, row_status, workspace):
    """Calls sv_distill on the current stream; grad: a tensor or None."""
    rows, dev, shape = described
    stream = torch._C._cuda_getCurrentRawStream(dev.index)
    teacher = _teacher(teacher_tokens, teacher_logprobs, shape, dev, tail)
    f32 = torch.float32
    weights_ptr = _per_row(weights, "weights", shape, f32, dev)
    if loss is None:
        loss = torch.empty(shape, dtype=f32, device=dev)
    ptrs = (_per_row(loss, "loss", shape, f32, dev), None, 0, 0)
    if grad is not None:
        ptrs = (ptrs[0], grad.data_ptr(), *_strides(grad)[2:])
    _check(_lib.load_logprobs().sv_distill(
        rows, *teacher, weights_ptr, *ptrs,
        _per_row(row_stats, "row_stats", shape, f32, dev, (SV_ROW_STATS,)),
        _per_row(row_status, "row_status", shape, torch.int32, dev),
        *_workspace(workspace, logits, shape.numel(), 0, stream), stream), "sv_distill")
    _wrote(row_status)
    return loss


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, call):
        tail, row_status, workspace = call.args
        call.row_stats = torch.empty((*call.described[2], SV_ROW_STATS), dtype=torch.float32,
                                     device=logits.device)
        ctx.save_for_backward(logits)
        ctx.call = call
        loss = _distill(call.described, logits, *call.inputs, None, tail, None, None, call.row_stats,
                        row_status, workspace)
        call.begun()
        call.described = None
        return loss

    @staticmethod
    def backward(ctx, grad_loss):
        return (_distill_backward_once if torch.is_grad_enabled() else _distill_backward)(
            ctx, grad_loss)


def _distill_backward(ctx, grad_loss):
    logits, rows, call = _saved(ctx)
    tokens, logprobs = call.inputs
    grad_loss, out = grad_loss.contiguous(), _grad_like(logits)
    _check(_lib.load_logprobs().sv_distill_backward(
        rows, tokens.data_ptr(), logprobs.data_ptr(), tokens.shape[-1], _TAILS[call.args[0]],
        call.row_stats.data_ptr(), grad_loss.data_ptr(), out.data_ptr(), *_strides(out)[2:],
        torch._C._cuda_getCurrentRawStream(logits.device.index)), "sv_distill_backward")
    return out, None


_distill_backward_once = torch.autograd.function.once_differentiable(_distill_backward)


def sv_distill_loss(logits, teacher_tokens, teacher_logprobs, *, temperature: float = 1.0,
                    tail: str = "renormalise", row_status=None, workspace=None, stream=None):
    """Divergence (float32, one for each row) of a teacher from softmax(logits / temperature),
    differentiable in the logits. The teacher's rows are k tokens (int32, -1 for none; a token given
    twice has both probabilities) and their log probabilities (float32): ``sv_token_logprobs``'
    ``top_tokens`` and ``top_logprobs``, at the same temperature. ``tail`` says what becomes of the
    probability that they leave: "renormalise" scales the k to sum 1 (their logits over the
    temperature do as well, then), "bucket" makes one outcome of all other tokens. Rows without a
    teacher have loss 0 and are not read. ``row_status`` and ``workspace`` as in
    ``sv_token_logprobs``."""
    described = _describe(logits, temperature)
    _refuse_tangents(logits)

    def call(_):
        if logits.requires_grad and torch.is_grad_enabled():
            return _DistillLoss.apply(logits, _Call(
                described, temperature, (teacher_tokens, teacher_logprobs), None,
                (tail, row_status, workspace)))
        return _distill(described, logits, teacher_tokens, teacher_logprobs, None, tail, None, None,
                        None, row_status, workspace)

    return _on(logits.device, stream, call, (logits, teacher_tokens, teacher_logprobs, row_status,
                                             workspace))


def sv_distill(logits, teacher_tokens, teacher_logprobs, *, weights=None, temperature: float = 1.0,
               tail: str = "renormalise", loss=None, grad=None, row_stats=None, row_status=None,
               workspace=None, stream=None):
    """``sv_distill_loss`` and its gradient at once: (loss, grad), grad being the logits' gradient of
    the sum of ``weights`` (float32, one for each row; default 1) times the losses. Continue with
    ``logits.backward(grad)``, or with the head's products. ``grad`` may be the logits themselves,
    whose values are then gone. Arguments otherwise as in ``sv_distill_loss``; ``row_stats``
    (float32 [..., SV_ROW_STATS]) receives what ``sv_distill_backward`` needs."""
    described = _describe(logits, temperature)
    if grad is not None:
        _check_grad(grad, logits)

    def call(_):
        g = _grad_like(logits) if grad is None else grad
        result = _distill(described, logits, teacher_tokens, teacher_logprobs, weights, tail, loss, g,
                          row_stats, row_status, workspace)
        _wrote(loss, grad, row_stats)
        return result, g

    return _on(logits.device, stream, call, (logits, teacher_tokens, teacher_logprobs, weights, loss,
                                             grad, row_stats, row_status, workspace))


def sv_distill_backward(logits, teacher_tokens, teacher_logprobs, row_stats, grad_loss, *,
                        temperature: float = 1.0, tail: str = "renormalise", grad=None,
                        stream=None):
    """The logits' gradient from that of ``sv_distill``'s losses (float32, one for each row), with the
    ``row_stats`` that it filled for the same logits and teacher."""
    rows, dev, shape = _describe(logits, temperature)
    teacher = _teacher(teacher_tokens, teacher_logprobs, shape, dev, tail)
    ptrs = (_per_row(row_stats, "row_stats", shape, torch.float32, dev, (SV_ROW_STATS,)),
            _per_row(grad_loss, "grad_loss", shape, torch.float32, dev))
    if grad is not None:
        _check_grad(grad, logits)

    def call(s):
        g = _grad_like(logits) if grad is None else grad
        _check(_lib.load_logprobs().sv_distill_backward(
            rows, *teacher, *ptrs, g.data_ptr(), *_strides(g)[2:], s), "sv_distill_backward")
        _wrote(grad)
        return g

    return _on(dev, stream, call, (logits, teacher_tokens, teacher_logprobs, row_stats, grad_loss,
                                   grad))
