"""Binding of the row operators of the C ABI (``include/spec_verify.h``): top
log-probabilities, distillation of the draft, beam search.

Argument marshalling only, like :mod:`.api`: tensors are checked for device,
dtype, shape and strides, and every computation runs in the library's CUDA
kernels on the current stream of the tensors' device (or ``stream``).

Logits are ``[B, K, V]`` or ``[R, V]`` (K = 1), bfloat16 or float32, with a
contiguous vocabulary axis and any other strides (0 repeats a row). ``status``
is an int32 CUDA tensor of one element or None; the calls leave the largest
device-side code there and never clear it.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _native
from .api import BF16, F32, MAX_V, SPEC_ERR_UNSUPPORTED, SPEC_OK, SpecError

MAX_TOP = 128
MAX_BEAMS = 32
MAX_BEAM_OUT = 64
MAX_B = 1 << 24
MAX_K_ROWS = 4096

_DTYPES = {torch.bfloat16: BF16, torch.float32: F32}
_F32, _I32 = torch.float32, torch.int32
_current_device = torch.cuda.current_device


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):   # the same number without the Stream object
    _raw_stream = torch._C._cuda_getCurrentRawStream


def _run(t: torch.Tensor, stream, body):
    """body(stream pointer) with the device of ``t`` current, and on ``stream``
    where one is given (so that outputs are allocated on the stream that
    writes them)."""
    index = t.device.index
    if stream is None:
        if index == _current_device():
            return body(_raw_stream(index))
        with torch.cuda.device(index):
            return body(_raw_stream(index))
    if stream.device != t.device:
        raise ValueError("stream must be a stream of the tensors' device")
    with torch.cuda.device(index), torch.cuda.stream(stream):
        return body(stream.cuda_stream)


def _check(rc: int):
    if rc != SPEC_OK:
        raise SpecError(rc, _native.last_error())


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _logits(z: torch.Tensor, name: str):
    """(B, K, V, dtype code, batch stride, row stride) of a logits tensor."""
    if not z.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    dt = _DTYPES.get(z.dtype)
    if dt is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {z.dtype}")
    shape = z.shape
    if len(shape) == 3:
        B, K, V = shape
        bs, rs, vs = z.stride()
    elif len(shape) == 2:
        (B, V), K = shape, 1
        (bs, vs), rs = z.stride(), 0
    else:
        raise ValueError(f"{name} must be [B, K, V] or [R, V]")
    if vs != 1 and V > 1:
        raise ValueError(f"{name}: the vocabulary axis must be contiguous")
    if B > MAX_B or K > MAX_K_ROWS or V > MAX_V:   # before the C ABI's 32-bit fields
        raise SpecError(SPEC_ERR_UNSUPPORTED, f"{name}: {tuple(shape)} is outside the supported range")
    return B, K, V, dt, bs, rs


def _tensor(t, name, dtype, shape, device, optional=True):
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is missing")
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on the logits' device")


def _status(status, device):
    if status is not None and (status.dtype != torch.int32 or status.numel() != 1 or status.device != device):
        raise ValueError("status must be an int32 tensor of one element on the logits' device")


# Tells autograd that a call has written into tensors of the caller's. All of them
# count: a detached alias shares its counter with a tensor that a backward pass may
# need, and so does a tensor without a gradient that another's backward pass keeps.
# Called after the write, so that a refused call leaves the counters alone.
_written = torch.autograd.graph.increment_version


def _out(out, name, dtype, shape, device):
    t = None if out is None else out.get(name)
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _tensor(t, f"out['{name}']", dtype, torch.Size(shape), device)
    return t


def top_logprobs(logits: torch.Tensor, M: int, inv_temperature: float = 1.0, out: Optional[dict] = None,
                 status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> dict:
    """The M (1..128) largest log-probabilities of every row
    (spec_top_logprobs): a dict with ``logprobs`` [B,K,M] float32, descending,
    ``ids`` [B,K,M] int32 and ``lse`` [B,K] float32 ([R,M] and [R] for [R,V]
    logits). Unfilled places (masked tokens) are -inf and -1. ``out`` may hold
    tensors to write into, under the same keys."""
    B, K, V, dt, bs, rs = _logits(logits, "logits")
    dev, lead = logits.device, tuple(logits.shape[:-1])
    _status(status, dev)
    if not 1 <= M <= MAX_TOP:
        raise SpecError(SPEC_ERR_UNSUPPORTED, f"top_logprobs: M must be in [1, {MAX_TOP}]")
    p = _native.RowsParams(B, K, V, dt, M, 0, inv_temperature, 0, bs, rs)

    def body(s):
        lp = _out(out, "logprobs", _F32, lead + (M,), dev)
        ids = _out(out, "ids", _I32, lead + (M,), dev)
        lse = _out(out, "lse", _F32, lead, dev)
        _check(_native.lib().spec_top_logprobs(ctypes.byref(p), logits.data_ptr(), lp.data_ptr(), ids.data_ptr(),
                                               lse.data_ptr(), _addr(status), s))
        if out is not None:
            _written((lp, ids, lse))
        return {"logprobs": lp, "ids": ids, "lse": lse}

    return _run(logits, stream, body)


def _distill_args(logits, logprobs, ids, weight, inv_temperature, tail, status):
    B, K, V, dt, bs, rs = _logits(logits, "logits")
    dev, lead = logits.device, logits.shape[:-1]
    M = logprobs.shape[-1] if logprobs.dim() else 0
    _tensor(logprobs, "logprobs", torch.float32, lead + (M,), dev, optional=False)
    _tensor(ids, "ids", torch.int32, lead + (M,), dev, optional=False)
    _tensor(weight, "weight", torch.float32, lead, dev)
    _status(status, dev)
    return _native.RowsParams(B, K, V, dt, M, 1 if tail else 0, inv_temperature, 0, bs, rs), dev, lead


def distill_loss(logits: torch.Tensor, logprobs: torch.Tensor, ids: torch.Tensor,
                 weight: Optional[torch.Tensor] = None, inv_temperature: float = 1.0, tail: bool = True,
                 out: Optional[dict] = None, status: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Distillation loss of the student's ``logits`` [B,K,V] from a teacher's
    top list (spec_distill_loss): ``logprobs`` and ``ids`` [B,K,M] as
    top_logprobs returns them, ``weight`` [B,K] or None (1). Returns ``loss``
    [B,K] float32 and ``stats`` [B,K,4] float32, which distill_grad takes. The
    loss is no part of an autograd graph, whether or not the logits are: its
    gradient comes from distill_grad or distill_step."""
    p, dev, lead = _distill_args(logits, logprobs, ids, weight, inv_temperature, tail, status)

    def body(s):
        loss = _out(out, "loss", _F32, lead, dev)
        stats = _out(out, "stats", _F32, lead + (4,), dev)
        _check(_native.lib().spec_distill_loss(ctypes.byref(p), logits.data_ptr(), logprobs.data_ptr(), ids.data_ptr(),
                                               _addr(weight), loss.data_ptr(), stats.data_ptr(), _addr(status), s))
        if out is not None:
            _written((loss, stats))
        return {"loss": loss, "stats": stats}

    return _run(logits, stream, body)


def _dlogits(out, logits):
    """The gradient's tensor and its two strides."""
    if out is None:
        out = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    elif out.dtype != logits.dtype or out.shape != logits.shape or out.device != logits.device:
        raise ValueError("dlogits must have the logits' dtype, shape and device")
    _, _, _, _, bs, rs = _logits(out, "dlogits")
    return out, bs, rs


def distill_grad(logits: torch.Tensor, logprobs: torch.Tensor, ids: torch.Tensor, stats: torch.Tensor,
                 grad_loss: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                 inv_temperature: float = 1.0, tail: bool = True, out: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Gradient of sum(grad_loss * loss) by the logits (spec_distill_grad),
    from distill_loss's ``stats`` and the same other arguments; ``grad_loss``
    [B,K] or None (1). ``out`` may be any tensor of the logits' shape and
    dtype, the logits themselves too (else it must not overlap them). Returns
    the gradient, which
    ``logits.backward(gradient)`` takes on through the draft model."""
    p, dev, lead = _distill_args(logits, logprobs, ids, weight, inv_temperature, tail, status)
    _tensor(stats, "stats", torch.float32, lead + (4,), dev, optional=False)
    _tensor(grad_loss, "grad_loss", torch.float32, lead, dev)

    def body(s):
        g, bs, rs = _dlogits(out, logits)
        _check(_native.lib().spec_distill_grad(ctypes.byref(p), logits.data_ptr(), logprobs.data_ptr(), ids.data_ptr(),
                                               _addr(weight), stats.data_ptr(), _addr(grad_loss), g.data_ptr(), bs, rs,
                                               _addr(status), s))
        if out is not None:
            _written(g)
        return g

    return _run(logits, stream, body)


def distill_step(logits: torch.Tensor, logprobs: torch.Tensor, ids: torch.Tensor,
                 weight: Optional[torch.Tensor] = None, inv_temperature: float = 1.0, tail: bool = True,
                 out: Optional[dict] = None, status: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Loss and gradient in one call (spec_distill_step): ``loss`` [B,K]
    float32 and ``dlogits`` [B,K,V], the gradient of loss.sum(); scale it by
    ``weight`` (a mean's 1/n, a loss scale). ``out['dlogits']`` may be the
    logits themselves, and must not overlap them otherwise."""
    p, dev, lead = _distill_args(logits, logprobs, ids, weight, inv_temperature, tail, status)

    def body(s):
        loss = _out(out, "loss", _F32, lead, dev)
        g, bs, rs = _dlogits(None if out is None else out.get("dlogits"), logits)
        _check(_native.lib().spec_distill_step(ctypes.byref(p), logits.data_ptr(), logprobs.data_ptr(), ids.data_ptr(),
                                               _addr(weight), loss.data_ptr(), g.data_ptr(), bs, rs, _addr(status), s))
        if out is not None:
            _written((loss, g))
        return {"loss": loss, "dlogits": g}

    return _run(logits, stream, body)


def beam_step(logits: torch.Tensor, scores: torch.Tensor, N: int, finished: Optional[torch.Tensor] = None,
              eos: int = -1, out: Optional[dict] = None, status: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> dict:
    """One step of beam search (spec_beam_step): the N best continuations of
    the W beams of every sequence, from ``logits`` [B,W,V], cumulative
    ``scores`` [B,W] float32 (-inf: no beam; at the first step all but one) and
    ``finished`` [B,W] int32 or None. Returns ``scores`` [B,N] float32,
    ``parent``, ``token`` and ``finished`` [B,N] int32."""
    if logits.dim() != 3:
        raise ValueError("logits must be [B, W, V]")
    B, W, V, dt, bs, rs = _logits(logits, "logits")
    dev = logits.device
    _tensor(scores, "scores", _F32, (B, W), dev, optional=False)
    _tensor(finished, "finished", _I32, (B, W), dev)
    _status(status, dev)
    if not 1 <= N <= MAX_BEAM_OUT:
        raise SpecError(SPEC_ERR_UNSUPPORTED, f"beam_step: N must be in [1, {MAX_BEAM_OUT}]")
    if not -1 <= eos < V:
        raise ValueError("eos must be -1 or a token")
    p = _native.RowsParams(B, W, V, dt, N, 0, 1.0, 0, bs, rs)

    def body(s):
        sc = _out(out, "scores", _F32, (B, N), dev)
        par = _out(out, "parent", _I32, (B, N), dev)
        tok = _out(out, "token", _I32, (B, N), dev)
        fin = _out(out, "finished", _I32, (B, N), dev)
        _check(_native.lib().spec_beam_step(ctypes.byref(p), logits.data_ptr(), scores.data_ptr(), _addr(finished),
                                            eos, sc.data_ptr(), par.data_ptr(), tok.data_ptr(), fin.data_ptr(),
                                            _addr(status), s))
        if out is not None:
            _written((sc, par, tok, fin))
        return {"scores": sc, "parent": par, "token": tok, "finished": fin}

    return _run(logits, stream, body)


def _merged(shape, stride):
    """One (count, stride) for several axes, or None where they do not merge."""
    n, st = 1, 0
    for c, k in zip(reversed(shape), reversed(stride)):
        if c == 1:
            continue
        if n > 1 and k != n * st:
            return None
        if n == 1:
            st = k
        n *= c
    return n, st


def _layout(t, batch_dim, length_dim, name):
    shape, stride, es = t.shape, t.stride(), t.element_size()
    outer = _merged(shape[:batch_dim], stride[:batch_dim])
    seg = _merged(shape[batch_dim + 2:length_dim], stride[batch_dim + 2:length_dim])
    unit = 1
    for c, k in zip(reversed(shape[length_dim + 1:]), reversed(stride[length_dim + 1:])):
        if c != 1 and k != unit:
            raise ValueError(f"{name}: the axes after the length axis must be contiguous")
        unit *= c
    if shape[length_dim] > 1 and unit and stride[length_dim] != unit:
        raise ValueError(f"{name}: the length axis must be contiguous with the axes after it")
    if outer is None or seg is None:
        raise ValueError(f"{name}: the axes before the batch, and those between beam and length, must each be "
                         "evenly spaced")
    st = [outer[1] * es, stride[batch_dim] * es, stride[batch_dim + 1] * es, seg[1] * es]
    return outer[0], shape[batch_dim], shape[batch_dim + 1], seg[0], shape[length_dim], unit * es, st


def beam_reorder(state: torch.Tensor, parent: torch.Tensor, lengths: Optional[torch.Tensor] = None,
                 batch_dim: int = 0, length_dim: int = -2, out: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """States in the order of the surviving beams (spec_beam_reorder): row
    (..., b, n, ...) becomes row (..., b, parent[b, n], ...), ``parent`` [B,N]
    int32, -1 leaves the row. Axis ``batch_dim`` is the sequence, the next one
    the beam. With ``lengths`` [B] int32 only the first lengths[b] entries of
    axis ``length_dim`` move; without, whole rows do, of a state cut out of a
    larger buffer along any one axis too. In place (``out`` None or ``state``), else into
    ``out``, whose beam axis has N rows and which must not overlap the state.
    Any dtype."""
    if not state.is_cuda:
        raise ValueError("state must be a CUDA tensor")
    dst = state if out is None else out
    nd, dev = state.dim(), state.device
    if dst is not state:
        if dst.dim() != nd or dst.dtype != state.dtype or dst.device != dev:
            raise ValueError("out must have the state's dtype, device and number of axes")
        if dst.is_conj() != state.is_conj() or dst.is_neg() != state.is_neg():   # bytes are moved, not values
            raise ValueError("out and state must both be conjugated or negated views, or neither")
    bd = batch_dim + nd if batch_dim < 0 else batch_dim
    if not 0 <= bd < nd - 1:
        raise ValueError("state must have a batch and a beam axis")
    if lengths is None:
        ld = bd + 2
        if ld == nd:   # [.., B, W]: one unit per row
            state_v, dst_v = state.unsqueeze(-1), dst.unsqueeze(-1)
        else:
            state_v, dst_v = state, dst
        # whole rows: any axis may divide them, the first that fits gives the longest segments
        while ld < state_v.dim() - 1 and (_try_layout(state_v, bd, ld) is None or
                                          (dst is not state and _try_layout(dst_v, bd, ld) is None)):
            ld += 1
    else:
        ld = length_dim + nd if length_dim < 0 else length_dim
        if not bd + 2 <= ld < nd:
            raise ValueError("length_dim must lie behind the beam axis")
        state_v, dst_v = state, dst
    O, B, W, H, T, unit, ss = _layout(state_v, bd, ld, "state")
    N, ds = W, ss
    if dst is not state:
        ds = _layout(dst_v, bd, ld, "out")[-1]
        N = dst.shape[bd + 1]
        if dst.shape[:bd + 1] != state.shape[:bd + 1] or dst.shape[bd + 2:] != state.shape[bd + 2:]:
            raise ValueError("out must have the state's shape, but for the beam axis")
    if parent.dim() != 2 or parent.shape[0] != B or (dst is not state and parent.shape[1] != N):
        raise ValueError("parent must be int32 [B, N]")
    N = parent.shape[1]
    _tensor(parent, "parent", _I32, (B, N), dev, optional=False)
    _tensor(lengths, "lengths", _I32, (B,), dev)
    _status(status, dev)
    if unit == 0:
        return dst
    if O > 65535 or H > 65535 or B > MAX_B or T >= 1 << 31 or unit > 1 << 30:   # before 32-bit fields
        raise SpecError(SPEC_ERR_UNSUPPORTED, "beam_reorder: the state's axes are outside the supported range")
    p = _native.ReorderParams(O, B, W, N, H, T, unit)
    p.src_stride[:] = ss
    p.dst_stride[:] = ds

    def body(s):
        _check(_native.lib().spec_beam_reorder(ctypes.byref(p), state.data_ptr(), dst.data_ptr(), parent.data_ptr(),
                                               _addr(lengths), _addr(status), s))
        _written(dst)
        return dst

    return _run(state, stream, body)


def _try_layout(t, bd, ld):
    try:
        return _layout(t, bd, ld, "")
    except ValueError:
        return None
