"""Binding of the tree operators of the C ABI (``include/spec_verify.h``):
attention of a tree of drafts over a cache held in pages, the accepted path,
and the upkeep of the pages.

Argument marshalling only, like :mod:`.rows`, with the same ``out``, ``status``
and ``stream`` arguments. A ``table`` [rows, M] int32 names a row's pages in
order (-1: none), ``refs`` [P] int32 counts the entries that name a page (0:
free), ``lengths`` int32 are tokens. One decoding step::

    t = sv.pages_resize(table, refs, lengths + N, page, out={"table": table, "refs": refs})
    ...                                        # in every layer: write the nodes' keys and values,
    a = sv.tree_attention(q, k, v, table, lengths, parents)
    ...                                        # on to the logits [B, N, V] of the nodes
    choice = sv.top_logprobs(logits, 1)["ids"][..., 0]
    r = sv.tree_accept(tokens, parents, choice)
    lengths = sv.pages_compact(cache, table, lengths, r["path"], page_dim=2)
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence, Union

import torch

from . import _native
from .api import BF16, SPEC_ERR_UNSUPPORTED, SpecError
from .rows import _addr, _check, _merged, _run, _written

MAX_NODES = 128
F16 = 2

_TYPES = {torch.bfloat16: BF16, torch.float16: F16}
_F32, _I32 = torch.float32, torch.int32
_MOST = (1 << 31) - 1
_I3 = ctypes.c_int64 * 3


def _need(t, name, shape, device, dtype=_I32):
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on {device}")


def _maybe(t, name, shape, device):
    if t is not None:
        _need(t, name, shape, device)


def _on_gpu(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _status(status, device):
    if status is not None and (status.dtype != _I32 or status.numel() != 1 or status.device != device):
        raise ValueError(f"status must be an int32 tensor of one element on {device}")


def _new(out, name, shape, device, dtype=_I32):
    t = None if out is None else out.get(name)
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(t, f"out['{name}']", torch.Size(shape), device, dtype)
    return t


def _small(what, *sizes):
    if max(sizes) > _MOST or min(sizes) < -_MOST:   # before the C ABI's 32-bit fields
        raise SpecError(SPEC_ERR_UNSUPPORTED, f"{what}: a size is outside the supported range")


def _parents(parents, B, N, device):
    """The batch stride of a tree per sequence [B, N], or of one [N] for all."""
    if parents is None:
        return 0
    if parents.dim() == 1:
        _need(parents, "parents", (N,), device)
        return 0
    _need(parents, "parents", (B, N), device)
    return N


def tree_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor,
                   parents: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                   scale: Optional[float] = None, out: Optional[dict] = None,
                   status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Attention of a tree's nodes over the cache (spec_tree_attention): ``q``
    [B,N,Hq,D], ``k`` and ``v`` [P,page,Hkv,D] bfloat16 or float16 with D
    contiguous (other axes in any order of strides), ``table`` [B,M],
    ``lengths`` [B] tokens before the nodes, whose own keys and values lie in
    slots lengths[b] + n. ``parents`` [B,N] or [N] int32 (None: a chain),
    ``counts`` [B] int32 or None (N). ``scale`` None is D ** -0.5. Returns ``out``
    [B,N,Hq,D] and ``lse`` [B,N,Hq] float32. No part of an autograd graph."""
    dev, dtype = _on_gpu(q, "q"), q.dtype
    dt = _TYPES.get(dtype)
    if dt is None:
        raise TypeError(f"q must be bfloat16 or float16, got {dtype}")
    qshape, kshape = q.shape, k.shape
    if len(qshape) != 4 or len(kshape) != 4 or v.shape != kshape:
        raise ValueError("q must be [B, N, Hq, D], k and v [P, page, Hkv, D]")
    if k.dtype != dtype or v.dtype != dtype or k.device != dev or v.device != dev:
        raise ValueError("q, k and v must have one dtype and device")
    B, N, Hq, D = qshape
    P, page, Hkv, Dk = kshape
    if Dk != D:
        raise ValueError("q, k and v must have the same head size")
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    if (qs[3] != 1 or ks[3] != 1 or vs[3] != 1) and D > 1:
        raise ValueError("q, k and v: the head's elements must be contiguous")
    if table.dim() != 2:
        raise ValueError("table must be [B, M]")
    M = table.shape[1]
    _need(table, "table", (B, M), dev)
    _need(lengths, "lengths", (B,), dev)
    _maybe(counts, "counts", (B,), dev)
    ps = _parents(parents, B, N, dev)
    _status(status, dev)
    _small("tree_attention", B, N, Hq, P, page, Hkv, D, M)
    p = _native.AttendParams(B, N, Hq, Hkv, D, dt, P, page, M, max(D, 1) ** -0.5 if scale is None else scale, _I3(*qs[:3]),
                             _I3(*ks[:3]), _I3(*vs[:3]), ps)

    def body(s):
        L = _native.lib()
        o = _new(out, "out", qshape, dev, dtype)
        lse = _new(out, "lse", (B, N, Hq), dev, _F32)
        size = L.spec_tree_attention_workspace_size(ctypes.byref(p))
        ws = torch.empty(size, dtype=torch.uint8, device=dev)
        _check(L.spec_tree_attention(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(), table.data_ptr(),
                                     lengths.data_ptr(), _addr(parents), _addr(counts), o.data_ptr(), lse.data_ptr(),
                                     ws.data_ptr(), size, _addr(status), s))
        if out is not None:
            _written((o, lse))
        return {"out": o, "lse": lse}

    return _run(q, stream, body)


def tree_accept(tokens: torch.Tensor, parents: Optional[torch.Tensor], choice: torch.Tensor,
                counts: Optional[torch.Tensor] = None, out: Optional[dict] = None,
                status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> dict:
    """The accepted path of a tree (spec_tree_accept): ``tokens`` [B,N] int32
    (node 0 the context's last token), ``parents`` [B,N], [N] or None (a chain),
    ``choice`` [B,N] int32 with any strides, the target's token after each
    node. Returns ``accepted_len`` [B], ``out_tokens`` [B,N] and ``path`` [B,N]
    int32, filled up with -1."""
    dev = _on_gpu(tokens, "tokens")
    if tokens.dim() != 2:
        raise ValueError("tokens must be [B, N]")
    B, N = tokens.shape
    _need(tokens, "tokens", (B, N), dev)
    if choice.dtype != _I32 or choice.shape != tokens.shape or choice.device != dev:
        raise ValueError(f"choice must be an int32 tensor {[B, N]} on {dev}")
    _maybe(counts, "counts", (B,), dev)
    ps = _parents(parents, B, N, dev)
    _status(status, dev)
    _small("tree_accept", B, N)

    def body(s):
        acc = _new(out, "accepted_len", (B,), dev)
        tok = _new(out, "out_tokens", (B, N), dev)
        path = _new(out, "path", (B, N), dev)
        _check(_native.lib().spec_tree_accept(B, N, tokens.data_ptr(), _addr(parents), ps, choice.data_ptr(),
                                              choice.stride(0), choice.stride(1), _addr(counts), acc.data_ptr(),
                                              tok.data_ptr(), path.data_ptr(), _addr(status), s))
        if out is not None:
            _written((acc, tok, path))
        return {"accepted_len": acc, "out_tokens": tok, "path": path}

    return _run(tokens, stream, body)


def _cache_params(t, page_dim, slot_dim, P, page):
    """The layout of a cache [.., P, .., page, ..] of the given pool (None: its own)."""
    nd = t.dim()
    pd = page_dim + nd if page_dim < 0 else page_dim
    sd = pd + 1 if slot_dim is None else slot_dim + nd if slot_dim < 0 else slot_dim
    if not 0 <= pd < sd < nd:
        raise ValueError("cache must have a page axis and a slot axis behind it")
    shape, stride, es = t.shape, t.stride(), t.element_size()
    if P is not None and shape[pd] != P or page is not None and shape[sd] != page:
        raise ValueError("caches and refs must have the same pages")
    if 0 in shape[sd + 1:]:   # nothing to move
        return _native.CacheParams(0, shape[pd], 0, shape[sd], es)
    if t.is_contiguous():   # (strides from the shape: those of axes of one entry say nothing)
        O, H, unit = math.prod(shape[:pd]), math.prod(shape[pd + 1:sd]), math.prod(shape[sd + 1:])
        seg = shape[sd] * unit
        return _params((O, shape[pd] * H * seg if O > 1 else 0), (H, seg if H > 1 else 0), shape[pd], H * seg, shape[sd], unit, es)
    unit = 1
    for c, k in zip(reversed(shape[sd + 1:]), reversed(stride[sd + 1:])):
        if c != 1 and k != unit:
            raise ValueError("cache: the axes after the slot axis must be contiguous")
        unit *= c
    if shape[sd] > 1 and stride[sd] != unit:
        raise ValueError("cache: the slot axis must be contiguous with the axes after it")
    outer, seg = _merged(shape[:pd], stride[:pd]), _merged(shape[pd + 1:sd], stride[pd + 1:sd])
    if outer is None or seg is None:
        raise ValueError("cache: the axes before the pages, and those between page and slot, must each be evenly spaced")
    return _params(outer, seg, shape[pd], stride[pd], shape[sd], unit, es)


def _params(outer, seg, pages, page_stride, slots, unit, es):
    _small("cache", outer[0], seg[0], pages, slots, unit * es)
    return _native.CacheParams(outer[0], pages, seg[0], slots, unit * es, _I3(outer[1] * es, page_stride * es, seg[1] * es))


_STEPS = 10000   # of a search for common bytes, before it is given up (caches with one layout take less than 100)


def _layout(t, p):
    """(first byte, extent, [(stride, entries)] from the widest on, bytes of a segment) of a cache."""
    axes = [(s, n) for s, n in zip(p.stride, (p.O, p.P, p.H)) if n > 1]
    axes.sort(reverse=True)
    seg = p.page * p.unit_bytes
    return t.data_ptr(), seg + sum(s * (n - 1) for s, n in axes), axes, seg


def _meet(a, b):
    """Whether two caches have a byte in common."""
    steps = {}
    for s, n in a[2]:
        steps[s] = [1 - n, 0]
    for s, n in b[2]:
        lo, hi = steps.get(s, (0, 0))
        steps[s] = [lo, hi + n - 1]
    axes = sorted(steps.items(), reverse=True)
    left = _STEPS

    def search(k, off):   # off: b's segment less a's, with the axes from k on still free
        nonlocal left
        left -= 1
        if left < 0:
            return True   # (not shown to be apart)
        if k == len(axes):
            return -b[3] < off < a[3]
        s, (lo, hi) = axes[k]
        least = off + sum(x * r[0] for x, r in axes[k + 1:])
        most = off + sum(x * r[1] for x, r in axes[k + 1:])
        first, last = max(lo, -((b[3] - 1 + most) // s)), min(hi, (a[3] - 1 - least) // s)
        return any(search(k + 1, off + d * s) for d in range(first, last + 1))

    return search(0, b[0] - a[0])


def _blocks(tensors):
    """Whether they are contiguous and one behind the other, as a cache per layer mostly is."""
    if not all(t.is_contiguous() for t in tensors):
        return False
    at = sorted((t.data_ptr(), t.nbytes) for t in tensors)
    return all(p + n <= q for (p, n), (q, _) in zip(at, at[1:]))


def _apart(layouts):
    """Whether no two caches have a byte in common; views of one buffer may lie between one another."""
    group, end = [], 0
    for x in sorted(layouts, key=lambda x: x[0]) + [(math.inf,)]:
        if x[0] < end:
            group.append(x)
            end = max(end, x[0] + x[1])
            continue
        if len(group) > 1 and not _between(group) and any(_meet(a, b) for i, a in enumerate(group) for b in group[:i]):
            return False
        if len(x) > 1:
            group, end = [x], x[0] + x[1]
    return True


def _between(group):
    """Whether one entry of the widest axis, which all have, holds the others' entries beside it."""
    widest = {x[2][0][0] if x[2] else 0 for x in group}
    s = widest.pop()
    if widest or s == 0:
        return False
    at = sorted((x[0] % s, x[1] - s * (x[2][0][1] - 1)) for x in group)
    return all(r + size <= nxt for (r, size), nxt in zip(at, [r for r, _ in at[1:]] + [at[0][0] + s]))


def _caches(cache, page_dim, slot_dim, P=None, ahead=False):
    """[(tensor, layout)] of one cache or several that share a table. ``ahead``: something
    else is written before the first of them."""
    tensors = [cache] if isinstance(cache, torch.Tensor) else list(cache)
    if not tensors:
        raise ValueError("no cache given")
    dev, found, page = _on_gpu(tensors[0], "cache"), [], None
    for t in tensors:
        if t.device != dev:
            raise ValueError("the caches must be on one device")
        found.append((t, _cache_params(t, page_dim, slot_dim, P, page)))
        P, page = found[0][1].P, found[0][1].page
    if ahead or len(found) > 1:
        for _, p in found:   # all are looked at before anything is written
            _check(_native.lib().spec_pages_copy(ctypes.byref(p), None, None, 0, None))
    if len(found) > 1 and not _blocks(tensors) and not _apart([_layout(t, p) for t, p in found if p.O and p.P and p.H]):
        raise ValueError("the caches must not overlap")
    return found, dev, P, page


Cache = Union[torch.Tensor, Sequence[torch.Tensor]]


def pages_compact(cache: Cache, table: torch.Tensor, lengths: torch.Tensor, path: torch.Tensor, page_dim: int = 0,
                  slot_dim: Optional[int] = None, out: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The kept nodes of a tree moved to the end of the context, in place
    (spec_pages_compact). ``cache`` is a tensor of any dtype with the pool's
    pages along ``page_dim`` and their slots along ``slot_dim`` (None: the next
    axis), or a sequence of such tensors (layers, keys, values), none over
    another, that share the table; ``table`` [B,M], ``lengths`` [B], ``path`` [B,N] as tree_accept
    returns it. Returns the new lengths [B] int32; ``out`` to write them into must not
    overlap ``lengths``."""
    found, dev, P, page = _caches(cache, page_dim, slot_dim)
    if path.dim() != 2 or table.dim() != 2:
        raise ValueError("path must be [B, N] and table [B, M]")
    (B, N), M = path.shape, table.shape[1]
    _need(path, "path", (B, N), dev)
    _need(table, "table", (B, M), dev)
    _need(lengths, "lengths", (B,), dev)
    _maybe(out, "out", (B,), dev)
    _status(status, dev)
    _small("pages_compact", B, N, M)

    def body(s):
        L = _native.lib()
        new = torch.empty(B, dtype=_I32, device=dev) if out is None else out
        for t, p in found:
            _check(L.spec_pages_compact(ctypes.byref(p), t.data_ptr(), B, N, M, table.data_ptr(), lengths.data_ptr(),
                                        path.data_ptr(), new.data_ptr(), _addr(status), s))
            _written(t)
        if out is not None:
            _written(out)
        return new

    return _run(path, stream, body)


def pages_resize(table: torch.Tensor, refs: torch.Tensor, lengths: torch.Tensor, page: int,
                 out: Optional[dict] = None, status: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Rows of exactly the pages of ``page`` slots that ``lengths`` ask for
    (spec_pages_resize): ``table`` [..,M] and ``refs`` [P] int32, ``lengths`` of
    the table's leading shape; length 0 frees a row. Returns the new ``table``
    and ``refs``; ``out`` may hold the given ones, to change them in place."""
    dev = _on_gpu(table, "table")
    if table.dim() < 1 or refs.dim() != 1:
        raise ValueError("table must be [.., M] and refs [P]")
    lead, M, P = table.shape[:-1], table.shape[-1], refs.shape[0]
    _need(table, "table", table.shape, dev)
    _need(refs, "refs", (P,), dev)
    _need(lengths, "lengths", lead, dev)
    _status(status, dev)
    R = lengths.numel()
    _small("pages_resize", R, M, P, page)
    p = _native.PagesParams(1, R, R, M, P, page)

    def body(s):
        t = _new(out, "table", table.shape, dev)
        r = _new(out, "refs", (P,), dev)
        ws = torch.empty(P, dtype=_I32, device=dev)
        _check(_native.lib().spec_pages_resize(ctypes.byref(p), table.data_ptr(), refs.data_ptr(), lengths.data_ptr(),
                                               t.data_ptr(), r.data_ptr(), ws.data_ptr(), _addr(status), s))
        if out is not None:
            _written((t, r))
        return {"table": t, "refs": r}

    return _run(table, stream, body)


def pages_fork(cache: Cache, table: torch.Tensor, refs: torch.Tensor, lengths: torch.Tensor, parent: torch.Tensor,
               page_dim: int = 0, slot_dim: Optional[int] = None, out: Optional[dict] = None,
               status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Rows of pages in the order of the surviving beams (spec_pages_fork and
    spec_pages_copy): row (b, n) continues row (b, parent[b, n]) of ``table``
    [B,W,M] and ``lengths`` [B,W]; ``parent`` [B,N] int32 as beam_step returns
    it, -1 continues its own row. Full pages are shared, pages that are not
    full copied in ``cache`` (as for pages_compact) for all rows but the first.
    Returns ``table`` [B,N,M], ``refs`` [P] and ``lengths`` [B,N]; ``out`` may
    hold tensors for them, of which only ``refs`` may be the given one."""
    if refs.dim() != 1 or table.dim() != 3 or parent.dim() != 2:
        raise ValueError("table must be [B, W, M], refs [P] and parent [B, N]")
    found, dev, P, page = _caches(cache, page_dim, slot_dim, refs.shape[0], ahead=True)
    (B, W, M), N = table.shape, parent.shape[1]
    _need(table, "table", (B, W, M), dev)
    _need(refs, "refs", (P,), dev)
    _need(lengths, "lengths", (B, W), dev)
    _need(parent, "parent", (B, N), dev)
    _status(status, dev)
    _small("pages_fork", B, W, N, M, B * N)
    p = _native.PagesParams(B, W, N, M, P, page)

    def body(s):
        L = _native.lib()
        t = _new(out, "table", (B, N, M), dev)
        r = _new(out, "refs", (P,), dev)
        ln = _new(out, "lengths", (B, N), dev)
        ws = torch.empty(2 * P + 4 * B * N, dtype=_I32, device=dev)   # (two parts of a page number each, then copies)
        copies = ws.data_ptr() + 8 * P
        _check(L.spec_pages_fork(ctypes.byref(p), table.data_ptr(), refs.data_ptr(), lengths.data_ptr(),
                                 parent.data_ptr(), t.data_ptr(), r.data_ptr(), ln.data_ptr(), copies, ws.data_ptr(),
                                 _addr(status), s))
        if out is not None:
            _written((t, r, ln))
        for c, cp in found:
            _check(L.spec_pages_copy(ctypes.byref(cp), c.data_ptr(), copies, B * N, s))
            _written(c)
        return {"table": t, "refs": r, "lengths": ln}

    return _run(table, stream, body)
