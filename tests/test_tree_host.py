"""CPU tests of the tree operators' boundary: struct layouts, refusals before any
launch, and the plain forms' own identities."""
import ctypes
import os
import subprocess
import tempfile

import numpy as np
import pytest
import torch

import speculative_decoding_token_verify_gb300 as sv
import tree_reference as ref
from speculative_decoding_token_verify_gb300 import _native, tree

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000
FAR = 1 << 34
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    _native.build()
    return _native.lib()


def test_struct_layouts_match_the_header():
    structs = {"spec_attend_params": _native.AttendParams, "spec_cache_params": _native.CacheParams,
               "spec_pages_params": _native.PagesParams}
    lines = []
    for name, cls in structs.items():
        lines.append(f'printf("%zu ", sizeof({name}));')
        lines += [f'printf("%zu ", offsetof({name}, {f}));' for f, _ in cls._fields_]
    prog = '#include <stdio.h>\n#include <stddef.h>\n#include "spec_verify.h"\nint main(void) {' + "\n".join(lines) + \
        'printf("%d %d %d %d %d %d", SPEC_MAX_NODES, SPEC_F16, SPEC_ERR_BAD_PAGE, SPEC_ERR_BAD_LENGTH, SPEC_ERR_NO_PAGES, SPEC_ERR_BAD_PATH); return 0; }'
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        with open(c, "w") as f:
            f.write(prog)
        subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe])
        got = list(map(int, subprocess.check_output([exe]).split()))
    want = []
    for cls in structs.values():
        want += [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]
    a = sv.api
    assert got == want + [sv.MAX_NODES, tree.F16, a.SPEC_ERR_BAD_PAGE, a.SPEC_ERR_BAD_LENGTH, a.SPEC_ERR_NO_PAGES, a.SPEC_ERR_BAD_PATH]


# ---- attention ------------------------------------------------------------------------------


def _attend(L, null=False, q=FAKE, k=FAKE + FAR, v=FAKE + 2 * FAR, table=FAKE, lengths=FAKE, out=FAKE + 3 * FAR, ws=FAKE + 4 * FAR,
            size=1 << 30, **kw):
    f = dict(B=2, N=4, Hq=8, Hkv=2, D=64, dtype=1, P=10, page=16, M=5, scale=0.125)
    f.update({x: y for x, y in kw.items() if x in f})
    p = _native.AttendParams(*f.values())
    p.q_stride[:] = kw.get("qs", [2048, 512, 64])
    p.k_stride[:] = kw.get("ks", [2048, 128, 64])
    p.v_stride[:] = kw.get("vs", [2048, 128, 64])
    p.parents_stride = kw.get("ps", 0)
    if kw.get("ask"):
        return L.spec_tree_attention_workspace_size(ctypes.byref(p))
    return L.spec_tree_attention(None if null else ctypes.byref(p), P(q), P(k), P(v), P(table), P(lengths), None, None, P(out),
                                 None, P(ws), size, None, None)


BAD = [(dict(B=-1), 1), (dict(N=-1), 1), (dict(M=-1), 1), (dict(P=-1), 1), (dict(dtype=0), 2), (dict(dtype=3), 2), (dict(B=65536), 2),
       (dict(N=129), 2), (dict(P=(1 << 30) + 1), 2), (dict(Hkv=0), 1), (dict(Hq=0), 1), (dict(Hq=9), 1), (dict(Hq=258, Hkv=2), 2),
       (dict(D=0), 2), (dict(D=136), 2), (dict(D=60), 2), (dict(page=4), 2), (dict(page=24), 2), (dict(page=0), 2), (dict(M=1 << 30), 2),
       (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(ps=3), 1), (dict(ps=-4), 1), (dict(qs=[2048, 512, 60]), 1),
       (dict(ks=[2048, 0, 64]), 1), (dict(vs=[-2048, 128, 64]), 1), (dict(vs=[1 << 40, 128, 64]), 1)]


@pytest.mark.parametrize("kw,code", BAD)
def test_attention_parameters_refused(L, kw, code):
    assert _attend(L, **kw) == code and L.spec_last_error()
    assert _attend(L, ask=True, **kw) == 0


def test_attention_pointers_refused(L):
    for kw in (dict(null=True), dict(q=0), dict(k=0), dict(v=0), dict(table=0), dict(lengths=0), dict(out=0), dict(ws=0), dict(size=0),
               dict(q=FAKE + 8), dict(k=FAKE + 2), dict(v=FAKE + 4), dict(out=FAKE + 8), dict(ws=FAKE + 4)):
        assert _attend(L, **kw) == 1, kw
    assert _attend(L, B=0, q=0) == 0 and _attend(L, N=0, q=0) == 0


def test_attention_output_over_an_input_refused(L):
    assert _attend(L, out=FAKE) == 1                       # the queries
    assert _attend(L, out=FAKE + FAR) == 1                 # the keys
    assert _attend(L, out=FAKE + 2 * FAR + 2048) == 1      # the values


# ---- pages ----------------------------------------------------------------------------------


def _resize(L, null=False, table=FAKE, refs=FAKE + FAR, lengths=FAKE + 2 * FAR, ot=None, orf=None, ws=FAKE + 3 * FAR, **kw):
    f = dict(B=2, W=3, N=3, M=4, P=100, page=16)
    f.update({x: y for x, y in kw.items() if x in f})
    p = _native.PagesParams(*f.values())
    return L.spec_pages_resize(None if null else ctypes.byref(p), P(table), P(refs), P(lengths), P(table if ot is None else ot),
                               P(refs if orf is None else orf), P(ws), None, None)


def _fork(L, null=False, table=FAKE, refs=FAKE + FAR, lengths=FAKE + 2 * FAR, parent=FAKE + 3 * FAR, ot=FAKE + 4 * FAR, orf=None,
          ol=FAKE + 5 * FAR, copies=FAKE + 6 * FAR, ws=FAKE + 7 * FAR, **kw):
    f = dict(B=2, W=3, N=3, M=4, P=100, page=16)
    f.update({x: y for x, y in kw.items() if x in f})
    p = _native.PagesParams(*f.values())
    return L.spec_pages_fork(None if null else ctypes.byref(p), P(table), P(refs), P(lengths), P(parent), P(ot),
                             P(refs if orf is None else orf), P(ol), P(copies), P(ws), None, None)


@pytest.mark.parametrize("kw,code", [(dict(B=-1), 1), (dict(W=-1), 1), (dict(N=-1), 1), (dict(M=-1), 1), (dict(P=-1), 1), (dict(page=0), 1),
                                     (dict(B=1 << 23), 2), (dict(P=(1 << 30) + 1), 2), (dict(M=1 << 29), 2), (dict(M=1 << 28, page=1), 0),
                                     (dict(page=1 << 30), 2)])
def test_pages_parameters_refused(L, kw, code):
    if code:
        assert _resize(L, **kw) == code and _fork(L, **kw) == code and L.spec_last_error()
    assert _resize(L, N=2) == 1


def test_pages_pointers_refused(L):
    for kw in (dict(null=True), dict(table=0), dict(refs=0), dict(lengths=0), dict(ws=0), dict(ot=FAKE + 4), dict(orf=FAKE + FAR + 4),
               dict(ot=FAKE + FAR), dict(orf=FAKE), dict(ws=FAKE), dict(ws=FAKE + FAR), dict(ot=FAKE + 2 * FAR), dict(orf=FAKE + 2 * FAR)):
        assert _resize(L, **kw) == 1, kw
    for kw in (dict(null=True), dict(table=0), dict(refs=0), dict(lengths=0), dict(parent=0), dict(ot=0), dict(ol=0), dict(copies=0),
               dict(ws=0), dict(ot=FAKE), dict(ol=FAKE + 2 * FAR), dict(ol=FAKE + 3 * FAR), dict(orf=FAKE + FAR + 8), dict(copies=FAKE),
               dict(copies=FAKE + 4 * FAR), dict(ws=FAKE + FAR - 4), dict(ws=FAKE + 6 * FAR)):
        assert _fork(L, **kw) == 1, kw
    assert _resize(L, B=0, P=0, table=0, refs=0) == 0 and _fork(L, B=0, P=0, table=0, refs=0) == 0


def _compact(L, null=False, cache=FAKE + FAR, table=FAKE, lengths=FAKE + 2 * FAR, path=FAKE + 3 * FAR, out=FAKE + 4 * FAR, B=2, N=4, M=5, **kw):
    f = dict(O=2, P=10, H=1, page=16, unit_bytes=64)
    f.update({x: y for x, y in kw.items() if x in f})
    p = _native.CacheParams(*f.values())
    p.stride[:] = kw.get("st", [10240, 1024, 0])
    if kw.get("copy"):
        return L.spec_pages_copy(None if null else ctypes.byref(p), P(cache), P(table), kw.get("count", 3), None)
    return L.spec_pages_compact(None if null else ctypes.byref(p), P(cache), B, N, M, P(table), P(lengths), P(path), P(out), None, None)


def test_cache_arguments_refused(L):
    for copy in (False, True):
        for kw, code in ((dict(null=True), 1), (dict(O=-1), 1), (dict(P=-1), 1), (dict(H=-1), 1), (dict(page=0), 1), (dict(O=65536), 2),
                         (dict(H=65536), 2), (dict(P=(1 << 30) + 1), 2), (dict(unit_bytes=0), 1), (dict(unit_bytes=(1 << 30) + 1), 1),
                         (dict(st=[10240, -1, 0]), 1), (dict(st=[10240, 1023, 0]), 1), (dict(st=[10239, 1024, 0]), 1),
                         (dict(st=[1 << 62, 1024, 0]), 1), (dict(H=2, st=[10240, 1024, 0]), 1), (dict(H=2, st=[40960, 2048, 1023]), 1),
                         (dict(cache=0), 1), (dict(table=0), 1)):
            assert _compact(L, copy=copy, **kw) == code, (copy, kw)
    for kw, code in ((dict(B=-1), 1), (dict(M=-1), 1), (dict(N=0), 2), (dict(N=129), 2), (dict(B=(1 << 24) + 1), 2), (dict(M=1 << 28), 2),
                     (dict(lengths=0), 1), (dict(path=0), 1), (dict(out=0), 1), (dict(out=FAKE + 2 * FAR), 1), (dict(out=FAKE + 3 * FAR + 4), 1),
                     (dict(out=FAKE + 8), 1)):
        assert _compact(L, **kw) == code, kw
    assert _compact(L, copy=True, count=-1) == 1 and _compact(L, copy=True, count=0, cache=0) == 0 and _compact(L, B=0, cache=0) == 0


def test_accept_arguments_refused(L):
    def call(B=2, N=4, tokens=FAKE, parents=0, ps=0, choice=FAKE + FAR, cb=4, cn=1, acc=FAKE + 2 * FAR, out=FAKE + 3 * FAR, path=FAKE + 4 * FAR):
        return L.spec_tree_accept(B, N, P(tokens), P(parents), ps, P(choice), cb, cn, None, P(acc), P(out), P(path), None, None)

    for kw, code in ((dict(B=-1), 1), (dict(N=0), 2), (dict(N=129), 2), (dict(B=(1 << 24) + 1), 2), (dict(parents=FAKE, ps=3), 1), (dict(ps=-1, parents=FAKE), 1),
                     (dict(cb=-1), 1), (dict(cn=-1), 1), (dict(cb=1 << 62), 1), (dict(cn=1 << 62), 1), (dict(tokens=0), 1), (dict(choice=0), 1),
                     (dict(acc=0), 1), (dict(out=0), 1), (dict(path=0), 1), (dict(out=FAKE + 4), 1), (dict(path=FAKE + FAR), 1),
                     (dict(acc=FAKE + FAR + 28), 1), (dict(path=FAKE + 3 * FAR + 28), 1), (dict(parents=FAKE + 4 * FAR + 4, ps=4), 1)):
        assert call(**kw) == code, kw
    assert call(B=0, tokens=0) == 0


def test_overlapping_caches_refused(monkeypatch):
    monkeypatch.setattr(tree, "_on_gpu", lambda t, name: t.device)
    t, i = torch.zeros((4, 16, 8)), torch.zeros((2, 4), dtype=torch.int32)
    for bad in ([t, t], [t, t[:, :8]], [t, torch.zeros((3, 16, 8))]):
        with pytest.raises(ValueError):
            tree._caches(bad, 0, None)
    with pytest.raises(sv.SpecError):
        tree._caches([t, torch.zeros((1, 16, 8)).expand(4, 16, 8)], 0, None)      # pages over one another
    assert len(tree._caches([t, torch.zeros((4, 16, 3)), torch.zeros((4, 16, 0))], 0, None)[0]) == 3


# ---- the binding ----------------------------------------------------------------------------


def test_binding_refuses_host_and_misshapen_tensors():
    i = torch.zeros((2, 4), dtype=torch.int32)
    q = torch.zeros((2, 4, 8, 64), dtype=torch.bfloat16)
    for f in (lambda: sv.tree_attention(q, q, q, i, i[:, 0]), lambda: sv.tree_accept(i, i, i), lambda: sv.pages_resize(i, i[0], i[:, 0], 16),
              lambda: sv.pages_compact(q, i, i[:, 0], i), lambda: sv.pages_compact([], i, i[:, 0], i),
              lambda: sv.pages_fork(q, i[None], i[0], i, i)):
        with pytest.raises(ValueError):
            f()


def test_cache_layouts():
    def of(t, pd, sd=None, pool=None, page=None):
        p = tree._cache_params(t, pd, sd, pool, page)
        return [p.O, p.P, p.H, p.page, p.unit_bytes, list(p.stride)]

    t = torch.zeros((3, 2, 10, 16, 4, 8), dtype=torch.bfloat16)
    assert of(t, 2) == [6, 10, 1, 16, 64, [10240, 1024, 0]]
    assert of(t, -4) == of(t, 2)
    assert of(t, 1, 3) == [3, 2, 10, 16, 64, [20480, 10240, 1024]]
    assert of(t[:, 0], 1) == [3, 10, 1, 16, 64, [20480, 1024, 0]]
    assert of(t[:, :, 2:5], 2, pool=3)[:2] == [6, 3]
    odd = t[:, :, :1].as_strided((3, 2, 1, 16, 4, 8), (1024, 512, 7, 32, 8, 1))    # an axis of one entry with any stride
    assert odd.is_contiguous() and of(odd, 2)[:5] == [6, 1, 1, 16, 64] and of(odd, 2)[5][0] == 1024
    assert of(t[..., :0], 2)[0] == 0 and of(t[..., :0], 2)[4] == 2
    for bad in (lambda: of(t[..., :4], 2), lambda: of(t[:, :, :, ::2], 2), lambda: of(t, 5), lambda: of(t, 2, 2), lambda: of(t, 2, 1),
                lambda: of(t, 2, pool=9), lambda: of(t, 2, page=8), lambda: of(t[:, :, :, :, :3], 2), lambda: of(t.transpose(0, 1)[:, :2], 2)):
        with pytest.raises(ValueError):
            bad()


# ---- the plain forms ------------------------------------------------------------------------


def test_plain_forms_agree_with_themselves():
    g = torch.Generator().manual_seed(0)
    # a chain over a cache is causal attention over the tokens in order
    T, D = 20, 8
    k, v, q = (torch.randn((T, D), generator=g, dtype=torch.float64) for _ in range(3))
    pool = torch.zeros((4, 8, 1, D), dtype=torch.float64), torch.zeros((4, 8, 1, D), dtype=torch.float64)
    order = [2, 0, 3]
    for t in range(T):
        pool[0][order[t // 8], t % 8, 0], pool[1][order[t // 8], t % 8, 0] = k[t], v[t]
    out, lse, e, _ = ref.attention(q[None, 15:, None], pool[0], pool[1], [order], [15], [[-1, 0, 1, 2, 3]], [5], 0.3)
    s = (0.3 * q @ k.T).masked_fill(torch.ones(T, T).triu(1).bool(), float("-inf"))
    assert np.allclose(out[0, :, 0], (torch.softmax(s, 1) @ v)[15:].numpy(), atol=1e-12)
    assert np.allclose(lse[0, :, 0], torch.logsumexp(s, 1)[15:].numpy(), atol=1e-12) and (e > 0).all()
    # a walk: greedy choices along a chain stop at the first that differs
    assert ref.accept([[9, 4, 5, 6]], [[-1, 0, 1, 2]], [[4, 5, 7, 8]], [4]) == ([2], [[4, 5, 7, -1]], [[0, 1, 2, -1]])
    # twins: the lowest child
    assert ref.accept([[9, 4, 4, 6]], [[-1, 0, 0, 2]], [[4, 6, 6, 8]], [4]) == ([1], [[4, 6, -1, -1]], [[0, 1, -1, -1]])
    table, refs, short = ref.resize([[0, 1], [2, -1]], [1, 1, 1, 0], [16, 32], 16)
    assert table == [[0, -1], [2, 1]] and refs == [1, 1, 1, 0] and not short
    new, refs, lens, copies = ref.fork([[[0, 1], [0, 2]]], [2, 1, 1, 0], [[20, 20]], [[1, 1]], 16)
    assert new == [[[0, 2], [0, 1]]] and refs == [2, 1, 1, 0] and copies == {(0, 1): (2, 1, 4)}
