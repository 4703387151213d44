"""CPU tests of the row operators' boundary: struct layouts, refusals before
any launch, and the reference's own identities."""
import ctypes
import os
import subprocess
import tempfile

import numpy as np
import pytest
import torch

import rows_reference as ref
import speculative_decoding_token_verify_gb300 as sv
from speculative_decoding_token_verify_gb300 import _native, rows

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    _native.build()
    return _native.lib()


def _rows(**kw):
    base = dict(B=4, K=3, V=100, dtype=0, M=8, tail=0, inv_temperature=1.0, reserved=0, batch_stride=300, row_stride=100)
    base.update(kw)
    return _native.RowsParams(*[base[n] for n, _ in _native.RowsParams._fields_])


def test_struct_layouts_match_the_header():
    prog = r"""
#include <stdio.h>
#include <stddef.h>
#include "spec_verify.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu %zu %zu %zu %d %d %d\n", sizeof(spec_rows_params), offsetof(spec_rows_params, inv_temperature),
         offsetof(spec_rows_params, batch_stride), offsetof(spec_rows_params, row_stride), sizeof(spec_reorder_params),
         offsetof(spec_reorder_params, unit_bytes), offsetof(spec_reorder_params, src_stride),
         offsetof(spec_reorder_params, dst_stride), SPEC_MAX_TOP, SPEC_MAX_BEAMS, SPEC_MAX_BEAM_OUT);
  return 0;
}
"""
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        with open(c, "w") as f:
            f.write(prog)
        subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe])
        got = list(map(int, subprocess.check_output([exe]).split()))
    R, O = _native.RowsParams, _native.ReorderParams
    assert got == [ctypes.sizeof(R), R.inv_temperature.offset, R.batch_stride.offset, R.row_stride.offset,
                   ctypes.sizeof(O), O.unit_bytes.offset, O.src_stride.offset, O.dst_stride.offset, sv.MAX_TOP,
                   sv.MAX_BEAMS, sv.MAX_BEAM_OUT]


BAD_ROWS = [(dict(reserved=1), 1), (dict(B=-1), 1), (dict(K=-1), 1), (dict(B=(1 << 24) + 1), 2), (dict(K=5000), 2),
            (dict(B=1 << 24, K=16), 2), (dict(V=0), 2), (dict(V=(1 << 20) + 1), 2), (dict(dtype=3), 2), (dict(M=0), 2),
            (dict(M=129), 2), (dict(tail=2), 1), (dict(inv_temperature=0.0), 1), (dict(inv_temperature=2e4), 1),
            (dict(inv_temperature=float("nan")), 1), (dict(batch_stride=-1), 1), (dict(row_stride=-5), 1),
            (dict(row_stride=1 << 62), 1)]


def _top(L, p, z=FAKE, lp=FAKE, ids=FAKE):
    return L.spec_top_logprobs(ctypes.byref(p) if p is not None else None, P(z), P(lp), P(ids), None, None, None)


def _loss(L, p, z=FAKE, lp=FAKE, ids=FAKE, loss=FAKE, stats=FAKE):
    return L.spec_distill_loss(ctypes.byref(p) if p is not None else None, P(z), P(lp), P(ids), None, P(loss), P(stats),
                               None, None)


def _grad(L, p, z=FAKE, stats=FAKE, g=FAKE + 65536, bs=300, rs=100):
    return L.spec_distill_grad(ctypes.byref(p) if p is not None else None, P(z), P(FAKE), P(FAKE), None, P(stats), None,
                               P(g), bs, rs, None, None)


def _step(L, p, z=FAKE, loss=FAKE, g=FAKE + 65536, bs=300, rs=100):
    return L.spec_distill_step(ctypes.byref(p) if p is not None else None, P(z), P(FAKE), P(FAKE), None, P(loss), P(g),
                               bs, rs, None, None)


def _beam(L, p, z=FAKE, scores=FAKE, fin=None, eos=-1, out=FAKE + 4096):
    return L.spec_beam_step(ctypes.byref(p) if p is not None else None, P(z), P(scores), P(fin) if fin else None, eos,
                            P(out), P(FAKE), P(FAKE), P(FAKE + 8192), None, None)


@pytest.mark.parametrize("kw,code", BAD_ROWS)
def test_row_parameters_refused(L, kw, code):
    for call in (_top, _loss, _grad, _step):
        assert call(L, _rows(**kw)) == code, call
    if "M" not in kw and "K" not in kw:
        assert _beam(L, _rows(**kw)) == code
    assert L.spec_last_error()


def test_pointers_refused(L):
    for call in (_top, _loss, _grad, _step, _beam):
        assert call(L, None) == 1
        assert call(L, _rows(), z=0) == 1
        assert call(L, _rows(), z=FAKE + 2) == 1          # float rows on an odd address
        assert call(L, _rows(dtype=1), z=FAKE + 1) == 1
    assert _top(L, _rows(), lp=0) == 1 and _top(L, _rows(), ids=0) == 1 and _top(L, _rows(tail=1)) == 1
    assert _loss(L, _rows(), lp=0) == 1 and _loss(L, _rows(), ids=0) == 1
    assert _loss(L, _rows(), loss=0) == 1 and _loss(L, _rows(), stats=0) == 1 and _loss(L, _rows(), stats=FAKE + 4) == 1
    assert _grad(L, _rows(), stats=0) == 1 and _grad(L, _rows(), stats=FAKE + 8) == 1 and _grad(L, _rows(), g=0) == 1
    assert _step(L, _rows(), loss=0) == 1 and _step(L, _rows(), g=0) == 1


def test_overlapping_gradients_refused(L):
    for call in (_grad, _step):
        assert call(L, _rows(), bs=0, rs=100) == 1        # sequences over one another
        assert call(L, _rows(), bs=300, rs=0) == 1
        assert call(L, _rows(), bs=299, rs=100) == 1
        assert call(L, _rows(), bs=300, rs=99) == 1
        assert call(L, _rows(), bs=100, rs=399) == 1      # batch inside, one short
        assert call(L, _rows(), g=FAKE, bs=600, rs=200) == 1   # in place with other strides
        assert call(L, _rows(), bs=-300, rs=100) == 1


def test_beam_arguments_refused(L):
    assert _beam(L, _rows(M=65)) == 2 and _beam(L, _rows(K=33)) == 2 and _beam(L, _rows(K=0)) == 1
    assert _beam(L, _rows(inv_temperature=2.0)) == 1 and _beam(L, _rows(tail=1)) == 1
    assert _beam(L, _rows(), eos=100) == 1 and _beam(L, _rows(), eos=-2) == 1
    assert _beam(L, _rows(), fin=FAKE, eos=-1) == 1
    assert _beam(L, _rows(), scores=0) == 1 and _beam(L, _rows(), out=0) == 1
    assert _beam(L, _rows(), scores=FAKE, out=FAKE) == 1          # in place with N != W


def test_reorder_arguments_refused(L):
    def call(src=FAKE, dst=FAKE, parent=FAKE, null=False, **kw):
        base = dict(O=2, B=3, W=4, N=4, H=2, T=8, unit_bytes=16)
        base.update({k: v for k, v in kw.items() if k in base})
        p = _native.ReorderParams(*[base[k] for k in ("O", "B", "W", "N", "H", "T", "unit_bytes")])
        p.src_stride[:] = kw.get("ss", [4096, 1024, 256, 128])
        p.dst_stride[:] = kw.get("ds", kw.get("ss", [4096, 1024, 256, 128]))
        return L.spec_beam_reorder(None if null else ctypes.byref(p), P(src), P(dst), P(parent), None, None, None)

    assert call(null=True) == 1
    for k in ("O", "B", "H", "T"):
        assert call(**{k: -1}) == 1
    for kw in (dict(O=65536), dict(H=65536), dict(W=0), dict(W=33), dict(N=0), dict(N=33), dict(B=(1 << 24) + 1)):
        assert call(**kw) == 2, kw
    assert call(unit_bytes=0) == 1 and call(src=0) == 1 and call(dst=0) == 1 and call(parent=0) == 1
    assert call(ss=[4096, -1, 256, 128]) == 1
    assert call(ss=[1 << 62, 1024, 256, 128]) == 1
    assert call(dst=FAKE + (1 << 20), ds=[4096, 1024, 256, 127]) == 1    # segments overlap
    assert call(dst=FAKE + (1 << 20), ds=[4096, 1024, 0, 128]) == 1
    assert call(ss=[4096, 1024, 256, 128], ds=[8192, 2048, 512, 256]) == 1   # in place, other strides
    assert call(N=5, ss=[8192, 2048, 256, 128]) == 1                     # in place, more beams
    assert call(ss=[4096, 1024, 0, 128], ds=[4096, 1024, 0, 128]) == 1
    assert call(O=0) == 0 and call(B=0, src=0) == 0 and call(T=0) == 0


def test_empty_calls_enqueue_nothing(L):
    assert _top(L, _rows(B=0), z=0) == 0 and _loss(L, _rows(K=0), z=0) == 0
    assert _grad(L, _rows(B=0)) == 0 and _step(L, _rows(B=0)) == 0 and _beam(L, _rows(B=0)) == 0


def test_binding_refuses_host_and_misshapen_tensors():
    z = torch.zeros((2, 3, 8))
    lp, ids = torch.zeros((2, 3, 4)), torch.zeros((2, 3, 4), dtype=torch.int32)
    for f in (lambda: sv.top_logprobs(z, 4), lambda: sv.distill_loss(z, lp, ids), lambda: sv.distill_step(z, lp, ids),
              lambda: sv.distill_grad(z, lp, ids, torch.zeros((2, 3, 4))), lambda: sv.beam_step(z, z[..., 0], 2),
              lambda: sv.beam_reorder(z, ids[..., 0])):
        with pytest.raises(ValueError):
            f()


class _Fake:
    """A tensor's outline: shapes beyond the C ABI's 32-bit fields."""
    is_cuda, dtype = True, torch.float32

    def __init__(self, shape):
        self.shape = torch.Size(shape)

    def stride(self):
        return (0,) * (len(self.shape) - 1) + (1,)


@pytest.mark.parametrize("shape", [(2 ** 32 + 1, 2, 10), (2, 4097, 10), (2, 2, 2 ** 32 + 5), (2 ** 33, 7)])
def test_binding_refuses_shapes_before_they_wrap(shape):
    with pytest.raises(sv.SpecError):
        rows._logits(_Fake(shape), "logits")


def test_layouts_of_states():
    t = torch.zeros((2, 3, 4, 5, 6, 8))
    assert rows._layout(t, 1, 4, "t") == (2, 3, 4, 5, 6, 32, [3 * 4 * 240 * 4, 960 * 4, 240 * 4, 48 * 4])
    assert rows._layout(t[:, :, :, :, :3], 1, 4, "t")[4] == 3
    with pytest.raises(ValueError):
        rows._layout(t[..., :5], 1, 4, "t")                  # units with gaps
    with pytest.raises(ValueError):
        rows._layout(t.transpose(4, 5), 1, 4, "t")
    u = torch.zeros((2, 7, 3, 4, 8))
    with pytest.raises(ValueError):
        rows._layout(u[:, :5], 2, 4, "u")                    # two outer axes that do not merge
    assert rows._layout(u[:, :5], 1, 4, "u")[0] == 2


def test_reference_identities():
    rng = np.random.default_rng(0)
    y = rng.normal(0, 2, 50)
    lp = y - ref.lse(y)
    at = np.argsort(-y)[:50].astype(np.int32)
    same = ref.distill(y, lp[at], at)                        # the teacher is the student
    assert abs(same["loss"]) < 1e-12 and np.abs(same["grad"]).max() < 1e-12
    top = at[:7]
    for tail in (True, False):
        r = ref.distill(y + rng.normal(0, 1, 50), lp[top], top, tail=tail)
        assert r["loss"] > 0 and abs(r["grad"].sum()) < 1e-12    # softmax gradients sum to zero
    a = ref.distill(y, lp[top], top)                         # the student holds the teacher's bucket masses
    assert abs(a["loss"]) < 1e-12 and np.abs(a["grad"]).max() < 1e-12
    L, ids, l, _, _ = ref.top(y, 60)
    assert (ids[:50] == at).all() and (ids[50:] == -1).all() and abs(np.exp(L[:50]).sum() - 1) < 1e-12
    z = np.stack([y, y])
    sc, par, tok, fin, _ = ref.beam(z, np.array([0.0, 0.0]), 4, None)
    assert par.tolist() == [0, 1, 0, 1] and tok[0] == tok[1] == at[0]
