"""Distillation loss and gradient on the GPU against the fp64 reference and
against differences of it."""
import numpy as np
import pytest

import rows_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = float("inf")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _sv():
    import speculative_decoding_token_verify_gb300 as sv
    sv.build()
    return sv


def _case(B, K, V, M, dtype, seed, s=1.0, noise=1.0, sigma=3.0):
    """A teacher's lists and a student some way off."""
    g = torch.Generator().manual_seed(seed)
    t = sigma * torch.randn((B, K, V), generator=g)
    y = (t + noise * torch.randn((B, K, V), generator=g)).to(DT[dtype])
    m = min(M, V)
    lp, ids = torch.full((B, K, M), -INF), torch.full((B, K, M), -1, dtype=torch.int32)
    val, at = torch.topk(t, m, dim=-1)
    lp[..., :m] = s * val - torch.logsumexp(s * t, -1, keepdim=True)
    ids[..., :m] = at.to(torch.int32)
    w = torch.rand((B, K), generator=g) + 0.1
    return y.to(DEV), lp.to(DEV), ids.to(DEV), w.to(DEV)


def _check(y, lp, ids, w=None, s=1.0, tail=True, grad_loss=None, status_want=0):
    """loss, stats, grad (from stats) and step against the reference."""
    sv = _sv()
    B, K, V = y.shape
    bf16 = y.dtype == torch.bfloat16
    kw = dict(weight=w, inv_temperature=s, tail=tail)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = {"loss": torch.full((B, K), 3.3e38, device=DEV), "stats": torch.full((B, K, 4), 3.3e38, device=DEV)}
    a = sv.distill_loss(y, lp, ids, out=out, status=status, **kw)
    g = sv.distill_grad(y, lp, ids, a["stats"], grad_loss, out=torch.full_like(y, 3e38), status=status, **kw)
    step = sv.distill_step(y, lp, ids, out={"dlogits": torch.full_like(y, 3e38)}, status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == status_want
    yn, lpn, idn = y.float().cpu().numpy(), lp.cpu().numpy(), ids.cpu().numpy()
    wn = np.ones((B, K)) if w is None else w.cpu().numpy().astype(np.float64)
    un = np.ones((B, K)) if grad_loss is None else grad_loss.cpu().numpy().astype(np.float64)
    an = {k: v.cpu().numpy().astype(np.float64) for k, v in a.items()}
    gn, sn = g.float().cpu().numpy().astype(np.float64), step["dlogits"].float().cpu().numpy().astype(np.float64)
    sl = step["loss"].cpu().numpy()
    for b in range(B):
        for k in range(K):
            r = ref.distill(yn[b, k], lpn[b, k], idn[b, k], wn[b, k], s, tail)
            for got in (an["loss"][b, k], sl[b, k]):
                if np.isfinite(r["loss"]):
                    assert abs(got - r["loss"]) <= r["loss_tol"], (b, k, got, r["loss"])
                else:
                    assert got == r["loss"]
            np.testing.assert_array_equal(np.isinf(an["stats"][b, k]), np.isinf(r["stats"]))
            fin = np.isfinite(r["stats"])
            off = np.abs(an["stats"][b, k][fin] - r["stats"][fin])
            assert np.all(off <= r["stats_tol"][fin]), (an["stats"][b, k], r["stats"])
            h = ref.half(bf16)
            for got, up in ((gn[b, k], un[b, k]), (sn[b, k], 1.0)):
                want, tol = r["grad"] * up, r["grad_tol"] * abs(up)
                tol = tol + h * (np.abs(want) + tol)
                bad = ~(np.abs(got - want) <= tol)
                assert not bad.any(), (b, k, np.nonzero(bad)[0][:5], got[bad][:5], want[bad][:5], tol[bad][:5])
    return a, g, step


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,K,V,M", [(2, 3, 1, 1), (2, 3, 2, 1), (1, 2, 7, 7), (3, 1, 9, 4), (2, 2, 33, 40),
                                     (2, 3, 1000, 16), (1, 1, 4097, 128), (2, 2, 32001, 100), (40, 1, 5003, 50)])
def test_against_reference(B, K, V, M, dtype, tail):
    y, lp, ids, w = _case(B, K, V, M, dtype, B * 1000 + V + M)
    _check(y, lp, ids, w, tail=tail, grad_loss=torch.rand((B, K), device=DEV) * 3)


@pytest.mark.parametrize("dtype,V", [("bf16", 128256), ("f32", 152064), ("bf16", 262147), ("f32", 300001)])
@pytest.mark.parametrize("tail", [True, False])
def test_long_rows(dtype, V, tail):
    y, lp, ids, w = _case(1, 3, V, 64, dtype, V)
    _check(y, lp, ids, w, tail=tail)


def test_longest_row():
    y, lp, ids, w = _case(1, 1, 1 << 20, 128, "f32", 1)
    _check(y, lp, ids, w)
    _check(y.to(torch.bfloat16), lp, ids, w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows(dtype):
    y, lp, ids, w = _case(300, 2, 2053, 20, dtype, 12)
    w[::3] = 0
    _check(y, lp, ids, w)


@pytest.mark.parametrize("dtype,V", [("bf16", 40003), ("f32", 40003), ("bf16", 262147), ("f32", 131077), ("bf16", 9),
                                     ("f32", 3), ("bf16", 16385)])
@pytest.mark.parametrize("tail", [True, False])
def test_many_rows_of_many_lengths(dtype, V, tail):
    """Batches that stream row behind row: four student rows repeated over 150
    sequences (stride 0), rows of weight zero and empty lists strewn in. Every
    copy of a row has the same bits; the first copies match the reference."""
    sv = _sv()
    B = 150
    y, lp, ids, w = _case(1, 4, V, 24, dtype, V)
    yy = y.expand(B, 4, V)
    lp, ids = lp.repeat(B, 1, 1), ids.repeat(B, 1, 1)
    w = w.repeat(B, 1)
    g = torch.Generator().manual_seed(V)
    off = torch.rand((B, 4), generator=g) < 0.3
    off[:1] = False
    off[40:60] = True                 # a long run of rows that are not read
    w[off.to(DEV)] = 0
    ids[-20:-10, 1] = -1
    dead = off.clone()
    dead[-20:-10, 1] = True
    a = sv.distill_loss(yy, lp, ids, w, tail=tail)
    st = sv.distill_step(yy, lp, ids, w, tail=tail, out={"dlogits": torch.full((B, 4, V), 3e38, dtype=DT[dtype],
                                                                            device=DEV)})
    torch.cuda.synchronize()
    live = (~dead).to(DEV)[..., None]
    zero = torch.zeros((), device=DEV)
    assert torch.equal(a["loss"], torch.where(live[..., 0], a["loss"][:1], zero))
    assert torch.equal(a["stats"], torch.where(live, a["stats"][:1], zero))
    assert torch.equal(st["loss"], torch.where(live[..., 0], st["loss"][:1], zero))
    assert torch.equal(st["dlogits"], torch.where(live, st["dlogits"][:1], zero.to(DT[dtype])))
    for k in range(4):
        r = ref.distill(y[0, k].float().cpu().numpy(), lp[0, k].cpu().numpy(), ids[0, k].cpu().numpy(), float(w[0, k]), 1.0,
                        tail)
        assert abs(float(a["loss"][0, k]) - r["loss"]) <= r["loss_tol"]
        assert abs(float(st["loss"][0, k]) - r["loss"]) <= r["loss_tol"]
        d = np.abs(st["dlogits"][0, k].float().cpu().numpy() - r["grad"])
        assert np.all(d <= r["grad_tol"] + ref.half(dtype == "bf16") * (np.abs(r["grad"]) + r["grad_tol"]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows_in_place(dtype):
    sv = _sv()
    for V in (2053, 70001):
        y, lp, ids, w = _case(2, 4, V, 24, dtype, V)
        y, lp, ids, w = (t.repeat((80,) + (1,) * (t.dim() - 1)) for t in (y, lp, ids, w))
        want = sv.distill_step(y, lp, ids, w)
        got = sv.distill_step(y, lp, ids, w, out={"dlogits": y})
        assert torch.equal(y, want["dlogits"]) and torch.equal(got["loss"], want["loss"])


@pytest.mark.parametrize("s", [0.1, 0.5, 2.0, 20.0])
@pytest.mark.parametrize("tail", [True, False])
def test_temperatures(s, tail):
    for dtype in ("bf16", "f32"):
        y, lp, ids, w = _case(2, 2, 3000, 30, dtype, 7, s=s)
        _check(y, lp, ids, w, s=s, tail=tail)


@pytest.mark.parametrize("tail", [True, False])
def test_peaked_rows(tail):
    """The list holds nearly all of the student's and the teacher's mass."""
    y, lp, ids, w = _case(2, 3, 6000, 32, "f32", 8)
    at = ids[..., 3:4].long()
    y.scatter_(-1, at, 40.0)
    lp[..., 0] = -1e-6
    lp[..., 1:] -= 20.0
    _check(y, lp, ids, w, tail=tail)


@pytest.mark.parametrize("tail", [True, False])
def test_lists_with_gaps_repeats_and_masks(tail):
    for dtype in ("bf16", "f32"):
        y, lp, ids, w = _case(3, 3, 2001, 24, dtype, 9)
        ids[0, 0, ::2] = -1                       # gaps
        ids[0, 1] = -1                            # an empty list
        ids[0, 2, 5] = ids[0, 2, 2]               # a token twice
        ids[1, 0, 1:] = ids[1, 0, 0]              # one token throughout
        lp[1, 0] = -4.0
        y[1, 1, ids[1, 1, 4].long()] = -INF       # a listed token the student masks
        y[1, 2, ::3] = -INF                       # masked vocabulary
        y[1, 2, ids[1, 2].long()] = 1.0
        w[2, 0] = 0
        y[2, 0] = float("nan")                    # not read
        y[2, 1, 1::2] = -3.38e38
        y[2, 1, ids[2, 1].long()] = 0.5
        lp[2, 2, 20:] = -INF                      # probability zero
        _check(y, lp, ids, w, tail=tail)


def test_only_listed_tokens_have_mass():
    y, lp, ids, w = _case(1, 2, 700, 10, "f32", 10)
    keep = torch.zeros_like(y).scatter_(-1, ids.long(), 1.0)
    y[keep == 0] = -INF
    _check(y, lp, ids, w, tail=True)
    _check(y, lp, ids, w, tail=False)


def test_rows_and_ids_that_are_wrong():
    sv = _sv()
    y, lp, ids, w = _case(2, 2, 900, 10, "f32", 11)
    ids2 = ids.clone()
    ids2[0, 1, 3] = 900
    ids2[1, 0, 0] = -7
    _check(y, lp, ids2, w, status_want=sv.api.SPEC_ERR_BAD_TOKEN)
    y2 = y.clone()
    y2[1, 1] = -INF
    _check(y2, lp, ids, w, status_want=sv.api.SPEC_ERR_BAD_ROW)
    clean = sv.distill_step(y, lp, ids, w)
    y2 = y.clone()
    y2[0, 1, 5] = float("nan")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = sv.distill_step(y2, lp, ids, w, status=status)
    torch.cuda.synchronize()
    assert int(status) == sv.api.SPEC_ERR_BAD_ROW and not torch.isfinite(got["loss"][0, 1])
    for b, k in ((0, 0), (1, 0), (1, 1)):
        assert torch.equal(got["loss"][b, k], clean["loss"][b, k])
        assert torch.equal(got["dlogits"][b, k], clean["dlogits"][b, k])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1037, 40003])
def test_strides_alignments_and_in_place(dtype, V):
    """Every start of the rows and of the gradient's rows; a row's sum is added
    in an order that its alignment sets, so bits are compared for one view."""
    sv = _sv()
    y, lp, ids, w = _case(3, 2, V, 20, dtype, 13)
    for off in range(5):
        wide = torch.full((3, 3, V + 9), 7.0, dtype=DT[dtype], device=DEV)
        view = wide[:, 1:, off:off + V]
        view.copy_(y)
        a, gwant, want = _check(view, lp, ids, w)
        stats = a["stats"]
        for goff in (off, (off + 1) % 5):
            gw = torch.full((3, 4, V + 11), 7.0, dtype=DT[dtype], device=DEV)
            gv = gw[:, :2, goff:goff + V]
            got = sv.distill_step(view, lp, ids, w, out={"dlogits": gv})
            assert torch.equal(got["dlogits"], want["dlogits"]) and torch.equal(got["loss"], want["loss"])
            gv.fill_(5.0)
            sv.distill_grad(view, lp, ids, stats, weight=w, out=gv)
            assert torch.equal(gv, gwant)
            gv.fill_(7.0)
            assert bool((gw == 7.0).all())          # nothing written beside the rows
        sv.distill_step(view, lp, ids, w, out={"dlogits": view})
        assert torch.equal(view, want["dlogits"])
        view.copy_(y)
        sv.distill_grad(view, lp, ids, stats, weight=w, out=view)
        assert torch.equal(view, gwant)
        view.fill_(7.0)
        assert bool((wide == 7.0).all())
    _check(y.transpose(0, 1).contiguous().transpose(0, 1), lp, ids, w)
    _check(y[:1, :1].expand(3, 2, V), lp, ids, w)   # a repeated student row


def test_gradient_against_differences():
    """Central differences of the reference's loss, in fp64: the step h = 1e-5
    leaves h^2 |f'''| / 6 < 1e-10 and 1e-16 * loss / h < 1e-10 per entry."""
    sv = _sv()
    for tail in (True, False):
        y, lp, ids, w = _case(1, 1, 40, 6, "f32", 14)
        got = sv.distill_step(y, lp, ids, w, inv_temperature=0.7, tail=tail)["dlogits"].cpu().numpy()[0, 0]
        yn, l, i = y.cpu().double().numpy()[0, 0], lp.cpu().numpy()[0, 0], ids.cpu().numpy()[0, 0]
        wt = float(w[0, 0])
        r = ref.distill(yn, l, i, wt, 0.7, tail)
        h = 1e-5
        for v in range(40):
            d = np.zeros(40)
            d[v] = h
            fd = (ref.distill(yn + d, l, i, wt, 0.7, tail)["loss"] - ref.distill(yn - d, l, i, wt, 0.7, tail)["loss"]) / (2 * h)
            assert abs(fd - got[v]) <= 1e-8 + r["grad_tol"][v] + ref.U * abs(fd)


def test_through_autograd():
    """The gradient goes on through the draft model as logits.backward()."""
    sv = _sv()
    y, lp, ids, w = _case(2, 3, 500, 12, "f32", 15)
    x = torch.randn((2, 3, 16), device=DEV)
    head = torch.randn((500, 16), device=DEV, requires_grad=True)
    logits = x @ head.t()
    r = sv.distill_step(logits.detach(), lp, ids, w)
    logits.backward(r["dlogits"])
    want = torch.einsum("bkv,bkd->vd", r["dlogits"].double(), x.double())
    err = (head.grad.double() - want).abs().max()
    # at most 6 products per entry, summed in fp32 or tf32-free fp32
    assert float(err) <= 8 * ref.U * float(torch.einsum("bkv,bkd->vd", r["dlogits"].double().abs(), x.double().abs()).max())


def test_streams_graphs_and_repeats():
    sv = _sv()
    y, lp, ids, w = _case(4, 2, 20011, 30, "bf16", 16)
    want = sv.distill_step(y, lp, ids, w)
    again = sv.distill_step(y, lp, ids, w)
    assert all(torch.equal(want[k], again[k]) for k in want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sv.distill_step(y, lp, ids, w, stream=s)
    s.synchronize()
    assert all(torch.equal(want[k], got[k]) for k in want)
    yy = y.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st = sv.distill_loss(yy, lp, ids, w)
        gr = sv.distill_grad(yy, lp, ids, st["stats"], weight=w)
        both = sv.distill_step(yy, lp, ids, w)
    yy.zero_()
    g.replay()
    yy.copy_(y)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(both["dlogits"], want["dlogits"]) and torch.equal(st["loss"], want["loss"])
    assert torch.equal(gr, sv.distill_grad(y, lp, ids, st["stats"], weight=w))
    empty = sv.distill_step(y[:0], lp[:0], ids[:0], w[:0])
    assert empty["dlogits"].shape == (0, 2, 20011)


def test_rows_without_a_batch_axis():
    sv = _sv()
    y, lp, ids, w = _case(6, 1, 3001, 12, "bf16", 17)
    want = sv.distill_step(y, lp, ids, w)
    two = [t[:, 0].contiguous() for t in (y, lp, ids, w)]
    got = sv.distill_step(*two)
    assert got["dlogits"].shape == (6, 3001) and got["loss"].shape == (6,)
    a = sv.distill_loss(*two)
    g = sv.distill_grad(two[0], two[1], two[2], a["stats"], weight=two[3])
    for r in range(6):   # another view of the same rows: the same alignments
        assert torch.equal(got["dlogits"][r], want["dlogits"][r, 0])
    assert torch.equal(got["loss"], want["loss"][:, 0]) and g.shape == (6, 3001)


def test_offsets_beyond_32_bits():
    """Student and gradient rows that start past 2^31 elements."""
    V = 5003
    buf = torch.zeros((2 ** 31 + 8 * V,), dtype=torch.bfloat16, device=DEV)
    far = buf.as_strided((2, 1, V), (2 ** 31 + 3 * V, V, 1))
    y, lp, ids, w = _case(2, 1, V, 16, "bf16", 18)
    far.copy_(y)
    _check(far, lp, ids, w)
    want = _sv().distill_step(far, lp, ids, w)
    got = _sv().distill_step(far, lp, ids, w, out={"dlogits": far})
    assert torch.equal(far, want["dlogits"]) and torch.equal(got["loss"], want["loss"])


def test_two_calls_and_two_graphs_at_once():
    """No call keeps anything that another could meet."""
    sv = _sv()
    a = _case(40, 2, 9001, 20, "bf16", 19)
    b = _case(3, 3, 60000, 100, "f32", 20)
    want = [sv.distill_step(*x) for x in (a, b)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got.append((sv.distill_step(*a, stream=s1), sv.distill_step(*b, stream=s2)))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sv.distill_step(*x))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    got.append(tuple(outs))
    for pair in got:
        for w, g in zip(want, pair):
            assert all(torch.equal(w[k], g[k]) for k in w)


def test_in_place_writes_are_seen_by_autograd():
    sv = _sv()
    y, lp, ids, w = _case(2, 2, 300, 8, "f32", 21)
    x = y.clone().requires_grad_()
    z = x * 1.0
    loss = (z * z).sum()              # keeps z for its backward pass
    sv.distill_step(z, lp, ids, w, out={"dlogits": z})
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_logits_at_the_mask_floor_are_masked():
    """fp32 -1e29 as a mask value gives what -inf gives, to the bit."""
    sv = _sv()
    y, lp, ids, w = _case(4, 3, 1501, 12, "f32", 31)
    listed = torch.zeros_like(y).scatter_(-1, ids.long(), 1.0) > 0
    mask = torch.zeros_like(listed)
    mask[0] = ~listed[0]                                   # only listed tokens have mass
    mask[1, 0] = True                                      # none has
    mask[1, 1, ::2] = True
    mask[2] = torch.rand(mask[2].shape, device=DEV) < 0.9
    mask[2, :, -1] = False
    for tail in (True, False):
        got = []
        for value in (-1e29, -INF):
            z = y.masked_fill(mask, value)
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            a = sv.distill_loss(z, lp, ids, w, tail=tail, status=status)
            g = sv.distill_grad(z, lp, ids, a["stats"], weight=w, tail=tail)
            step = sv.distill_step(z, lp, ids, w, tail=tail)
            got.append((a["loss"], a["stats"], g, step["loss"], step["dlogits"], status))
        for at, inf in zip(*got):
            assert torch.equal(at, inf)
        assert int(got[0][-1]) == sv.api.SPEC_ERR_BAD_ROW


@pytest.mark.parametrize("s", [0.05, 1.0, 20.0])
@pytest.mark.parametrize("value", [-1e9, -3e9, -1e10, -7e15, -1e20, -9e28, 2e10])
def test_logits_far_out(value, s):
    """Masks of ordinary size (-1e9, -1e20) and whole rows out there."""
    for dtype, V in (("f32", 3001), ("bf16", 40003)):
        y, lp, ids, w = _case(3, 3, V, 12, dtype, 32, s=s)
        listed = torch.zeros(y.shape, device=DEV).scatter_(-1, ids.long(), 1.0) > 0
        gen = torch.Generator().manual_seed(33)
        mask = (torch.rand(y.shape, generator=gen) < 0.9).to(DEV)
        mask[..., -1] = False
        mask[1] = ~listed[1]                                   # all unlisted tokens
        mask[2] = True                                         # all tokens,
        mask[2, 2, ids[2, 2, 0].long()] = False                # or all but a listed one
        z = y.masked_fill(mask, value)
        z[2, 1] = (value * (1 + torch.rand((V,), generator=gen))).to(z)   # a row spread out there
        for tail in (True, False):
            _check(z, lp, ids, w, s=s, tail=tail)


@pytest.mark.parametrize("s", [1e-4, 1e4])
@pytest.mark.parametrize("tail", [True, False])
def test_extreme_temperatures(s, tail):
    for dtype, V in (("f32", 3001), ("bf16", 40003)):
        y, lp, ids, w = _case(2, 3, V, 12, dtype, 35, s=s)
        _check(y, lp, ids, w, s=s, tail=tail)


@pytest.mark.parametrize("bad", [float("nan"), INF])
def test_spoilt_rows_far_out(bad):
    sv = _sv()
    y, lp, ids, w = _case(1, 3, 2001, 10, "f32", 37)
    y[:] = -1e20
    clean = sv.distill_step(y, lp, ids, w)
    unlisted = next(v for v in range(2001) if v not in ids[0, 1].tolist())
    y[0, 1, unlisted] = bad
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = sv.distill_step(y, lp, ids, w, status=status)
    torch.cuda.synchronize()
    assert int(status) == sv.api.SPEC_ERR_BAD_ROW and not torch.isfinite(got["loss"][0, 1])
    for k in (0, 2):
        assert torch.equal(got["loss"][0, k], clean["loss"][0, k])
        assert torch.equal(got["dlogits"][0, k], clean["dlogits"][0, k])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,M,noise", [(2003, 1, 0.1), (2003, 5, 0.02), (40003, 1, 0.3), (40003, 30, 0.01), (300, 150, 0.01)])
def test_small_divergences(V, M, noise, dtype):
    """Lists of little mass. With Z = So + Sl the sums' relative errors enter the
    divergence as P dZ + p_T (dZ - dSo) = (q_T - p_T) dSo + (1 - q_T) dSl, each at
    most DS; beside them stand the list's sum, two roundings of the result and 1e-9
    for the terms in two floats."""
    sv = _sv()
    y, lp, ids, _ = _case(2, 4, V, min(M, 128), dtype, 38, noise=noise, sigma=1.0)
    got = sv.distill_loss(y, lp, ids)["loss"].cpu().numpy().astype(np.float64)
    step = sv.distill_step(y, lp, ids)["loss"].cpu().numpy().astype(np.float64)
    yn, lpn, idn = y.float().cpu().numpy().astype(np.float64), lp.cpu().numpy().astype(np.float64), ids.cpu().numpy()
    for b in range(2):
        for k in range(4):
            want = ref.distill(yn[b, k], lpn[b, k], idn[b, k])["loss"]
            q = np.exp(yn[b, k] - ref.lse(yn[b, k]))
            listed = q[idn[b, k]].sum()
            P = np.exp(lpn[b, k]).sum()
            tol = (abs(P - listed) + listed) * ref.DS + 2 * ref.U * abs(want) + 1e-9
            tol += ref.DP * P * (1 + abs(np.log((1 - P) / (1 - listed))))
            assert abs(got[b, k] - want) <= tol and abs(step[b, k] - want) <= tol, (got[b, k], step[b, k], want, tol)
