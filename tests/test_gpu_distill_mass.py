"""Distillation lists whose probabilities sum to more than 1 (a token listed
twice, lists put together by hand): the gradient against automatic
differentiation of the loss in fp64, which shares no formula with the row
references."""
import numpy as np
import pytest

import rows_reference as ref

torch = pytest.importorskip("torch")
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def divergence(y, lp, ids, s, tail):
    """The loss of one row in fp64, written from its definition: y [V], lp and ids [M]."""
    keep = ids >= 0
    lp, ids = lp[keep], ids[keep].long()
    logq = torch.log_softmax(s * y, 0)
    P = lp.exp().sum()
    if not tail:
        lp = lp - P.log()
    kl = (lp.exp() * (lp - logq[ids])).sum()
    free = torch.ones(y.shape[0], dtype=torch.bool)
    free[ids] = False
    if tail and P < 1 and bool(free.any()):
        pT = 1 - P
        kl = kl + pT * (pT.log() - torch.logsumexp(logq[free], 0))
    return kl


def gradient(y, lp, ids, s, tail):
    y = y.clone().requires_grad_()
    loss = divergence(y, lp, ids, s, tail)
    return float(loss.detach()), torch.autograd.grad(loss, y)[0]


def _case(K, V, M, dtype, masses, repeats, seed, s):
    """K student rows, lists of the given masses, with or without a token listed twice."""
    g = torch.Generator().manual_seed(seed)
    t = 3 * torch.randn((K, V), generator=g)
    y = (t + torch.randn((K, V), generator=g)).to(DT[dtype])
    m = min(M, V)
    val, at = torch.topk(t, m, dim=-1)
    ids = at.to(torch.int32)
    if repeats:
        ids[:, m - 1] = ids[:, 0]
        ids[:, m // 2] = ids[:, 0]
    lp = s * val.double()
    lp = lp - torch.logsumexp(lp, -1, keepdim=True) + torch.log(torch.tensor(masses, dtype=torch.float64))[:, None]
    return y, lp.float(), ids


def test_differentiation_against_differences():
    """h = 1e-5 leaves h^2 |f'''| / 6 < 1e-10 and 1e-15 |f| / h < 1e-9 per entry (|f| < 10)."""
    masses = [0.7, 1.0 + 1e-4, 1.2, 2.5]
    for repeats in (False, True):
        y, lp, ids = _case(4, 40, 6, "f32", masses, repeats, 1, 0.7)
        y, lp = y.double(), lp.double()
        for tail in (True, False):
            for k in range(4):
                _, g = gradient(y[k], lp[k], ids[k], 0.7, tail)
                for v in range(40):
                    d = torch.zeros(40, dtype=torch.float64)
                    d[v] = 1e-5
                    f = [float(divergence(x, lp[k], ids[k], 0.7, tail)) for x in (y[k] + d, y[k] - d)]
                    assert abs((f[0] - f[1]) / 2e-5 - float(g[v])) <= 2e-9
                assert abs(float(g.sum())) < 1e-12   # a softmax's gradient sums to zero


def _tolerance(y, lp, ids, s, tail, w, half):
    """Per entry. c = P beyond mass 1 (else 1), p_T = 0 there. Listed entries are
    c q - p: q's sum (DS), argument (2 U |arg|), exponential (2^-22), and c / Z's
    roundings; p's own. Unlisted ones c q_T r: q_T from two sums, r a sum and an
    exponential. Factors' roundings: at most ten of U. Masses up to 1 + 2^-15 take
    c = 1: off by (P - 1) q."""
    keep = ids >= 0
    i, p = ids[keep].long(), lp[keep].double().exp()
    P = float(p.sum())
    y = y.double()
    m = float(y.max())
    q = torch.softmax(s * y, 0)
    free = torch.ones(y.shape[0], dtype=torch.bool)
    free[i] = False
    c = P if tail else 1.0
    target = torch.zeros_like(q).index_add_(0, i, p if tail else p / P)
    arg = (s * (y - m)).abs()
    tol = c * q * (ref.DS + 2 * ref.U * arg + 2.0 ** -22 + 10 * ref.U) + 6 * ref.U * target
    if bool(free.any()):
        mo = float(y[free].max())
        argo = (s * (y - mo)).abs()
        tol = torch.where(free, c * q * (3 * ref.DS + 4 * ref.U * abs(s * (m - mo)) + 2 * ref.U * argo + 2.0 ** -22 + 10 * ref.U),
                          tol)
        if tail and 1 < P <= 1 + 2.0 ** -15 * (1 + 1e-3):
            tol = tol + (P - 1) * q
    return abs(w) * s * tol


@pytest.mark.gpu
@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,M,s", [(40, 6, 0.7), (9, 9, 1.0), (2001, 24, 1.0), (16001, 128, 0.5), (128256, 64, 2.0)])
def test_mass_above_one(V, M, s, dtype, tail):
    import speculative_decoding_token_verify_gb300 as sv
    sv.build()
    masses = [1.2, 3.0, 1.001, 1.0 + 1e-4, 1.0 + 2e-5]
    K = len(masses)
    for repeats in (False, True):
        y, lp, ids = _case(K, V, M, dtype, masses, repeats, V + M, s)
        w = torch.linspace(0.25, 1.0, K)
        up = torch.linspace(1.5, 0.5, K)
        yd, lpd, idd = y[None].to(DEV), lp[None].to(DEV), ids[None].to(DEV)
        kw = dict(weight=w[None].to(DEV), inv_temperature=s, tail=tail)
        a = sv.distill_loss(yd, lpd, idd, **kw)
        g = sv.distill_grad(yd, lpd, idd, a["stats"], up[None].to(DEV), **kw)
        step = sv.distill_step(yd, lpd, idd, **kw)
        torch.cuda.synchronize()
        half = ref.half(dtype == "bf16")
        for k in range(K):
            loss, want = gradient(y[k].double(), lp[k].double(), ids[k], s, tail)
            P = float(lp[k].double().exp().sum())
            # the terms' sums in two floats; ln Z's error times the list's mass; two roundings
            lt = float(w[k]) * ((P if tail else 1.0) * ref.DS + 4 * ref.U * abs(loss) + 1e-8 * (1 + P))
            for got in (a["loss"], step["loss"]):
                assert abs(float(got[0, k]) - float(w[k]) * loss) <= lt, (repeats, k)
            for got, f in ((step["dlogits"], float(w[k])), (g, float(w[k]) * float(up[k]))):
                tol = _tolerance(y[k], lp[k], ids[k], s, tail, f, half)
                exact = want * f
                tol = tol + half * (exact.abs() + tol) + 1e-37
                off = (got[0, k].double().cpu() - exact).abs()
                assert bool((off <= tol).all()), (repeats, k, float((off / tol).max()), int((off / tol).argmax()))


def test_reference_holds_up_to_mass_one():
    """The row references' gradient is that of the loss for masses up to 1."""
    y, lp, ids = _case(3, 50, 7, "f32", [0.3, 0.9, 1.0 - 1e-6], True, 2, 1.0)
    for k in range(3):
        for tail in (True, False):
            loss, g = gradient(y[k].double(), lp[k].double(), ids[k], 1.0, tail)
            r = ref.distill(y[k].numpy(), lp[k].numpy(), ids[k].numpy(), tail=tail)
            assert abs(r["loss"] - loss) < 1e-9 and np.abs(r["grad"] - g.numpy()).max() < 1e-9


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_little_teacher_mass_left(dtype):
    """M equal probabilities that leave the unlisted tokens 1e-7 or so of the
    teacher's mass, and a student that leaves them none: the gradient there is
    -p_T r, as good as the list's sum (DP of P)."""
    import speculative_decoding_token_verify_gb300 as sv
    sv.build()
    V, lists = 300, [2, 3, 5, 7, 11, 23, 45, 64, 90, 91, 128]
    for M in lists:
        l = np.float32(-np.log(M))
        while M * np.exp(float(l)) >= 1.0:
            l = np.nextafter(l, np.float32(-100))
        lp = torch.full((1, 1, M), float(l))
        ids = torch.arange(M, dtype=torch.int32)[None, None] * 2
        y = torch.full((1, 1, V), -60.0)
        y[..., ids[0, 0].long()] = 1.0
        y = y.to(DT[dtype])
        a = sv.distill_loss(y.to(DEV), lp.to(DEV), ids.to(DEV))
        g = sv.distill_grad(y.to(DEV), lp.to(DEV), ids.to(DEV), a["stats"])
        step = sv.distill_step(y.to(DEV), lp.to(DEV), ids.to(DEV))["dlogits"]
        r = ref.distill(y[0, 0].float().numpy(), lp[0, 0].numpy(), ids[0, 0].numpy())
        tol = r["grad_tol"] + ref.half(dtype == "bf16") * (np.abs(r["grad"]) + r["grad_tol"])
        for got in (g, step):
            off = np.abs(got[0, 0].float().cpu().double().numpy() - r["grad"])
            assert np.all(off <= tol), (M, float((off / tol).max()))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,M", [(40, 6), (2001, 24), (40003, 128)])
def test_renormalised_lists_of_any_level(V, M, dtype):
    """With tail = 0 only differences of the list's log-probabilities count: levels
    whose probabilities all leave fp32's range."""
    import speculative_decoding_token_verify_gb300 as sv
    sv.build()
    levels = [-600.0, -103.0, -90.0, 89.0, 300.0]
    K = len(levels)
    for repeats in (False, True):
        y, lp, ids = _case(K, V, M, dtype, [1.0] * K, repeats, V + M, 1.0)
        lp = (lp.double() + torch.tensor(levels, dtype=torch.float64)[:, None]).float()
        ids[0, M // 2] = -1
        lp[1, M - 1] = -float("inf")
        w = torch.linspace(0.25, 1.0, K)
        yd, lpd, idd = y[None].to(DEV), lp[None].to(DEV), ids[None].to(DEV)
        kw = dict(weight=w[None].to(DEV), tail=False)
        a = sv.distill_loss(yd, lpd, idd, **kw)
        g = sv.distill_grad(yd, lpd, idd, a["stats"], **kw)
        step = sv.distill_step(yd, lpd, idd, **kw)
        half = ref.half(dtype == "bf16")
        for k in range(K):
            keep = (ids[k] >= 0) & (lp[k] > -float("inf"))
            l, i = lp[k][keep].double(), ids[k][keep]
            loss, want = gradient(y[k].double(), l, i, 1.0, False)
            f = float(w[k])
            lt = f * (ref.DS + 4 * ref.U * abs(loss) + 2e-8)
            for got in (a["loss"], step["loss"]):
                assert abs(float(got[0, k]) - f * loss) <= lt, (repeats, k, float(got[0, k]), f * loss)
            tol = _tolerance(y[k], l, i, 1.0, False, f, half)
            exact = want * f
            tol = tol + half * (exact.abs() + tol) + 1e-37
            for got in (step["dlogits"], g):
                off = (got[0, k].double().cpu() - exact).abs()
                assert bool((off <= tol).all()), (repeats, k, float((off / tol).max()))
    lp.fill_(-float("inf"))                   # no probability at all: an empty list
    a = sv.distill_loss(yd, lp[None].to(DEV), idd, **kw)
    assert not a["loss"].any() and not a["stats"].any()
