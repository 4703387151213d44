"""Plain fp64 references (numpy) of the row operators, one row at a time, and
the tolerances their fp32 kernels are held to.

Tolerances. S is a row's sum of exponentials. Its relative error is at most
DS = 4e-6: an exponential's own error (2^-22), its argument's two roundings
(2^-24 |y| ln 2 in all, 1e-6 at |y| = 24; smaller terms carry no mass), and the
additions on a term's way into the sum (at most 32, each 2^-24 of the partial
sum, 1.9e-6): 3.2e-6. An argument y = (z - M) s log2e carries two roundings, so an
exponential of its own (a gradient's q) is off by |y| 2^-23 ln 2 besides.
The list's sum P is formed from exponentials of relative error DP = 2e-10, and
p_T = 1 - P is off by DP P: e^r, |r| <= 0.35, is summed as 1 + r + r^2/2 + r^3/6
with every rounding carried, and r^4 Q(r) <= 6.3e-4 in plain fp32, of at most
four roundings (its factors r^2, r^4, Q and the product): 6.3e-4 * 4 * 2^-24 =
1.5e-10; the reduced argument and the final sum add less than 1e-11.
U = 2^-24 is half a step of fp32 and `half(dtype)` that of the output."""
import numpy as np

DS = 4e-6
DP = 2e-10
U = 2.0 ** -24
TINY = 2.0 ** -125   # two steps (a quotient and a difference) that lose what is below fp32's normal range, 2^-126
FLOOR = float(np.float32(-1e29))   # logits up to it count as masked


def half(bf16):
    return 2.0 ** -8 if bf16 else 2.0 ** -24


def _masked(z):
    z = np.asarray(z, np.float64)
    return np.where(z <= FLOOR, -np.inf, z)


def max_lnsum(z, s=1.0):
    """m = max z and ln sum e^{s (z - m)}: apart, because s m of 1e20 has no room for the other in fp64."""
    z = _masked(z)
    m = z.max()
    return (m, 0.0) if m == -np.inf else (m, np.log(np.exp(s * (z - m)).sum()))


def lse(z, s=1.0):
    m, lnS = max_lnsum(z, s)
    return s * m + lnS


def order(z, m):
    """Indices of the m largest unmasked logits, equal ones by index."""
    z = _masked(z)
    at = np.argsort(-z, kind="stable")[:m]
    return at[z[at] > -np.inf]


def top(z, M, s=1.0):
    """(logprobs [M], ids [M], lse, tolerance of logprobs, tolerance of lse)."""
    z = _masked(z)
    m, lnS = max_lnsum(z, s)
    L = s * m + lnS
    at = order(z, M)
    lp, ids, tol = np.full(M, -np.inf), np.full(M, -1, np.int32), np.zeros(M)
    lp[:len(at)] = s * (z[at] - m) - lnS if len(at) else 0.0
    ids[:len(at)] = at
    if not len(at):
        return lp, ids, L, tol, 0.0
    # roundings: z - M, its product with s, ln S, the difference
    tol[:len(at)] = DS + U * (3 * np.abs(s * (z[at] - m)) + 2 * abs(lnS) + np.abs(lp[:len(at)]))
    return lp, ids, L, tol, DS + U * (2 * abs(s * m) + 2 * abs(lnS) + 2 * abs(L))


def distill(y, lp, ids, w=1.0, s=1.0, tail=True, up=1.0):
    """dict(loss, stats, grad) with tolerances under loss_tol, stats_tol, grad_tol (without the output's rounding)."""
    y, lp, ids = _masked(y), np.asarray(lp, np.float64), np.asarray(ids)
    V = y.shape[0]
    keep = (ids >= 0) & (ids < V)
    ids, lp = ids[keep], lp[keep]
    p = np.exp(lp)
    P = p.sum()
    zero = dict(loss=0.0, stats=np.zeros(4), grad=np.zeros(V), loss_tol=0.0, stats_tol=np.zeros(4), grad_tol=np.zeros(V))
    if w == 0 or not len(ids) or (not tail and P == 0):
        return zero
    m, lnS = max_lnsum(y, s)
    if m == -np.inf:
        return {**zero, "loss": np.inf if w > 0 else -np.inf}
    lq = s * (y - m) - lnS
    q = np.exp(lq)
    out = np.ones(V, bool)
    out[ids] = False
    mo = y[out].max() if out.any() else -np.inf
    pT = max(0.0, 1.0 - P) if tail else 0.0
    ln, pn = (lp, p) if tail else (lp - np.log(P), p / P)
    pos = pn > 0
    kl = float((pn[pos] * (ln[pos] - lq[ids[pos]])).sum())
    target = np.zeros(V)
    np.add.at(target, ids, pn)
    g, gt, kl_tol = q.copy(), np.zeros(V), 0.0
    inv = np.exp(-lnS)
    stats, st = np.array([m, inv, -np.inf, 0.0]), np.array([0.0, inv * (DS + 2 * U), 0.0, 0.0])

    def arg(z, ref_):   # |argument| where an exponential is more than 0
        return np.where(np.isfinite(z), np.abs(s * (z - ref_)), 0.0)

    if mo > -np.inf:
        lnSo = max_lnsum(np.where(out, y, -np.inf), s)[1]
        lqT = s * (mo - m) + lnSo - lnS
        qT = np.exp(lqT)
        r = np.where(out, np.exp(s * (y - mo) - lnSo), 0.0)
        if pT > 0:
            kl += pT * (np.log(pT) - lqT)
        excess = qT - pT
        # q_T: two sums, and the exponential between the two maxima
        et = qT * (2 * DS + 4 * U * abs(s * (m - mo)))
        if pT > 0:   # and the list's sum
            et += DP * P
            kl_tol += DP * P * (1 + abs(np.log(pT) - lqT))
        g = np.where(out, excess * r, q)
        gt = r * (et + abs(excess) * (DS + 2 * U * arg(y, mo) + 2.0 ** -22 + 8 * U))
        k = np.exp(-lnSo)
        stats[2:], st[2:] = [mo, excess * k], [0.0, k * (et + abs(excess) * (DS + 2 * U)) + TINY]
    elif tail:
        g = P * q
    g = np.where(out, g, g - target)
    # listed: q's sum, argument and products, and p's rounding
    gt = np.where(out, gt, q * max(1.0, P) * (DS + 2 * U * arg(y, m) + 2.0 ** -22 + 8 * U) + 6 * U * target)
    f = abs(w * up * s)
    return dict(loss=w * kl, loss_tol=abs(w) * (3 * DS + 4 * U * abs(kl) + kl_tol) if np.isfinite(kl) else 0.0, stats=stats,
                stats_tol=st, grad=w * up * s * g, grad_tol=f * gt + 1e-37 * (1 + f))


def beam(z, scores, N, finished=None, eos=-1):
    """One sequence: (scores [N] f64, parent, token, finished, tolerance)."""
    W, V = z.shape
    pool = []
    for w in range(W):
        if not scores[w] > -np.inf:
            continue
        if finished is not None and finished[w]:
            pool.append((-float(scores[w]), w * V + eos, 0.0))
            continue
        m, lnS = max_lnsum(z[w])
        for v in order(z[w], N):
            sc = float(scores[w]) + ((float(z[w][v]) - m) - lnS)
            pool.append((-sc, w * V + int(v), DS))
    pool.sort()
    pool = pool[:N]
    sc, par = np.full(N, -np.inf), np.full(N, -1, np.int32)
    tok, fin, tol = np.full(N, -1, np.int32), np.zeros(N, np.int32), np.zeros(N)
    for i, (s, place, d) in enumerate(pool):
        sc[i], par[i], tok[i] = -s, place // V, place % V
        fin[i] = tok[i] == eos
        tol[i] = d + 2 * U * abs(s)
    return sc, par, tok, fin, tol


def reorder(state, parent, lengths=None):
    """state [O, B, W, H, T, X] -> new state [O, B, N.., H, T, X] in place of the first N beams."""
    new = state.copy()
    T = state.shape[4]
    for b in range(state.shape[1]):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        for i, p in enumerate(parent[b]):
            if 0 <= p < state.shape[2]:
                new[:, b, i, :, :n] = state[:, b, p, :, :n]
    return new
