"""The draft model's training and beam drafting operators: cases, plain forms and exact values.

Operators over rows of vocabulary logits, next to the verification pass:

* ``top``      -- a row's top M log-probabilities (what a teacher hands to its student);
* ``loss``, ``grad``, ``step`` -- distillation of the draft from those: per-row divergence, its
                  gradient by the draft's logits, and both in one call;
* ``beam``     -- one step of beam search: the best N continuations of W beams;
* ``reorder``  -- the beams' cached states put in the order of the surviving beams, in place.

``own = False`` computes each in elementary torch operations; ``own = True`` calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
INF = float("inf")


# ---- cases ------------------------------------------------------------------------------------

def listed():
    return [
        # the smallest vocabulary of the tests, a handful of rows: one decoding step's latency
        {"name": "top B4 K4 V1024 f32", "op": "top", "B": 4, "K": 4, "V": 1024, "M": 16, "dtype": "f32", "temp": 1.0},
        # teacher lists of a whole verification batch (the target rows of the drafts, bonus rows skipped)
        {"name": "top B256 K8 V128256", "op": "top", "B": 256, "K": 8, "V": 128256, "M": 64, "dtype": "bf16", "temp": 1.0},
        # the held-out loss of a small draft batch
        {"name": "loss B8 K5 V32000", "op": "loss", "B": 8, "K": 5, "V": 32000, "M": 32, "dtype": "bf16", "tail": True, "temp": 1.0},
        # the held-out loss of a large batch, long drafts and a large vocabulary, lists renormalised
        {"name": "loss B128 K15 V152064", "op": "loss", "B": 128, "K": 15, "V": 152064, "M": 64, "dtype": "bf16", "tail": False, "temp": 1.0},
        # backward pass alone (the loss ran earlier), mid-size batch
        {"name": "grad B64 K5 V128256", "op": "grad", "B": 64, "K": 5, "V": 128256, "M": 64, "dtype": "bf16", "tail": True, "temp": 1.0},
        # a vocabulary with one token added: no two rows start alike
        {"name": "grad B32 K4 V32001 f32", "op": "grad", "B": 32, "K": 4, "V": 32001, "M": 20, "dtype": "f32", "tail": True, "temp": 0.5},
        # one training step of the draft on a verification batch
        {"name": "step B256 K8 V128256", "op": "step", "B": 256, "K": 8, "V": 128256, "M": 64, "dtype": "bf16", "tail": True, "temp": 1.0},
        # a small online step, odd vocabulary
        {"name": "step B16 K4 V32001", "op": "step", "B": 16, "K": 4, "V": 32001, "M": 100, "dtype": "bf16", "tail": True, "temp": 2.0},
        # one user's beams: latency
        {"name": "beam B1 W4 V32000", "op": "beam", "B": 1, "W": 4, "N": 4, "V": 32000, "dtype": "bf16", "first": False},
        # a batch of wide beams, twice the beams kept for the host to finish hypotheses
        {"name": "beam B64 W8 V128256", "op": "beam", "B": 64, "W": 8, "N": 16, "V": 128256, "dtype": "bf16", "first": False},
        # a small draft model's cache
        {"name": "reorder L2 B4 W4", "op": "reorder", "L": 2, "B": 4, "W": 4, "H": 2, "T": 128, "D": 64, "dtype": "bf16"},
        # a batch's cache, contexts of many lengths
        {"name": "reorder L4 B32 W8", "op": "reorder", "L": 4, "B": 32, "W": 8, "H": 8, "T": 1024, "D": 128, "dtype": "bf16"},
    ]


def draw(rng):
    def logu(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["top", "top", "loss", "grad", "step", "step", "beam", "beam", "reorder"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    es = 2 if dtype == "bf16" else 4
    if op == "reorder":
        W = rng.randint(2, 16)
        H, D = rng.randint(1, 8), rng.choice([64, 128, 80, 33])
        T, L = logu(16, 2048), rng.randint(1, 4)
        B = max(1, min(logu(1, 32), int(1.5e9 // (L * W * H * T * D * es))))
        return {"op": op, "L": L, "B": B, "W": W, "H": H, "T": T, "D": D, "dtype": dtype}
    V = logu(1000, 160000)
    if op == "beam":
        W = rng.randint(1, 16)
        N = rng.randint(1, 2 * W)
        B = max(1, min(logu(1, 64), int(2e8 // (W * V * es))))
        return {"op": op, "B": B, "W": W, "N": N, "V": V, "dtype": dtype, "first": rng.random() < 0.15}
    K = rng.randint(1, 15)
    B = max(1, min(logu(1, 256), int(4e8 // (K * V * es))))
    c = {"op": op, "B": B, "K": K, "V": V, "M": logu(1, 128), "dtype": dtype, "temp": rng.choice([1.0, 1.0, 0.5, 2.0])}
    if op != "top":
        c["tail"] = rng.random() < 0.6
    return c


# ---- inputs -----------------------------------------------------------------------------------

def _rows(g, n, V, sigma):
    """Normal logits at a temperature per row, a likely token on every other row."""
    t = torch.randn((n, V), generator=g, device=DEV)
    t *= sigma / (0.5 + 1.5 * torch.rand((n, 1), generator=g, device=DEV))
    at = torch.randint(0, V, (n, 1), generator=g, device=DEV)
    lift = 12.0 * (torch.arange(n, device=DEV)[:, None] % 2).float()
    return t.scatter_add_(1, at, lift)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    dt = DT[case["dtype"]]
    if op == "reorder":
        L, B, W, H, T, D = (case[k] for k in "LBWHTD")
        state = torch.empty((L, B, W, H, T, D), dtype=dt, device=DEV)
        for i in range(L):
            state[i] = torch.randn((B, W, H, T, D), generator=g, device=DEV, dtype=dt)
        # survivors: the best beam goes on more than once, some beams stay where they are
        r = torch.rand((B, W), generator=g, device=DEV)
        parent = torch.randint(0, W, (B, W), generator=g, device=DEV)
        parent = torch.where(r < 0.3, torch.arange(W, device=DEV)[None], parent)
        parent = torch.where(r > 0.97, -1, parent).to(torch.int32)
        lengths = torch.randint(T // 2, T + 1, (B,), generator=g, device=DEV).to(torch.int32)
        return {"case": case, "state": state, "parent": parent, "lengths": lengths}
    B, V = case["B"], case["V"]
    if op == "beam":
        W = case["W"]
        z = torch.empty((B, W, V), dtype=dt, device=DEV)
        for b in range(0, B, 16):
            n = min(16, B - b)
            z[b:b + n] = _rows(g, n * W, V, 3.0).view(n, W, V).to(dt)
        z[..., V - V // 64:] = -INF  # the padded end of the vocabulary
        scores = -4.0 * torch.rand((B, W), generator=g, device=DEV)
        finished = (torch.rand((B, W), generator=g, device=DEV) < 0.1).to(torch.int32)
        if case["first"]:
            scores[:, 1:] = -INF
            scores[:, 0] = 0.0
            finished.zero_()
        return {"case": case, "logits": z, "scores": scores, "finished": finished, "eos": 2}
    K, M, s = case["K"], case["M"], 1.0 / case["temp"]
    rows = K + 1 if op == "top" else K
    z = torch.empty((B, rows, V), dtype=dt, device=DEV)
    logp = torch.empty((B, K, M), device=DEV)
    ids = torch.empty((B, K, M), dtype=torch.int32, device=DEV)
    m = min(M, V - V // 64)
    step = max(1, int(3e8 // (4 * rows * V)))
    for b in range(0, B, step):
        n = min(step, B - b)
        t = _rows(g, n * rows, V, 3.0)
        t[:, V - V // 64:] = -INF
        if op == "top":
            t[torch.rand(n * rows, generator=g, device=DEV) < 0.02] = -INF  # rows past a sequence's end
            z[b:b + n] = t.view(n, rows, V).to(dt)
            continue
        # the teacher's list, and a student some way off
        lse = torch.logsumexp(s * t, dim=-1, keepdim=True)
        val, at = torch.topk(t, m, dim=-1)
        logp[b:b + n], ids[b:b + n] = -INF, -1
        logp[b:b + n, :, :m] = (s * val - lse).view(n, K, m)
        ids[b:b + n, :, :m] = at.view(n, K, m).to(torch.int32)
        t += torch.randn(t.shape, generator=g, device=DEV)
        z[b:b + n] = t.view(n, rows, V).to(dt)
    if op == "top":
        return {"case": case, "logits": z[:, :K], "M": M, "s": s}
    weight = torch.rand((B, K), generator=g, device=DEV) / (B * K)
    weight[torch.rand((B, K), generator=g, device=DEV) < 0.1] = 0.0  # positions past the accepted ones
    state = {"case": case, "logits": z, "logp": logp, "ids": ids, "weight": weight, "s": s, "tail": case["tail"]}
    if op == "grad":
        state["stats"] = _stats(z, logp, ids, weight, s, case["tail"])["stats"]
        state["grad_loss"] = torch.rand((B, K), generator=g, device=DEV) + 0.5
    return state


# ---- the plain forms --------------------------------------------------------------------------

def _order(z):
    """One whole number per value: larger values first, and of equal ones the lowest index."""
    i = (z + 0.0).view(torch.int32)
    i = torch.where(i < 0, i ^ 0x7FFFFFFF, i).to(torch.int64)
    return (i << 21) + ((1 << 21) - 1 - torch.arange(z.shape[-1], device=z.device))


def _top(z, M):
    """Values and indices of the top M of the last axis; -inf and -1 where there are fewer."""
    m = min(M, z.shape[-1])
    key = torch.topk(_order(z), m, dim=-1).values
    at = (1 << 21) - 1 - (key & ((1 << 21) - 1))
    val = torch.gather(z, -1, at)
    at = torch.where(val == -INF, -1, at)
    if m < M:
        pad = z.shape[:-1] + (M - m,)
        val = torch.cat([val, torch.full(pad, -INF, device=z.device)], -1)
        at = torch.cat([at, torch.full(pad, -1, device=z.device)], -1)
    return val, at.to(torch.int32)


def _plain_top(z, M, s):
    z = z.float()
    mx = z.amax(-1, keepdim=True)
    safe = torch.where(mx == -INF, 0.0, mx)
    total = torch.exp(s * (z - safe)).sum(-1, keepdim=True)
    val, ids = _top(z, M)
    lse = s * safe + torch.log(total)
    logp = torch.where(ids < 0, -INF, s * (val - safe) - torch.log(total))
    return {"logprobs": logp, "ids": ids, "lse": lse[..., 0]}


def _list(logp, ids, tail):
    """Listed places, their probabilities, their sum, and the unlisted mass, in 64 bits."""
    here = ids >= 0
    p = torch.where(here, torch.exp(logp.double()), 0.0)
    P = p.sum(-1)
    if tail:
        return here, p, P, (1.0 - P).clamp(min=0.0)
    return here, p / P[..., None].clamp(min=1e-300), P, torch.zeros_like(P)


def _unlisted(y, ids, here):
    mark = torch.zeros(y.shape, dtype=torch.int32, device=y.device)
    return mark.scatter_add_(-1, ids.clamp(min=0).long(), here.int()) == 0


def _stats(y, logp, ids, weight, s, tail):
    """The loss and what its gradient needs of a row: (maximum, 1/sum, the unlisted tokens' maximum and factor)."""
    y = y.float()
    here, p, P, pt = _list(logp, ids, tail)
    live = (weight != 0) & here.any(-1)
    at = ids.clamp(min=0).long()
    mx = y.amax(-1)
    total = torch.exp(s * (y - mx[..., None])).sum(-1).double()
    out = torch.where(_unlisted(y, ids, here), y, -INF)
    mo = out.amax(-1)
    some = mo > -INF
    so = torch.exp(s * (out - torch.where(some, mo, 0.0)[..., None])).sum(-1).double()
    del out
    lq_t = torch.where(some, s * (mo - mx).double() + torch.log(so) - torch.log(total), -INF)
    logq = s * (torch.gather(y, -1, at) - mx[..., None]).double() - torch.log(total)[..., None]
    logp = logp.double() if tail else logp.double() - torch.log(P)[..., None]
    kl = torch.where(here & (p > 0), p * (logp - logq), 0.0).sum(-1)
    kl = kl + torch.where(some & (pt > 0), pt * (torch.log(pt) - lq_t), 0.0)
    factor = torch.where(some, (torch.exp(lq_t) - pt) / so, 0.0)
    stats = torch.stack([mx.double(), 1.0 / total, mo.double(), factor], -1)
    return {"loss": torch.where(live, weight * kl, 0.0).float(), "stats": torch.where(live[..., None], stats, 0.0).float()}


def _plain_grad(y, logp, ids, stats, scale, s, tail):
    here, p, P, _ = _list(logp, ids, tail)
    live = (stats[..., 1] != 0) & (scale != 0)
    mx, inv, mo, factor = (stats[..., i, None] for i in range(4))
    if tail:
        inv = torch.where(mo == -INF, P[..., None].float(), 1.0) * inv
    mo = torch.where(mo == -INF, 0.0, mo)
    y32 = y.float()
    free = _unlisted(y, ids, here)
    g = torch.where(free, torch.exp(s * (y32 - mo)) * factor, torch.exp(s * (y32 - mx)) * inv)
    del y32, free
    g = g.scatter_add_(-1, ids.clamp(min=0).long(), -p.float()) * (scale * s)[..., None]
    return torch.where(live[..., None], g, 0.0).to(y.dtype)


def _plain_beam(z, scores, finished, eos, N):
    B, W, V = z.shape
    n = min(N, V)
    val, ids = _top(z.float(), n)
    z64 = z.double()  # scores of two beams can lie closer than 32 bits tell apart
    mx = z64.amax(-1, keepdim=True)
    lse = mx + torch.log(torch.exp(z64 - mx).sum(-1, keepdim=True))
    del z64
    total = scores.double()[..., None] + (val.double() - lse)
    total = torch.where(ids < 0, -INF, total)
    done = (finished != 0)[..., None]
    first = torch.arange(n, device=z.device) == 0
    total = torch.where(done, torch.where(first, scores.double()[..., None], -INF), total)
    ids = torch.where(done, eos, ids)
    total = torch.where((scores == -INF)[..., None], -INF, total).view(B, W * n)
    flat = (torch.arange(W, device=z.device)[:, None] * V + ids.long()).view(B, W * n)
    order = torch.argsort(flat, dim=-1, stable=True)
    total, flat = torch.gather(total, -1, order), torch.gather(flat, -1, order)
    total, order = torch.sort(total, dim=-1, descending=True, stable=True)
    flat = torch.gather(flat, -1, order)
    if total.shape[1] < N:
        pad = (B, N - total.shape[1])
        total = torch.cat([total, torch.full(pad, -INF, dtype=total.dtype, device=z.device)], -1)
        flat = torch.cat([flat, torch.zeros(pad, dtype=flat.dtype, device=z.device)], -1)
    total, flat = total[:, :N], flat[:, :N]
    none = total == -INF
    parent = torch.where(none, -1, flat // V).to(torch.int32)
    token = torch.where(none, -1, flat % V).to(torch.int32)
    over = (~none & (token == eos)).to(torch.int32)
    return {"scores": total.float(), "parent": parent, "token": token, "finished": over}


def _plain_reorder(state, parent, lengths):
    L, B, W, H, T, D = state.shape
    src = torch.where(parent < 0, torch.arange(W, device=state.device), parent.long())
    live = (torch.arange(T, device=state.device)[None] < lengths[:, None]).view(1, B, 1, 1, T, 1)
    moved = torch.gather(state, 2, src.view(1, B, W, 1, 1, 1).expand(state.shape))
    return state.copy_(torch.where(live, moved, state))


def run(state):
    op = state["case"]["op"]
    if own:
        import speculative_decoding_token_verify_gb300 as sv

        if op == "top":
            return sv.top_logprobs(state["logits"], state["M"], inv_temperature=state["s"])
        if op == "beam":
            return sv.beam_step(state["logits"], state["scores"], state["case"]["N"], finished=state["finished"],
                                eos=state["eos"])
        if op == "reorder":
            return sv.beam_reorder(state["state"], state["parent"], lengths=state["lengths"], batch_dim=1)
        y, logp, ids = state["logits"], state["logp"], state["ids"]
        kw = {"weight": state["weight"], "inv_temperature": state["s"], "tail": state["tail"]}
        if op == "loss":
            return sv.distill_loss(y, logp, ids, **kw)
        if op == "grad":
            return sv.distill_grad(y, logp, ids, state["stats"], state["grad_loss"], **kw)
        return sv.distill_step(y, logp, ids, **kw)
    if op == "top":
        return _plain_top(state["logits"], state["M"], state["s"])
    if op == "beam":
        return _plain_beam(state["logits"], state["scores"], state["finished"], state["eos"], state["case"]["N"])
    if op == "reorder":
        return _plain_reorder(state["state"], state["parent"], state["lengths"])
    y, logp, ids, w, s, tail = (state[k] for k in ("logits", "logp", "ids", "weight", "s", "tail"))
    if op == "grad":
        return _plain_grad(y, logp, ids, state["stats"], w * state["grad_loss"], s, tail)
    r = _stats(y, logp, ids, w, s, tail)
    if op == "loss":
        return {"loss": r["loss"], "stats": r["stats"]}
    return {"loss": r["loss"], "dlogits": _plain_grad(y, logp, ids, r["stats"], w, s, tail)}


# ---- work -------------------------------------------------------------------------------------

def work(case):
    op, es = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op == "reorder":
        # rows that change places, read and written: about 0.7 (1 - 1/W) of them, three quarters long
        moved = 0.7 * (1 - 1 / case["W"]) * 0.75
        return {"bytes": 2 * moved * es * math.prod(case[k] for k in "LBWHTD"), "flops": 0}
    V = case["V"]
    if op == "beam":
        live = case["B"] * (1 if case["first"] else 0.9 * case["W"])
        return {"bytes": live * V * es + case["B"] * (case["W"] * 8 + case["N"] * 16), "flops": 4 * live * V}
    R, M = case["B"] * case["K"], case["M"]
    if op == "top":
        return {"bytes": R * (V * es + 8 * M + 4), "flops": 4 * R * V}
    live = 0.9 * R  # rows of weight zero need no reading
    if op == "loss":
        return {"bytes": live * (V * es + 8 * M) + R * 24, "flops": 4 * live * V}
    return {"bytes": live * (V * es + 8 * M) + R * (V * es + 28), "flops": (4 if op == "grad" else 7) * live * V}


# ---- exact values, in 64 bits, row after row --------------------------------------------------

def _ranked(values, places):
    """(value, place) pairs without -inf, best first, equal ones by place."""
    pairs = [(-v, p) for v, p in zip(values, places) if v > -INF]
    pairs.sort()
    return [(-v, p) for v, p in pairs]


def _exact_top(st):
    z, M, s = st["logits"], st["M"], st["s"]
    B, K, V = z.shape
    logp = torch.full((B, K, M), -INF, dtype=torch.float64, device=DEV)
    ids = torch.full((B, K, M), -1, dtype=torch.int32, device=DEV)
    lse = torch.empty((B, K), dtype=torch.float64, device=DEV)
    m = min(M, V)
    for b in range(B):
        x = z[b].to(torch.float64)
        lse[b] = torch.logsumexp(x * s, dim=1)
        val, at = x.sort(dim=1, descending=True, stable=True)
        val, at = val[:, :m], at[:, :m]
        ok = ~torch.isneginf(val)
        logp[b, :, :m] = torch.where(ok, val * s - torch.where(ok.any(1), lse[b], 0.0)[:, None], -INF)
        ids[b, :, :m] = torch.where(ok, at, -1).to(torch.int32)
    return {"logprobs": logp, "ids": ids, "lse": lse}


def _exact_distill(st, op):
    y, w, s, tail = st["logits"], st["weight"].double(), st["s"], st["tail"]
    B, K, V = y.shape
    logp, ids = st["logp"].double(), st["ids"].long()
    loss = torch.zeros((B, K), dtype=torch.float64, device=DEV)
    stats = torch.zeros((B, K, 4), dtype=torch.float64, device=DEV)
    grads = torch.zeros((B, K, V), dtype=torch.float64, device=DEV) if op != "loss" else None
    up = w * st["grad_loss"].double() if op == "grad" else w
    alive = ((w != 0) & (ids >= 0).any(-1)).cpu()
    for b in range(B):
        for k in range(K):
            if not alive[b, k]:
                continue
            keep = ids[b, k] >= 0
            where, lp = ids[b, k][keep], logp[b, k][keep]
            row = s * y[b, k].double()
            lq = torch.log_softmax(row, 0)
            listed_ = torch.zeros(V, dtype=torch.bool, device=DEV)
            listed_[where] = True
            free = row.masked_fill(listed_, -INF)
            peak = free.max()
            some = peak > -INF
            rest = torch.logsumexp(lq.masked_fill(listed_, -INF), 0)
            share = torch.where(some, torch.softmax(free, 0), 0.0)  # of the unlisted mass
            mass = lp.exp().sum()
            left = (1 - mass).clamp(min=0) if tail else torch.zeros_like(mass)
            if not tail:
                lp = lp - mass.log()
            target = lp.exp()
            d = (target * (lp - lq[where])).sum() + torch.where(some & (left > 0), left * (left.log() - rest), 0.0)
            loss[b, k] = w[b, k] * d
            excess = torch.where(some, rest.exp() - left, 0.0)
            stats[b, k] = torch.stack([row.max() / s, lq.max().exp(), peak / s, excess * share.max()])
            if grads is not None:
                q = lq.exp() * torch.where(some, 1.0, target.sum())
                x = torch.where(listed_, q, excess * share).index_add(0, where, -target)
                grads[b, k] = s * up[b, k] * x
    if op == "loss":
        return {"loss": loss, "stats": stats}
    return grads if op == "grad" else {"loss": loss, "dlogits": grads}


def _exact_beam(st, N):
    z, eos = st["logits"], st["eos"]
    B, W, V = z.shape
    out = {"scores": torch.full((B, N), -INF, dtype=torch.float64)}
    for k in ("parent", "token", "finished"):
        out[k] = torch.full((B, N), 0 if k == "finished" else -1, dtype=torch.int32)
    sc, over = st["scores"].double().cpu(), st["finished"].cpu()
    for b in range(B):
        x = torch.log_softmax(z[b].double(), dim=-1)
        val, at = x.sort(dim=-1, descending=True, stable=True)
        val, at = val[:, :N].cpu(), at[:, :N].cpu()
        pool = []
        for w in range(W):
            if sc[b, w] == -INF:
                continue
            if over[b, w]:
                pool += _ranked([float(sc[b, w])], [w * V + eos])
            else:
                pool += _ranked((val[w] + sc[b, w]).tolist(), (w * V + at[w]).tolist())
        pool = _ranked([v for v, _ in pool], [p for _, p in pool])[:N]
        for n, (v, place) in enumerate(pool):
            out["scores"][b, n] = v
            out["parent"][b, n], out["token"][b, n] = place // V, place % V
            out["finished"][b, n] = int(place % V == eos)
    return out


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "top":
        return _exact_top(st)
    if op == "beam":
        return _exact_beam(st, case["N"])
    if op == "reorder":
        return None  # values are moved, not computed
    return _exact_distill(st, op)
