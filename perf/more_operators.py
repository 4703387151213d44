"""Verifying trees of drafts over a paged cache: cases, plain forms and exact values.

The operators of one decoding step whose drafts form a tree, next to the verification pass:

* ``attend``  -- attention of the tree's nodes over a cache held in pages (one node: a decoding step);
* ``accept``  -- the walk down the tree along the target's choices;
* ``compact`` -- the accepted nodes' keys and values moved together at the end of the context;
* ``fork``    -- rows of pages in the order of the surviving beams: full pages shared, partial ones copied;
* ``resize``  -- pages given to rows that grew, and taken from rows that shrank or ended.

A table [rows, M] of page numbers (-1: none) says where a row's tokens lie; refs [P] counts the table entries that
name a page (0: free). ``own = False`` computes each in elementary torch operations; ``own = True`` calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
INF = float("inf")


# ---- cases ------------------------------------------------------------------------------------

def listed():
    return [
        # one user's next token without drafts: latency
        {"name": "attend B1 N1 L2048", "op": "attend", "B": 1, "N": 1, "L": 2048, "Hkv": 8, "G": 4, "D": 128, "page": 16, "dtype": "bf16"},
        # a verification batch: eight drafts and the last token, contexts of many lengths
        {"name": "attend B64 N9 L8192", "op": "attend", "B": 64, "N": 9, "L": 8192, "Hkv": 8, "G": 4, "D": 128, "page": 16, "dtype": "bf16"},
        # wide trees over long contexts: arithmetic counts
        {"name": "attend B8 N64 L32768", "op": "attend", "B": 8, "N": 64, "L": 32768, "Hkv": 8, "G": 8, "D": 128, "page": 64, "dtype": "bf16"},
        # odd head counts and widths, a few short contexts
        {"name": "attend B5 N33 L1000 f16", "op": "attend", "B": 5, "N": 33, "L": 1000, "Hkv": 3, "G": 5, "D": 80, "page": 32, "dtype": "f16"},
        # one user's tree of eight drafts: latency
        {"name": "accept B1 N9", "op": "accept", "B": 1, "N": 9},
        # a batch of the widest trees
        {"name": "accept B256 N128", "op": "accept", "B": 256, "N": 128},
        # one user's accepted drafts in a small draft model's cache
        {"name": "compact B1 N9 O4", "op": "compact", "B": 1, "N": 9, "O": 4, "L": 512, "Hkv": 2, "D": 64, "page": 16, "dtype": "bf16"},
        # a batch's accepted drafts, keys and values of many layers
        {"name": "compact B64 N33 O32", "op": "compact", "B": 64, "N": 33, "O": 32, "L": 256, "Hkv": 8, "D": 128, "page": 16, "dtype": "bf16"},
        # four beams of one user
        {"name": "fork B1 W4 O4", "op": "fork", "B": 1, "W": 4, "O": 4, "L": 512, "Hkv": 2, "D": 64, "page": 16, "dtype": "bf16"},
        # a batch of wide beams over shared prompts
        {"name": "fork B32 W8 O16", "op": "fork", "B": 32, "W": 8, "O": 16, "L": 4096, "Hkv": 4, "D": 128, "page": 16, "dtype": "bf16"},
        # a few rows that grew by a tree
        {"name": "resize R4 M64", "op": "resize", "R": 4, "M": 64, "page": 16, "spare": 1.5},
        # a serving batch of long contexts over a large pool, requests ending and beginning
        {"name": "resize R512 M1024", "op": "resize", "R": 512, "M": 1024, "page": 16, "spare": 1.2},
    ]


def draw(rng):
    def logu(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["attend", "attend", "attend", "attend", "accept", "compact", "fork", "resize"])
    if op == "accept":
        return {"op": op, "B": logu(1, 256), "N": logu(1, 128)}
    if op == "resize":
        M = logu(16, 1024)
        return {"op": op, "R": logu(1, 512), "M": M, "page": rng.choice([8, 16, 32]), "spare": rng.choice([1.05, 1.2, 1.5])}
    c = {"op": op, "Hkv": rng.randint(1, 8), "D": rng.choice([64, 128, 128, 80, 40]), "page": rng.choice([16, 16, 32, 64, 128]),
         "dtype": rng.choice(["bf16", "bf16", "f16"])}
    if op == "attend":
        c |= {"N": rng.choice([1, logu(1, 64), logu(1, 64)]), "G": rng.randint(1, 8), "L": logu(16, 32768)}
        page = 2 * 2 * c["Hkv"] * c["D"] * c["L"]
        rows = c["N"] * c["G"] * c["Hkv"]
        # no more bytes, and no more arithmetic, than the listed ones
        c["B"] = max(1, min(logu(1, 64), int(1.3e9 // page), int(8 * 32768 * 64 * 64 * 128 // (c["L"] * rows * c["D"]))))
        return c
    c["O"] = rng.randint(1, 32)
    c["L"] = logu(16, 1024)
    unit = 2 * c["O"] * c["Hkv"] * c["D"]
    if op == "compact":
        c["N"] = logu(2, 64)
        c["B"] = max(1, min(logu(1, 64), int(2e9 // (unit * (c["L"] + c["N"] + c["page"])))))
    else:
        c["W"] = rng.randint(2, 16)
        c["B"] = max(1, min(logu(1, 32), int(2e9 // (unit * (2 * c["L"] + 4 * c["W"] * c["page"])))))
    return c


# ---- inputs -----------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _lengths(g, B, L):
    """Lengths from a quarter of L up to L, always of the same sum."""
    at = torch.randperm(B, generator=g, device=DEV)
    return (L * (0.25 + 0.75 * (at + 1).double() / B)).long().clamp(min=1).to(torch.int32)


def _mean_length(B, L):
    return L * (0.25 + 0.375 * (B + 1) / B)


def _tree(g, B, N):
    """Parents of trees of drafts, node 0 the last token: often the node before, else any earlier one."""
    n = torch.arange(N, device=DEV)
    far = (torch.rand((B, N), generator=g, device=DEV) * n).long()
    par = torch.where(torch.rand((B, N), generator=g, device=DEV) < 0.4, (n - 1).expand(B, N), far)
    return torch.where(n == 0, -1, torch.minimum(par, (n - 1).expand(B, N))).to(torch.int32)


def _cache(g, shape, dt):
    out = torch.empty(shape, dtype=dt, device=DEV)
    for i in range(shape[0]):
        out[i] = torch.randn(shape[1:], generator=g, device=DEV, dtype=dt)
    return out


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "accept":
        B, N = case["B"], case["N"]
        parents = _tree(g, B, N)
        # a small alphabet, so that drafts repeat among siblings and are often right
        tokens = torch.randint(0, 5, (B, N), generator=g, device=DEV).to(torch.int32)
        choice = torch.randint(0, 5, (B, N), generator=g, device=DEV).to(torch.int32)
        return {"case": case, "tokens": tokens, "parents": parents, "choice": choice}
    if op == "resize":
        R, M, page = case["R"], case["M"], case["page"]
        had = torch.randint(0, M + 1, (R,), generator=g, device=DEV)
        P = int(case["spare"] * R * M / 2) + M + 8
        m = torch.arange(M, device=DEV)
        held = m < had[:, None]
        pages = torch.randperm(max(P, R * M), generator=g, device=DEV)[:R * M].view(R, M) % P
        table = torch.where(held, pages, -1).to(torch.int32)
        refs = torch.zeros(P, dtype=torch.int32, device=DEV)
        refs.scatter_add_(0, pages.flatten(), held.flatten().to(torch.int32))
        # most rows grow by up to a tree's pages, some end, some were just admitted
        grow = (had * page + torch.randint(-page, 5 * page, (R,), generator=g, device=DEV)).clamp(min=0, max=M * page)
        r = torch.rand((R,), generator=g, device=DEV)
        fresh = torch.randint(0, M * page // 2 + 1, (R,), generator=g, device=DEV)
        lengths = torch.where(r < 0.1, 0, torch.where(r > 0.9, fresh, grow)).to(torch.int32)
        return {"case": case, "table": table, "refs": refs, "lengths": lengths, "page": page}
    B, L, page, dt = case["B"], case["L"], case["page"], DT[case["dtype"]]
    Hkv, D = case["Hkv"], case["D"]
    if op == "fork":
        W, O = case["W"], case["O"]
        M = -(-L // page) + 1
        length = _lengths(g, B, L).long()
        last = (length - 1) // page                          # the last page that holds a token
        own_from = (last - torch.randint(0, 3, (B,), generator=g, device=DEV)).clamp(min=0)
        m = torch.arange(M, device=DEV)
        shared = (m < own_from[:, None])[:, None].expand(B, W, M)
        mine = ((m >= own_from[:, None]) & (m <= last[:, None] + 1))[:, None].expand(B, W, M)   # one page ahead
        first = shared & (torch.arange(W, device=DEV) == 0)[:, None]
        need = (first | mine)
        number = torch.cumsum(need.flatten().long(), 0).view(B, W, M) - 1
        number = torch.where(shared, number[:, :1], number)
        P = B * (M + 4 * W) + 8
        order = torch.randperm(P, generator=g, device=DEV)
        table = torch.where(shared | mine, order[number.clamp(min=0)], -1).to(torch.int32)
        refs = torch.zeros(P, dtype=torch.int32, device=DEV)
        refs.scatter_add_(0, table.clamp(min=0).flatten().long(), (table >= 0).flatten().to(torch.int32))
        r = torch.rand((B, W), generator=g, device=DEV)
        parent = torch.randint(0, W, (B, W), generator=g, device=DEV)
        parent = torch.where(r < 0.3, torch.arange(W, device=DEV)[None], parent)
        parent = torch.where(r > 0.97, -1, parent).to(torch.int32)
        return {"case": case, "cache": _cache(g, (O, P, page, Hkv, D), dt), "table": table, "refs": refs, "parent": parent,
                "lengths": length[:, None].expand(B, W).to(torch.int32).contiguous()}
    N = case["N"]
    M = -(-(L + N) // page)
    P = B * M + 3
    table = torch.randperm(P, generator=g, device=DEV)[:B * M].view(B, M).to(torch.int32)
    lengths = _lengths(g, B, L)
    if op == "compact":
        keep = torch.rand((B, N), generator=g, device=DEV) < 0.25
        keep[:, 0] = True
        n = torch.arange(N, device=DEV).expand(B, N)
        path = torch.sort(torch.where(keep, n, N), dim=1).values
        path = torch.where(path == N, -1, path).to(torch.int32)
        return {"case": case, "cache": _cache(g, (case["O"], P, page, Hkv, D), dt), "table": table, "lengths": lengths, "path": path}
    G = case["G"]
    k, v = _cache(g, (P, page, Hkv, D), dt), _cache(g, (P, page, Hkv, D), dt)
    v += 0.25                                                # values have a mean
    q = (2.0 * torch.randn((B, N, Hkv * G, D), generator=g, device=DEV)).to(dt)
    return {"case": case, "q": q, "k": k, "v": v, "table": table, "lengths": lengths, "parents": _tree(g, B, N), "scale": D ** -0.5}


# ---- the plain forms --------------------------------------------------------------------------

def _lineage(parents):
    """[B, N, N]: whether node j is node n or one of its ancestors."""
    B, N = parents.shape
    n = torch.arange(N, device=parents.device)
    step = (parents.long()[..., None] == n).float() + torch.eye(N, device=parents.device)   # its powers hold binomials: at most 2^127
    return torch.linalg.matrix_power(step, max(N - 1, 1)) > 0


def _plain_attend(q, k, v, table, lengths, parents, scale):
    B, N, H, D = q.shape
    Hkv, T = k.shape[2], table.shape[1] * k.shape[1]
    at = table.clamp(min=0).long()
    keys = k[at].view(B, T, Hkv, D).float().permute(0, 2, 3, 1)
    node = torch.arange(T, device=q.device) - lengths.long()[:, None]                       # [B, T]
    seen = torch.gather(_lineage(parents), 2, node.clamp(0, N - 1)[:, None].expand(B, N, T))
    seen = (node < 0)[:, None] | (seen & (node < N)[:, None])                               # [B, N, T]
    rows = q.float().view(B, N, Hkv, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    s = ((rows @ keys) * scale).view(B, Hkv, N, H // Hkv, T)
    s = s.masked_fill_(~seen[:, None, :, None], -INF)
    mx = s.amax(-1, keepdim=True)
    s = s.sub_(mx).exp_()
    total = s.sum(-1, keepdim=True)
    vals = torch.where((node < N)[..., None, None], v[at].view(B, T, Hkv, D).float(), 0.0).permute(0, 2, 1, 3)
    out = (s.view(B, Hkv, -1, T) @ vals).view(B, Hkv, N, H // Hkv, D) / total
    lse = (mx + torch.log(total))[..., 0]
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(B, N, H, D).to(q.dtype), "lse": lse.permute(0, 2, 1, 3).reshape(B, N, H)}


def _plain_accept(tokens, parents, choice):
    B, N = tokens.shape
    n = torch.arange(N, device=tokens.device)
    right = tokens == torch.gather(choice, 1, parents.clamp(min=0).long())
    twin = (parents[:, None] == parents[..., None]) & (tokens[:, None] == tokens[..., None]) & (n[None] < n[:, None])
    good = (right & ~twin.any(-1) & (parents >= 0)) | (n == 0)
    on = (good[:, None] | ~_lineage(parents)).all(-1)
    path = torch.sort(torch.where(on, n, N), dim=1).values
    said = torch.where(path < N, torch.gather(choice, 1, path.clamp(max=N - 1)), -1)
    return {"accepted_len": (on.sum(1) - 1).to(torch.int32), "out_tokens": said, "path": torch.where(path < N, path, -1).to(torch.int32)}


def _plain_compact(cache, table, lengths, path):
    O, P, page, H, D = cache.shape
    B, N = path.shape
    i = torch.arange(N, device=path.device)
    here = lengths.long()[:, None]

    def place(at):   # of tokens `at` [B, N] of the rows, among all slots of the pool
        return torch.gather(table.long(), 1, (at // page).clamp(max=table.shape[1] - 1)) * page + at % page

    kept = path >= 0
    src = place(here + path.clamp(min=0).long())
    # entries that are not kept rewrite a kept one's place with its own value
    dst, src = torch.where(kept, place(here + i), place(here)), torch.where(kept, src, src[:, :1])
    flat = cache.view(O, P * page, H, D)
    flat[:, dst.flatten()] = flat[:, src.flatten()]
    return {"lengths": lengths + kept.sum(1).to(torch.int32), "cache": cache}


def _counted(refs, pages, on, by):
    return refs.scatter_add(0, pages.clamp(min=0).flatten().long(), by * on.flatten().to(torch.int32))


def _given(refs, want):
    """Free pages, lowest first, for the places in `want`, in order; -1 where there are none left."""
    rank = torch.cumsum(want.flatten().long(), 0).view(want.shape) - 1
    free = torch.argsort((refs != 0).to(torch.int32), stable=True)
    got = torch.where(rank < (refs == 0).sum(), free[rank.clamp(0, refs.numel() - 1)], -1)
    return torch.where(want, got, -1).to(torch.int32)


def _plain_fork(cache, table, refs, lengths, parent):
    O, P, page, H, D = cache.shape
    B, W, M = table.shape
    N = parent.shape[1]
    src = torch.where(parent < 0, torch.arange(N, device=table.device), parent.long())
    lens = torch.gather(lengths, 1, src)
    old = torch.gather(table, 1, src[..., None].expand(B, N, M))
    full = (lens // page).long()
    new = torch.where(torch.arange(M, device=table.device) < full[..., None], old, -1)
    base = _counted(_counted(refs, table, table >= 0, -1), new, new >= 0, 1)
    # the page that holds a row's last tokens is kept by the first row that wants it, if nothing else names it
    at = full.clamp(max=M - 1)[..., None]
    last = torch.where(lens % page > 0, torch.gather(old, 2, at)[..., 0], -1)
    row = torch.arange(B * N, device=table.device)
    where = last.clamp(min=0).flatten().long()
    first = torch.full((P,), B * N, device=table.device).scatter_reduce(0, where, torch.where(last.flatten() >= 0, row, B * N), "amin")
    keeps = ((last >= 0).flatten() & (first[where] == row) & (base[where] == 0)).view(B, N)
    copies = (last >= 0) & ~keeps
    base = _counted(base, last, keeps, 1)
    page_to = _given(base, copies)
    out = torch.where(keeps, last, page_to)
    new = new.scatter(2, at, torch.where((last >= 0)[..., None], out[..., None], torch.gather(new, 2, at)))
    # rows without a copy rewrite one that has, or else a page's own bytes
    done = page_to >= 0
    some = torch.argmax(done.flatten().to(torch.int32))
    any_ = done.any()
    to = torch.where(done.flatten(), page_to.flatten(), torch.where(any_, page_to.flatten()[some], 0)).long()
    of = torch.where(done.flatten(), last.flatten(), torch.where(any_, last.flatten()[some], 0)).long()
    valid = torch.where(done.flatten(), (lens % page).flatten(), torch.where(any_, (lens % page).flatten()[some], 0))
    live = (torch.arange(page, device=table.device) < valid[:, None])[None, :, :, None, None]
    cache[:, to] = torch.where(live, cache[:, of], cache[:, to])
    return {"table": new, "refs": _counted(base, page_to, done, 1), "lengths": lens, "cache": cache}


def _plain_resize(table, refs, lengths, page):
    need = (lengths.long() + page - 1) // page
    inside = torch.arange(table.shape[1], device=table.device) < need[:, None]
    refs = _counted(refs, table, (table >= 0) & ~inside, -1)
    fresh = _given(refs, inside & (table < 0))
    out = torch.where(inside, torch.where(table < 0, fresh, table), -1)
    return {"table": out, "refs": _counted(refs, fresh, fresh >= 0, 1)}


def run(state):
    op = state["case"]["op"]
    if own:
        import speculative_decoding_token_verify_gb300 as sv

        if op == "attend":
            return sv.tree_attention(state["q"], state["k"], state["v"], state["table"], state["lengths"],
                                     parents=state["parents"], scale=state["scale"])
        if op == "accept":
            return sv.tree_accept(state["tokens"], state["parents"], state["choice"])
        if op == "compact":
            lengths = sv.pages_compact(state["cache"], state["table"], state["lengths"], state["path"], page_dim=1)
            return {"lengths": lengths, "cache": state["cache"]}
        if op == "fork":
            r = sv.pages_fork(state["cache"], state["table"], state["refs"], state["lengths"], state["parent"], page_dim=1)
            return {"table": r["table"], "refs": r["refs"], "lengths": r["lengths"], "cache": state["cache"]}
        r = sv.pages_resize(state["table"], state["refs"], state["lengths"], state["page"])
        return {"table": r["table"], "refs": r["refs"]}
    if op == "attend":
        return _plain_attend(*(state[x] for x in ("q", "k", "v", "table", "lengths", "parents", "scale")))
    if op == "accept":
        return _plain_accept(state["tokens"], state["parents"], state["choice"])
    if op == "compact":
        return _plain_compact(state["cache"], state["table"], state["lengths"], state["path"])
    if op == "fork":
        return _plain_fork(state["cache"], state["table"], state["refs"], state["lengths"], state["parent"])
    return _plain_resize(state["table"], state["refs"], state["lengths"], state["page"])


# ---- work -------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "accept":
        return {"bytes": 4 * case["B"] * (5 * case["N"] + 1), "flops": 0}
    if op == "resize":
        pool = int(case["spare"] * case["R"] * case["M"] / 2) + case["M"] + 8
        return {"bytes": 8 * (case["R"] * case["M"] + pool) + 4 * case["R"], "flops": 0}
    B, L, Hkv, D, page = (case[x] for x in ("B", "L", "Hkv", "D", "page"))
    unit = 2 * Hkv * D
    if op == "compact":
        # a quarter of the nodes behind the first are kept, and nearly all of those move
        moved = B * 0.25 * (case["N"] - 1)
        return {"bytes": 2 * moved * unit * case["O"] + 4 * B * (case["N"] + 2), "flops": 0}
    if op == "fork":
        W, M = case["W"], -(-L // page) + 1
        # beams that are no one's first: of W beams about 0.7 W / e + ... = 0.35 W, each half a page
        copied = 0.35 * B * W * page / 2 * (page - 1) / page
        return {"bytes": 2 * copied * unit * case["O"] + 8 * (B * W * M + B * (M + 4 * W)) + 12 * B * W, "flops": 0}
    N, H = case["N"], Hkv * case["G"]
    keys = B * (_mean_length(B, L) + N)
    return {"bytes": 2 * keys * unit + 2 * 2 * B * N * H * D + 4 * B * N * (H + 1), "flops": 4 * keys * N * H * D}


# ---- exact values, row after row --------------------------------------------------------------

def _exact_attend(st):
    q, k, v = st["q"], st["k"], st["v"]
    B, N, H, D = q.shape
    page, Hkv = k.shape[1:3]
    out = torch.zeros((B, N, H, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, N, H), dtype=torch.float64, device=DEV)
    parents, lengths, table = st["parents"].tolist(), st["lengths"].tolist(), st["table"].tolist()
    for b in range(B):
        L = lengths[b]
        T = L + N
        pages = table[b][:(T + page - 1) // page]
        kb = torch.cat([k[p] for p in pages])[:T].double()
        vb = torch.cat([v[p] for p in pages])[:T].double()
        bias = torch.full((N, T), -INF, dtype=torch.float64)
        bias[:, :L] = 0
        for n in range(N):
            j = n
            while j >= 0:
                bias[n, L + j] = 0
                j = parents[b][j]
        bias = bias.to(DEV)
        for h in range(H):
            s = st["scale"] * (q[b, :, h].double() @ kb[:, h * Hkv // H].T) + bias
            lse[b, :, h] = torch.logsumexp(s, 1)
            out[b, :, h] = torch.softmax(s, 1) @ vb[:, h * Hkv // H]
    return {"out": out, "lse": lse}


def _exact_accept(st):
    tokens, parents, choice = (st[x].tolist() for x in ("tokens", "parents", "choice"))
    N = len(tokens[0])
    got = {"accepted_len": [], "out_tokens": [], "path": []}
    for tok, par, cho in zip(tokens, parents, choice):
        path = [0]
        while True:
            after = [c for c in range(path[-1] + 1, N) if par[c] == path[-1] and tok[c] == cho[path[-1]]]
            if not after:
                break
            path.append(after[0])
        got["accepted_len"].append(len(path) - 1)
        got["out_tokens"].append([cho[n] for n in path] + [-1] * (N - len(path)))
        got["path"].append(path + [-1] * (N - len(path)))
    return {x: torch.tensor(y, dtype=torch.int32) for x, y in got.items()}


def _exact_fork(st, page):
    table, lengths, parent, refs = (st[x].tolist() for x in ("table", "lengths", "parent", "refs"))
    M = len(table[0][0])
    for beams in table:
        for row in beams:
            for p in row:
                refs[p] -= p >= 0
    new, lens, wants = [], [], {}
    for b, order in enumerate(parent):
        for n, w in enumerate(order):
            w = n if w < 0 else w
            whole, part = divmod(lengths[b][w], page)
            new.append(table[b][w][:whole] + [-1] * (M - whole))
            lens.append(lengths[b][w])
            for p in new[-1]:
                refs[p] += p >= 0
            if part:
                wants.setdefault(table[b][w][whole], []).append((len(new) - 1, whole))
    late = []
    for p, who in wants.items():
        if refs[p] == 0:
            r, m = who.pop(0)
            new[r][m] = p
            refs[p] = 1
        late += who
    free = (p for p, c in enumerate(list(refs)) if c == 0)
    for r, m in sorted(late):
        new[r][m] = next(free, -1)
        if new[r][m] >= 0:
            refs[new[r][m]] = 1
    B, N = len(parent), len(parent[0])
    i32 = torch.int32
    return {"table": torch.tensor(new, dtype=i32).view(B, N, M), "refs": torch.tensor(refs, dtype=i32),
            "lengths": torch.tensor(lens, dtype=i32).view(B, N), "cache": None}


def _exact_resize(st):
    table, refs, lengths, page = st["table"].tolist(), st["refs"].tolist(), st["lengths"].tolist(), st["page"]
    need = [-(-n // page) for n in lengths]
    for row, n in zip(table, need):
        for m in range(n, len(row)):
            if row[m] >= 0:
                refs[row[m]] -= 1
                row[m] = -1
    free = (p for p, c in enumerate(list(refs)) if c == 0)
    for row, n in zip(table, need):
        for m in range(n):
            if row[m] < 0:
                row[m] = next(free, -1)
                if row[m] >= 0:
                    refs[row[m]] += 1
    return {"table": torch.tensor(table, dtype=torch.int32), "refs": torch.tensor(refs, dtype=torch.int32)}


def exact(case, seed):
    if case["op"] == "compact":
        return None  # values are moved, not computed
    st = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(st)
    if case["op"] == "accept":
        return _exact_accept(st)
    return _exact_fork(st, case["page"]) if case["op"] == "fork" else _exact_resize(st)
