"""Plain 64-bit forms of the tree operators, for the tests: one row after another,
in numpy and Python lists."""
import numpy as np
import torch

NEG = float("-inf")


def lineage(parents, n):
    """Nodes n, parents[n], .. up to a root."""
    seen = []
    while n >= 0:
        seen.append(n)
        n = parents[n]
    return seen


def attention(q, k, v, table, lengths, parents, counts, scale):
    """out, lse and the errors that rounding allows (see bounds()). q [B,N,Hq,D], k and v
    [P,page,Hkv,D] in any dtype, parents a list per sequence."""
    B, N, Hq, D = q.shape
    page, Hkv = k.shape[1], k.shape[2]
    u = torch.finfo(q.dtype).eps / 2
    q, dt = q.double().cpu().numpy(), q.dtype
    out = np.zeros((B, N, Hq, D))
    lse = np.full((B, N, Hq), NEG)
    e_out, e_lse = np.zeros_like(out), np.zeros_like(lse)
    for b in range(B):
        L, count = int(lengths[b]), int(counts[b])
        pages = [int(table[b][t // page]) for t in range(L + count)]
        slots = [t % page for t in range(L + count)]
        kb = k[pages, slots].double().cpu().numpy()      # [T, Hkv, D]
        vb = v[pages, slots].double().cpu().numpy()
        for n in range(count):
            see = list(range(L)) + [L + j for j in lineage(parents[b], n)]
            for h in range(Hq):
                kk, vv = kb[see, h * Hkv // Hq], vb[see, h * Hkv // Hq]
                with np.errstate(all="ignore"):
                    s = scale * (kk @ q[b, n, h])
                    m = s.max()
                    w = np.exp(s - m)
                    p = w / w.sum()
                    out[b, n, h] = p @ vv
                    lse[b, n, h] = m + np.log(w.sum())
                    # a score: D products that are exact in fp32, added with at most 2^-22 of
                    # their magnitude lost an addition (tensor cores cut, they do not round)
                    ds = abs(scale) * (np.abs(kk) @ np.abs(q[b, n, h])).max() * (D + 8) * 2.0 ** -23
                    mean = p @ np.abs(vv)
                    # the output's rounding, each probability's, the scores' and 2^x's (2^-21),
                    # and fp32 sums over the keys
                    rel = u + 2 * ds + 2.0 ** -21 + (64 + len(see) / 16) * 2.0 ** -23
                    e_out[b, n, h] = u * np.abs(out[b, n, h]) + rel * mean * (1 + u) + (2.0 ** -24 if dt == torch.float16 else 0)
                    e_lse[b, n, h] = ds + 2.0 ** -21 + (64 + len(see) / 16) * 2.0 ** -24 + 2.0 ** -22 * abs(lse[b, n, h])
    return out, lse, e_out, e_lse


def accept(tokens, parents, choice, counts):
    B, N = len(tokens), len(tokens[0])
    acc, out, paths = [], [], []
    for b in range(B):
        path = [0] if counts[b] else []
        while path:
            after = [c for c in range(path[-1] + 1, counts[b])
                     if parents[b][c] == path[-1] and tokens[b][c] == choice[b][path[-1]]]
            if not after:
                break
            path.append(after[0])
        acc.append(max(len(path) - 1, 0))
        out.append([choice[b][n] for n in path] + [-1] * (N - len(path)))
        paths.append(path + [-1] * (N - len(path)))
    return acc, out, paths


def resize(table, refs, lengths, page):
    """table [R][M], refs [P], lengths [R] lists; new lists and whether pages ran out."""
    table, refs = [list(r) for r in table], list(refs)
    P = len(refs)
    table = [[e if 0 <= e < P else -1 for e in r] for r in table]
    need = [-(-min(max(n, 0), len(r) * page) // page) for n, r in zip(lengths, table)]
    for row, n in zip(table, need):
        for m in range(n, len(row)):
            if row[m] >= 0:
                refs[row[m]] -= 1
                row[m] = -1
    free = iter([p for p in range(P) if refs[p] == 0])
    short = False
    for row, n in zip(table, need):
        for m in range(n):
            if row[m] < 0:
                row[m] = next(free, -1)
                if row[m] >= 0:
                    refs[row[m]] = 1
                else:
                    short = True
    return table, refs, short


def fork(table, refs, lengths, parent, page):
    """table [B][W][M], lengths [B][W], parent [B][N]: new table, refs, lengths, copies {(b, n): (from, to, slots)}."""
    refs, P = list(refs), len(refs)
    table = [[[e if 0 <= e < P else -1 for e in r] for r in beams] for beams in table]
    W, M = len(table[0]), len(table[0][0])
    for beams in table:
        for row in beams:
            for e in row:
                if e >= 0:
                    refs[e] -= 1
    new, lens, want = [], [], []
    for b, order in enumerate(parent):
        new.append([])
        lens.append([])
        for n, w in enumerate(order):
            if not 0 <= w < W:
                w = n if n < W else None
            row, L = (table[b][w], min(max(lengths[b][w], 0), M * page)) if w is not None else ([-1] * M, 0)
            full, part = divmod(L, page)
            row = [row[m] if m < full or m == full and part else -1 for m in range(M)]
            if part and row[full] >= 0:
                want.append((b, n, full, row[full], part))
                row[full] = -1
            for e in row:
                if e >= 0:
                    refs[e] += 1
            new[-1].append(row)
            lens[-1].append(L)
    base, seen, copies, late = list(refs), set(), {}, []
    for b, n, m, e, part in want:
        if base[e] == 0 and e not in seen:
            new[b][n][m] = e
            refs[e] = 1
        else:
            late.append((b, n, m, e, part))
        seen.add(e)
    free = iter([p for p in range(P) if refs[p] == 0])
    for b, n, m, e, part in late:
        to = next(free, -1)
        new[b][n][m] = to
        if to >= 0:
            refs[to] = 1
            copies[b, n] = (e, to, part)
    return new, refs, lens, copies
