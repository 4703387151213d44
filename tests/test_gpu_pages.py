"""Pages resized, forked and compacted, and the walk down a tree, against plain
lists; and one decoding step of all tree operators together."""
import pytest

torch = pytest.importorskip("torch")

import tree_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _sv():
    import speculative_decoding_token_verify_gb300 as sv
    sv.build()
    return sv


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---- accept -------------------------------------------------------------------------------


def _tree(g, N, far=0.5):
    return [-1] + [int(torch.randint(0, n, (1,), generator=g)) if torch.rand(1, generator=g) < far else n - 1 for n in range(1, N)]


@pytest.mark.parametrize("B,N,words", [(1, 1, 2), (1, 9, 2), (3, 32, 2), (5, 33, 3), (40, 64, 1), (7, 127, 2), (129, 128, 4), (2, 128, 1)])
def test_accept(B, N, words):
    sv = _sv()
    g = torch.Generator().manual_seed(N)
    parents = [_tree(g, N, 0.2 if words == 1 else 0.7) for _ in range(B)]
    tokens = torch.randint(0, words, (B, N), generator=g).tolist()
    choice = torch.randint(0, words, (B, N), generator=g).tolist()
    counts = torch.randint(0, N + 1, (B,), generator=g).tolist()
    for cnt in (None, counts):
        st = _i32([0])
        r = sv.tree_accept(_i32(tokens), _i32(parents), _i32(choice), counts=None if cnt is None else _i32(cnt), status=st)
        want = ref.accept(tokens, parents, choice, cnt or [N] * B)
        assert r["accepted_len"].tolist() == want[0] and r["out_tokens"].tolist() == want[1] and r["path"].tolist() == want[2]
        assert int(st) == 0
    # a chain, one tree for all, choices with strides
    chain = [[n - 1 for n in range(N)]] * B
    want = ref.accept(tokens, chain, choice, [N] * B)
    wide = torch.full((B, N, 3), -9, dtype=torch.int32, device=DEV)
    wide[..., 0] = _i32(choice)
    for par in (None, _i32(chain[0])):
        r = sv.tree_accept(_i32(tokens), par, wide[..., 0])
        assert r["path"].tolist() == want[2] and r["out_tokens"].tolist() == want[1]
    one = torch.full((1, 1), 0, dtype=torch.int32, device=DEV).expand(B, N)
    want = ref.accept(tokens, chain, [[0] * N] * B, [N] * B)
    assert sv.tree_accept(_i32(tokens), None, one)["path"].tolist() == want[2]


def test_accept_bad_values():
    sv = _sv()
    tokens, choice = [[0, 0, 0, 0]], [[0, 0, 0, 0]]
    for par, cnt, code in (([-1, 0, 2, 1], 4, 9), ([-1, 0, 3, 1], 4, 9), ([-1, 0, -5, 1], 4, 9), ([0, 0, 1, 2], 4, 9),
                           ([-1, 0, 1, 2], 9, 11), ([-1, 0, 1, 2], -1, 11), ([-1, 0, 1 << 30, 1], 4, 9)):
        st = _i32([0])
        r = sv.tree_accept(_i32(tokens), _i32([par]), _i32(choice), counts=_i32([cnt]), status=st)
        fixed = [p if -1 <= p < n else -1 for n, p in enumerate(par)]
        want = ref.accept(tokens, [fixed], choice, [min(max(cnt, 0), 4)])
        assert int(st) == code and r["path"].tolist() == want[2] and r["accepted_len"].tolist() == want[0]


def test_accept_out_and_empty():
    sv = _sv()
    out = {"path": torch.full((2, 5), 7, dtype=torch.int32, device=DEV)}
    r = sv.tree_accept(_i32([[0] * 5] * 2), None, _i32([[1] * 5] * 2), out=out)
    assert r["path"] is out["path"] and r["path"].tolist() == [[0, -1, -1, -1, -1]] * 2
    r = sv.tree_accept(torch.empty((0, 5), dtype=torch.int32, device=DEV), None, torch.empty((0, 5), dtype=torch.int32, device=DEV))
    assert r["path"].shape == (0, 5)


# ---- resize -------------------------------------------------------------------------------


def _pool(g, R, M, P, full=0.5, shared=True):
    """A table whose rows hold some pages (shared ones among them), and its counts."""
    had = (torch.rand(R, generator=g) * (M + 1) * 2 * full).long().clamp(max=M)
    if shared:
        pages = torch.randint(0, P, (R, M), generator=g)
    else:
        pages = torch.randperm(P, generator=g)[:R * M].view(R, M)
    table = torch.where(torch.arange(M) < had[:, None], pages, -1)
    refs = torch.bincount(table[table >= 0], minlength=P)
    return table.tolist(), refs.tolist(), had


@pytest.mark.parametrize("R,M,P,page", [(1, 1, 1, 16), (1, 1, 4, 1), (3, 5, 40, 16), (4, 64, 300, 16), (33, 31, 700, 8), (100, 1, 90, 16),
                                        (7, 1000, 5000, 16), (200, 100, 30000, 32), (2000, 3, 5000, 16), (64, 512, 66000, 16)])
@pytest.mark.parametrize("seed", [0, 1])
def test_resize(R, M, P, page, seed):
    sv = _sv()
    g = torch.Generator().manual_seed(seed)
    table, refs, had = _pool(g, R, M, P)
    grow = had * page + torch.randint(-3 * page, 3 * page + 1, (R,), generator=g)
    lengths = torch.where(torch.rand(R, generator=g) < 0.2, 0, grow).clamp(min=0, max=M * page).tolist()
    want = ref.resize(table, refs, lengths, page)
    st = _i32([0])
    t, f = _i32(table), _i32(refs)
    r = sv.pages_resize(t, f, _i32(lengths), page, status=st)
    assert r["table"].tolist() == want[0] and r["refs"].tolist() == want[1]
    assert int(st) == (12 if want[2] else 0)
    assert t.tolist() == table and f.tolist() == refs
    r = sv.pages_resize(t, f, _i32(lengths), page, out={"table": t, "refs": f})      # in place
    assert r["table"] is t and t.tolist() == want[0] and f.tolist() == want[1]
    sv.pages_resize(t, f, _i32(lengths), page, out={"table": t, "refs": f})          # nothing left to do
    again = ref.resize(want[0], want[1], lengths, page)
    assert t.tolist() == again[0] and f.tolist() == again[1]
    r = sv.pages_resize(t, f, _i32([0] * R), page)                                   # all given back
    assert (r["table"] == -1).all() and r["refs"].sum() == 0


def test_resize_bad_values_and_exhaustion():
    sv = _sv()
    for table, refs, lengths, code in (
            ([[0, 9, -1]], [1, 0, 0, 0], [48], 10), ([[0, -2, -1]], [1, 0, 0, 0], [32], 10), ([[0, 1 << 30, -1]], [1, 0, 0, 0], [16], 10),
            ([[0, -1, -1]], [1, 0, 0, 0], [49], 11), ([[0, -1, -1]], [1, 0, 0, 0], [-5], 11), ([[0, -1, -1]], [1, 0, 0, 0], [(1 << 31) - 1], 11),
            ([[-1, -1, -1], [-1, -1, -1]], [0, 1, 0, 0], [40, 40], 12), ([[-1, -1]], [1], [32], 12)):
        st = _i32([0])
        r = sv.pages_resize(_i32(table), _i32(refs), _i32(lengths), 16, status=st)
        want = ref.resize(table, refs, lengths, 16)
        assert r["table"].tolist() == want[0] and r["refs"].tolist() == want[1] and int(st) == code


def test_resize_shapes():
    sv = _sv()
    r = sv.pages_resize(_i32([[[0, -1], [-1, -1]]]), _i32([1, 0, 0]), _i32([[20, 3]]), 16)    # [B, W, M]
    assert r["table"].tolist() == [[[0, 1], [2, -1]]] and r["refs"].tolist() == [1, 1, 1]
    r = sv.pages_resize(torch.empty((0, 4), dtype=torch.int32, device=DEV), _i32([0, 1]), torch.empty(0, dtype=torch.int32, device=DEV), 16)
    assert r["refs"].tolist() == [0, 1]
    st = _i32([0])
    r = sv.pages_resize(_i32([[-1]]), torch.empty(0, dtype=torch.int32, device=DEV), _i32([4]), 16, status=st)
    assert r["table"].tolist() == [[-1]] and int(st) == 12


# ---- fork ---------------------------------------------------------------------------------


def _beams(g, B, W, M, page, P=None, shared=2):
    """Beams that share full pages, with a private page at the end and one ahead."""
    lengths = [[int(torch.randint(0, M * page + 1, (1,), generator=g))] * W for _ in range(B)]
    P = P or B * (M + W * (shared + 3)) + 2 * B * W
    order = iter(torch.randperm(P, generator=g).tolist())
    table, refs = [], [0] * P
    for b in range(B):
        full = lengths[b][0] // page
        common = [next(order) for _ in range(max(full - shared, 0))]
        rows = []
        for _ in range(W):
            row = list(common)
            while len(row) < min(M, full + 2):
                row.append(next(order))
            rows.append(row + [-1] * (M - len(row)))
            for e in row:
                refs[e] += 1
        table.append(rows)
    return table, refs, lengths, P


LAYOUTS = {
    "slots before heads": (lambda P, page: (3, P, page, 2, 24), 1, None),
    "heads before slots": (lambda P, page: (2, 2, P, 3, page, 8), 2, 4),
    "no outer axis": (lambda P, page: (P, page, 40), 0, None),
    "odd units": (lambda P, page: (2, P, 3, page, 5), 1, 3),
}


@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("B,W,N,M,page", [(1, 1, 1, 1, 16), (1, 4, 4, 6, 16), (3, 3, 3, 9, 8), (5, 1, 8, 4, 16), (2, 8, 3, 5, 32), (9, 16, 16, 40, 16)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8])
def test_fork(layout, B, W, N, M, page, dtype):
    sv = _sv()
    shape, pd, sd = LAYOUTS[layout]
    g = torch.Generator().manual_seed(B * W + N)
    table, refs, lengths, P = _beams(g, B, W, M, page)
    parent = torch.randint(0, W, (B, N), generator=g)
    parent[torch.rand((B, N), generator=g) < 0.2] = -1
    parent = parent.tolist()
    new, nrefs, lens, copies = ref.fork(table, refs, lengths, parent, page)
    cache = torch.randint(-100, 100, shape(P, page), generator=g).to(dtype).to(DEV)
    want = cache.clone()
    s = (sd if sd is not None else pd + 1)
    for src, to, slots in copies.values():
        want.select(pd, to).narrow(s - 1, 0, slots).copy_(cache.select(pd, src).narrow(s - 1, 0, slots))
    st = _i32([0])
    r = sv.pages_fork(cache, _i32(table), _i32(refs), _i32(lengths), _i32(parent), page_dim=pd, slot_dim=sd, status=st)
    assert int(st) == 0
    assert r["table"].tolist() == new and r["refs"].tolist() == nrefs and r["lengths"].tolist() == lens
    assert torch.equal(cache, want)
    # every reference is an entry
    t = r["table"].flatten().long()
    assert torch.equal(torch.bincount(t[t >= 0], minlength=P).int(), r["refs"])


def test_fork_of_shared_last_pages():
    """Pages that are not full but named by others are copied for all, and one page is kept by one row only."""
    sv = _sv()
    page = 16
    table, refs = [[[0, 1], [0, 1]], [[2, 1], [3, -1]]], [2, 4, 1, 1] + [0] * 8       # page 1: three rows and one more entry elsewhere
    lengths, parent = [[20, 20], [25, 16]], [[0, 1], [0, 1]]
    want = ref.fork(table, refs, lengths, parent, page)
    cache = torch.arange(12 * page, device=DEV).view(12, page, 1).to(torch.int32)
    keep = cache.clone()
    r = sv.pages_fork(cache, _i32(table), _i32(refs), _i32(lengths), _i32(parent))
    assert r["table"].tolist() == want[0] and r["refs"].tolist() == want[1]
    assert len(want[3]) == 3
    for src, to, slots in want[3].values():
        keep[to, :slots] = keep[src, :slots]
    assert torch.equal(cache, keep)


def test_fork_several_caches_and_refs_in_place():
    sv = _sv()
    g = torch.Generator().manual_seed(3)
    table, refs, lengths, P = _beams(g, 2, 4, 5, 16)
    parent = [[2, 2, 0, 2], [1, 1, 1, 0]]
    want = ref.fork(table, refs, lengths, parent, 16)
    caches = [torch.randn((P, 16, 2, 8), device=DEV) for _ in range(3)]
    kept = [c.clone() for c in caches]
    f = _i32(refs)
    v = [c._version for c in caches], f._version
    r = sv.pages_fork(caches, _i32(table), f, _i32(lengths), _i32(parent), out={"refs": f})
    assert r["refs"] is f and f.tolist() == want[1] and r["table"].tolist() == want[0]
    assert f._version > v[1] and all(c._version > o for c, o in zip(caches, v[0]))
    for c, k in zip(caches, kept):
        for src, to, slots in want[3].values():
            k[to, :slots] = k[src, :slots]
        assert torch.equal(c, k)


def test_fork_bad_values_and_exhaustion():
    sv = _sv()
    page, cache = 16, torch.zeros((6, 16, 4), device=DEV)
    good = dict(table=[[[0, 1], [2, 3]]], refs=[1, 1, 1, 1, 0, 0], lengths=[[20, 20]], parent=[[1, 1]])
    for change, code in (({}, 0), ({"parent": [[2, 1]]}, 9), ({"parent": [[-2, 1 << 30]]}, 9), ({"lengths": [[20, 99]]}, 11),
                         ({"lengths": [[-1, 20]], "parent": [[0, 1]]}, 11), ({"table": [[[0, 1], [9, 3]]]}, 10), ({"table": [[[0, 1], [2, -1]]]}, 10),
                         ({"refs": [1, 1, 1, 2, 5, 5]}, 0),                    # the dropped row's two pages are free again
                         ({"refs": [2, 2, 1, 2, 5, 5]}, 12), ({"refs": [2, 1, 1, 2, 5, 5]}, 12)):
        a = {**good, **change}
        st = _i32([0])
        r = sv.pages_fork(cache, _i32(a["table"]), _i32(a["refs"]), _i32(a["lengths"]), _i32(a["parent"]), status=st)
        want = ref.fork(a["table"], a["refs"], a["lengths"], a["parent"], page)
        assert int(st) == code, change
        assert r["table"].tolist() == want[0] and r["refs"].tolist() == want[1] and r["lengths"].tolist() == want[2]


def test_fork_large():
    sv = _sv()
    g = torch.Generator().manual_seed(8)
    table, refs, lengths, P = _beams(g, 32, 8, 260, 16)
    parent = torch.randint(-1, 8, (32, 8), generator=g).tolist()
    want = ref.fork(table, refs, lengths, parent, 16)
    cache = torch.randn((P, 16, 8), device=DEV)
    r = sv.pages_fork(cache, _i32(table), _i32(refs), _i32(lengths), _i32(parent))
    assert r["table"].tolist() == want[0] and r["refs"].tolist() == want[1]


# ---- compact --------------------------------------------------------------------------------


def _compacted(cache, pd, sd, table, lengths, path, page):
    want = cache.clone()
    for b, L in enumerate(lengths):
        for i, p in enumerate(path[b]):
            if p < 0:
                break
            src, to = L + p, L + i
            want.select(pd, table[b][to // page]).select(sd - 1, to % page).copy_(
                cache.select(pd, table[b][src // page]).select(sd - 1, src % page))
    return want


@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("N,page", [(1, 16), (2, 1), (9, 16), (33, 8), (64, 4), (128, 64), (128, 16)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.uint8])
def test_compact(layout, N, page, dtype):
    sv = _sv()
    shape, pd, sd = LAYOUTS[layout]
    g = torch.Generator().manual_seed(N)
    lengths = [0, 1, page, 3 * page - 1, 50, 77]
    B, M = len(lengths), -(-(77 + 3 * page + N) // page)
    P = B * M + 2
    table = torch.randperm(P, generator=g)[:B * M].view(B, M).tolist()
    path = []
    for b in range(B):
        p = [n for n in range(N) if torch.rand(1, generator=g) < (0.3, 0.9, 0.0, 1.0, 0.5, 0.1)[b]]
        path.append(p + [-1] * (N - len(p)))
    cache = torch.randint(0, 200, shape(P, page), generator=g).to(dtype).to(DEV)
    want = _compacted(cache, pd, sd if sd is not None else pd + 1, table, lengths, path, page)
    st = _i32([0])
    r = sv.pages_compact(cache, _i32(table), _i32(lengths), _i32(path), page_dim=pd, slot_dim=sd, status=st)
    assert int(st) == 0 and torch.equal(cache, want)
    assert r.tolist() == [L + sum(x >= 0 for x in p) for L, p in zip(lengths, path)]


def test_compact_bad_values():
    sv = _sv()
    for path, lengths, table, kept, code in (
            ([0, 2, 2, 3], 8, [0, 1], 2, 13), ([0, 3, 1, -1], 8, [0, 1], 2, 13), ([1, 9, -1, -1], 8, [0, 1], 1, 13), ([-3, 0, 1, 2], 8, [0, 1], 0, 13),
            ([0, 2, -1, 3], 8, [0, 1], 2, 0), ([0, 2, 3, -1], -2, [0, 1], 0, 11), ([0, 2, 3, -1], 33, [0, 1], 0, 11),
            ([0, 2, 3, -1], 13, [0, -1], 3, 10), ([0, 2, 3, -1], 13, [0, 5], 3, 10), ([1, 2, 3, -1], 30, [0, 1], 3, 10)):
        cache = torch.arange(48, device=DEV).to(torch.int32).view(3, 16, 1)
        flat = [None if not 0 <= p < 3 else p for p in table]
        want = cache.clone()
        for i in range(kept):
            a, z = lengths + path[i], lengths + i
            if a // 16 < 2 and z // 16 < 2 and flat[a // 16] is not None and flat[z // 16] is not None:
                want[flat[z // 16], z % 16] = cache[flat[a // 16], a % 16]
        st = _i32([0])
        r = sv.pages_compact(cache, _i32([table]), _i32([lengths]), _i32([path]), status=st)
        assert int(st) == code and torch.equal(cache, want) and r.tolist() == [lengths + kept]


def test_compact_several_far_and_out():
    """Caches that share a table; pages whose bytes lie past 2^32; lengths into a tensor of the caller's."""
    sv = _sv()
    P = (5 << 30) // (16 * 4096 * 2)
    big = torch.empty((P, 16, 4096), dtype=torch.bfloat16, device=DEV)
    small = torch.randn((P, 16, 3), device=DEV)
    big[P - 2:] = torch.randn((2, 16, 4096), device=DEV).bfloat16()
    table, lengths, path = [[P - 1, P - 2]], [10], [[0, 3, 4, 9, -1, -1, -1, -1, -1, -1]]
    want = [_compacted(c[P - 2:], 0, 1, [[1, 0]], lengths, path, 16) for c in (big, small)]
    out = _i32([0])
    assert sv.pages_compact([big, small], _i32(table), _i32(lengths), _i32(path), out=out) is out
    assert out.tolist() == [14] and torch.equal(big[P - 2:], want[0]) and torch.equal(small[P - 2:], want[1])


def test_streams_and_graphs():
    sv = _sv()
    g = torch.Generator().manual_seed(5)
    table, refs, lengths, P = _beams(g, 4, 4, 30, 16)
    parent = torch.randint(0, 4, (4, 4), generator=g).tolist()
    cache = torch.randn((2, P, 16, 8), device=DEV)
    t, f, ln, par = _i32(table), _i32(refs), _i32(lengths), _i32(parent)
    want = sv.pages_fork(cache.clone(), t, f, ln, par, page_dim=1)
    grown = sv.pages_resize(t, f, ln + 0, 16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = sv.pages_fork(cache.clone(), t, f, ln, par, page_dim=1, stream=s)
    s.synchronize()
    assert torch.equal(r["table"], want["table"])
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            outs.append((sv.pages_fork(cache, t, f, ln, par, page_dim=1), sv.pages_resize(t, f, ln, 16)))
        graphs.append(gr)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for a, b in outs:
            assert all(torch.equal(a[k], want[k]) for k in want) and all(torch.equal(b[k], grown[k]) for k in grown)
            for v in list(a.values()) + list(b.values()):
                v.zero_()


def test_on_a_stream_of_its_own():
    """Every call with stream=, beside work on the current stream; outputs written there."""
    sv = _sv()
    s = torch.cuda.Stream()
    tokens, choice = _i32([[5, 1, 2, 3]] * 3), _i32([[1, 2, 9, 9]] * 3)
    table, refs, lengths = _i32([[0, 1], [2, -1], [3, -1]]), _i32([1, 1, 1, 1, 0, 0]), _i32([20, 9, 3])
    cache = torch.arange(96, device=DEV, dtype=torch.int32).view(6, 16, 1)
    want = [sv.tree_accept(tokens, None, choice), sv.pages_resize(table, refs, lengths, 16)]
    kept = cache.clone()
    path = want[0]["path"]
    new = sv.pages_compact(kept, table, lengths, path)
    s.wait_stream(torch.cuda.current_stream())
    got = [sv.tree_accept(tokens, None, choice, stream=s), sv.pages_resize(table, refs, lengths, 16, stream=s)]
    other = sv.pages_compact(cache, table, lengths, got[0]["path"], stream=s)
    s.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(a[k], b[k]) for k in b)
    assert torch.equal(other, new) and torch.equal(cache, kept)
    with pytest.raises(ValueError):
        sv.tree_accept(tokens.cpu(), None, choice)


def test_writes_are_seen_by_autograd():
    sv = _sv()
    cache = torch.zeros((4, 16, 2), device=DEV)
    w = torch.ones((4, 16, 2), device=DEV, requires_grad=True)
    y = (w * cache).sum()
    sv.pages_compact(cache, _i32([[0, 1]]), _i32([4]), _i32([[1, 2]]))
    with pytest.raises(RuntimeError):
        y.backward()                        # the cache that it kept was written
    table, refs = _i32([[0, -1]]), _i32([1, 0, 0, 0])
    v = table._version, refs._version
    sv.pages_resize(table, refs, _i32([20]), 16)
    assert (table._version, refs._version) == v
    sv.pages_resize(table, refs, _i32([20]), 16, out={"table": table, "refs": refs})
    assert table._version > v[0] and refs._version > v[1]


# ---- together -------------------------------------------------------------------------------


def test_a_decoding_step_of_trees():
    """Pages for the nodes, their keys and values, attention, a head, the walk, the
    cache made compact; then the next step over the new context gives what a cache that
    holds only the accepted tokens gives."""
    sv = _sv()
    g = torch.Generator(device=DEV).manual_seed(0)
    B, N, Hq, Hkv, D, page, M, V, layers = 3, 12, 4, 2, 64, 16, 8, 50, 2
    P = B * M
    cache = torch.full((layers, 2, P, page, Hkv, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    table = torch.full((B, M), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(P, dtype=torch.int32, device=DEV)
    lengths = _i32([37, 16, 0])
    words = torch.randn((layers, 2, V, Hkv, D), generator=g, device=DEV).bfloat16()      # keys and values of each token
    heads = torch.randn((Hq * D, V), generator=g, device=DEV)
    text = [[int(x) for x in torch.randint(0, V, (n,), generator=torch.Generator().manual_seed(n))] for n in lengths.tolist()]

    def write(b, tokens, at):
        for i, tok in enumerate(tokens):
            cache[:, :, table[b, (at + i) // page].long(), (at + i) % page] = words[:, :, tok]

    def logits(tokens, parents, lengths):
        x = torch.randn((V, Hq, D), generator=torch.Generator().manual_seed(7)).to(DEV).bfloat16()[tokens.long()]
        for layer in range(layers):
            x = sv.tree_attention(x, cache[layer, 0], cache[layer, 1], table, lengths, parents)["out"]
        return (x.float().flatten(2) @ heads).contiguous()

    sv.pages_resize(table, refs, lengths, page, out={"table": table, "refs": refs})
    for b in range(B):
        write(b, text[b], 0)
    tokens = torch.randint(0, V, (B, N), generator=g, device=DEV).to(torch.int32)
    parents = _i32([-1, 0, 0, 0, 1, 1, 2, 4, 7, 8, 3, 10])
    for step in range(3):
        sv.pages_resize(table, refs, lengths + N, page, out={"table": table, "refs": refs})
        for b in range(B):
            write(b, tokens[b].tolist(), int(lengths[b]))
        z = logits(tokens, parents, lengths)
        choice = sv.top_logprobs(z, 1)["ids"][..., 0]
        assert torch.equal(choice, z.argmax(-1).int())
        # drafts that are right along a path of their own: node 2, then 6
        tokens[:, 2] = choice[:, 0]
        for b in range(B):
            write(b, tokens[b].tolist(), int(lengths[b]))
        z = logits(tokens, parents, lengths)
        choice = sv.top_logprobs(z, 1)["ids"][..., 0]
        r = sv.tree_accept(tokens, parents, choice)
        want = ref.accept(tokens.tolist(), [parents.tolist()] * B, choice.tolist(), [N] * B)
        assert r["path"].tolist() == want[2] and min(want[0]) >= 1
        old = lengths.tolist()
        lengths = sv.pages_compact(cache, table, lengths, r["path"], page_dim=2)
        sv.pages_resize(table, refs, lengths, page, out={"table": table, "refs": refs})
        for b in range(B):
            text[b] += [int(tokens[b, n]) for n in want[2][b] if n >= 0]
            assert lengths[b] == old[b] + want[0][b] + 1 == len(text[b])
            for t, tok in enumerate(text[b]):
                assert torch.equal(cache[:, :, table[b, t // page].long(), t % page], words[:, :, tok])
        assert int(refs.sum()) == int(((lengths + page - 1) // page).sum())
        # the walk's last token opens the next tree, random drafts after it
        last = torch.gather(r["out_tokens"], 1, r["accepted_len"].long()[:, None])
        tokens = torch.randint(0, V, (B, N), generator=g, device=DEV).to(torch.int32)
        tokens[:, :1] = last
    # beams: two of each sequence over one prompt, forked twice
    wide = table[:, None].expand(B, 2, M).contiguous()
    refs += refs                                             # every entry is named twice
    wl = lengths[:, None].expand(B, 2).contiguous()
    f = sv.pages_fork(cache, wide, refs, wl, _i32([[0, 1]] * B), page_dim=2)
    for b in range(B):
        for w in range(2):
            for t, tok in enumerate(text[b]):
                assert torch.equal(cache[:, :, f["table"][b, w, t // page].long(), t % page], words[:, :, tok])
    t = f["table"].flatten().long()
    assert torch.equal(torch.bincount(t[t >= 0], minlength=P).int(), f["refs"])
    last = ((wl - 1) // page).long()[..., None]
    ends = torch.gather(f["table"], 2, last)[..., 0]
    assert ((ends[:, 0] != ends[:, 1]) | (wl[:, 0] % page == 0)).all()
