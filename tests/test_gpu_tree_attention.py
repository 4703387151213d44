"""Attention of a tree's nodes over pages against 64-bit values: head layouts,
lengths around pages and tiles, trees, counts, strides, what a row must not see."""
import math

import pytest

torch = pytest.importorskip("torch")
import numpy as np  # noqa: E402

import tree_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F16 = torch.bfloat16, torch.float16
NAN = float("nan")


def _sv():
    import speculative_decoding_token_verify_gb300 as sv
    sv.build()
    return sv


def _tree(g, N, kind):
    if kind == "chain":
        return [n - 1 for n in range(N)]
    if kind == "star":
        return [-1] + [0] * (N - 1)
    if kind == "roots":
        return [-1] * N
    return [-1] + [int(torch.randint(0, n, (1,), generator=g)) if torch.rand(1, generator=g) < 0.6 else n - 1
                   for n in range(1, N)]


def _case(seed, dtype, N, Hq, Hkv, D, page, lengths, counts=None, kind="random", M=None, spare=3, poison=True, scale_q=2.0):
    """Random inputs on the GPU; slots that no node may see hold NaN."""
    g = torch.Generator().manual_seed(seed)
    B = len(lengths)
    counts_ = counts or [N] * B
    most = max(L + c for L, c in zip(lengths, counts_))
    M = M or max(1, -(-most // page))
    P = B * M + spare
    pages = torch.randperm(P, generator=g)[:B * M].view(B, M)
    q = (scale_q * torch.randn((B, N, Hq, D), generator=g)).to(dtype)
    k = torch.randn((P, page, Hkv, D), generator=g).to(dtype)
    v = (torch.randn((P, page, Hkv, D), generator=g) + 0.25).to(dtype)
    if poison:
        live = torch.zeros((P, page), dtype=torch.bool)
        for b in range(B):
            for t in range(lengths[b] + counts_[b]):
                live[pages[b, t // page], t % page] = True
        bad = torch.tensor([NAN, math.inf, -math.inf]).to(dtype)
        at = (~live).nonzero()
        k[at[:, 0], at[:, 1]] = bad[torch.randint(0, 3, (len(at), 1, 1), generator=g)]
        v[at[:, 0], at[:, 1]] = bad[torch.randint(0, 3, (len(at), 1, 1), generator=g)]
    parents = [_tree(g, N, kind) for _ in range(B)]
    table = pages.to(torch.int32)
    return dict(q=q, k=k, v=v, table=table, lengths=lengths, counts=counts, counts_=counts_, parents=parents)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _check(c, got, scale):
    out, lse, e_out, e_lse = ref.attention(c["q"], c["k"], c["v"], c["table"], c["lengths"], c["parents"], c["counts_"], scale)
    o, s = got["out"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
    assert np.array_equal(np.isnan(o), np.isnan(out)) and np.array_equal(np.isnan(s), np.isnan(lse))
    inf = ~np.isfinite(out)
    assert np.array_equal(o[inf & ~np.isnan(out)], out[inf & ~np.isnan(out)])
    with np.errstate(invalid="ignore"):
        d = np.abs(o - out)
    d[inf] = 0
    e_out[inf] = 0
    assert (d <= e_out).all(), (d - e_out).max()
    none = np.isneginf(lse)
    assert np.array_equal(none, np.isneginf(s))
    fine = ~none & ~np.isnan(lse)
    assert (np.abs(s[fine] - lse[fine]) <= e_lse[fine]).all(), np.abs(s[fine] - lse[fine]).max()


def _run(sv, c, scale=None, parents="each", **kw):
    par = None if parents is None else _i32(c["parents"]) if parents == "each" else _i32(c["parents"][0])
    return sv.tree_attention(c["q"].to(DEV), c["k"].to(DEV), c["v"].to(DEV), c["table"].to(DEV), _i32(c["lengths"]), par,
                             counts=None if c["counts"] is None else _i32(c["counts"]), scale=scale, **kw)


SHAPES = [  # N, Hq, Hkv, D, page
    (1, 1, 1, 8, 8), (1, 8, 2, 64, 16), (1, 32, 8, 128, 16), (9, 8, 2, 128, 16), (5, 6, 2, 80, 32), (33, 15, 3, 40, 64),
    (64, 16, 2, 128, 128), (128, 4, 4, 64, 16), (3, 7, 1, 120, 256), (17, 24, 2, 96, 8), (2, 128, 1, 64, 16),
    (43, 3, 1, 128, 512), (128, 20, 2, 72, 32),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "N%d-H%d.%d-D%d-page%d" % s)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_shapes(shape, dtype):
    sv = _sv()
    N, Hq, Hkv, D, page = shape
    c = _case(N + Hq + D, dtype, N, Hq, Hkv, D, page, [0, 1, 37, 128, 300])
    status = _i32([0])
    got = _run(sv, c, status=status)
    _check(c, got, D ** -0.5)
    assert int(status) == 0


@pytest.mark.parametrize("length", [0, 1, 7, 8, 15, 16, 17, 63, 64, 65, 119, 120, 127, 128, 129, 255, 256, 257, 383, 640, 1000])
@pytest.mark.parametrize("N", [1, 6, 40])
def test_lengths(length, N):
    sv = _sv()
    c = _case(length + N, BF16, N, 8, 2, 64, 16, [length, length + 3, max(length - 1, 0)])
    _check(c, _run(sv, c), 0.125)


@pytest.mark.parametrize("kind", ["chain", "star", "roots", "random"])
@pytest.mark.parametrize("N", [1, 2, 31, 32, 33, 64, 65, 127, 128])
def test_trees(kind, N):
    sv = _sv()
    c = _case(N, BF16, N, 4, 2, 64, 16, [100, 3], kind=kind)
    _check(c, _run(sv, c), 0.125)
    if kind == "chain":
        _check(c, _run(sv, c, parents=None), 0.125)
    c["parents"][1] = c["parents"][0]
    _check(c, _run(sv, c, parents="one"), 0.125)


def test_nodes_that_do_not_exist():
    """counts: rows of missing nodes are 0 and -inf, and nobody sees their slots."""
    sv = _sv()
    c = _case(5, BF16, 20, 8, 2, 128, 16, [50, 0, 0, 127, 200, 16], counts=[20, 0, 3, 1, 19, 0])
    got = _run(sv, c, out={"out": torch.full((6, 20, 8, 128), NAN, dtype=BF16, device=DEV),
                           "lse": torch.full((6, 20, 8), NAN, device=DEV)})
    _check(c, got, 128 ** -0.5)
    assert (got["out"][1] == 0).all() and (got["lse"][1] == -math.inf).all() and (got["out"][2, 3:] == 0).all()


@pytest.mark.parametrize("N,L", [(12, 60), (40, 120), (128, 250)])
def test_branches_do_not_see_one_another(N, L):
    """NaN and infinities in a node's key or value reach its descendants alone."""
    sv = _sv()
    c = _case(N, BF16, N, 8, 2, 64, 16, [L, L + 1])
    for b in range(2):
        for i, (t, x) in enumerate([("k", NAN), ("v", NAN), ("v", math.inf), ("v", -math.inf), ("k", math.inf)]):
            n = N - 1 - i
            s = c["lengths"][b] + n
            c[t][c["table"][b, s // 16], s % 16, i % 2, (7 * i) % 64] = x
        c["q"][b, N - 5] = c["q"][b, N - 5].abs()
    got = _run(sv, c)
    out, lse, _, _ = ref.attention(c["q"], c["k"], c["v"], c["table"], c["lengths"], c["parents"], c["counts_"], 0.125)
    clean = np.isfinite(out).all(-1) & np.isfinite(lse)
    assert clean.any() and not clean.all()
    o = got["out"].double().cpu().numpy()
    assert np.array_equal(np.isfinite(o[clean]), np.isfinite(out[clean]))
    # rows whose scores are finite: the values' infinities and NaN in their places
    score = np.isfinite(lse)
    assert np.array_equal(np.isnan(o[score]), np.isnan(out[score]))
    assert np.array_equal(np.isinf(o[score]), np.isinf(out[score]))


def test_context_values_reach_every_row():
    sv = _sv()
    c = _case(3, BF16, 4, 4, 2, 64, 16, [200, 70], kind="star")
    c["v"][c["table"][0, 2], 5, 1, 9] = math.inf
    c["v"][c["table"][1, 1], 5, 0, 9] = NAN
    _check(c, _run(sv, c), 0.125)


def test_rows_spoil_themselves_alone():
    sv = _sv()
    c = _case(4, BF16, 6, 8, 2, 64, 16, [100])
    c["q"][0, 2, 3] = NAN
    got = _run(sv, c)
    assert got["out"][0, 2, 3].isnan().all()
    keep = torch.ones((6, 8), dtype=torch.bool)
    keep[2, 3] = False
    assert got["out"][0].cpu()[keep].isfinite().all() and got["lse"][0].cpu()[keep].isfinite().all()


@pytest.mark.parametrize("scale_q,scale", [(0.0, None), (30.0, None), (2.0, 0.0), (2.0, -0.3), (2.0, 4.0)])
def test_flat_and_peaked_rows(scale_q, scale):
    sv = _sv()
    c = _case(8, F16, 10, 6, 3, 64, 16, [700, 90], scale_q=scale_q)
    _check(c, _run(sv, c, scale=scale), 0.125 if scale is None else scale)


def test_rising_scores():
    """The running maximum moves with every key."""
    sv = _sv()
    c = _case(9, BF16, 5, 4, 1, 64, 16, [900])
    c["q"] = torch.ones_like(c["q"])
    for t in range(905):
        c["k"][c["table"][0, t // 16], t % 16] = 0.0
        c["k"][c["table"][0, t // 16], t % 16, :, :4] = t / 16.0
    _check(c, _run(sv, c, scale=1.0), 1.0)
    for t in range(905):
        c["k"][c["table"][0, t // 16], t % 16] *= -1
    _check(c, _run(sv, c, scale=1.0), 1.0)


def test_strides():
    """Keys and values in one pool, heads before slots, queries cut out of a fused projection."""
    sv = _sv()
    c = _case(10, BF16, 9, 8, 2, 64, 16, [130, 20, 77])
    want = _run(sv, c)
    P = c["k"].shape[0]
    both = torch.full((P, 2, 16, 2, 64), NAN, dtype=BF16, device=DEV)
    both[:, 0], both[:, 1] = c["k"].to(DEV), c["v"].to(DEV)
    heads = torch.empty((P, 2, 16, 64), dtype=BF16, device=DEV)
    heads.copy_(c["v"].to(DEV).transpose(1, 2))
    wide = torch.full((P, 16, 2, 200), NAN, dtype=BF16, device=DEV)[..., 8:72]
    wide.copy_(c["k"].to(DEV))
    fused = torch.full((9, 3, 12, 64), NAN, dtype=BF16, device=DEV)     # nodes first
    q = fused[:, :, :8].transpose(0, 1)
    q.copy_(c["q"].to(DEV))
    for kk, vv in ((both[:, 0], both[:, 1]), (both[:, 0], heads.transpose(1, 2)), (wide, heads.transpose(1, 2))):
        got = sv.tree_attention(q, kk, vv, c["table"].to(DEV), _i32(c["lengths"]), _i32(c["parents"]))
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


def test_offsets_past_32_bits():
    sv = _sv()
    c = _case(11, BF16, 3, 4, 2, 64, 16, [50, 33])
    want = _run(sv, c)
    P = (5 << 30) // (16 * 2 * 64 * 2)
    k = torch.empty((P, 16, 2, 64), dtype=BF16, device=DEV)
    v = torch.empty((P, 16, 2, 64), dtype=BF16, device=DEV)
    far = c["table"] + (P - c["k"].shape[0])
    k[P - c["k"].shape[0]:] = c["k"].to(DEV)
    v[P - c["k"].shape[0]:] = c["v"].to(DEV)
    got = sv.tree_attention(c["q"].to(DEV), k, v, far.to(DEV), _i32(c["lengths"]), _i32(c["parents"]))
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


@pytest.mark.parametrize("B,N,Hq,Hkv,most", [(1, 1, 8, 1, 20000), (1, 9, 8, 2, 20000), (3, 40, 16, 2, 9000), (150, 2, 4, 2, 600)])
def test_long_and_many(B, N, Hq, Hkv, most):
    """Rows split over many CTAs, and many short ones."""
    sv = _sv()
    g = torch.Generator().manual_seed(B)
    lengths = [int(x) for x in torch.randint(0, most, (B,), generator=g)]
    lengths[0] = most
    c = _case(B, BF16, N, Hq, Hkv, 64, 16, lengths, poison=False)
    keep = sorted({0, B // 2, B - 1})
    got, again = _run(sv, c), _run(sv, c)
    assert torch.equal(got["out"], again["out"]) and torch.equal(got["lse"], again["lse"])    # the same bits on every run
    for key in ("q", "table"):
        c[key] = c[key][keep]
    for key in ("lengths", "parents", "counts_"):
        c[key] = [c[key][b] for b in keep]
    c["counts"] = None
    _check(c, {x: y[keep] for x, y in got.items()}, 0.125)


@pytest.mark.parametrize("N,Hq,Hkv,B,most", [(100, 8, 2, 40, 700), (33, 16, 1, 30, 400), (7, 4, 4, 200, 300), (128, 128, 1, 3, 200)])
def test_ragged_batches(N, Hq, Hkv, B, most):
    """Several tiles of rows, nodes that do not exist, many sequences a CTA; branches with NaN."""
    sv = _sv()
    g = torch.Generator().manual_seed(N)
    lengths = [int(x) for x in torch.randint(0, most, (B,), generator=g)]
    counts = [int(x) for x in torch.randint(0, N + 1, (B,), generator=g)]
    counts[1], lengths[2] = 0, 0
    c = _case(N, BF16, N, Hq, Hkv, 64, 16, lengths, counts=counts)
    for b in range(0, B, 3):      # a node's value that only it and its descendants see
        if counts[b] > 1:
            t = lengths[b] + counts[b] - 1
            c["v"][c["table"][b, t // 16], t % 16, 0, b % 64] = NAN if b % 2 else math.inf
    st = _i32([0])
    got = _run(sv, c, status=st)
    assert int(st) == 0
    keep = sorted({0, 1, 2, 3, B // 2, B - 1}) if B > 5 else list(range(B))
    for key in ("q", "table"):
        c[key] = c[key][keep]
    for key in ("lengths", "parents", "counts_"):
        c[key] = [c[key][b] for b in keep]
    _check(c, {x: y[keep] for x, y in got.items()}, 0.125)


def test_shared_and_repeated_pages():
    """Sequences over one prompt, a page twice in a row, keys and values in one tensor."""
    sv = _sv()
    c = _case(25, BF16, 6, 8, 2, 64, 16, [150, 160, 90], poison=False)
    t = c["table"]
    t[1, :9], t[2, :5] = t[0, :9], t[0, :5]          # full pages of the first sequence
    t[2, 3] = t[2, 1]
    _check(c, _run(sv, c), 0.125)
    same = {**c, "v": c["k"]}
    k = c["k"].to(DEV)
    got = sv.tree_attention(c["q"].to(DEV), k, k, t.to(DEV), _i32(c["lengths"]), _i32(c["parents"]))
    _check(same, got, 0.125)


def test_one_large_page():
    sv = _sv()
    c = _case(21, BF16, 5, 8, 2, 64, 1 << 20, [3000, 129], poison=False, spare=0)
    _check(c, _run(sv, c), 0.125)


def test_repeated_under_load():
    """Many calls in a row, beside another stream's products: always the same bits and no code."""
    sv = _sv()
    c = _case(22, BF16, 20, 16, 2, 128, 16, [5000, 300, 70, 0])
    a = (c["q"].to(DEV), c["k"].to(DEV), c["v"].to(DEV), c["table"].to(DEV), _i32(c["lengths"]), _i32(c["parents"]))
    want = sv.tree_attention(*a)
    st, x = _i32([0]), torch.randn((2048, 2048), device=DEV).bfloat16()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = []
    for i in range(60):
        with torch.cuda.stream(s):
            y = x @ x
        outs.append(sv.tree_attention(*a, status=st))
    torch.cuda.synchronize()
    assert int(st) == 0 and y.isfinite().all()
    assert all(torch.equal(o["out"], want["out"]) and torch.equal(o["lse"], want["lse"]) for o in outs)


def test_waits_give_up():
    """With no polls allowed every wait gives up: a code, and nothing left behind."""
    sv = _sv()
    from speculative_decoding_token_verify_gb300 import _native
    for N, lengths in ((1, [5]), (9, [900, 30, 0]), (64, [2000, 100])):
        c = _case(23, BF16, N, 8, 2, 64, 16, lengths)
        want, st = _run(sv, c), _i32([0])
        torch.cuda.synchronize()
        old = _native.lib().spec_debug_set_wait_limit(0)
        try:
            _run(sv, c, status=st)
            torch.cuda.synchronize()
        finally:
            _native.lib().spec_debug_set_wait_limit(old)
        assert int(st) == 4
        st.zero_()
        got = _run(sv, c, status=st)
        assert int(st) == 0 and torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


def test_empty():
    sv = _sv()
    c = _case(12, BF16, 3, 4, 2, 64, 16, [5])
    for B, N in ((0, 3), (1, 0)):
        r = sv.tree_attention(c["q"][:B, :N].to(DEV), c["k"].to(DEV), c["v"].to(DEV), c["table"][:B].to(DEV), _i32(c["lengths"][:B]))
        assert r["out"].shape == (B, N, 4, 64) and r["lse"].shape == (B, N, 4)
    r = sv.tree_attention(c["q"].to(DEV), c["k"][:0].to(DEV), c["v"][:0].to(DEV), c["table"][:, :0].to(DEV), _i32([0]), counts=_i32([0]))
    assert (r["out"] == 0).all() and (r["lse"] == -math.inf).all()


def test_bad_device_values():
    """Lengths, counts, parents and pages out of range: clamped or reported, never followed."""
    sv = _sv()

    def status(change, want):
        c = _case(13, BF16, 4, 4, 2, 64, 16, [40, 30])
        t = {"lengths": _i32(c["lengths"]), "counts": _i32([4, 4]), "parents": _i32(c["parents"]), "table": c["table"].to(DEV)}
        good = sv.tree_attention(c["q"].to(DEV), c["k"].to(DEV), c["v"].to(DEV), t["table"], t["lengths"], t["parents"], counts=t["counts"])
        change(t)
        st = _i32([0])
        r = sv.tree_attention(c["q"].to(DEV), c["k"].to(DEV), c["v"].to(DEV), t["table"], t["lengths"], t["parents"],
                              counts=t["counts"], status=st)
        assert int(st) == want
        assert torch.equal(r["out"][1], good["out"][1])         # the other sequence
        return r, c

    status(lambda t: None, 0)
    r, _ = status(lambda t: t["lengths"].__setitem__(0, -3), 11)
    status(lambda t: t["lengths"].__setitem__(0, 1 << 30), 11)
    status(lambda t: t["lengths"].__setitem__(0, (1 << 31) - 1), 11)
    r, _ = status(lambda t: t["counts"].__setitem__(0, -1), 11)
    assert (r["out"][0] == 0).all()
    status(lambda t: t["counts"].__setitem__(0, 1 << 30), 11)
    status(lambda t: t["parents"].__setitem__((0, 2), 2), 9)
    status(lambda t: t["parents"].__setitem__((0, 2), -7), 9)
    status(lambda t: t["table"].__setitem__((0, 1), -1), 10)
    status(lambda t: t["table"].__setitem__((0, 0), 1 << 30), 10)
    status(lambda t: t["table"].__setitem__((0, 2), -(1 << 31)), 10)


def test_out_and_autograd():
    """Outputs into the caller's tensors, whose versions move; queries that want a gradient."""
    sv = _sv()
    c = _case(24, BF16, 5, 8, 2, 64, 16, [40])
    want = _run(sv, c)
    o = {"out": torch.empty((1, 5, 8, 64), dtype=BF16, device=DEV), "lse": torch.empty((1, 5, 8), device=DEV)}
    v = o["out"]._version, o["lse"]._version
    q = c["q"].to(DEV).requires_grad_(True)
    r = sv.tree_attention(q, c["k"].to(DEV), c["v"].to(DEV), c["table"].to(DEV), _i32(c["lengths"]), _i32(c["parents"]), out=o)
    assert r["out"] is o["out"] and r["lse"] is o["lse"] and not r["out"].requires_grad
    assert o["out"]._version > v[0] and o["lse"]._version > v[1]
    assert torch.equal(r["out"], want["out"]) and torch.equal(r["lse"], want["lse"])
    with pytest.raises(ValueError):
        sv.tree_attention(q, c["k"].to(DEV), c["v"].to(DEV), c["table"].to(DEV), _i32(c["lengths"]), out={"out": o["out"][:, :4]})
    with pytest.raises(TypeError):
        sv.tree_attention(q.float(), c["k"].to(DEV), c["v"].to(DEV), c["table"].to(DEV), _i32(c["lengths"]))
    with pytest.raises(sv.SpecError):
        sv.tree_attention(q.expand(3, 5, 8, 64), c["k"].to(DEV), c["v"].to(DEV), c["table"].expand(3, -1).contiguous().to(DEV),
                          _i32(c["lengths"] * 3))         # a stride of 0


def test_streams_and_graphs():
    sv = _sv()
    c, d = _case(14, BF16, 9, 8, 2, 64, 16, [3000, 40]), _case(15, BF16, 9, 8, 2, 64, 16, [64, 2500])
    want = [_run(sv, x) for x in (c, d)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = _run(sv, c, stream=s)
    s.synchronize()
    assert torch.equal(r["out"], want[0]["out"])
    args = [(x["q"].to(DEV), x["k"].to(DEV), x["v"].to(DEV), x["table"].to(DEV), _i32(x["lengths"]), _i32(x["parents"])) for x in (c, d)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a in args:
        with torch.cuda.stream(s):
            sv.tree_attention(*a)
        s.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            outs.append(sv.tree_attention(*a))
        graphs.append(gr)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):       # two graphs at once
        for o in outs:
            o["out"].zero_()
            o["lse"].zero_()
        torch.cuda.synchronize()
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o["out"], w["out"]) and torch.equal(o["lse"], w["lse"])
    args[0][4].fill_(30)     # other lengths in the captured call
    graphs[0].replay()
    torch.cuda.synchronize()
    again = sv.tree_attention(*args[0])
    assert torch.equal(outs[0]["out"], again["out"])
