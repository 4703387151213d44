"""Beam steps and the reordering of states on the GPU against the fp64
reference, and a run of them with the verification pass."""
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


def _poisoned(B, N):
    out = {k: torch.full((B, N), 0x7F7F7F7F, dtype=torch.int32, device=DEV) for k in ("parent", "token", "finished")}
    out["scores"] = torch.full((B, N), 3.3e38, device=DEV)
    return out


def _check(z, scores, N, finished=None, eos=-1, status_want=0):
    sv = _sv()
    B, W, V = z.shape
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = sv.beam_step(z, scores, N, finished=finished, eos=eos, out=_poisoned(B, N), status=status)
    torch.cuda.synchronize()
    assert int(status) == status_want
    zn, sn = z.float().cpu().numpy(), scores.cpu().numpy()
    fn = None if finished is None else finished.cpu().numpy()
    o = {k: v.cpu().numpy() for k, v in out.items()}
    for b in range(B):
        sc, par, tok, fin, tol = ref.beam(zn[b], sn[b], N, None if fn is None else fn[b], eos)
        np.testing.assert_array_equal(o["parent"][b], par, err_msg=f"item {b}")
        np.testing.assert_array_equal(o["token"][b], tok, err_msg=f"item {b}")
        np.testing.assert_array_equal(o["finished"][b], fin)
        full = par >= 0
        assert np.all(o["scores"][b][~full] == -INF)
        assert np.all(np.abs(o["scores"][b][full] - sc[full]) <= tol[full])
    return out


def _case(B, W, V, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    z = (3 * torch.randn((B, W, V), generator=g)).to(DT[dtype]).to(DEV)
    scores = (-5 * torch.rand((B, W), generator=g)).to(DEV)
    return z, scores, g


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,W,V,N", [(1, 1, 1, 1), (2, 1, 2, 4), (3, 2, 5, 4), (2, 3, 9, 64), (4, 4, 1000, 4),
                                     (1, 4, 32000, 8), (5, 8, 4097, 16), (2, 32, 2001, 64), (1, 5, 128256, 10),
                                     (70, 2, 333, 3), (1, 1, 128256, 64), (1, 31, 32001, 64), (2, 12, 20000, 24),
                                     (100, 3, 4099, 6), (200, 2, 2051, 4), (700, 1, 1031, 2), (1, 32, 40000, 64)])
def test_against_reference(B, W, V, N, dtype):
    z, scores, _ = _case(B, W, V, dtype, B + W + V)
    _check(z, scores, N)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_finished_first_and_dead_beams(dtype):
    z, scores, g = _case(6, 4, 700, dtype, 1)
    fin = torch.zeros((6, 4), dtype=torch.int32, device=DEV)
    scores[0, 1:] = -INF              # the first step
    scores[1] = -INF                  # nothing left
    fin[2, 1] = 1
    scores[2, 1] = -0.25              # a finished beam ahead
    fin[3] = 1                        # all finished: fewer continuations than places
    fin[4, 0] = 7
    z[4, 1, 9] = 40.0                 # a live beam that ends
    z[5, 2] = -INF                    # a beam with every token masked
    z[2, 1] = float("nan")            # a finished beam's logits are not read
    z[0, 2] = float("nan")            # nor a dead one's
    _check(z, scores, 4, fin, eos=9)
    _check(z, scores, 9, fin, eos=9)


def test_masks_and_ties():
    sv = _sv()
    z, scores, _ = _case(3, 4, 512, "bf16", 2)
    z[0] = 0.5                        # every token equal
    scores[0] = -1.0                  # every beam too: lowest beam, lowest token
    z[1] = z[1, 0]                    # identical beams
    scores[1] = -2.0
    z[2, :, 3:] = -INF                # few tokens
    _check(z, scores, 16)
    z[2, :, :3] = -3.38e38
    out = _check(z, scores, 16)
    assert (out["parent"][2] == -1).all()
    assert sv.MAX_BEAMS == 32


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [3001, 60000])
def test_scores_closer_than_fp32_sums_tell_apart(dtype, V):
    """Beams whose rows hold the same logits in another order, at scores one
    fp32 step (6e-8) apart: fp32 sums of the two rows may differ by more."""
    B, W = 24, 4
    g = torch.Generator().manual_seed(V)
    z = torch.empty((B, W, V), dtype=DT[dtype])
    scores = torch.empty((B, W))
    for b in range(B):
        row = (2 * torch.randn(V, generator=g)).to(DT[dtype])
        base = np.float32(-0.9)
        steps = torch.randperm(W, generator=g).tolist()
        for w in range(W):
            z[b, w] = row[torch.randperm(V, generator=g)]
            s = base
            for _ in range(steps[w]):
                s = np.nextafter(s, np.float32(0))
            scores[b, w] = float(s)
    for N in (2, 4, 6):
        _check(z.to(DEV), scores.to(DEV), N)
    for n in (1, 2, 3):   # one cluster
        _check(z[:n].to(DEV), scores[:n].to(DEV), 4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_longest_rows_and_most_beams(dtype):
    z, scores, _ = _case(1, 32, 1 << 20, dtype, 7)
    z[0, 3] = z[0, 2]                 # identical beams at equal scores
    scores[0, 3] = scores[0, 2]
    _check(z, scores, 64)
    z[0, 5:9] = 0.25                  # rows of equal logits among the best
    scores[0, 5:9] = 20.0
    _check(z, scores, 64)


def test_spoilt_beams():
    sv = _sv()
    z, scores, _ = _case(3, 3, 400, "f32", 4)
    want = sv.beam_step(z[:, :2].contiguous(), scores[:, :2].contiguous(), 4)
    z[0, 2, 7] = float("nan")
    z[1, 2, 7] = INF
    scores[2, 2] = float("nan")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = sv.beam_step(z, scores, 4, status=status)
    torch.cuda.synchronize()
    assert int(status) == sv.api.SPEC_ERR_BAD_ROW
    assert all(torch.equal(got[k], want[k]) for k in want)


def test_strides_in_place_streams_and_graphs():
    sv = _sv()
    z, scores, _ = _case(4, 4, 5001, "bf16", 5)
    fin = torch.zeros((4, 4), dtype=torch.int32, device=DEV)
    want = sv.beam_step(z, scores, 4, finished=fin, eos=2)
    wide = torch.zeros((4, 6, 5010), dtype=torch.bfloat16, device=DEV)
    wide[:, 1:5, 3:5004] = z
    got = _check(wide[:, 1:5, 3:5004], scores, 4, fin, eos=2)
    assert all(torch.equal(got[k], want[k]) for k in ("parent", "token", "finished"))
    sc2, fin2 = scores.clone(), fin.clone()
    got = sv.beam_step(z, sc2, 4, finished=fin2, eos=2, out={"scores": sc2, "finished": fin2})
    assert got["scores"] is sc2 and all(torch.equal(got[k], want[k]) for k in want)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    zf, sf = z.flip(0), scores.flip(0)
    wantf = sv.beam_step(zf, sf, 4, finished=fin, eos=2)
    torch.cuda.synchronize()
    a = sv.beam_step(z, scores, 4, finished=fin, eos=2, stream=s1)   # two calls at once
    b = sv.beam_step(zf, sf, 4, finished=fin, eos=2, stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(a[k], want[k]) and torch.equal(b[k], wantf[k]) for k in want)
    zz = z.clone()
    graphs, outs = [], []
    for _ in range(2):                # two graphs, replayed at once
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sv.beam_step(zz, scores, 4, finished=fin, eos=2))
        graphs.append(g)
    torch.cuda.synchronize()
    for g, s in zip(graphs, (s1, s2)):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o[k], want[k]) for o in outs for k in want)


# ---- reordering ---------------------------------------------------------------------------------

def _state(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-100, 100, shape, generator=g).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 64), (torch.float32, 33), (torch.bfloat16, 33), (torch.uint8, 7),
                                     (torch.int64, 3), (torch.bfloat16, 2)])
@pytest.mark.parametrize("W", [1, 2, 4, 5, 8, 13, 32])
def test_reorder(dtype, D, W):
    sv = _sv()
    O, B, H, T = 2, 5, 3, 37
    state = _state((O, B, W, H, T, D), dtype, W)
    parent = torch.randint(-1, W, (B, W), generator=torch.Generator().manual_seed(W), dtype=torch.int32)
    parent[0] = torch.arange(W)
    parent[1] = 0
    parent[2] = torch.arange(W).flip(0)
    lengths = torch.tensor([5, 37, 0, 36, 100], dtype=torch.int32)
    lengths[4] = 100 if W % 2 else -3
    kind = np.uint16 if dtype == torch.bfloat16 else None
    for ln in (None, lengths):
        s = state.clone()
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = sv.beam_reorder(s, parent.to(DEV), lengths=None if ln is None else ln.to(DEV), batch_dim=1,
                              length_dim=4, status=status)
        torch.cuda.synchronize()
        assert got is s and int(status) == 0
        host = (state.view(torch.int16) if kind else state).cpu().numpy()
        want = ref.reorder(host, parent.numpy(), None if ln is None else ln.numpy())
        np.testing.assert_array_equal((s.view(torch.int16) if kind else s).cpu().numpy(), want)


@pytest.mark.parametrize("off", [0, 1, 2, 3, 7, 15])
@pytest.mark.parametrize("T,D", [(64, 33), (16, 40), (48, 1), (5, 3), (1, 1)])
def test_reorder_of_bytes_at_every_alignment(off, T, D):
    """Segments that start and lengths that end anywhere in a vector; beams a
    multiple of 16 bytes apart, or not; nothing beside the rows is touched."""
    sv = _sv()
    O, B, W, H = 2, 3, 4, 2
    for pad in (0, 5):
        row = H * T * D
        beam = (row + 15) // 16 * 16 + pad
        buf = torch.randint(0, 256, (off + O * B * W * beam + 32,), dtype=torch.uint8, device=DEV)
        s = buf.as_strided((O, B, W, H, T, D), (B * W * beam, W * beam, beam, T * D, D, 1), off)
        parent = torch.tensor([[3, 0, 1, 2], [0, 0, 3, -1], [1, 1, 1, 1]], dtype=torch.int32, device=DEV)
        ln = torch.tensor([T, T // 2, max(T - 1, 0)], dtype=torch.int32, device=DEV)
        host = buf.cpu().numpy().copy()
        view = np.lib.stride_tricks.as_strided(host[off:], s.shape, s.stride())
        view[...] = ref.reorder(view, parent.cpu().numpy(), ln.cpu().numpy())
        before = s.clone()
        sv.beam_reorder(s, parent, lengths=ln, batch_dim=1, length_dim=4)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(buf.cpu().numpy(), host)
        out = torch.randint(0, 256, (off + 3 + O * B * W * beam,), dtype=torch.uint8, device=DEV)
        for shift in (0, 3):
            d = out.as_strided(s.shape, s.stride(), off + shift)
            want = torch.from_numpy(ref.reorder(before.cpu().numpy(), parent.cpu().numpy(), ln.cpu().numpy()))
            d.copy_(before)
            sv.beam_reorder(before.contiguous(), parent, lengths=ln, batch_dim=1, length_dim=4, out=d)
            torch.cuda.synchronize()
            assert torch.equal(d.cpu(), want)


def test_reorder_out_of_place_and_fewer_beams():
    sv = _sv()
    state = _state((4, 6, 50), torch.float32, 1)                    # [B, W, X]
    parent = torch.tensor([[5, 0, -1], [1, 1, 1], [0, 1, 2], [3, 9, -4]], dtype=torch.int32, device=DEV)
    out = torch.full((4, 3, 50), 9.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.beam_reorder(state, parent, out=out, status=status)
    torch.cuda.synchronize()
    assert int(status) == sv.api.SPEC_ERR_BAD_PARENT
    want = torch.full((4, 3, 50), 9.0, device=DEV)
    for b in range(4):
        for n in range(3):
            p = int(parent[b, n])
            if 0 <= p < 6:
                want[b, n] = state[b, p]
    assert torch.equal(out, want)
    s = state.clone()
    sv.beam_reorder(s[:3], parent[:3].contiguous())
    w = state.clone()
    for b in range(3):
        for n in range(3):
            p = int(parent[b, n])
            if p >= 0:
                w[b, n] = state[b, p]
    assert torch.equal(s, w)                                        # beams past N stay
    tok = _state((3, 4), torch.int32, 2)                            # [B, W]: one value per beam
    par = torch.tensor([[3, 2, 1, 0]] * 3, dtype=torch.int32, device=DEV)
    assert torch.equal(sv.beam_reorder(tok.clone(), par), tok.flip(1))


def test_reorder_strided_views_and_large_offsets():
    sv = _sv()
    big = _state((3, 2, 5, 4, 6, 24), torch.bfloat16, 3)
    view = big[:, :, 1:4, 1:, :, :16]                               # beams, heads and units cut out
    with pytest.raises(ValueError):
        sv.beam_reorder(view, torch.zeros((2, 3), dtype=torch.int32, device=DEV), batch_dim=1, length_dim=4,
                        lengths=torch.zeros(2, dtype=torch.int32, device=DEV))
    view = big[:, :, 1:4, 1:]
    parent = torch.tensor([[2, 0, 1], [1, 1, 0]], dtype=torch.int32, device=DEV)
    ln = torch.tensor([6, 3], dtype=torch.int32, device=DEV)
    host = big.view(torch.int16).cpu().numpy().copy()
    host[:, :, 1:4, 1:] = ref.reorder(host[:, :, 1:4, 1:], parent.cpu().numpy(), ln.cpu().numpy())
    sv.beam_reorder(view, parent, lengths=ln, batch_dim=1, length_dim=4)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(big.view(torch.int16).cpu().numpy(), host)
    x = torch.zeros(2 ** 32 + 4096, dtype=torch.uint8, device=DEV)  # beams 2^32 bytes apart
    s = x.as_strided((1, 2, 1024), (2 ** 33, 2 ** 32, 1))
    s[0, 1] = torch.arange(1024, device=DEV).to(torch.uint8)
    sv.beam_reorder(s, torch.tensor([[1, 1]], dtype=torch.int32, device=DEV))
    assert torch.equal(s[0, 0], s[0, 1]) and int(s[0, 0].long().sum()) > 0


def test_reorder_in_a_graph_and_on_a_stream():
    sv = _sv()
    state = _state((2, 3, 4, 2, 50, 16), torch.bfloat16, 5)
    parent = torch.tensor([[1, 0, 3, 3], [0, 0, 0, 0], [3, 2, 1, 0]], dtype=torch.int32, device=DEV)
    ln = torch.tensor([50, 7, 0], dtype=torch.int32, device=DEV)
    kw = dict(lengths=ln, batch_dim=1, length_dim=4)
    once = sv.beam_reorder(state.clone(), parent, **kw)
    twice = sv.beam_reorder(once.clone(), parent, **kw)
    s = torch.cuda.Stream()
    a = state.clone()
    torch.cuda.synchronize()
    sv.beam_reorder(a, parent, stream=s, **kw)
    s.synchronize()
    assert torch.equal(a, once)
    b = state.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.beam_reorder(b, parent, **kw)
    b.copy_(state)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(b, once)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(b, twice)


# ---- a run of them ------------------------------------------------------------------------------

def test_beam_drafts_verified_and_distilled():
    """Draft by beams with a small recurrent draft, verify the best beam
    against target rows, then take one distillation step on the draft's rows:
    each operator's inputs are the one before's outputs."""
    sv = _sv()
    B, W, K, V, D = 5, 4, 6, 1500, 32
    g = torch.Generator(device=DEV).manual_seed(1)
    emb = torch.randn((V, D), generator=g, device=DEV)
    head = torch.randn((V, D), generator=g, device=DEV) * 0.5
    state = torch.randn((B, 1, D), generator=g, device=DEV).repeat(1, W, 1)
    scores = torch.full((B, W), -INF, device=DEV)
    scores[:, 0] = 0
    toks = torch.zeros((B, W, K), dtype=torch.int32, device=DEV)
    rows = torch.zeros((B, W, K, V), device=DEV)
    for i in range(K):
        z = torch.einsum("bwd,vd->bwv", state, head)
        step = sv.beam_step(z, scores, W)
        want = [ref.beam(z[b].cpu().numpy(), scores[b].cpu().numpy(), W) for b in range(B)]
        np.testing.assert_array_equal(step["parent"].cpu().numpy(), np.stack([x[1] for x in want]))
        np.testing.assert_array_equal(step["token"].cpu().numpy(), np.stack([x[2] for x in want]))
        scores = step["scores"]
        rows[:, :, i] = z
        for t in (state, toks, rows):
            t_before = t.cpu().numpy().copy()
            sv.beam_reorder(t, step["parent"])
            new = t.cpu().numpy()
            for b in range(B):
                np.testing.assert_array_equal(new[b], t_before[b][step["parent"][b].cpu().numpy()])
        toks[:, :, i] = step["token"]
        state = 0.9 * state + emb[step["token"].long()]
    draft = toks[:, 0].contiguous()
    zd = rows[:, 0].contiguous()
    zt = torch.randn((B, K + 1, V), generator=g, device=DEV) * 2
    zt[:, :K] += zd
    out = sv.verify(zt, None, draft, None, mode="greedy")
    n = out["accepted_len"].cpu().numpy()
    arg = zt.argmax(-1).cpu().numpy()
    for b in range(B):
        k = 0
        while k < K and int(draft[b, k]) == arg[b, k]:
            k += 1
        assert n[b] == k
    t = sv.top_logprobs(zt[:, :K], 20)
    weight = (torch.arange(K, device=DEV)[None] <= out["accepted_len"][:, None]).float() / B
    r = sv.distill_step(zd, t["logprobs"], t["ids"], weight)
    ln, idn = t["logprobs"].cpu().numpy(), t["ids"].cpu().numpy()
    for b in range(B):
        for k in range(K):
            x = ref.distill(zd[b, k].cpu().numpy(), ln[b, k], idn[b, k], float(weight[b, k]))
            assert abs(float(r["loss"][b, k]) - x["loss"]) <= x["loss_tol"]
            d = np.abs(r["dlogits"][b, k].cpu().numpy() - x["grad"])
            assert np.all(d <= x["grad_tol"] + ref.U * (np.abs(x["grad"]) + x["grad_tol"]))


def test_logits_at_the_mask_floor_are_masked():
    """fp32 -1e29 as a mask value gives what -inf gives, to the bit."""
    sv = _sv()
    z, scores, _ = _case(3, 4, 2003, "f32", 78)
    mask = torch.zeros_like(z, dtype=torch.bool)
    mask[0, 1] = True
    mask[0, 2, 5:] = True
    mask[1] = True
    mask[2, :, ::3] = True
    got = []
    for value in (-1e29, -float("inf")):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = sv.beam_step(z.masked_fill(mask, value), scores, 8, status=status)
        got.append((out["scores"], out["parent"], out["token"], out["finished"], status))
    for at, inf in zip(*got):
        assert torch.equal(at, inf)


@pytest.mark.parametrize("value", [-1e9, -3e9, -1e10, -7e15, -1e20, -9e28, 2e10])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logits_far_out(dtype, value):
    """Masks of ordinary size (-1e9, -1e20) and whole rows out there."""
    for V in (2003, 40003):
        z, scores, g = _case(4, 4, V, dtype, 79)
        mask = (torch.rand(z.shape, generator=g) < 0.95).to(DEV)
        mask[1, 1] = True
        mask[1, 2] = True
        mask[1, 2, 7:9] = False
        mask[2] = True
        z = z.masked_fill(mask, value)
        z[3, 1] = (value * (1 + torch.rand((V,), generator=g))).to(z)
        _check(z, scores, 8)


@pytest.mark.parametrize("V", [9, 2003, 40003])
@pytest.mark.parametrize("bad", [float("nan"), INF])
def test_spoilt_beams_far_out(V, bad):
    sv = _sv()
    z = torch.full((1, 2, V), -1e20, device=DEV)
    z[0, 1, V // 2] = bad
    scores = torch.tensor([[-1.0, 5.0]], device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = sv.beam_step(z, scores, 3, status=status)
    torch.cuda.synchronize()
    assert int(status) == sv.api.SPEC_ERR_BAD_ROW
    assert out["parent"].tolist() == [[0, 0, 0]] and out["token"].tolist() == [[0, 1, 2]]
