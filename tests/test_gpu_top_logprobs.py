"""Top log-probabilities on the GPU against the fp64 reference: every length,
alignment, stride, tie and mask where a list can go wrong."""
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


def _poisoned(lead, M):
    return {"logprobs": torch.full(lead + (M,), 3.3e38, device=DEV),
            "ids": torch.full(lead + (M,), 0x7F7F7F7F, dtype=torch.int32, device=DEV),
            "lse": torch.full(lead, 3.3e38, device=DEV)}


def _check(z, M, s=1.0):
    """top_logprobs of z [B, K, V] (any strides) against the reference."""
    sv = _sv()
    lead = tuple(z.shape[:-1])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = sv.top_logprobs(z, M, inv_temperature=s, out=_poisoned(lead, M), status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    rows = z.float().cpu().numpy().reshape(-1, z.shape[-1])
    lp, ids = out["logprobs"].cpu().numpy().reshape(-1, M), out["ids"].cpu().numpy().reshape(-1, M)
    L = out["lse"].cpu().numpy().reshape(-1)
    for r in range(rows.shape[0]):
        want, at, wl, tol, ltol = ref.top(rows[r], M, s)
        np.testing.assert_array_equal(ids[r], at, err_msg=f"row {r}")
        full = at >= 0
        assert np.all(lp[r][~full] == -INF)
        assert np.all(np.abs(lp[r][full] - want[full]) <= tol[full]), (r, lp[r][full] - want[full])
        assert L[r] == wl if wl == -INF else abs(L[r] - wl) <= ltol, (r, L[r], wl)
    return out


def _rows(kind, n, V, g):
    z = 3.0 * torch.randn((n, V), generator=g)
    if kind == "equal":
        z[:] = 1.25
    elif kind == "zeros":           # both signs of zero tie
        z = torch.where(torch.rand((n, V), generator=g) < 0.5, 0.0, -0.0)
    elif kind == "ties":            # few distinct values
        z = torch.round(z)
    elif kind == "two values":      # the list ends inside the larger value's tokens
        z = (torch.rand((n, V), generator=g) < 0.6).float()
    elif kind == "ascending":
        z = torch.sort(z, dim=-1).values
    elif kind == "descending":
        z = torch.sort(z, dim=-1, descending=True).values
    elif kind == "masked":
        z[torch.rand((n, V), generator=g) < 0.9] = -INF
    elif kind == "lowest":          # masks of a type's lowest value
        z[torch.rand((n, V), generator=g) < 0.5] = -3.38e38
    elif kind == "few":             # fewer tokens than places
        keep = torch.rand((n, V), generator=g) < 3.0 / V
        z = torch.where(keep, z, torch.tensor(-INF))
    elif kind == "empty":
        z[::2] = -INF
        z[1::4] = -3.38e38
    elif kind == "spikes":
        z[:, V // 2] += 60.0
    elif kind == "block":           # every large value in one stretch
        z[:, V // 3: V // 3 + max(1, V // 8)] += 30.0
    elif kind == "wide":            # large and small magnitudes
        z = z * 1e4
    return z


KINDS = ["normal", "equal", "zeros", "ties", "two values", "ascending", "descending", "masked", "lowest", "few",
         "empty", "spikes", "block", "wide"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V,M", [(5000, 17), (40000, 128)])
def test_kinds_of_rows(kind, dtype, V, M):
    g = torch.Generator().manual_seed(V + M)
    _check(_rows(kind, 6, V, g).view(2, 3, V).to(DT[dtype]).to(DEV), M)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 33, 63, 65, 127, 129, 1000, 1024, 1025, 4095, 4097])
def test_lengths(V, dtype):
    g = torch.Generator().manual_seed(V)
    for M in (1, 2, 64, 128):
        _check(_rows("normal", 5, V, g).view(5, 1, V).to(DT[dtype]).to(DEV), M)


@pytest.mark.parametrize("rows", [1, 3, 40, 700])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_row_counts(rows, dtype):
    """Few rows are split over several CTAs, many are not."""
    g = torch.Generator().manual_seed(rows)
    V = 32001 if rows > 100 else 128256
    _check(_rows("normal", rows, V, g).view(rows, 1, V).to(DT[dtype]).to(DEV), 50)


@pytest.mark.parametrize("kind", ["equal", "ties", "few", "empty", "block", "ascending"])
def test_split_rows(kind):
    g = torch.Generator().manual_seed(9)
    _check(_rows(kind, 2, 152064, g).view(2, 1, 152064).to(torch.bfloat16).to(DEV), 64)


@pytest.mark.parametrize("s", [1e-4, 0.25, 3.0, 1e4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_temperatures(s, dtype):
    g = torch.Generator().manual_seed(3)
    _check(_rows("normal", 4, 9001, g).view(2, 2, 9001).to(DT[dtype]).to(DEV), 20, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_alignments(dtype):
    g = torch.Generator().manual_seed(4)
    V, M = 1037, 33
    base = _rows("normal", 4 * 5, V + 3, g).view(4, 5, V + 3).to(DT[dtype]).to(DEV)
    for off in range(4):
        _check(base[:, :3, off:off + V], M)          # padded rows, every start
    _check(base[:, :, :V].transpose(0, 1), M)        # batch inside
    _check(base[1:2, :, :V].expand(3, 5, V), M)      # a repeated sequence
    _check(base[:, 2:3, :V].expand(4, 2, V), M)      # a repeated row
    sv = _sv()
    two = sv.top_logprobs(base[:, 0, :V], M)
    three = sv.top_logprobs(base[:, :1, :V], M)
    assert all(torch.equal(two[k], three[k][:, 0]) for k in two)


def test_offsets_beyond_32_bits():
    """Rows that start past 2^32 bytes and 2^31 elements."""
    V = 4096
    z = torch.zeros((2 ** 31 + 10 * V,), dtype=torch.bfloat16, device=DEV)
    rows = z.as_strided((2, 1, V), (2 ** 31 + V + 5, V, 1))
    g = torch.Generator().manual_seed(5)
    rows.copy_(_rows("normal", 2, V, g).view(2, 1, V))
    _check(rows, 16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_longest_rows(dtype):
    """V = 2^20, split over a cluster and, repeated, one CTA a row."""
    sv = _sv()
    V = 1 << 20
    g = torch.Generator().manual_seed(8)
    z = _rows("normal", 2, V, g).view(2, 1, V).to(DT[dtype]).to(DEV)
    z[1, 0, :] = torch.sort(z[1, 0]).values          # ascending: the filter lets everything through
    out = _check(z, 128)
    many = sv.top_logprobs(z.expand(2, 400, V), 128)
    assert torch.equal(many["ids"], out["ids"].expand_as(many["ids"]))
    assert torch.equal(many["logprobs"], many["logprobs"][:, :1].expand_as(many["logprobs"]))


def test_spoilt_rows_stay_alone():
    sv = _sv()
    g = torch.Generator().manual_seed(6)
    V, M = 3001, 8
    z = _rows("normal", 6, V, g).to(DEV)
    clean = sv.top_logprobs(z[:, None], M)
    z2 = z.clone()
    z2[1, 77] = float("nan")
    z2[4, 5] = INF
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = sv.top_logprobs(z2[:, None], M, status=status)
    torch.cuda.synchronize()
    assert int(status) == sv.api.SPEC_ERR_BAD_ROW
    for r in (0, 2, 3, 5):
        assert all(torch.equal(out[k][r], clean[k][r]) for k in out)
    for r in (1, 4):
        assert not torch.isfinite(out["lse"][r]).any()
        assert not torch.isfinite(out["logprobs"][r]).any()
        assert ((out["ids"][r] >= -1) & (out["ids"][r] < V)).all()


def test_none_rows_and_repeats():
    sv = _sv()
    z = torch.randn((0, 4, 100), device=DEV)
    out = sv.top_logprobs(z, 5)
    assert out["ids"].shape == (0, 4, 5)
    z = torch.randn((3, 4, 20000), device=DEV)
    a, b = sv.top_logprobs(z, 100), sv.top_logprobs(z, 100)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_other_stream_and_graph():
    sv = _sv()
    z = torch.randn((4, 3, 30000), device=DEV)
    want = sv.top_logprobs(z, 40)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sv.top_logprobs(z, 40, stream=s)
    s.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    g = torch.cuda.CUDAGraph()
    zz = z.clone()
    with torch.cuda.graph(g):
        out = sv.top_logprobs(zz, 40)
    zz.copy_(z.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], want[k].flip(0)) for k in want)


@pytest.mark.parametrize("V", [3, 1037, 40003])
def test_logits_at_the_mask_floor_are_masked(V):
    """fp32 -1e29 as a mask value gives what -inf gives, to the bit."""
    sv = _sv()
    g = torch.Generator().manual_seed(77)
    z = 3.0 * torch.randn((6, V), generator=g).to(DEV)
    mask = torch.zeros_like(z, dtype=torch.bool)
    mask[0] = True
    mask[1, 1:] = True
    mask[2, ::2] = True
    mask[3, : V // 2] = True
    a = sv.top_logprobs(z.masked_fill(mask, -1e29), 8)
    b = sv.top_logprobs(z.masked_fill(mask, -INF), 8)
    for key in ("logprobs", "ids", "lse"):
        assert torch.equal(a[key], b[key]), key


@pytest.mark.parametrize("s", [0.05, 1.0, 20.0])
@pytest.mark.parametrize("value", [-1e9, -3e9, -1e10, -7e15, -1e20, -9e28, 2e10])
def test_logits_far_out(value, s):
    """Masks of ordinary size (-1e9, -1e20) and whole rows out there."""
    for dtype, V, n in (("f32", 1037, 1), ("bf16", 40003, 1), ("bf16", 40003, 120)):
        g = torch.Generator().manual_seed(34)
        z = 3.0 * torch.randn((n, 5, V), generator=g)
        mask = torch.rand(z.shape, generator=g) < 0.95
        mask[:, 1] = True
        mask[:, 1, 5:9] = False
        mask[:, 2] = True
        mask[:, 2, -1] = False
        mask[:, 3] = True
        z = z.masked_fill(mask, value)
        z[:, 4] = value * (1 + torch.rand((n, V), generator=g))
        _check(z.to(DT[dtype]).to(DEV), 16, s)


@pytest.mark.parametrize("s", [1e-4, 1e4])
def test_extreme_temperatures(s):
    for dtype, V, n in (("f32", 1037, 2), ("bf16", 40003, 2), ("f32", 40003, 130)):
        z = 3.0 * torch.randn((n, 5, V), generator=torch.Generator().manual_seed(36))
        _check(z.to(DT[dtype]).to(DEV), 16, s)


@pytest.mark.parametrize("V", [9, 1037, 40003])
@pytest.mark.parametrize("bad", [float("nan"), INF])
def test_spoilt_rows_far_out(V, bad):
    sv = _sv()
    z = torch.full((3, V), -1e20, device=DEV)
    z[1, V // 2] = bad
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = sv.top_logprobs(z, 4, status=status)
    torch.cuda.synchronize()
    assert int(status) == sv.api.SPEC_ERR_BAD_ROW and not torch.isfinite(out["lse"][1])
    for r in (0, 2):
        assert out["ids"][r].tolist() == [0, 1, 2, 3]
        assert torch.equal(out["logprobs"][r], out["logprobs"][r, :1].expand(4))
        assert abs(float(out["logprobs"][r, 0]) + np.log(V)) <= ref.DS + 4 * ref.U * np.log(V)
