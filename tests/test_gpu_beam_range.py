"""Beam steps whose scores leave fp32's range, or come near its ends."""
from fractions import Fraction

import numpy as np
import pytest

import rows_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = float("inf")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,N", [(9, 8), (2003, 12), (40003, 12), (40003, 64)])
def test_scores_below_the_range_count_as_none(V, N, dtype):
    """Beam 0 at -1e38 has one token at 3e38: every other continuation of it
    would lie near -4e38. Beam 1 has three tokens, beam 2 none."""
    import speculative_decoding_token_verify_gb300 as sv
    sv.build()
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    B = 3
    z = torch.randn((B, 3, V), generator=torch.Generator().manual_seed(V)).to(dt)
    z[:, 0, 5] = 3e38
    z[:, 1, 3:] = -INF
    z[:, 2] = -INF
    scores = torch.tensor([[-1e38, -2.0, -1.0]] * B)
    scores[1, 0] = -3.4e38
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = sv.beam_step(z.to(DEV), scores.to(DEV), N, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    o = {k: v.cpu().numpy() for k, v in got.items()}
    for b in range(B):
        live = z[b, 1].float().numpy()
        sc, par, tok, _, tol = ref.beam(live[None], scores[b, 1:2].numpy(), 3)
        want_parent = [1, 1, 1, 0] + [-1] * (N - 4)
        want_token = tok.tolist() + [5] + [-1] * (N - 4)
        np.testing.assert_array_equal(o["parent"][b], want_parent)
        np.testing.assert_array_equal(o["token"][b], want_token)
        assert np.all(np.abs(o["scores"][b, :3] - sc) <= tol)
        assert o["scores"][b, 3] == np.float32(scores[b, 0]) and np.all(o["scores"][b, 4:] == -INF)
        assert not o["finished"][b].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,N", [(4, 8), (9, 24), (300, 64), (4099, 8), (40003, 64)])
def test_logits_near_the_mask_floor(V, N, dtype):
    """Fill values just above -1e29 are logits: a beam of nothing else, whose
    maximum lies there, says nothing about the others' fills, which are listed
    where places are left (V = 4, 9: all continuations fit)."""
    import speculative_decoding_token_verify_gb300 as sv
    sv.build()
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    z = torch.full((3, V), -9.9e28).to(dt)
    z[0, 3] = -4.1875
    z[2, 3] = -4.1875
    z[2, :2] = -float("inf")
    scores = torch.tensor([-4.75, -2.5, -1.375])
    got = sv.beam_step(z[None].to(DEV), scores[None].to(DEV), N)
    # in exact arithmetic: at this size fp64 scores of the three beams round alike
    pool = []
    for w in range(3):
        m, lnS = ref.max_lnsum(z[w].float().numpy())
        for v in range(V):
            x = float(z[w, v].float())
            if x > -INF:
                pool.append((Fraction(m) + Fraction(lnS) - Fraction(x) - Fraction(float(scores[w])), w * V + v))
    pool = sorted(pool)[:N]
    want = [p for _, p in pool] + [-1] * (N - len(pool))
    place = torch.where(got["parent"] < 0, -1, got["parent"] * V + got["token"])[0].tolist()
    assert place == want
    sc = np.array([-float(s) for s, _ in pool])
    off = np.abs(got["scores"][0, :len(pool)].cpu().double().numpy() - sc)
    assert np.all(off <= ref.DS + 2 * ref.U * np.abs(sc))
