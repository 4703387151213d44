"""Beam steps whose scores leave fp32's range."""
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
