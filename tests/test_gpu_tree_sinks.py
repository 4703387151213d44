"""Long contexts behind one large score: thousands of probabilities far below a row's largest
still make up a part of its output. (Many sequences over one prompt's pages, so that a CTA walks whole
contexts: pieces of few tiles have a reference each.)"""
import math

import pytest

torch = pytest.importorskip("torch")
import numpy as np  # noqa: E402

from test_gpu_tree_attention import BF16, DEV, F16, _case, _i32, _sv  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("place", ["first token", "middle", "node"])
@pytest.mark.parametrize("nats", [12.0, 17.0, 20.0])
@pytest.mark.parametrize("N,D", [(1, 64), (40, 128)])
def test_one_large_score(dtype, place, nats, N, D):
    """One key `nats` above 32767 others, its own value 0."""
    sv = _sv()
    B, L, Hq, Hkv = 40, 32768 - (place == "node"), 32, 8
    c = _case(int(nats) + N, dtype, N, Hq, Hkv, D, 64, [L], kind="roots", poison=False)
    c["q"], c["k"] = torch.zeros_like(c["q"]), torch.zeros_like(c["k"])
    c["q"][..., 0] = 1.0
    c["v"] = (1.0 + 0.25 * c["v"].float()).to(dtype)
    for t in {"first token": [0], "middle": [20011], "node": list(range(L, L + N))}[place]:
        c["k"][c["table"][0, t // 64], t % 64, :, 0] = nats          # (exact in both types)
        c["v"][c["table"][0, t // 64], t % 64] = 0.0
    got = sv.tree_attention(c["q"].to(DEV).expand(B, -1, -1, -1).contiguous(), c["k"].to(DEV), c["v"].to(DEV),
                            c["table"].to(DEV).expand(B, -1).contiguous(), _i32([L] * B), _i32(c["parents"][0]), scale=1.0)
    out, lse = got["out"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
    at = c["table"][0].long()
    v, s = (c[x][at].double().reshape(-1, Hkv, D).numpy() for x in ("v", "k"))
    w = np.exp(s[:L + N, 0, 0] - nats)
    u = torch.finfo(dtype).eps / 2
    W0, sum0, abs0, all0 = w[:L].sum(), np.tensordot(w[:L], v[:L], 1), np.tensordot(w[:L], np.abs(v[:L]), 1), np.abs(v[:L]).sum(0)
    for n in range(N):
        W, own = W0 + w[L + n], v[L + n]
        want, mean, every = (sum0 + w[L + n] * own) / W, (abs0 + w[L + n] * np.abs(own)) / W, (all0 + np.abs(own)) / W
        # the scores are exact. Roundings: the output's (and fp16's least step), each probability's, 2^x's
        # (2^-21), sums over the keys in fp32; in fp16 a probability's is at least half of
        # 2^-24 where the largest is at least 2^7
        rel = u + 2.0 ** -21 + (64 + L / 16) * 2.0 ** -23
        tol = u * want + rel * mean * (1 + u) + ((2.0 ** -25 + 2.0 ** -32 * every) if dtype == F16 else 0)
        d = np.abs(out[:, n] - np.repeat(want, Hq // Hkv, 0))
        assert (d <= np.repeat(tol, Hq // Hkv, 0)).all(), (n, (d / np.repeat(want, Hq // Hkv, 0)).max())
        assert np.abs(lse[:, n] - (nats + math.log(W))).max() <= 2.0 ** -21 + (64 + L / 16) * 2.0 ** -24 + 2.0 ** -22 * 40
