"""Scores of any size that fp32 holds: one-hot rows, ties and near ties at 2^13 to 2^100. The products
are exact (powers of two), so that the 64-bit softmax of the same scores is what the
formula asks for."""
import math

import pytest

torch = pytest.importorskip("torch")
import numpy as np  # noqa: E402

from test_gpu_tree_attention import BF16, DEV, F16, _case, _i32, _sv  # noqa: E402

pytestmark = pytest.mark.gpu

SIZES = [(BF16, e) for e in (13, 24, 31, 40, 100)] + [(F16, e) for e in (13, 24, 30)]


@pytest.mark.parametrize("dtype,e", SIZES, ids=lambda x: str(x).replace("torch.", ""))
@pytest.mark.parametrize("kind", ["ties", "near ties", "rising", "falling", "shuffled"])
@pytest.mark.parametrize("B,N,L", [(1, 5, 900), (30, 5, 900), (40, 40, 300)])
@pytest.mark.parametrize("sign,scale", [(1, 1.0), (-1, 0.6), (1, -0.6)])
def test_far_scores(dtype, e, kind, B, N, L, sign, scale):
    sv = _sv()
    Hq, Hkv, D = 8, 2, 64
    g = torch.Generator().manual_seed(e + N)
    c = _case(e + N, dtype, N, Hq, Hkv, D, 16, [L], kind="roots", poison=False)
    T = L + N
    up = 15 if dtype == F16 and e > 16 else e // 2
    q, k = torch.zeros_like(c["q"]), torch.zeros_like(c["k"])
    q[..., 0], q[..., 1] = sign * 2.0 ** (e - up), 2.0 ** (e - 20)
    first, second = torch.full((T,), 2.0 ** up), torch.zeros(T)
    if kind == "near ties":
        second = torch.randint(0, 4, (T,), generator=g).float()
    elif kind != "ties":         # numbers of the type itself, every one of them, below 2^up
        one = torch.tensor([2.0 ** up], dtype=dtype).view(torch.int16)
        first = (one - (T - 1) + torch.arange(T, dtype=torch.int16)).view(dtype).float()
        first = first.flip(0) if kind == "falling" else first[torch.randperm(T, generator=g)] if kind == "shuffled" else first
    at = c["table"][0].long()
    place = at[torch.arange(T) // 16], torch.arange(T) % 16
    k[..., 0][place] = first.to(dtype)[:, None].expand(T, Hkv)
    k[..., 1][place] = second.to(dtype)[:, None].expand(T, Hkv)
    q[:, 1::3, 3] = 0.0                                              # rows of ordinary scores between them
    got = sv.tree_attention(q.to(DEV).expand(B, -1, -1, -1).contiguous(), k.to(DEV), c["v"].to(DEV),
                            c["table"].to(DEV).expand(B, -1).contiguous(), _i32([L] * B), _i32(c["parents"][0]), scale=scale)
    out, lse = got["out"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
    v = c["v"][at].double().reshape(-1, Hkv, D)[:T].numpy()
    f32 = float(np.float32(scale))
    u = torch.finfo(dtype).eps / 2
    for n in range(N):
        see = list(range(L)) + [L + n]
        for h in range(Hq):
            s = f32 * (float(q[0, n, h, 0]) * first.double() + float(q[0, n, h, 1]) * second.double()).numpy()[see]
            w = np.exp(s - s.max())
            W, vv = w.sum(), v[see, h // 4]
            want, mean, every = w @ vv / W, w @ np.abs(vv) / W, np.abs(vv).sum(0) / W
            # as for ordinary scores, and 2^-24 of an exponent of up to 40, and where scores do not
            # differ from their reference by subtraction (2^12 and below) a reference's rounding
            rel = u + 2.0 ** -18 + 2.0 ** -11 + (64 + len(see) / 16) * 2.0 ** -23
            tol = u * np.abs(want) + rel * mean * (1 + u) + ((2.0 ** -25 + 2.0 ** -32 * every) if dtype == F16 else 0)
            d = np.abs(out[:, n, h] - want)
            assert (d <= tol).all(), (n, h, np.nanmax(d), np.isnan(out[:, n, h]).any())
            assert (np.abs(lse[:, n, h] - (s.max() + math.log(W))) <= 2.0 ** -22 * abs(s.max()) + 2.0 ** -11).all(), (n, h)
