"""NaN and infinities in the values of nodes that lie on both sides of a tile's end, where a
sequence may be cut into pieces: few sequences (every tile its own piece) and many (cuts
anywhere)."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_tree_attention import BF16, F16, NAN, _case, _check, _i32, _run, _sv  # noqa: E402

pytestmark = pytest.mark.gpu


def _spoil(c, b, n, value, columns):
    t = c["lengths"][b] + n
    c["v"][c["table"][b, t // 16], t % 16, :, columns] = value


def _first(c, got, keep):
    c = dict(c, counts=None)
    for key in ("q", "table"):
        c[key] = c[key][keep]
    for key in ("lengths", "parents", "counts_"):
        c[key] = [c[key][b] for b in keep]
    return c, {x: y[keep] for x, y in got.items()}


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B", [1, 3, 90])
@pytest.mark.parametrize("L,N,Hq,Hkv,D", [(120, 40, 8, 2, 64), (125, 9, 8, 8, 128), (250, 128, 8, 2, 64), (250, 128, 32, 2, 72),
                                          (127, 2, 4, 4, 40), (255, 33, 15, 3, 80), (1, 128, 4, 1, 64)])
def test_early_nodes(B, L, N, Hq, Hkv, D, dtype):
    """The first nodes' values, which lie before the tile's end, and those on both sides of it."""
    sv = _sv()
    c = _case(L + N + B, dtype, N, Hq, Hkv, D, 16, [L + 128 * (b % 5) if B > 3 else L for b in range(B)])
    side = (L // 128 + 1) * 128 - L                 # the first node behind the tile's end
    for b in range(B):
        _spoil(c, b, 0, math.inf, slice(0, 2))
        _spoil(c, b, min(1, N - 1), NAN, slice(5, 6))
        if side < N:
            _spoil(c, b, side, -math.inf, slice(7, 9))
        if 1 < side - 1 < N:
            _spoil(c, b, side - 1, -math.inf, slice(30, 33))
    st = _i32([0])
    got = _run(sv, c, status=st)
    assert int(st) == 0
    assert (got["out"][..., :2] == math.inf).all() and got["out"].isnan().any()      # every node sees node 0
    _check(*_first(c, got, sorted({0, B // 2, B - 1})), D ** -0.5)


def test_pieces_of_no_weight():
    """An infinity in a piece whose probabilities are below fp32's range: the formula's
    probability is not 0, and a cut changes nothing."""
    sv = _sv()
    c = _case(2, BF16, 40, 8, 2, 64, 16, [120])
    c["q"] = torch.ones_like(c["q"])
    c["k"] = torch.where(c["k"].isfinite(), 0.25 * c["k"], c["k"])
    for t in range(128):                            # scores lower by 400
        c["k"][c["table"][0, t // 16], t % 16, :, :8] -= 50.0
    _spoil(c, 0, 0, math.inf, slice(3, 4))
    _spoil(c, 0, 0, NAN, slice(40, 41))
    got = _run(sv, c, scale=1.0)
    assert got["out"].isinf().any()
    _check(c, got, 1.0)
