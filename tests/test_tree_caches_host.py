"""Caches of one call that lie over one another, on the CPU: every pair of layouts against the
set of its bytes."""
import itertools
import random

import pytest
import torch

from speculative_decoding_token_verify_gb300 import tree


def _layouts(tensors, page_dim, slot_dim=None):
    return [tree._layout(t, tree._cache_params(t, page_dim, slot_dim, None, None)) for t in tensors]


def _bytes(x):
    first, extent, axes, seg = x
    starts = [first]
    for s, n in axes:
        starts = [b + s * i for b in starts for i in range(n)]
    got = {b + i for b in starts for i in range(seg)}
    assert max(got) - first + 1 == extent and len(got) == len(starts) * seg
    return got


def test_views_of_one_buffer():
    layers = torch.zeros((4, 2, 6, 16, 3, 8), dtype=torch.float16)          # [layer, keys and values, page, slot, head, D]
    between = torch.zeros((6, 4, 2, 16, 3, 8), dtype=torch.float16)         # pages first
    heads = torch.zeros((6, 3, 16, 20), dtype=torch.float16)                # [page, head, slot, elements]
    good = [([layers[i, j] for i in range(4) for j in range(2)], 0, None), ([layers[:, 0], layers[:, 1]], 1, None),
            ([layers[:2], layers[2:]], 2, None), ([between[:, i, j] for i in range(4) for j in range(2)], 0, None),
            ([between[:, :2], between[:, 2:]], 0, 3), ([between[:, :1], between[:, 1:]], 0, 3),
            ([heads[:, :2], heads[:, 2:]], 0, 2), ([heads[:, 0], heads[:, 1:], torch.zeros_like(heads)], 0, -2),
            ([layers[0, 0], torch.zeros_like(layers[0, 0]), layers[3, 1]], 0, None)]
    bad = [([layers, layers], 2, None), ([layers[:2], layers[1:3]], 2, None), ([layers[:3], layers[2:]], 2, None),
           ([layers[:, 0], layers[1:, 0]], 1, None), ([layers[:, 0], layers[2:]], 2, 3), ([between[:, :3], between[:, 2:]], 0, 3),
           ([heads[:, :2], heads[:, 1:]], 0, 2), ([layers[0, 0], layers[1, 0], layers[0, 1], layers[:1, 0]], 0, None)]
    for tensors, pd, sd in good:
        assert tree._apart(_layouts(tensors, pd, sd)), [t.shape for t in tensors]
        assert tree._blocks(tensors) <= tree._apart(_layouts(tensors, pd, sd))
    for tensors, pd, sd in bad[:4] + bad[5:7]:
        assert not tree._blocks(tensors) and not tree._apart(_layouts(tensors, pd, sd)), [t.shape for t in tensors]
    a, b = _layouts([layers[:, 0]], 1), _layouts([layers[2:]], 2)            # the pages along different axes
    assert not tree._apart(a + b)
    a, b = _layouts([layers[i, j] for i in (0, 1) for j in (0, 1)], 0), _layouts([layers[:1, 0]], 1)
    assert tree._apart(a) and not tree._apart(a + b) and not tree._apart(b + a)
    assert tree._blocks([layers[i, j] for i in range(4) for j in range(2)]) and not tree._blocks([layers[0, 0], layers[0, 0]])


def test_against_the_bytes():
    rng = random.Random(1)
    seen = {True: 0, False: 0}
    for _ in range(3000):
        made = []
        for _ in range(rng.randint(2, 4)):
            seg, axes, extent = rng.randint(1, 6), [], 0
            extent = seg
            for _ in range(rng.randint(0, 3)):
                s, n = extent + rng.choice([0, 0, 1, 5, 12, 30]), rng.randint(2, 4)
                axes.insert(0, (s, n))
                extent += s * (n - 1)
            made.append((1000 + rng.randint(0, 60), extent, axes, seg))
        if rng.random() < 0.5:       # one layout, moved
            made = [(1000 + rng.randint(0, 80),) + made[0][1:] for _ in made]
        sets = [_bytes(x) for x in made]
        want = not any(a & b for a, b in itertools.combinations(sets, 2))
        got = tree._apart(made)
        assert got == want, made
        seen[want] += 1
    assert min(seen.values()) > 300


def test_many_layers_take_no_search(monkeypatch):
    """A cache per layer, as tensors of their own or views of one: sorted, not compared in pairs."""
    monkeypatch.setattr(tree, "_meet", lambda a, b: pytest.fail("compared"))
    page = 2 * 16 * 8 * 128
    own = [(4096 + i * 50 * page, 50 * page, [(page, 50)], page) for i in range(160)]
    between = [(4096 + i * page, 49 * 160 * page + page, [(160 * page, 50)], page) for i in range(160)]
    for x in (own, between):
        random.Random(0).shuffle(x)
        assert tree._apart(x)
