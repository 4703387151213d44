"""Calls on caches that are refused leave everything as it was."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _sv():
    import speculative_decoding_token_verify_gb300 as sv
    sv.build()
    return sv


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("several", [False, True])
@pytest.mark.parametrize("kind", ["pages over one another", "outer entries over one another", "outer axis too long"])
def test_fork_refused_before_it_writes(kind, several):
    """One cache or two whose pages the copy cannot move: tables, counts and lengths stay."""
    sv = _sv()
    if kind == "pages over one another":
        cache, pd = torch.zeros((1, 16, 4), device=DEV).expand(6, 16, 4), 0
    elif kind == "outer entries over one another":
        cache, pd = torch.zeros((1, 6, 16, 4), device=DEV).expand(3, 6, 16, 4), 1
    else:
        cache, pd = torch.zeros((65536, 6, 16, 1), dtype=torch.uint8, device=DEV), 1
    table, refs, lengths, parent = _i32([[[0, 1], [2, 3]]]), _i32([1, 1, 1, 1, 0, 0]), _i32([[20, 20]]), _i32([[1, 1]])
    out = {"table": torch.full((1, 2, 2), 77, dtype=torch.int32, device=DEV), "refs": refs,
           "lengths": torch.full((1, 2), 77, dtype=torch.int32, device=DEV)}
    versions = [t._version for t in out.values()]
    caches = [torch.zeros_like(cache, memory_format=torch.contiguous_format), cache] if several else cache
    if several and kind == "outer axis too long":
        caches[0] = torch.zeros((6, 6, 16, 1), dtype=torch.uint8, device=DEV)
    with pytest.raises(sv.SpecError):
        sv.pages_fork(caches, table, refs, lengths, parent, page_dim=pd, out=out)
    assert refs.tolist() == [1, 1, 1, 1, 0, 0] and (out["table"] == 77).all() and (out["lengths"] == 77).all()
    assert [t._version for t in out.values()] == versions
    # the same call on a cache that it takes
    good = torch.zeros((6, 16, 4), device=DEV)
    r = sv.pages_fork(good, table, refs, lengths, parent, out=out)
    assert r["refs"] is refs and int(refs.sum()) == 4 and r["lengths"].tolist() == [[20, 20]]


@pytest.mark.parametrize("call", ["compact", "fork"])
def test_caches_over_one_another(call):
    """Caches that share some layers, from different first bytes on, and views between one another."""
    sv = _sv()
    layers = torch.randn((4, 2, 6, 16, 2, 8), device=DEV)          # [layer, keys and values, page, slot, head, D]
    kept = layers.clone()
    table, refs, lengths = _i32([[[0, 1], [2, 3]]]), _i32([1, 1, 1, 1, 0, 0]), _i32([[20, 20]])

    def run(caches, page_dim):
        if call == "compact":
            return sv.pages_compact(caches, table[0], lengths[0], _i32([[1, 3, -1, -1], [0, 2, 3, -1]]), page_dim=page_dim)
        return sv.pages_fork(caches, table, refs, lengths, _i32([[1, 1]]), page_dim=page_dim)

    for caches, pd in (([layers[0:2], layers[1:3]], 2), ([layers[:, 0], layers[2:, 0]], 1), ([layers, layers[3:]], 2)):
        with pytest.raises(ValueError, match="overlap"):
            run(caches, pd)
        assert torch.equal(layers, kept)
    one = layers.clone()
    run(one, 2)
    assert not torch.equal(one, layers)
    for caches, pd in (([layers[:, 0], layers[:, 1]], 1), ([layers[3:], layers[:3]], 2), ([layers[i, j] for j in (1, 0) for i in range(4)], 0)):
        layers.copy_(kept)
        run(caches, pd)
        assert torch.equal(layers, one)
    mixed = kept.permute(2, 0, 1, 3, 4, 5).contiguous()             # pages first, the layers between one another
    run([mixed[:, i, j] for i in range(4) for j in range(2)], 0)
    assert torch.equal(mixed, one.permute(2, 0, 1, 3, 4, 5))


@pytest.mark.parametrize("path,length,table,code", [
    ([0, 1, 2, 3], 15, [0, -1], 10), ([0, 1, 2, 3], 15, [0, 9], 10), ([0, 1, 2, 3], 30, [0, 1], 10), ([0, 1, -1, -1], 30, [0, 1], 0),
    ([0, 1, 3, -1], 13, [0, 1], 0), ([0, 1, 3, -1], 15, [0, -1], 10), ([0, -1, -1, -1], 15, [0, -1], 0), ([-1, -1, -1, -1], 32, [0, 1], 0),
    ([0, -1, -1, -1], 32, [0, 1], 10), ([0, 1, 2, 3], 16, [-1, 1], 0)])
def test_compact_without_a_page(path, length, table, code):
    """Kept nodes without a page, moved or not: the status tells, the lengths count them."""
    sv = _sv()
    cache = torch.arange(48, device=DEV).to(torch.int32).view(3, 16, 1)
    want, kept = cache.clone(), sum(p >= 0 for p in path)
    for i in range(kept):
        a, z = length + path[i], length + i
        if a // 16 < 2 and 0 <= table[a // 16] < 3 and 0 <= table[z // 16] < 3:
            want[table[z // 16], z % 16] = cache[table[a // 16], a % 16]
    st = _i32([0])
    r = sv.pages_compact(cache, _i32([table]), _i32([length]), _i32([path]), status=st)
    assert int(st) == code and r.tolist() == [length + kept] and torch.equal(cache, want)
