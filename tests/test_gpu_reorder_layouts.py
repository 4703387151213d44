"""Reordering whole rows (no lengths) of states cut out of larger buffers: any
axis behind the beam may be the one that is not full."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _sv():
    import speculative_decoding_token_verify_gb300 as sv
    sv.build()
    return sv


def _want(state, parent, bd):
    """The reordered state by indexing."""
    new = state.clone()
    for b in range(parent.shape[0]):
        for n in range(parent.shape[1]):
            p = int(parent[b, n])
            if p >= 0:
                new.select(bd, b).select(bd, n).copy_(state.select(bd, b).select(bd, p))
    return new


CUTS = {
    "tokens": ((2, 3, 4, 5, 11, 8), 1, lambda t: t[:, :, :, :, :7]),          # [L, B, W, H, T of Tmax, D]
    "tokens, no layers": ((3, 4, 5, 11, 6), 0, lambda t: t[:, :, :, 2:9]),
    "tokens first": ((2, 3, 4, 11, 5, 8), 1, lambda t: t[:, :, :, :7]),      # [L, B, W, T of Tmax, H, D]
    "heads": ((2, 3, 4, 6, 7, 8), 1, lambda t: t[:, :, :, 1:5]),
    "units": ((2, 3, 4, 5, 7, 9), 1, lambda t: t[..., :8]),
    "two head axes": ((3, 4, 2, 5, 9, 2, 8), 0, lambda t: t[:, :, :, :, :6]),
    "beams": ((2, 3, 6, 5, 7, 8), 1, lambda t: t[:, :, 1:5]),
    "history": ((3, 4, 12), 0, lambda t: t[:, :, :7]),
    "one token": ((2, 3, 4, 5, 11, 8), 1, lambda t: t[:, :, :, :, 3:4]),
}


@pytest.mark.parametrize("cut", list(CUTS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int32])
def test_states_cut_out_of_buffers(cut, dtype):
    sv = _sv()
    shape, bd, view = CUTS[cut]
    g = torch.Generator().manual_seed(1)
    buf = torch.randint(-99, 99, shape, generator=g).to(dtype).to(DEV)
    keep = buf.clone()
    state = view(buf)
    parent = torch.tensor([[1, 0, 3, 3], [2, 2, -1, 0], [0, 1, 2, 3]], dtype=torch.int32, device=DEV)
    want = _want(state, parent, bd)
    out = torch.zeros_like(buf)
    got = sv.beam_reorder(state, parent, batch_dim=bd, out=view(out).copy_(state))      # out of place, cut alike
    assert torch.equal(got, want)
    dense = torch.empty(state.shape, dtype=dtype, device=DEV).copy_(state)              # into a dense tensor
    assert torch.equal(sv.beam_reorder(state, parent, batch_dim=bd, out=dense), want)
    assert torch.equal(buf, keep)
    back = view(out).copy_(state)                                                       # and from one
    assert torch.equal(sv.beam_reorder(state.contiguous(), parent, batch_dim=bd, out=back), want)
    view(keep).copy_(want)
    assert sv.beam_reorder(state, parent, batch_dim=bd) is state                        # in place
    assert torch.equal(buf, keep)                                                       # nothing beside it


def test_many_heads_and_tokens():
    """More heads times tokens than a call has segments for."""
    sv = _sv()
    buf = torch.randint(-99, 99, (1, 2, 40, 2100, 8), dtype=torch.int8, device=DEV)
    state = buf[:, :, :, :2000]
    parent = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
    want = state.flip(1)
    sv.beam_reorder(state, parent)
    assert torch.equal(state, want)


def test_states_that_no_axis_splits_are_refused():
    sv = _sv()
    t = torch.zeros((2, 2, 4, 6, 8, 10), device=DEV)
    parent = torch.zeros((2, 2), dtype=torch.int32, device=DEV)
    for bad in (t[:, :, ::2, :3, :5], t[..., ::2], t.transpose(3, 5)):
        with pytest.raises(ValueError):
            sv.beam_reorder(bad, parent)
    with pytest.raises(ValueError):
        sv.beam_reorder(torch.zeros((2, 2, 4, 6, 8, 10), device=DEV), parent, out=t.transpose(3, 5).expand(2, 2, 4, 10, 8, 6))


def test_views_that_stand_for_other_values_are_refused():
    """A conjugated or negated view's memory is not its values."""
    sv = _sv()
    parent = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
    z = torch.randn((1, 2, 5), dtype=torch.complex64, device=DEV)
    with pytest.raises(ValueError):
        sv.beam_reorder(z.conj(), parent, out=torch.empty_like(z))
    with pytest.raises(ValueError):
        sv.beam_reorder(torch._neg_view(z.real.contiguous()), parent, out=torch.empty((1, 2, 5), device=DEV))
    want = z.flip(1)
    w = z.conj()
    assert torch.equal(sv.beam_reorder(w, parent), want.conj()) and torch.equal(z, want)   # both alike: in place
