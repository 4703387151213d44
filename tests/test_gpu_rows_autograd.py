"""The row operators' writes into tensors of the caller's move the version
counter that autograd checks, whichever alias was handed over."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _sv():
    import speculative_decoding_token_verify_gb300 as sv
    sv.build()
    return sv


def _lists(B, K, V, M, seed):
    g = torch.Generator().manual_seed(seed)
    t = 2 * torch.randn((B, K, V), generator=g)
    val, at = torch.topk(torch.log_softmax(t, -1), M, dim=-1)
    return (t + torch.randn(t.shape, generator=g)).to(DEV), val.to(DEV), at.to(torch.int32).to(DEV)


def _write(kind, z):
    """One call that overwrites z [2, 3, 40] through a detached alias."""
    sv = _sv()
    y, lp, ids = _lists(2, 3, 40, 4, 1)
    out = z.detach()
    if kind == "step":
        sv.distill_step(out, lp, ids, out={"dlogits": out})
    elif kind == "grad":
        a = sv.distill_loss(y, lp, ids)
        sv.distill_grad(y, lp, ids, a["stats"], out=out)
    elif kind == "reorder":
        sv.beam_reorder(out, torch.tensor([[1, 0, 2], [0, 0, 1]], dtype=torch.int32, device=DEV))
    elif kind == "reorder out":
        sv.beam_reorder(y, torch.tensor([[1, 0, 2], [0, 0, 1]], dtype=torch.int32, device=DEV), out=out)
    elif kind == "top":
        sv.top_logprobs(y, 40, out={"logprobs": out})
    elif kind == "loss":
        sv.distill_loss(y, lp, ids, out={"loss": out.view(-1)[:6].view(2, 3)})
    elif kind == "beam":
        sv.beam_step(y, torch.zeros((2, 3), device=DEV), 3, out={"scores": out.view(-1)[:6].view(2, 3)})


@pytest.mark.parametrize("kind", ["step", "grad", "reorder", "reorder out", "top", "loss", "beam"])
def test_writes_through_a_detached_alias_are_seen(kind):
    x = _lists(2, 3, 40, 4, 2)[0].requires_grad_()
    z = x.tanh()                          # keeps its result for the backward pass
    _write(kind, z)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.sum().backward()


def test_a_tensor_without_gradient_that_another_tensor_s_backward_keeps():
    sv = _sv()
    cache = torch.randn((2, 3, 8), device=DEV)
    w = torch.randn((8, 5), device=DEV, requires_grad=True)
    y = cache @ w                         # keeps the cache
    sv.beam_reorder(cache, torch.tensor([[1, 0, 2], [0, 0, 1]], dtype=torch.int32, device=DEV))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_calls_that_write_nothing_leave_the_counter():
    """Inputs, and tensors handed to a call that is refused."""
    sv = _sv()
    y, lp, ids = _lists(2, 3, 40, 4, 3)
    bad = torch.zeros((2, 3, 40), device=DEV).expand(2, 3, 40)
    over = torch.zeros((40,), device=DEV).expand(2, 3, 40)
    was = [t._version for t in (y, lp, ids, bad, over)]
    sv.distill_step(y, lp, ids)
    sv.top_logprobs(y, 5)
    sv.beam_reorder(y, torch.zeros((2, 3), dtype=torch.int32, device=DEV), out=torch.empty_like(y))
    loss = torch.zeros((2, 3), device=DEV)
    with pytest.raises(sv.SpecError):
        sv.distill_step(y, lp, ids, out={"loss": loss, "dlogits": over})   # rows over one another
    with pytest.raises(sv.SpecError):
        sv.beam_reorder(over, torch.zeros((2, 3), dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        sv.distill_loss(y, lp, ids, out={"loss": loss, "stats": bad})
    torch.cuda.synchronize()
    assert [t._version for t in (y, lp, ids, bad, over)] == was and loss._version == 0


def test_inference_tensors():
    sv = _sv()
    parent = torch.tensor([[1, 0, 2], [0, 0, 1]], dtype=torch.int32, device=DEV)
    with torch.inference_mode():
        s = torch.randn((2, 3, 8), device=DEV)
        want = torch.gather(s, 1, parent.long()[..., None].expand_as(s))
        sv.beam_reorder(s, parent)
        assert torch.equal(s, want)
    want = torch.gather(s, 1, parent.long()[..., None].expand_as(s))
    sv.beam_reorder(s, parent)
    assert torch.equal(s, want)
