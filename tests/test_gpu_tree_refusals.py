"""Sizes at the ends of what the tree operators' binding can be asked for are refused as the
library refuses them."""
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


@pytest.mark.parametrize("scale", [None, 1.0])
def test_heads_of_no_elements(scale):
    sv = _sv()
    q, k = torch.empty((1, 2, 4, 0), dtype=torch.bfloat16, device=DEV), torch.empty((3, 16, 2, 0), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(sv.SpecError) as e:
        sv.tree_attention(q, k, k, _i32([[0, 1]]), _i32([5]), scale=scale)
    assert e.value.code == sv.api.SPEC_ERR_UNSUPPORTED


@pytest.mark.parametrize("page,code", [(0, 1), (-1, 1), (-(1 << 31), 2), (16 - (1 << 32), 2), ((1 << 32) + 16, 2), (1 << 31, 2)])
def test_pages_of_no_size(page, code):
    sv = _sv()
    table, refs = _i32([[0, -1]]), _i32([1, 0, 0])
    with pytest.raises(sv.SpecError) as e:
        sv.pages_resize(table, refs, _i32([20]), page, out={"table": table, "refs": refs})
    assert e.value.code == code
    assert table.tolist() == [[0, -1]] and refs.tolist() == [1, 0, 0]
