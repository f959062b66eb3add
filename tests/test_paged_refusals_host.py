"""Refusals of paged_tree_attention, on tensors that claim to be a GPU's: what
its documentation does not allow is a ValueError, of whatever shape it is.  No
CUDA call is made."""
import pytest

torch = pytest.importorskip("torch")
fake_tensor = pytest.importorskip("torch._subclasses.fake_tensor")

import entropy_bounded_softmax_gb300 as cs

# (Their addresses, which the checks look at, are not real.)
pytestmark = pytest.mark.filterwarnings("ignore:.*data pointer.*")


@pytest.fixture
def args():
    with fake_tensor.FakeTensorMode():
        def half(*shape):
            return torch.empty(shape, dtype=torch.bfloat16, device="cuda")

        pages = half(5, 16, 2, 64)
        yield dict(query=half(2, 3, 4, 64), key_pages=pages, value_pages=pages,
                   page_table=torch.zeros(2, 3, dtype=torch.int32,
                                          device="cuda"),
                   lengths=torch.zeros(2, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("shape", [(), (1,), (3,), (9,), (3, 4), (1, 3, 3),
                                   (2, 1, 3, 3)], ids=str)
def test_masks_of_other_shapes(args, shape):
    mask = torch.ones(shape, dtype=torch.bool, device="cuda")
    with pytest.raises(ValueError, match="mask must be"):
        cs.paged_tree_attention(**args, mask=mask)


@pytest.mark.parametrize("T", [0, 3])
@pytest.mark.parametrize("bad", [
    dict(key_pages=None), dict(key_pages=3), dict(value_pages=[1]),
    dict(page_table=None), dict(lengths=None), dict(lengths=7)], ids=str)
def test_arguments_of_other_types(args, T, bad):
    """Also where there is no new token, so that nothing is looked at."""
    args["query"] = args["query"][:, :T]
    with pytest.raises(ValueError):
        cs.paged_tree_attention(**{**args, **bad})
