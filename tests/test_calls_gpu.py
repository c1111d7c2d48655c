"""Arguments that the extension module reads itself."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    from tiled_staged_matmul_gb300 import binding
    return binding


def test_a_truth_value_that_raises(b):
    class Neither:
        def __bool__(self):
            raise ValueError("neither")

    x = torch.randn((4, 8), device="cuda")
    ids, w = b.moe_choose(x, 2, renormalize=1)
    for flag, text in ((Neither(), "neither"), (torch.ones(2), "ambiguous")):
        with pytest.raises((ValueError, RuntimeError), match=text):
            b.moe_choose(x, 2, renormalize=flag)
        with pytest.raises((ValueError, RuntimeError), match=text):
            b.moe_choose_grad(w, x, ids, renormalize=flag)
    assert torch.equal(b.moe_choose(x, 2, renormalize=torch.ones(1))[1], w)
