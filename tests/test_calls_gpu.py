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


def test_a_tensor_whose_address_may_not_be_taken(b):
    """As tracers mark theirs: an error, raised under the interpreter's lock."""
    x = torch.randn((4, 8), device="cuda")
    ids, w = b.moe_choose(x, 2)
    q = b.quantize_fp4(x)
    marked, codes = x.clone(), q.codes.clone()
    for t in (marked, codes):
        torch._C._set_throw_on_mutable_data_ptr(t)
    for call in (lambda: b.moe_choose(marked, 2), lambda: b.moe_choose_grad(w, marked, ids), lambda: b.quantize_fp4(marked),
                 lambda: b.gemm_fp4(q._replace(codes=codes), q)):
        with pytest.raises(RuntimeError):
            call()
    assert torch.equal(b.moe_choose(x, 2)[0], ids)
