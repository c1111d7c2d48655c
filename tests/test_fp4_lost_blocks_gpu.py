"""Quantisation of rows whose neighbouring blocks end in every way: codes are kept in
some lanes of a warp and dropped in others.  Compared code by code with the definition
in 64 bits."""
import pytest
import torch

from test_fp4_gpu import TORCH, b, check_quantised  # noqa: F401  (b: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("M,K", [(40, 1), (40, 47), (33, 1024), (9, 2050), (5, 4097), (3, 16384)])
def test_blocks_of_every_kind_side_by_side(b, M, K, dtype, block):  # noqa: F811
    """Ordinary values, zeros, values that round to a block scale of 0 beside the row's
    largest, and (in blocks of 32, where they take their block alone) what is not finite."""
    g = torch.Generator().manual_seed(M + K)
    units = -(-K // 16)
    kind = torch.randint(0, 5, (M, units), generator=g)
    size = torch.tensor([1.0, 0.0, 2.0 ** -13, 8.0, 1.0])[kind]
    x = (torch.randn((M, 16 * units), generator=g) * size.repeat_interleave(16, 1))
    if block == 32:
        lost = torch.where(kind == 4, torch.randint(0, 16, (M, units), generator=g), -1)
        bad = torch.tensor([float("nan"), float("inf"), -float("inf")])[torch.randint(0, 3, (M, units), generator=g)]
        at = torch.arange(16) == lost[:, :, None]
        x = torch.where(at, bad[:, :, None], x.view(M, units, 16)).view(M, -1)
    x = x[:, :K].to(TORCH[dtype])
    check_quantised(b, x.float(), block, b.quantize_fp4(x.cuda(), block=block))
