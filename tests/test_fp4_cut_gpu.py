"""4-bit products whose tiles are cut along K: over a cluster of CTAs, over single
CTAs and over pairs, plain and grouped.

Random codes with the scales 1/2, 1 and 2 (times 1/2 ... 2 of the other operand's):
every product is a multiple of 2^-4, and the sums of these sizes stay below 2^20 by
far (a thousand standard deviations), so that f32 holds them exactly in any order."""
import pytest
import torch

pytestmark = pytest.mark.gpu

PRIOR = 41.0
# (M, N, K): the kernel's kind (32, 64, 128 rows, pair), CTAs of a cluster, cut over workers
CUT = {(5, 300, 9000): (0, 8, False), (64, 1500, 8192): (1, 4, False), (100, 2000, 6000): (2, 4, False),
       (16, 19600, 8192): (0, 1, True), (33, 19600, 8192): (1, 1, True), (120, 19600, 8192): (2, 1, True),
       (512, 10240, 16384): (2, 1, True), (1024, 5000, 28672): (3, 1, True)}


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    from tiled_staged_matmul_gb300 import binding
    return binding


def operand(b, rows, K, block, seed):
    """Codes and scales made on the GPU (K even), and their values in f64."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pitch = -(-K // 32) * 16
    codes = torch.randint(0, 256, (rows, pitch), generator=g, dtype=torch.uint8, device="cuda")[:, :K // 2]
    blocks = -(-K // block)
    R, C = -(-rows // 128), -(-blocks // 4)
    kinds = torch.tensor([48, 56, 64] if block == 16 else [126, 127, 128], dtype=torch.uint8, device="cuda")
    tiles = kinds[torch.randint(0, 3, (R, C, 512), generator=g, device="cuda")]
    value = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    value = torch.cat((value, -value))
    v = torch.empty((rows, K), dtype=torch.float64, device="cuda")
    v[:, 0::2], v[:, 1::2] = value[(codes & 15).long()], value[(codes >> 4).long()]
    i = torch.arange(rows, device="cuda")[:, None]
    k = torch.arange(blocks, device="cuda")[None, :]
    byte = tiles[i // 128, k // 4, 16 * (i % 32) + 4 * (i % 128 // 32) + k % 4]
    scale = torch.tensor([0.5, 1.0, 2.0], dtype=torch.float64, device="cuda")[(byte.int() - int(kinds[0])) // int(kinds[1] - kinds[0])]
    for j in range(blocks):
        v[:, j * block:(j + 1) * block] *= scale[:, j:j + 1]
    return b.Fp4Rows(codes, tiles, None, block), v


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("size", list(CUT))
def test_sums(b, size, block):
    M, N, K = size
    A, va = operand(b, M, K, block, 1)
    B, vb = operand(b, N, K, block, 2)
    want = (va @ vb.T).float()
    del vb
    out = torch.full((M, N + 3), PRIOR, device="cuda")
    for _ in range(3):
        b.gemm_fp4(A, B, out[:, :N])
        b.check(b.gemm_get_device_status(0))
        assert torch.equal(out[:, :N], want)
        assert (out[:, N:] == PRIOR).all()
        out.fill_(PRIOR)
    # Captured, and replayed without a pause.
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.gemm_fp4(A, B, out[:, :N])
    for _ in range(4):
        graph.replay()
    assert torch.equal(out[:, :N], want)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("cap,N,K,counts", [
    (16, 300, 9000, [16, 0, 5]), (60, 500, 12000, [60, 33, 0, 1]), (128, 200, 14000, [128, 1]),
    (300, 700, 16384, [300, 0, 257, 1]), (520, 512, 16384, [512])])
def test_groups(b, cap, N, K, counts, block):
    """Few tiles of a long K: cut on the device, by the counts."""
    G = len(counts)
    a = [operand(b, cap, K, block, 3 + e) for e in range(G)]
    w = [operand(b, N, K, block, 30 + e) for e in range(G)]
    A = b.Fp4Rows(torch.stack([x[0].codes for x in a]), torch.stack([x[0].block_scales for x in a]), None, block)
    B = b.Fp4Rows(torch.stack([x[0].codes for x in w]), torch.stack([x[0].block_scales for x in w]), None, block)
    out = torch.full((G, cap, N), PRIOR, device="cuda")
    n = torch.tensor(counts, dtype=torch.int32, device="cuda")
    for _ in range(3):
        out.fill_(PRIOR)
        b.grouped_gemm_fp4(A, B, n, out)
        b.check(b.gemm_get_device_status(0))
        for e, c in enumerate(counts):
            assert torch.equal(out[e, :c], (a[e][1][:c] @ w[e][1].T).float()), e
            assert (out[e, c:] == PRIOR).all()
