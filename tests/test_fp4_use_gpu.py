"""The choice of experts and the 4-bit operators as programs use them: calls at
once on several streams and in several graphs, a process whose first calls are
captured, rows gigabytes apart, more tokens than a launch has warps.

What is compared bit for bit is the same call alone, or (products of short codes
and powers of two) sums that f32 holds exactly."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import fp4_util as fp4
import test_choose_gpu as choice
import test_fp4_gpu as products

pytestmark = pytest.mark.gpu

PRIOR = 41.0
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    from tiled_staged_matmul_gb300 import binding
    return binding


def calls(b):
    """Calls of every way a product is launched (K cut over a cluster, over the
    SMs, over pairs of SMs, whole tiles, groups), quantisation and the choice."""
    g = torch.Generator().manual_seed(1)
    all_ = []
    for M, N, K, block in ((1, 1000, 4096, 16), (97, 14333, 2000, 32), (300, 5000, 2100, 16), (40, 20000, 256, 16),
                           (600, 4000, 500, 32)):
        a = b.quantize_fp4(torch.randn((M, K), generator=g).cuda(), block=block)
        w = b.quantize_fp4(torch.randn((N, K), generator=g).cuda(), block=block)
        all_.append(lambda a=a, w=w: b.gemm_fp4(a, w, activation="gelu"))
    for cap, N, K in ((40, 300, 600), (260, 500, 700)):
        a = b.quantize_fp4(torch.randn((6, cap, K), generator=g).cuda())
        w = b.quantize_fp4(torch.randn((6, N, K), generator=g).cuda())
        counts = torch.tensor([cap, 0, 3, cap - 1, 17, 33], dtype=torch.int32, device="cuda")
        all_.append(lambda a=a, w=w, n=counts: b.grouped_gemm_fp4(a, w, n, out_dtype=torch.bfloat16))
    x = torch.randn((1500, 900), generator=g).cuda()
    all_.append(lambda: b.quantize_fp4(x, block=32).codes)
    logits = torch.randn((5000, 64), generator=g).cuda()
    all_.append(lambda: b.moe_choose(logits, 6, score="sigmoid", groups=8, keep_groups=3)[1])
    ids, dw = b.moe_choose(logits, 6)
    all_.append(lambda: b.moe_choose_grad(dw, logits, ids))
    return all_


def test_calls_at_once_on_several_streams(b):
    todo = calls(b)
    want = [f() for f in todo]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    outs = []
    for i in range(12):
        for j, f in enumerate(todo):
            with torch.cuda.stream(streams[(i + j) % 4]):
                outs.append((j, f()))
    torch.cuda.synchronize()
    b.check(b.gemm_get_device_status(0))
    for j, o in outs:
        assert torch.equal(o, want[j]), j


def test_graphs_at_once(b):
    """Two graphs of all the calls, replayed together on two streams, beside
    eager calls on a third."""
    todo = calls(b)
    want = [f() for f in todo]
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append([f() for f in todo])
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(8):
        for o in outs:
            for v in o:
                v.zero_()
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        with torch.cuda.stream(streams[2]):
            eager = [f() for f in todo]
        torch.cuda.synchronize()
        for o in (*outs, eager):
            for j, v in enumerate(o):
                assert torch.equal(v, want[j]), j
    b.check(b.gemm_get_device_status(0))


FIRST = """
import torch
from tiled_staged_matmul_gb300 import binding as b
g = torch.Generator().manual_seed(1)
x, w = torch.randn((70, 900), generator=g).cuda(), torch.randn((333, 900), generator=g).cuda()
logits = torch.randn((70, 20), generator=g).cuda()
graph = torch.cuda.CUDAGraph()
def run():
    ids, weights = b.moe_choose(logits, 3)
    return [b.gemm_fp4(b.quantize_fp4(x), b.quantize_fp4(w)), b.moe_choose_grad(weights, logits, ids)]
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    out = run()
graph.replay()
for got, want in zip(out, run()):
    assert torch.equal(got, want)
b.check(b.gemm_get_device_status(0))
print("same")
"""


def test_the_first_calls_of_a_process_are_captured(b):
    run = subprocess.run([sys.executable, "-c", FIRST], cwd=os.path.dirname(HERE), capture_output=True, text=True,
                         timeout=300)
    assert run.returncode == 0 and "same" in run.stdout, run.stderr[-2000:]


def spread(x, pitch):
    """The rows of x (on the CPU) with this pitch, in elements, on the GPU."""
    far = torch.empty((x.shape[0] - 1) * pitch + x.shape[1], dtype=x.dtype, device="cuda")
    view = far.as_strided(x.shape, (pitch, 1))
    view.copy_(x)
    return view


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("pa,pb", [(2 ** 31 + 16, 2 ** 25 + 32), (2 ** 31 + 17, 2 ** 25 + 32), (2 ** 31 + 16, 2 ** 25 + 1)])
def test_products_of_rows_far_apart(b, pa, pb, block):
    """Operands past 2^32 bytes, read in place and copied first; C past 2^33."""
    M, N, K = 3, 150, 300
    A, va = products.whole_operand(b, M, K, block, 1)
    B, vb = products.whole_operand(b, N, K, block, 2)
    far = [rows._replace(codes=spread(rows.codes.cpu(), pitch)) for rows, pitch in ((A, pa), (B, pb))]
    pitch = 2 ** 31 + 3
    buf = torch.empty(2 * pitch + N + 1, dtype=torch.bfloat16, device="cuda")
    C = buf.as_strided((M, N + 1), (pitch, 1))
    C.fill_(PRIOR)
    b.gemm_fp4(*far, C[:, :N])
    b.check(b.gemm_get_device_status(0))
    assert torch.equal(C[:, :N], torch.from_numpy((va @ vb.T).astype(np.float32)).bfloat16().cuda())
    assert (C[:, N] == PRIOR).all()


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("pitch", [2 ** 30 + 16, 2 ** 30 + 5])
def test_quantisation_of_rows_far_apart(b, pitch, block):
    x = torch.randn((4, 700), generator=torch.Generator().manual_seed(3))
    products.check_quantised(b, x, block, b.quantize_fp4(spread(x, pitch), block=block))


def test_choice_of_rows_far_apart(b):
    x = torch.randn((4, 60), generator=torch.Generator().manual_seed(4)).half()
    want, ww = b.moe_choose(x.cuda(), 5)
    dw = torch.randn((4, 5), generator=torch.Generator().manual_seed(5)).cuda()
    for pitch in (2 ** 31 + 8, 2 ** 31 + 1):
        far = spread(x, pitch)
        ids, w = b.moe_choose(far, 5)
        assert torch.equal(ids, want) and torch.equal(w, ww)
        out = spread(torch.zeros_like(x), pitch)
        b.moe_choose_grad(dw, far, ids, out)
        assert torch.equal(out, b.moe_choose_grad(dw, x.cuda(), want))


def test_more_tokens_than_a_launch_has_warps(b):
    """152 SMs x 64 blocks x 4 tokens are 38912."""
    g = torch.Generator().manual_seed(6)
    x = torch.randn((80001, 8), generator=g).cuda()
    bias = torch.randn(8, generator=g).cuda()
    ids, w = b.moe_choose(x, 2, score="sigmoid", bias=bias, renormalize=True)
    d = b.moe_choose_grad(w, x, ids, score="sigmoid", renormalize=True)
    for i in range(0, 80001, 20000):
        part = x[i:i + 20000].contiguous()
        i2, w2 = b.moe_choose(part, 2, score="sigmoid", bias=bias, renormalize=True)
        assert torch.equal(ids[i:i + 20000], i2) and torch.equal(w[i:i + 20000], w2)
        assert torch.equal(d[i:i + 20000], b.moe_choose_grad(w2, part, i2, score="sigmoid", renormalize=True))
    # (Parts of 20000 are a launch's one round; these are checked against 64 bits.)
    want, _ = choice.reference(x[:300].cpu().double().numpy(), 2, score="sigmoid", bias=bias.cpu().double().numpy(),
                               renormalize=True)
    assert np.array_equal(ids[:300].cpu().numpy(), want)


def test_slices_of_an_operand(b):
    """Rows and matrices of a larger operand, as a program cuts them."""
    A, va = products.whole_operand(b, 300, 400, 16, 1)
    B, vb = products.whole_operand(b, 260, 400, 16, 2)
    part = A._replace(codes=A.codes[128:256], block_scales=A.block_scales[1:2])
    want = torch.from_numpy((va[128:256] @ vb.T).astype(np.float32)).cuda()
    assert torch.equal(b.gemm_fp4(part, B), want)
    # A row for each tile of scales; every output a slice of one buffer.
    out = torch.full((3, 400), PRIOR, device="cuda")
    for i in range(3):
        one = A._replace(codes=A.codes[128 * i:128 * i + 1], block_scales=A.block_scales[i:i + 1])
        b.gemm_fp4(one, B, out[i:i + 1, 70:330])
    assert torch.equal(out[:, 70:330], torch.from_numpy((va[::128] @ vb.T).astype(np.float32)).cuda())
    assert (out[:, :70] == PRIOR).all() and (out[:, 330:] == PRIOR).all()


def test_outputs_that_overlap_an_input_are_refused(b):
    x = torch.randn((20, 64), device="cuda")
    ids, w = b.moe_choose(x, 3)
    with pytest.raises(b.GemmError):
        b.moe_choose_grad(w, x, ids, x)
    a = b.quantize_fp4(torch.randn((8, 8192), device="cuda"))
    with pytest.raises(b.GemmError):
        b.gemm_fp4(a, a, a.block_scales.view(torch.float32).reshape(-1)[:64].view(8, 8))
    with pytest.raises(b.GemmError):
        b.gemm_fp4(a, a, a.codes.view(torch.float32)[:, :8])


def test_numbers_past_32_bits_are_refused(b):
    x = torch.randn((4, 8), device="cuda")
    a = b.quantize_fp4(x)
    with pytest.raises(ValueError):
        b.moe_choose(x, 2, group_best=2 ** 32 + 1)
    with pytest.raises(ValueError):
        b.gemm_fp4(a, a, activation=2 ** 32)
