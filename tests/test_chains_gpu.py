"""Long runs of the experts' and 8-bit calls with nothing between them.  Each
of their kernels starts while the one before still runs and waits for its end
itself, so what would show a missing wait is a run over the same buffers, pass
after pass, that no other kernel, copy or synchronisation interrupts.  Every
pass has its own inputs and its own place for the result, which has to be what
the same pass gives with a synchronisation after every call."""
import pytest
import torch

pytestmark = pytest.mark.gpu

PASSES = 40
HEAD_START = 50_000_000  # cycles: the calls are all queued before the first kernel runs


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    from tiled_staged_matmul_gb300 import binding
    return binding


class Layer:
    """An int8 experts' layer over buffers that every pass uses again."""

    def __init__(self, b, tokens, topk, groups, capacity, width, hidden):
        g = torch.Generator(device="cuda").manual_seed(tokens)
        codes = lambda *s: torch.randint(-128, 128, s, generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
        rand = lambda *s: torch.rand(s, generator=g, device="cuda")
        self.b, self.groups, self.capacity = b, groups, capacity
        self.W1, self.W2 = codes(groups, width, hidden), codes(groups, hidden, width)
        self.s1, self.s2 = rand(groups, hidden) * 1e-3, rand(groups, width) * 1e-3
        empty = lambda dtype, *s: torch.empty(s, dtype=dtype, device="cuda")
        self.q, self.qs = empty(torch.int8, tokens, width), empty(torch.float32, tokens)
        self.rows, self.rs = empty(torch.int8, groups, capacity, width), empty(torch.float32, groups, capacity, 1)
        self.a = empty(torch.float16, groups, capacity, hidden)
        self.qa, self.qas = empty(torch.int8, groups, capacity, hidden), empty(torch.float32, groups, capacity)
        self.y = empty(torch.float16, groups, capacity, width)
        # (Only what a pass has written may be read in it.)
        for t in (self.q, self.qs, self.rows, self.rs, self.a, self.qa, self.qas, self.y):
            t.fill_(77)
        self.inputs = [((rand(tokens, width) * 4 - 2).half(),
                        torch.randint(0, groups, (tokens, topk), generator=g, device="cuda", dtype=torch.int32),
                        rand(tokens, topk)) for _ in range(PASSES)]
        torch.cuda.synchronize()

    def calls(self, x, ids, weights, out):
        b = self.b
        slots, counts = b.moe_route(ids, self.groups, self.capacity)
        yield
        b.quantize_rows(x, q=self.q, scales=self.qs)
        yield
        b.moe_dispatch(self.q, slots, self.groups, self.capacity, self.rows)
        yield
        b.moe_dispatch(self.qs[:, None], slots, self.groups, self.capacity, self.rs)
        yield
        b.grouped_gemm_s8(self.rows, self.W1, self.rs[..., 0], self.s1, counts, self.a, activation="silu")
        yield
        b.quantize_rows(self.a, counts, self.qa, self.qas)
        yield
        b.grouped_gemm_s8(self.qa, self.W2, self.qas, self.s2, counts, self.y)
        yield
        b.moe_combine(self.y, slots, weights, out)
        yield
        # (the next pass's buffers, read once more: a late read would show)
        b.moe_combine_grad(x, self.y, slots, weights, self.grad)

    grad = None


LAYERS = [(5, 2, 4, 5, 128, 96), (64, 2, 8, 40, 512, 336), (1500, 3, 8, 700, 1024, 720)]


def outputs(layer, width):
    layer.grad = torch.zeros_like(layer.y)
    return [torch.empty((x.shape[0], width), dtype=torch.float16, device="cuda") for x, _, _ in layer.inputs]


@pytest.mark.parametrize("shape", LAYERS)
def test_passes_without_a_pause(b, shape):
    layer = Layer(b, *shape)
    want, got = outputs(layer, shape[4]), outputs(layer, shape[4])
    for inputs, out in zip(layer.inputs, want):
        for _ in layer.calls(*inputs, out):
            torch.cuda.synchronize()
    torch.cuda.synchronize()
    torch.cuda._sleep(HEAD_START)
    for inputs, out in zip(layer.inputs, got):
        for _ in layer.calls(*inputs, out):
            pass
    torch.cuda.synchronize()
    b.check(b.gemm_get_device_status(0))
    assert all(bool(torch.isfinite(o).all()) and bool((o != 0).any()) for o in want)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("shape", LAYERS)
def test_passes_in_a_graph(b, shape):
    layer = Layer(b, *shape)
    n = 6
    want, got = outputs(layer, shape[4])[:n], outputs(layer, shape[4])[:n]
    held = [tuple(t.clone() for t in layer.inputs[i]) for i in range(n)]
    for _ in layer.calls(*held[0], got[0]):
        pass
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for inputs, out in zip(held, got):
            for _ in layer.calls(*inputs, out):
                pass
    for turn in range(PASSES // n):
        fresh = layer.inputs[turn * n:(turn + 1) * n]
        for mine, theirs in zip(held, fresh):
            for p, q in zip(mine, theirs):
                p.copy_(q)
        graph.replay()
        graph.replay()
        for inputs, out in zip(fresh, want):
            for _ in layer.calls(*inputs, out):
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), turn
    b.check(b.gemm_get_device_status(0))


# A row of products, each on the last one's quantised result: few rows, single
# CTAs (one size with its tiles cut along K), pairs.
@pytest.mark.parametrize("M,N", [(1, 2048), (24, 2048), (100, 2048), (128, 4096), (700, 2048), (1500, 2048)])
def test_products_on_products(b, M, N):
    g = torch.Generator(device="cuda").manual_seed(M)
    W = torch.randint(-128, 128, (N, N), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    ws = torch.rand(N, generator=g, device="cuda") * 1e-3
    x = [torch.randn((M, N), generator=g, device="cuda").half() for _ in range(PASSES)]
    q, qs = torch.empty((M, N), dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    h = torch.empty((M, N), dtype=torch.float16, device="cuda")

    def run(out, wait):
        torch.cuda._sleep(HEAD_START)
        for i in range(PASSES):
            b.quantize_rows(x[i], q=q, scales=qs)
            wait()
            b.gemm_s8(q, W, qs, ws, h, activation="gelu")
            wait()
            b.quantize_rows(h, q=q, scales=qs)
            wait()
            b.gemm_s8(q, W, qs, ws, out[i])
            wait()
        torch.cuda.synchronize()
        return out

    want = run([torch.empty((M, N), device="cuda") for _ in range(PASSES)], torch.cuda.synchronize)
    got = run([torch.empty((M, N), device="cuda") for _ in range(PASSES)], lambda: None)
    b.check(b.gemm_get_device_status(0))
    assert all(bool(torch.isfinite(o).all()) for o in want)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
