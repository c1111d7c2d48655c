"""Calls on another stream than torch's current one, which allocate, fill or
copy something themselves: all of that has to be ordered with the kernels on
the given stream, whatever the current stream is still busy with.

The current stream is given a long wait, then work on memory that it has let go
of, of just the sizes that the call allocates: an output taken from there would
be written over, and a fill or copy queued there would come too late."""
import pytest
import torch

pytestmark = pytest.mark.gpu

TOKENS, TOPK, GROUPS, CAPACITY, WIDTH, COLS = 70, 3, 6, 40, 256, 144


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    from tiled_staged_matmul_gb300 import binding
    return binding


@pytest.fixture(scope="module")
def data(b):
    g = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")
    codes = lambda *s: torch.randint(-128, 128, s, generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    d = {"wide_ids": torch.randint(0, GROUPS, (TOKENS, 2 * TOPK), generator=g, device="cuda", dtype=torch.int32)}
    d["ids"] = d["wide_ids"][:, ::2]
    d["slots"], d["counts"] = b.moe_route(d["ids"], GROUPS, CAPACITY)
    d["weights"] = rand(TOKENS, TOPK)
    d["x"], d["rows"] = rand(TOKENS, WIDTH).half(), rand(GROUPS, CAPACITY, WIDTH).half()
    d["A"], d["B"] = codes(GROUPS, CAPACITY, WIDTH), codes(GROUPS, WIDTH, COLS)
    torch.cuda.synchronize()
    return d


CALLS = {
    "moe_route": lambda b, d, s: b.moe_route(d["ids"], GROUPS, CAPACITY, stream=s),
    "moe_dispatch": lambda b, d, s: [b.moe_dispatch(d["x"], d["slots"], GROUPS, CAPACITY, stream=s)],
    "moe_dispatch_grad": lambda b, d, s: [b.moe_dispatch_grad(d["rows"], d["slots"], stream=s)],
    "moe_combine": lambda b, d, s: [b.moe_combine(d["rows"], d["slots"], d["weights"], stream=s)],
    "moe_combine_grad": lambda b, d, s: b.moe_combine_grad(d["x"], d["rows"], d["slots"], d["weights"], stream=s),
    "quantize_rows": lambda b, d, s: b.quantize_rows(d["x"], stream=s),
    "gemm_s8": lambda b, d, s: [b.gemm_s8(d["A"][0], d["B"][0], stream=s)],
    "grouped_gemm_s8": lambda b, d, s: [b.grouped_gemm_s8(d["A"], d["B"], None, None, d["counts"], stream=s)],
}


def check(call, handle):
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(2):  # (the second with memory that the stream has used before)
        busy = [torch.empty(t.untyped_storage().nbytes(), dtype=torch.uint8, device="cuda") for t in want]
        torch.cuda._sleep(100_000_000)
        for t in busy:
            t.fill_(0x5a)
        del busy, t
        got = call(s.cuda_stream if handle else s)
        s.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        del got


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", list(CALLS))
def test_what_a_call_prepares_is_on_its_stream(b, data, name, handle):
    check(lambda s: CALLS[name](b, data, s), handle)


def test_the_default_stream_by_its_handle(b, data):
    want = CALLS["moe_dispatch"](b, data, None)[0]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        got = CALLS["moe_dispatch"](b, data, 0)[0]
    torch.cuda.default_stream().synchronize()
    side.synchronize()
    assert torch.equal(got, want)


OLDER = {
    "gemm": lambda b, d, s: [b.gemm(d["x"], d["W"][0], stream=s)],
    "grouped_gemm": lambda b, d, s: [b.grouped_gemm(d["rows"], d["W"], d["counts"], stream=s)],
    "grouped_gemm, strided counts": lambda b, d, s: [b.grouped_gemm(d["rows"], d["W"], d["wide_counts"][::2], stream=s)],
    "rowsum": lambda b, d, s: [b.rowsum(d["x"], stream=s)],
    "gemv": lambda b, d, s: [b.gemv(d["x"], d["rows"][0, 0], stream=s)],
}


@pytest.mark.parametrize("name", list(OLDER))
def test_so_do_the_matrix_calls(b, data, name):
    data["W"] = torch.randn((GROUPS, WIDTH, COLS), generator=torch.Generator(device="cuda").manual_seed(5),
                            device="cuda").half()
    data["wide_counts"] = data["counts"].repeat_interleave(2)
    torch.cuda.synchronize()
    check(lambda s: OLDER[name](b, data, s), False)
