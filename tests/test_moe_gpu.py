"""Token rows to their experts and back, against plain definitions in 64 bits.

Slots and counts are whole numbers and must be equal; copied rows must be
equal bit for bit; sums are held to the bound of their own arithmetic: n
products summed in f32 (unit roundoff 2^-24) err by at most (n + 1) 2^-24
times the sum of their magnitudes, and one rounding to the output type adds
its unit roundoff of the result (2^-11 for f16, 2^-8 for bf16, 2^-24 for
f32) or half its smallest subnormal."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROUNDOFF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    from tiled_staged_matmul_gb300 import binding
    return binding


def route_reference(ids, groups, capacity):
    """One choice after the other."""
    slots = np.full(ids.shape, -1, dtype=np.int32)
    seen = np.zeros(groups, dtype=np.int64)
    flat, out = ids.reshape(-1), slots.reshape(-1)
    for i, e in enumerate(flat.tolist()):
        if 0 <= e < groups:
            if seen[e] < capacity:
                out[i] = e * capacity + seen[e]
            seen[e] += 1
    return slots, np.minimum(seen, capacity).astype(np.int32)


def draw_ids(tokens, topk, groups, seed, bad=True):
    g = np.random.default_rng(seed)
    p = np.exp(g.standard_normal(groups))
    ids = g.choice(groups, size=(tokens, topk), p=p / p.sum())
    if bad and ids.size:
        ids.reshape(-1)[g.integers(0, ids.size, size=max(1, ids.size // 17))] = -1
        ids.reshape(-1)[g.integers(0, ids.size)] = groups
    return ids


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("tokens,topk,groups,capacity", [
    (0, 2, 4, 8), (1, 1, 1, 1), (1, 6, 64, 1), (3, 0, 5, 4), (16, 2, 8, 0), (16, 2, 8, 3), (512, 2, 8, 200),
    (513, 2, 8, 1000), (1, 1023, 7, 500), (1, 1025, 7, 500), (341, 6, 64, 40), (4096, 6, 64, 512),
    (999, 3, 1024, 5), (5000, 4, 1, 1 << 20), (40000, 8, 33, 9000), (170001, 2, 1000, 200)])
def test_route(b, tokens, topk, groups, capacity, wide):
    ids = draw_ids(tokens, topk, groups, tokens + topk)
    dev = torch.from_numpy(ids.astype(np.int64 if wide else np.int32)).cuda()
    if wide and ids.size:
        dev.view(-1)[0] = 1 << 40  # past 32 bits: no expert, not expert 0
        ids.reshape(-1)[0] = -1
    slots, counts = b.moe_route(dev, groups, capacity)
    want_slots, want_counts = route_reference(ids, groups, capacity)
    assert np.array_equal(slots.cpu().numpy(), want_slots)
    assert np.array_equal(counts.cpu().numpy(), want_counts)


def test_route_all_to_one_expert_and_none(b):
    for tokens in (1, 700, 20000):
        ids = torch.full((tokens, 2), 3, dtype=torch.int64, device="cuda")
        slots, counts = b.moe_route(ids, 5, tokens)
        flat = torch.arange(2 * tokens, device="cuda").view(tokens, 2)
        want = torch.where(flat < tokens, 3 * tokens + flat, torch.full_like(flat, -1))
        assert torch.equal(slots.long(), want)
        assert counts.tolist() == [0, 0, 0, tokens, 0]
        slots, counts = b.moe_route(torch.full_like(ids, -1), 5, tokens)
        assert bool((slots == -1).all()) and counts.tolist() == [0] * 5


def make_slots(b, tokens, topk, groups, capacity, seed):
    """Slots with dropped choices, tokens without any, and rows no one names."""
    ids = draw_ids(tokens, topk, groups, seed)
    if tokens > 2:
        ids[1] = -1
    slots, counts = route_reference(ids, groups, capacity)
    return slots, torch.from_numpy(slots).cuda()


SHAPES = [(1, 1, 1, 1, 1), (1, 4, 8, 1, 8), (7, 2, 3, 5, 33), (64, 6, 16, 20, 256), (33, 2, 8, 40, 1000),
          (257, 3, 5, 100, 2048), (100, 9, 12, 77, 136), (50, 14, 20, 30, 4104)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "int8"])
@pytest.mark.parametrize("tokens,topk,groups,capacity,width", SHAPES)
def test_dispatch_copies_the_named_rows_only(b, tokens, topk, groups, capacity, width, dtype):
    dt = TYPES.get(dtype, torch.int8)
    slots, dslots = make_slots(b, tokens, topk, groups, capacity, 5)
    g = torch.Generator().manual_seed(width)
    x = torch.randint(-100, 100, (tokens, width), generator=g).to(dt)
    for pad_x, pad_r in ((0, 0), (3, 0), (16, 16), (0, 5)):
        bx = torch.full((tokens, width + pad_x), 111, dtype=dt, device="cuda")
        bx[:, :width] = x.cuda()
        br = torch.full((groups, capacity, width + pad_r), 99, dtype=dt, device="cuda")
        out = b.moe_dispatch(bx[:, :width], dslots, groups, capacity, br[:, :, :width])
        assert out.data_ptr() == br.data_ptr()
        want = torch.full((groups * capacity, width + pad_r), 99, dtype=dt)
        for t in range(tokens):
            for j in range(topk):
                if slots[t, j] >= 0:
                    want[slots[t, j], :width] = x[t]
        assert torch.equal(br.cpu().view(groups * capacity, -1), want)
    fresh = b.moe_dispatch(x.cuda(), dslots, groups, capacity)
    named = np.zeros(groups * capacity, bool)
    named[slots[slots >= 0]] = True
    assert bool((fresh.view(groups * capacity, -1).cpu()[torch.from_numpy(~named)] == 0).all())


def test_dispatch_keeps_nan_and_infinity_bits(b):
    x = torch.tensor([[float("nan"), float("inf"), -0.0, 1e-7]], dtype=torch.float16, device="cuda")
    slots = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    rows = b.moe_dispatch(x, slots, 3, 1)
    assert torch.equal(rows[2, 0].view(torch.int16), x[0].view(torch.int16))
    assert torch.equal(rows[0, 0].view(torch.int16), x[0].view(torch.int16))


def combine_reference(rows, slots, w):
    """(sum, sum of magnitudes) in f64."""
    T, k = slots.shape
    H = rows.shape[1]
    out, mag = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            if slots[t, j] >= 0:
                v = w[t, j] * rows[slots[t, j]]
                out[t] += v
                mag[t] += np.abs(v)
    return out, mag


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens,topk,groups,capacity,width", SHAPES)
def test_combine_and_dispatch_grad(b, tokens, topk, groups, capacity, width, dtype):
    dt = TYPES[dtype]
    slots, dslots = make_slots(b, tokens, topk, groups, capacity, 6)
    g = torch.Generator().manual_seed(tokens)
    # rows no slot names hold NaN: they may not be read into a sum
    named = torch.zeros(groups * capacity, dtype=torch.bool)
    named[torch.from_numpy(slots[slots >= 0]).long()] = True
    rows = torch.randn((groups * capacity, width), generator=g).to(dt)
    rows[~named] = float("nan")
    w = torch.randn((tokens, topk), generator=g)
    w[torch.from_numpy(slots) < 0] = float("inf")  # the weight of a dropped choice does not count
    r64, w64 = rows.double().numpy(), w.double().numpy()
    for pad_r, pad_o, weights in ((0, 0, True), (3, 1, True), (16, 8, False), (0, 0, False)):
        br = torch.full((groups, capacity, width + pad_r), float("nan"), dtype=dt, device="cuda")
        br[:, :, :width] = rows.view(groups, capacity, width).cuda()
        bo = torch.full((tokens, width + pad_o), 77.0, dtype=dt, device="cuda")
        if weights:
            b.moe_combine(br[:, :, :width], dslots, w.cuda(), bo[:, :width])
        else:
            b.moe_dispatch_grad(br[:, :, :width], dslots, bo[:, :width])
        want, mag = combine_reference(r64, slots, w64 if weights else np.ones_like(w64))
        got = bo[:, :width].double().cpu().numpy()
        bound = (topk + 1) * 2.0 ** -24 * mag + ROUNDOFF[dt] * (np.abs(want) + 2.0 ** -20 * mag) + TINY[dt]
        assert np.all(np.abs(got - want) <= bound)
        assert bool((bo[:, width:] == 77.0).all())
    none = b.moe_combine(br[:, :, :width], torch.full_like(dslots, -1))
    assert bool((none == 0).all())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens,topk,groups,capacity,width", SHAPES)
def test_combine_grad(b, tokens, topk, groups, capacity, width, dtype):
    dt = TYPES[dtype]
    slots, dslots = make_slots(b, tokens, topk, groups, capacity, 7)
    g = torch.Generator().manual_seed(tokens + 1)
    rows = torch.randn((groups * capacity, width), generator=g).to(dt)
    dout = torch.randn((tokens, width), generator=g).to(dt)
    w = torch.randn((tokens, topk), generator=g)
    r64, d64, w64 = rows.double().numpy(), dout.double().numpy(), w.double().numpy()
    for pad, weights in ((0, True), (5, True), (8, False)):
        bd = torch.full((tokens, width + pad), float("nan"), dtype=dt, device="cuda")
        bd[:, :width] = dout.cuda()
        br = torch.full((groups, capacity, width + pad), float("nan"), dtype=dt, device="cuda")
        br[:, :, :width] = rows.view(groups, capacity, width).cuda()
        bg = torch.full((groups, capacity, width + pad), 55.0, dtype=dt, device="cuda")
        drows, dw = b.moe_combine_grad(bd[:, :width], br[:, :, :width], dslots, w.cuda() if weights else None,
                                       bg[:, :, :width])
        got = bg.double().cpu().numpy().reshape(groups * capacity, width + pad)
        want = np.full_like(got, 55.0)
        tol = np.zeros_like(got)
        want_w, tol_w = np.zeros((tokens, topk)), np.zeros((tokens, topk))
        for t in range(tokens):
            for j in range(topk):
                s = slots[t, j]
                if s >= 0:
                    v = (w64[t, j] if weights else 1.0) * d64[t]
                    want[s, :width] = v
                    tol[s, :width] = (2.0 ** -23 + ROUNDOFF[dt]) * np.abs(v) + TINY[dt]
                    want_w[t, j] = np.dot(d64[t], r64[s])
                    tol_w[t, j] = (width + 1) * 2.0 ** -24 * np.dot(np.abs(d64[t]), np.abs(r64[s]))
        assert np.all(np.abs(got - want) <= tol)
        assert np.all(np.abs(dw.double().cpu().numpy() - want_w) <= tol_w)


def test_gradients_are_those_of_the_forward_calls(b):
    """Differences: both calls are linear in each argument, so the difference
    quotient over a unit step is the derivative up to the sums' rounding."""
    tokens, topk, groups, capacity, width = 40, 3, 6, 16, 96
    slots, dslots = make_slots(b, tokens, topk, groups, capacity, 8)
    g = torch.Generator(device="cuda").manual_seed(3)

    def rnd(*shape):
        return torch.randint(-8, 9, shape, generator=g, device="cuda").float()  # sums exact in f32

    rows, w, dout = rnd(groups, capacity, width), rnd(tokens, topk), rnd(tokens, width)
    drows, dw = b.moe_combine_grad(dout, rows, dslots, w)
    for _ in range(3):
        er, ew = rnd(groups, capacity, width), rnd(tokens, topk)
        diff = (b.moe_combine(rows + er, dslots, w) - b.moe_combine(rows - er, dslots, w)) / 2
        assert float((diff.double() * dout).sum()) == float((er.double() * drows).sum())
        diff = (b.moe_combine(rows, dslots, w + ew) - b.moe_combine(rows, dslots, w - ew)) / 2
        assert float((diff.double() * dout).sum()) == float((ew.double() * dw).sum())
    x, ex, gr = rnd(tokens, width), rnd(tokens, width), rnd(groups, capacity, width)
    dx = b.moe_dispatch_grad(gr, dslots)
    diff = (b.moe_dispatch(x + ex, dslots, groups, capacity) - b.moe_dispatch(x - ex, dslots, groups, capacity)) / 2
    assert float((diff.double() * gr).sum()) == float((ex.double() * dx).sum())


def test_slots_past_the_rows_are_skipped(b):
    """Slots made for a larger buffer: nothing is read or written past the rows there are."""
    slots = torch.tensor([[0, 7], [5, 1], [2**31 - 1, -5]], dtype=torch.int32, device="cuda")
    x = torch.ones((3, 64), device="cuda")
    rows = b.moe_dispatch(x, slots, 2, 2)
    assert rows.sum(2).view(-1).tolist() == [64.0, 64.0, 0.0, 0.0]
    assert b.moe_combine(rows, slots).sum(1).tolist() == [64.0, 64.0, 0.0]
    drows, dw = b.moe_combine_grad(x, rows, slots)
    assert drows.sum(2).view(-1).tolist() == [64.0, 64.0, 0.0, 0.0]
    assert dw.tolist() == [[64.0, 0.0], [0.0, 64.0], [0.0, 0.0]]


def test_offsets_past_32_bits(b):
    """Rows whose element offsets pass 2^31 (and byte offsets 2^32)."""
    groups, capacity, width = 2, 1 << 17, 8200
    rows = torch.empty((groups, capacity, width), dtype=torch.float16, device="cuda")
    last = groups * capacity - 1
    x = torch.randn((2, width), device="cuda").half()
    slots = torch.tensor([[last, 0], [capacity, last - 1]], dtype=torch.int32, device="cuda")
    b.moe_dispatch(x, slots, groups, capacity, rows)
    flat = rows.view(-1, width)
    assert torch.equal(flat[last], x[0]) and torch.equal(flat[capacity], x[1]) and torch.equal(flat[last - 1], x[1])
    out = b.moe_combine(rows, slots, torch.tensor([[1.0, 0.0], [0.5, 0.5]], device="cuda"))
    assert torch.equal(out, x)


def test_runs_on_the_given_stream_and_repeats(b):
    ids = torch.from_numpy(draw_ids(3000, 4, 32, 1)).cuda()
    x = torch.randn((3000, 512), device="cuda").bfloat16()
    w = torch.rand((3000, 4), device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    seen = []
    for _ in range(3):
        slots, counts = b.moe_route(ids, 32, 300, stream=s)
        with torch.cuda.stream(s):
            rows = b.moe_dispatch(x, slots, 32, 300, stream=s)
            out = b.moe_combine(rows, slots, w, stream=s)
            drows, dw = b.moe_combine_grad(x, rows, slots, w, stream=s)
        s.synchronize()
        seen.append((slots, counts, rows, out, drows, dw))
    for other in seen[1:]:
        assert all(torch.equal(p, q) for p, q in zip(seen[0], other))


def test_capture_in_a_graph(b):
    ids = torch.from_numpy(draw_ids(64, 2, 8, 2)).cuda()
    x = torch.randn((64, 256), device="cuda").half()
    rows = torch.zeros((8, 32, 256), dtype=torch.float16, device="cuda")
    b.moe_route(ids, 8, 32)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        slots, counts = b.moe_route(ids, 8, 32)
        b.moe_dispatch(x, slots, 8, 32, rows)
        out = b.moe_combine(rows, slots)
    ids.copy_(torch.from_numpy(draw_ids(64, 2, 8, 9)).cuda())
    graph.replay()
    torch.cuda.synchronize()
    want, want_counts = route_reference(ids.cpu().numpy(), 8, 32)
    assert np.array_equal(slots.cpu().numpy(), want) and np.array_equal(counts.cpu().numpy(), want_counts)
    kept = torch.from_numpy((want >= 0).sum(1)).cuda()[:, None]
    assert torch.equal(out, (x.float() * kept).half())


def test_refusals(b):
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(b.GemmError):
        b.moe_route(ids, 2000, 4)
    with pytest.raises(ValueError):
        b.moe_route(ids.float(), 4, 4)
    slots, _ = b.moe_route(ids, 4, 8)
    x = torch.zeros((4, 16), device="cuda")
    with pytest.raises(ValueError):
        b.moe_dispatch(x[:3], slots, 4, 8)
    with pytest.raises(ValueError):
        b.moe_dispatch(x, slots, 4, 8, torch.zeros((4, 8, 16), device="cuda").half())
    with pytest.raises(TypeError):
        b.moe_combine(torch.zeros((4, 8, 16), dtype=torch.int8, device="cuda"), slots)
    rows = torch.zeros((4, 8, 16), device="cuda")
    with pytest.raises(ValueError):
        b.moe_combine(rows, slots, torch.zeros((4, 2), device="cuda").half())
    with pytest.raises(b.GemmError):  # written onto what it reads
        b.moe_combine_grad(x, rows, slots, None, rows)
    host = torch.zeros((4, 16))
    assert b.moe_dispatch_rows(host.data_ptr(), 4, slots.data_ptr(), rows.data_ptr(), 4, 2, 32, 16, 16, 16) \
        == b.GEMM_ERR_INVALID_VALUE
    # an allocation that ends before the last row
    assert b.moe_dispatch_rows(x.data_ptr(), 4, slots.data_ptr(), rows.data_ptr(), 4, 2, 1 << 28, 16, 16, 16) \
        == b.GEMM_ERR_INVALID_VALUE


@pytest.mark.parametrize("topk", [31, 32, 33, 70])
def test_more_choices_than_a_warp_has_lanes(b, topk):
    groups, capacity, width = 80, 4, 40
    g = torch.Generator().manual_seed(topk)
    ids = torch.stack([torch.randperm(groups, generator=g)[:topk] for _ in range(6)]).int()
    x = torch.randn((6, width), generator=g)
    w = torch.rand((6, topk), generator=g)
    slots, counts = b.moe_route(ids.cuda(), groups, capacity)
    want, kept = route_reference(ids.numpy(), groups, capacity)
    assert np.array_equal(slots.cpu().numpy(), want) and np.array_equal(counts.cpu().numpy(), kept)
    rows = b.moe_dispatch(x.cuda(), slots, groups, capacity)
    plain = torch.zeros((groups * capacity, width))
    for t in range(6):
        for j in range(topk):
            if want[t, j] >= 0:
                plain[want[t, j]] = x[t]
    assert torch.equal(rows.cpu().view(-1, width), plain)
    out = b.moe_combine(rows, slots, w.cuda()).cpu().double()
    keep = torch.from_numpy(want >= 0).double() * w.double()
    total = keep.sum(1, keepdim=True) * x.double()
    assert ((out - total).abs() <= (topk + 2) * 2.0 ** -24 * total.abs()).all()


def test_a_dropped_choice_adds_nothing_whatever_its_weight(b):
    slots = torch.tensor([[0, -1], [-1, -1], [1, 5]], dtype=torch.int32, device="cuda")  # (4 rows)
    rows = torch.randn((1, 4, 24), generator=torch.Generator().manual_seed(3)).cuda()
    nan, inf = float("nan"), float("inf")
    w = torch.tensor([[2.0, nan], [inf, nan], [0.5, -inf]], device="cuda")
    out = b.moe_combine(rows, slots, w)
    assert torch.equal(out[0], 2 * rows[0, 0]) and torch.equal(out[2], 0.5 * rows[0, 1])
    assert (out[1] == 0).all()


@pytest.mark.parametrize("n", [1023, 1024, 1025, 8191, 8192, 8193, 16384, 16385, 24576, 32768, 32769, 40001])
@pytest.mark.parametrize("groups,wide", [(1, False), (8, True), (1000, False)])
def test_route_over_chunks(b, n, groups, wide):
    """Numbers of choices around those where the work is cut differently."""
    g = torch.Generator().manual_seed(n + groups)
    ids = torch.randint(-1, groups + 1, (n, 1), generator=g, dtype=torch.int64 if wide else torch.int32)
    capacity = n // groups + 3
    slots, counts = b.moe_route(ids.cuda(), groups, capacity)
    want, kept = route_reference(ids.numpy(), groups, capacity)
    assert np.array_equal(slots.cpu().numpy(), want)
    assert np.array_equal(counts.cpu().numpy(), kept)


def many_slots(tokens, topk, groups, capacity, seed):
    """Slots of random choices with room for about two thirds of them."""
    ids = draw_ids(tokens, topk, groups, seed)
    slots = np.full(ids.size, -1, dtype=np.int64)
    for e in range(groups):
        at = np.flatnonzero(ids.reshape(-1) == e)[:capacity]
        slots[at] = e * capacity + np.arange(at.size)
    return torch.from_numpy(slots.reshape(ids.shape))


# As many tokens as make one warp take two rows of two pieces at a time (155648
# pieces in all on 152 SMs), and more warps' work than one grid has warps (77824).
MANY = [(700, 5, 9, 300, 2048), (2500, 3, 4, 1300, 1001), (1300, 7, 16, 400, 1032), (90001, 2, 5, 30000, 40),
        (40003, 3, 7, 12000, 24)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens,topk,groups,capacity,width", MANY)
def test_many_tokens(b, tokens, topk, groups, capacity, width, dtype):
    """Every call on one set of slots, against sums in 64 bits on the GPU."""
    dt = TYPES[dtype]
    slots = many_slots(tokens, topk, groups, capacity, 11).cuda()
    dslots = slots.int()
    g = torch.Generator(device="cuda").manual_seed(tokens)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    R = groups * capacity
    at, on = slots.clamp(min=0), slots >= 0
    named = torch.zeros(R, dtype=torch.bool, device="cuda")
    named[slots[on]] = True
    x, dout, w = rnd(tokens, width).to(dt), rnd(tokens, width).to(dt), rnd(tokens, topk)
    rows = rnd(R, width).to(dt)
    rows[~named] = float("nan")
    w[~on] = float("nan")
    token = torch.arange(tokens, device="cuda")[:, None].expand(-1, topk)

    out = torch.full((groups, capacity, width), 99.0, dtype=dt, device="cuda")
    b.moe_dispatch(x, dslots, groups, capacity, out)
    want = torch.full((R, width), 99.0, dtype=dt, device="cuda")
    want[slots[on]] = x[token[on]]
    assert torch.equal(out.view(R, width), want)

    view = rows.view(groups, capacity, width)
    for weights in (w, None):
        total, mag = (torch.zeros((tokens, width), dtype=torch.float64, device="cuda") for _ in range(2))
        for j in range(topk):
            c = torch.where(on[:, j], w[:, j].double() if weights is not None else 1.0, 0.0)[:, None]
            v = torch.where(on[:, j, None], rows[at[:, j]].double(), 0.0) * c
            total += v
            mag += v.abs()
        got = b.moe_combine(view, dslots, weights) if weights is not None else b.moe_dispatch_grad(view, dslots)
        bound = (topk + 1) * 2.0 ** -24 * mag + ROUNDOFF[dt] * (total.abs() + 2.0 ** -20 * mag) + TINY[dt]
        assert bool(((got.double() - total).abs() <= bound).all())

    drows, dw = b.moe_combine_grad(dout, view, dslots, w,
                                   torch.full((groups, capacity, width), 55.0, dtype=dt, device="cuda"))
    want = torch.full((R, width), 55.0, dtype=torch.float64, device="cuda")
    exact = w[on].double()[:, None] * dout[token[on]].double()
    want[slots[on]] = exact
    tol = torch.zeros_like(want)
    tol[slots[on]] = (2.0 ** -23 + ROUNDOFF[dt]) * exact.abs() + TINY[dt]
    assert bool(((drows.view(R, width).double() - want).abs() <= tol).all())
    for j in range(topk):
        r = torch.where(on[:, j, None], rows[at[:, j]].double(), 0.0)
        d = dout.double()
        assert bool(((dw[:, j].double() - (d * r).sum(1)).abs()
                     <= (width + 2) * 2.0 ** -24 * (d.abs() * r.abs()).sum(1)).all())
