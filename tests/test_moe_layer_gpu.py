"""The example's mixture-of-experts layer, its gradients and its int8 form,
against the definition in 64 bits.

The bound of every result is carried along with the reference: a rounding to
f16 adds 2^-11 of the value (and half the smallest subnormal, 2^-25), a sum of
n products in f32 (n + 4) 2^-24 of its terms' magnitudes, a quantised value half
its row's scale (with 2^-20 of it for the scale's own rounding), and an earlier
error goes through the next product with the magnitudes of its other factor.
|silu'| < 1.1 and |silu''| < 0.55 everywhere; silu and its derivative are
computed in f32 from errors of a few units, 2^-20 of their value together."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U16, U32, TINY = 2.0 ** -11, 2.0 ** -24, 2.0 ** -25


@pytest.fixture(scope="module")
def layer_type():
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    from examples.moe_layer import MoELayer
    return MoELayer


def f16(v, e):
    return e + U16 * (v.abs() + e) + TINY


def product(a, ea, b, eb=None):
    """a @ b and the bound of its error."""
    n = a.shape[-1]
    e = ea @ b.abs() + (n + 4) * U32 * ((a.abs() + ea) @ b.abs())
    if eb is not None:
        e = e + (a.abs() + ea) @ eb * (1 + (n + 4) * U32) + (n + 4) * U32 * ((a.abs() + ea) @ b.abs())
    return a @ b, e


def silu(h, eh):
    s = torch.sigmoid(h)
    a = h * s
    return a, 1.1 * eh + 2.0 ** -20 * (a.abs() + 1.1 * eh)


def setup(tokens, topk, groups, width, hidden, seed):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g)
    W1 = (rand(groups, width, hidden) * width ** -0.5).half()
    W2 = (rand(groups, hidden, width) * hidden ** -0.5).half()
    x = rand(tokens, width).half()
    popularity = torch.linspace(1.5, 0.0, groups)
    ids = (rand(tokens, groups) + popularity).topk(topk).indices.int()
    weights = torch.softmax(rand(tokens, topk), 1).contiguous()
    return W1, W2, x, ids, weights


def placed(ids, groups, capacity):
    """For each expert the (token, choice) pairs that it keeps, in order."""
    kept = [[] for _ in range(groups)]
    for t, row in enumerate(ids.tolist()):
        for j, e in enumerate(row):
            if len(kept[e]) < capacity:
                kept[e].append((t, j))
    return [(torch.tensor([t for t, _ in k], dtype=torch.long), torch.tensor([j for _, j in k], dtype=torch.long))
            for k in kept]


def check(got, want, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    over = ((got - want).abs() - bound).max().item() if want.numel() else 0.0
    assert over <= 0, f"{what}: {over} past the bound"
    # The bound is of use: on the whole well below the result.
    assert not want.numel() or bound.norm() < 0.2 * want.norm(), what


CASES = [
    # tokens, topk, groups, capacity, width, hidden
    (1, 2, 4, 4, 64, 96),        # one token, experts without any
    (37, 2, 4, 24, 136, 72),     # sizes that are odd for the tiles; a dropped tail
    (200, 3, 8, 64, 256, 192),
]


@pytest.mark.parametrize("tokens,topk,groups,capacity,width,hidden", CASES)
def test_training_step(layer_type, tokens, topk, groups, capacity, width, hidden):
    W1, W2, x, ids, weights = setup(tokens, topk, groups, width, hidden, seed=tokens)
    layer = layer_type(W1.cuda(), W2.cuda(), capacity)
    out, saved = layer.forward(x.cuda(), ids.cuda(), weights.cuda())
    dout = torch.randn((tokens, width), generator=torch.Generator().manual_seed(7)).half()
    dx, dweights, dW1, dW2 = layer.backward(dout.cuda(), saved)

    X, D, R = x.double(), dout.double(), weights.double()
    o, eo = torch.zeros_like(X), torch.zeros_like(X)
    gx, egx = torch.zeros_like(X), torch.zeros_like(X)
    gr, egr = torch.zeros_like(R), torch.zeros_like(R)
    g1, eg1 = torch.zeros(W1.shape).double(), torch.zeros(W1.shape).double()
    g2, eg2 = torch.zeros(W2.shape).double(), torch.zeros(W2.shape).double()
    for e, (t, j) in enumerate(placed(ids, groups, capacity)):
        A, B = W1[e].double(), W2[e].double()
        none = torch.zeros(len(t), width).double()
        h, eh = product(X[t], none, A)
        eh = f16(h, eh)
        a, ea = silu(h, eh)
        ea = f16(a, ea)
        y, ey = product(a, ea, B)
        ey = f16(y, ey)
        r = R[t, j][:, None]
        o.index_add_(0, t, r * y)
        eo.index_add_(0, t, r * ey + (topk + 2) * U32 * r * (y.abs() + ey))
        # back
        dy = r * D[t]
        edy = f16(dy, 2 * U32 * dy.abs())
        gr[t, j] = (D[t] * y).sum(1)
        egr[t, j] = (D[t].abs() * ey).sum(1) + (width + 4) * U32 * (D[t].abs() * (y.abs() + ey)).sum(1)
        da, eda = product(dy, edy, B.T)
        s = torch.sigmoid(h)
        slope = s * (1 + h * (1 - s))
        dh = da * slope
        eslope = 0.55 * eh + 2.0 ** -20
        edh = f16(dh, eda * (slope.abs() + eslope) + da.abs() * eslope)
        dxr, edxr = product(dh, edh, A.T)
        edxr = f16(dxr, edxr)
        gx.index_add_(0, t, dxr)
        egx.index_add_(0, t, edxr + (topk + 2) * U32 * (dxr.abs() + edxr))
        g2[e], eg2[e] = product(a.T, ea.T, dy, edy)
        g1[e], eg1[e] = product(X[t].T, none.T, dh, edh)
    check(out, o, f16(o, eo), "out")
    check(dx, gx, f16(gx, egx), "dx")
    check(dweights, gr, egr, "dweights")
    check(dW1, g1, eg1, "dW1")
    check(dW2, g2, eg2, "dW2")

    # The formulas themselves, against differences of the definition in 64
    # bits, along one direction of everything that has a gradient.
    g = torch.Generator().manual_seed(11)
    step = [torch.randn(v.shape, generator=g).double() for v in (X, R, g1, g2)]

    def loss(s):
        total = torch.zeros(()).double()
        for e, (t, j) in enumerate(placed(ids, groups, capacity)):
            h = (X + s * step[0])[t] @ (W1[e].double() + s * step[2][e])
            y = h * torch.sigmoid(h) @ (W2[e].double() + s * step[3][e])
            total = total + ((R + s * step[1])[t, j][:, None] * y * D[t]).sum()
        return total.item()

    eps = 1e-5
    slope = (loss(eps) - loss(-eps)) / (2 * eps)
    along = sum((a * b).sum().item() for a, b in zip((gx, gr, g1, g2), step))
    size = sum((a * b).abs().sum().item() for a, b in zip((gx, gr, g1, g2), step))
    assert abs(slope - along) <= 1e-6 * size


@pytest.mark.parametrize("tokens,topk,groups,capacity,width,hidden", CASES)
def test_int8_serving(layer_type, tokens, topk, groups, capacity, width, hidden):
    W1, W2, x, ids, weights = setup(tokens, topk, groups, width, hidden, seed=100 + tokens)
    layer = layer_type(W1.cuda(), W2.cuda(), capacity)
    layer.quantise()
    got = layer.serve(x.cuda(), ids.cuda(), weights.cuda())

    X, R = x.double(), weights.double()

    def half_scale(v, e):
        return (0.5 + 2.0 ** -20) * ((v.abs() + e).max(-1, keepdim=True).values / 127) * (1 + 2.0 ** -20)

    o, eo = torch.zeros_like(X), torch.zeros_like(X)
    for e, (t, j) in enumerate(placed(ids, groups, capacity)):
        A, B = W1[e].double(), W2[e].double()
        ex = half_scale(X[t], 0.0).expand(-1, width) if len(t) else torch.zeros(0, width).double()
        ewa = half_scale(A.T, 0.0).T.expand(width, -1)
        ewb = half_scale(B.T, 0.0).T.expand(hidden, -1)
        h, eh = product(X[t], ex, A, ewa)
        a, ea = silu(h, eh)
        ea = f16(a, ea)
        if len(t):
            ea = ea + half_scale(a, ea)
        y, ey = product(a, ea, B, ewb)
        ey = f16(y, ey)
        r = R[t, j][:, None]
        o.index_add_(0, t, r * y)
        eo.index_add_(0, t, r * ey + (topk + 2) * U32 * r * (y.abs() + ey))
    got = got.cpu().double()
    bound = f16(o, eo)
    assert torch.isfinite(got).all()
    assert ((got - o).abs() <= bound).all()
    # The worst case of every rounding is far from what they do together: as
    # independent errors they come to a few hundredths of the result.
    assert (got - o).norm() <= 0.05 * o.norm()


def test_example_runs(layer_type, capsys):
    from examples import moe_layer
    moe_layer.main()
    lines = capsys.readouterr().out.strip().splitlines()
    assert len(lines) == 2 and all("int8" in line for line in lines)
