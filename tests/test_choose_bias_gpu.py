"""Biases of any size in the choice of experts.  Choices are compared for equality
with those of 64 bits."""
import pytest
import torch

from test_choose_gpu import INF, b, check  # noqa: F401  (b: a fixture)

pytestmark = pytest.mark.gpu

LOW, HIGH = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
# The choices and groups of a call: among candidates in a lane each, and (few kept lanes that
# hold more experts than a warp has lanes) one after another.
FORMS = [(64, 6, 8, 4), (64, 6, 8, 1), (256, 8, 8, 2), (512, 9, 4, 1), (12, 3, 6, 2)]


def group_biases(E, groups, keep, g):
    """Biases that leave f32 in a group's sum, or begin outside it."""
    per = E // groups
    small = 0.1 * torch.randn(E, generator=g)
    whole = small.view(groups, per)
    for hidden in sorted({1, groups - keep, min(groups - keep + 1, groups), groups}):
        for first in (0, groups - hidden):
            bias = whole.clone()
            bias[first:first + hidden] = LOW
            yield bias.flatten()
    for pinned in (1, keep, keep + 1, groups):
        for at in (0, per - 1):
            bias = whole.clone()
            bias[groups - pinned:, at] = INF
            yield bias.flatten()
    bias = whole.clone()
    bias[groups - 1] = INF
    yield bias.flatten()
    # Sums of 1.2 to 2 times the largest number, in another order than the groups'.
    bias = whole.clone()
    order = torch.randperm(groups, generator=g)
    bias[:, 0] = HIGH
    bias[:, 1 % per] = HIGH * (0.2 + 0.8 * order.float() / groups)
    yield bias.flatten()
    yield -bias.flatten()


@pytest.mark.parametrize("E,k,groups,keep", FORMS)
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_sums_outside_f32(b, score, best, E, k, groups, keep):  # noqa: F811
    g = torch.Generator().manual_seed(E + keep)
    x = torch.randn((21, E), generator=g)
    for bias in group_biases(E, groups, keep, g):
        check(b, x, k, score=score, bias=bias, groups=groups, keep=keep, best=best, renormalize=True)


@pytest.mark.parametrize("E,k", [(64, 6), (256, 8), (1000, 31), (40, 32), (2, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_infinite_biases(b, score, E, k):  # noqa: F811
    """From one to all experts, spread over the warp's lanes or together."""
    g = torch.Generator().manual_seed(E)
    x = torch.randn((21, E), generator=g)
    for pinned in sorted({1, k - 1, k, min(k + 1, E), min(k + 5, E), E}):
        for at in (torch.randperm(E, generator=g)[:pinned], torch.arange(E - pinned, E),
                   (torch.arange(pinned) * E) // max(pinned, 1)):
            bias = 0.1 * torch.randn(E, generator=g)
            bias[at] = INF
            check(b, x, k, score=score, bias=bias)
            bias[at[::2]] = HIGH
            check(b, x, k, score=score, bias=bias)


@pytest.mark.parametrize("size", [100.0, 1000.0, 1e5])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_that_cancel_in_pairs(b, score, size):  # noqa: F811
    """Groups of two with biases of +size and -size: their sums are those of two scores,
    each added to a bias that rounds it."""
    T = 1 << 20
    x = torch.randn((T, 4), generator=torch.Generator().manual_seed(int(size)))
    x[0] = torch.tensor([-0.35108897, 1.4023322, 0.89841217, 0.020195935])
    for bias in (torch.tensor([size, -size, -size, size]), torch.tensor([-size, size, size, -size]),
                 torch.tensor([size, -size, size, -size])):
        d, c = x.double(), bias.double()
        s = torch.softmax(d, 1) if score == "softmax" else 1 / (1 + torch.exp(-d))
        c = s + c
        v = c.view(T, 2, 2).sum(2)
        first = torch.where(v[:, 1] > v[:, 0], 2, 0)
        want = first + (c.gather(1, first[:, None] + 1) > c.gather(1, first[:, None]))[:, 0]
        ids, _ = b.moe_choose(x.cuda(), 1, score=score, bias=bias.cuda(), groups=2, keep_groups=1)
        assert torch.equal(ids.cpu()[:, 0].long(), want)


@pytest.mark.parametrize("size", [1000.0, 1e5])
@pytest.mark.parametrize("E,k,groups,keep", FORMS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_that_cancel_in_groups(b, score, E, k, groups, keep, size):  # noqa: F811
    """A group's largest two cancel but for their scores; the other experts lie below."""
    g = torch.Generator().manual_seed(E * 3 + keep)
    x = torch.randn((600, E), generator=g)
    bias = torch.full((groups, E // groups), -2 * size)
    bias[:, 0], bias[:, -1] = -size, size
    check(b, x, k, score=score, bias=bias.flatten(), groups=groups, keep=keep)
    # Of one group only, which then decides about the others.
    only = 0.1 * torch.randn((groups, E // groups), generator=g)
    only[groups // 2] = bias[groups // 2]
    check(b, x, k, score=score, bias=only.flatten(), groups=groups, keep=keep)


def test_what_64_bits_cannot_tell_apart(b):  # noqa: F811
    """Scores are compared as 64 bits hold them: with a bias sigmoids of logits past 37
    are all 1 and go to the lower number; without one the logits decide."""
    x = torch.zeros((3, 16))
    x[:, 3], x[:, 9], x[:, 12] = 40.0, 45.0, 38.0
    assert b.moe_choose(x.cuda(), 3, score="sigmoid")[0].tolist() == [[9, 3, 12]] * 3
    assert b.moe_choose(x.cuda(), 3, score="sigmoid", bias=torch.zeros(16).cuda())[0].tolist() == [[3, 9, 12]] * 3
    # (Sums of a group's two best are sums of scores, with a bias or without.)
    y = torch.zeros((3, 8))
    y[:, 2], y[:, 3], y[:, 4], y[:, 5] = 40.0, 41.0, 44.0, 45.0
    for bias in (None, torch.zeros(8).cuda()):
        ids, _ = b.moe_choose(y.cuda(), 2, score="sigmoid", bias=bias, groups=4, keep_groups=1)
        assert sorted(ids[0].tolist()) == [2, 3]
    ids, _ = b.moe_choose(y.cuda(), 2, score="sigmoid", groups=4, keep_groups=1, group_best=1)
    assert ids.tolist() == [[5, 4]] * 3
