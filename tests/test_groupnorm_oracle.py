"""Pins of the group norm oracle: closed forms, invariants, and its gradients against central
differences."""
import pytest
import torch

from oracle import groupnorm as OG

F = torch.float64


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F)


def test_two_valued_groups():
    # values m +- 3 with eps = 7: rstd = 1/4, z = +-3/4
    x = torch.tensor([2.0 ** 30 + 3, 2.0 ** 30 - 3], dtype=F).repeat(4)[None, :, None].expand(1, 8, 2)
    y, mean, rstd = OG.fwd(x.contiguous(), torch.ones(2, dtype=F), torch.zeros(2, dtype=F), 2, 7.0,
                           "none")
    assert (mean == 2.0 ** 30).all() and (rstd == 0.25).all() and (y.abs() == 0.75).all()


def test_one_group_of_one_channel_is_per_channel():
    x = randn(1, 2, 50, 6)
    y, mean, rstd = OG.fwd(x, torch.ones(6, dtype=F), torch.zeros(6, dtype=F), 6, 0.0, "none")
    assert torch.allclose(mean, x.mean(1)) and torch.allclose(y.mean(1), torch.zeros(2, 6, dtype=F),
                                                              atol=1e-14)
    assert torch.allclose(y.square().mean(1), torch.ones(2, 6, dtype=F))


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_slope_against_differences(kind):
    z = torch.linspace(-9, 9, 401, dtype=F)
    num = (OG.act(z + 1e-5, kind) - OG.act(z - 1e-5, kind)) / 2e-5
    assert (num - OG.slope(z, kind)).abs().max() < 1e-9


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
@pytest.mark.parametrize("n,s,c,groups", [(2, 3, 8, 2), (1, 5, 6, 1), (3, 4, 9, 3)])
def test_gradients_against_differences(n, s, c, groups, kind):
    args = [randn(1, n, s, c), 1 + 0.1 * randn(2, c), 0.1 * randn(3, c)]
    dy, eps = randn(4, n, s, c), 1e-3

    def loss(x, w, b):
        return (dy * OG.fwd(x, w, b, groups, eps, kind)[0]).sum()

    mean, rstd = OG.stats(args[0], groups, eps)
    got = OG.bwd(dy, args[0], mean, rstd, *args[1:], groups, kind)
    for i, grad in enumerate(got):
        num = torch.zeros_like(args[i])
        for at in range(num.numel()):
            step = torch.zeros_like(num)
            step.view(-1)[at] = 1e-5
            up = loss(*[a + step if j == i else a for j, a in enumerate(args)])
            down = loss(*[a - step if j == i else a for j, a in enumerate(args)])
            num.view(-1)[at] = (up - down) / 2e-5
        assert (num - grad).abs().max() < 1e-7


def test_gradient_invariants():
    x, dy = randn(5, 2, 7, 12), randn(6, 2, 7, 12)
    w, b = 1 + 0.1 * randn(7, 12), randn(8, 12)
    mean, rstd = OG.stats(x, 3, 0.0)
    dx, _, _ = OG.bwd(dy, x, mean, rstd, w, b, 3, "silu")
    xhat = (x - OG.wide(mean, 12)) * OG.wide(rstd, 12)
    assert OG.group_mean(dx, 3).abs().max() < 1e-14          # shifts of x change nothing
    assert OG.group_mean(dx * xhat, 3).abs().max() < 1e-14   # nor do scalings, at eps = 0
