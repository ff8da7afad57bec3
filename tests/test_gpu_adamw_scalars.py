"""AdamW's device scalars and eps at the ends of their ranges."""

import pytest
import torch

from mixture_experts_expert_amd import MoEAdamW, moe_grad_norm

pytestmark = pytest.mark.gpu

DEV = "cuda"


def optimizer(state, step, n=5000, g=0.5, **kw):
    return MoEAdamW([torch.ones(n, device=DEV)], [torch.full((n,), g, device=DEV)], lr=1e-3, weight_decay=0.0, state=state,
                    step=step, **kw)


@pytest.mark.parametrize("state", ["f32", "q8"])
@pytest.mark.parametrize("step", [-1, -7, -(1 << 31)])
def test_a_step_number_below_0_counts_as_0(state, step):
    a, b = optimizer(state, step), optimizer(state, 0)
    for o in (a, b):
        o.step_()
    assert a.step.item() == 1 and torch.equal(a.params[0], b.params[0]) and torch.isfinite(a.params[0]).all()
    assert all(torch.equal(x, y) for x, y in zip(sum(a.moments.values(), []), sum(b.moments.values(), [])))


@pytest.mark.parametrize("state", ["f32", "q8"])
def test_the_last_step_number_stays(state):
    top = (1 << 31) - 1
    for step in (top - 1, top):
        o = optimizer(state, step)
        o.step_()
        assert o.step.item() == top
        # the corrections have become 1: m 0.05, root sqrt(0.05 / 4), each within 8u and the rounding of p
        want = 1 - 1e-3 * 0.05 / (0.0125 ** 0.5 + 1e-8)
        assert (o.params[0].double() - want).abs().max() < 2.0 ** -22


def test_the_smallest_eps():
    """Nothing to divide by but eps: an element without a gradient stays, and 2^-126 is a divisor like any other."""
    for eps in (2.0 ** -126, 2.0 ** -100):
        o = MoEAdamW([torch.ones(64, device=DEV)], [torch.zeros(64, device=DEV)], lr=1e-3, weight_decay=0.0, eps=eps)
        o.step_()
        assert (o.params[0] == 1).all()
        # v underflows to 0, m does not: p = 1 - 1e-3 * 2^-80 / eps, off by m's and the division's 8u
        o.grads[0].fill_(2.0 ** -80)
        o.step.zero_()
        o.step_()
        move = 1e-3 * 2.0 ** -80 / eps
        assert ((o.params[0].double() - (1 - move)).abs() <= 2.0 ** -20 * (1 + move)).all()


def test_the_norm_within_its_bound():
    """Eight squares are added in float32, each addition and each product off by u of the sum so far: 8u of their sum at
    most, 4u of its root, and the last rounding: 5u.  Groups of eight that a search found to round far to one side, all
    alike so that nothing averages out, and random ones."""
    u = 2.0 ** -24
    g = torch.Generator().manual_seed(0)
    x = (1 + torch.rand((1 << 16, 8), generator=g))
    s = torch.zeros(1 << 16, dtype=torch.float64)
    for j in range(8):                           # a fused product and addition, rounded to float32 (or both apart: as good)
        s = (s + x[:, j].double().square()).float().double()
    off = (s.sqrt() / x.double().square().sum(1).sqrt() - 1).abs()
    assert off.max() > 1.5 * u
    for row in off.topk(4).indices.tolist() + [0]:
        for dt in (torch.float32, torch.bfloat16):
            grad = x[row].repeat(1 << 12).to(dt).to(DEV)
            opt = MoEAdamW([torch.zeros(grad.numel(), device=DEV)], [grad], max_norm=1.0)
            moe_grad_norm(opt.table, opt.norm)
            want = grad.double().square().sum().sqrt().item()
            assert abs(opt.norm.item() - want) <= 5 * u * want
