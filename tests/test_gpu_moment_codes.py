"""8-bit moments rounded to nearest: every root's value is the one that is
wanted, the lowest code's too (which is wanted below half-way to the next one and
nowhere else), from moe_moment_codes and from a step.

A root is float32, off by 2u of itself from moe_moment_codes and by 16u from a
step (u = 2^-24; the bounds of test_gpu_adamw.py), 32 steps at most: within 2^-14
of a step from the middle between two codes it may go to either."""

import numpy as np
import pytest
import torch

from mixture_experts_expert_amd import MoEAdamW, moe_moment_codes, moe_moment_values
from oracle import moments as M

pytestmark = pytest.mark.gpu

DEV = "cuda"


def codes(m, v):
    n = m.numel()
    c = [torch.zeros(k, dtype=torch.uint8, device=DEV) for k in (n, -(-n // 32), n, -(-n // 32))]
    moe_moment_codes(m, v, *c)
    return c


def values(c):
    n = c[0].numel()
    m, r = (torch.empty(n, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    moe_moment_values(*c, m, r)
    return m.double().cpu().numpy(), r.double().cpu().numpy()


def check(got, root):
    """Values held against exact roots (a multiple of 32 of them)."""
    want, slack = M.root_nearest(root), 2.0 ** -14
    lo, hi = M.root_nearest(root * (1 - slack / 32)), M.root_nearest(root * (1 + slack / 32))
    sure = lo == hi
    assert sure.mean() > 0.99
    assert (got == want)[sure].all(), (got[sure & (got != want)][:4], want[sure & (got != want)][:4])
    assert ((got == lo) | (got == hi))[~sure].all()
    assert ((got > 0) == (root > 0)).all()


@pytest.mark.parametrize("spread", [0.5, 3.0, 8.0])      # 8: many roots of a group below the smallest code
def test_codes_of_given_moments(spread):
    g = torch.Generator(device=DEV).manual_seed(int(10 * spread))
    n = 1 << 16
    root = torch.randn(n, generator=g, device=DEV).abs() * torch.exp(spread * torch.randn(n, generator=g, device=DEV))
    v = root.square()
    v[::97] = 0
    m = torch.randn(n, generator=g, device=DEV) * torch.exp(spread * torch.randn(n, generator=g, device=DEV))
    got_m, got_r = values(codes(m, v))
    check(got_r, np.sqrt(v.double().cpu().numpy()))
    assert (got_m == M.first_nearest(m.double().cpu().numpy())).all()
    lowest = got_r.reshape(-1, 32) == M.LOWEST_ROOT * M._scale(got_r.reshape(-1, 32).max(1), 1.9375)[:, None]
    assert spread < 8 or lowest.mean() > 0.01


@pytest.mark.parametrize("spread", [0.5, 8.0])
def test_codes_after_a_step(spread):
    g = torch.Generator(device=DEV).manual_seed(3)
    n = 1 << 15
    rnd = lambda: torch.randn(n, generator=g, device=DEV) * torch.exp(spread * torch.randn(n, generator=g, device=DEV))  # noqa: E731
    c = codes(rnd(), rnd().square())
    grad = rnd()
    _, r = values(c)
    opt = MoEAdamW([torch.zeros(n, device=DEV)], [grad], betas=(0.9, 0.95), state="q8", rounding="nearest", step=5,
                   moments=dict(m=[c[0]], m_scales=[c[1]], v=[c[2]], v_scales=[c[3]]))
    opt.step_()
    check(values(c)[1], np.sqrt(0.95 * r * r + 0.05 * grad.double().cpu().numpy() ** 2))
