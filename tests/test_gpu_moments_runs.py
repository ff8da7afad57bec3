"""MoEAdamW over two thousand steps with moments in 8 bits, beside itself with
moments in 32: moments and parameters follow.

The bars are those of test_oracle_moments.py, and for their reasons: v's
mean within 1%, the median root and the movement within 5%."""

import pytest
import torch

from gpu_support import say
from mixture_experts_expert_amd import MoEAdamW

pytestmark = pytest.mark.gpu

DEV = "cuda"
SIZES = [4096, 5000, 96]            # whole chunks, and ends


@pytest.mark.parametrize("beta2", [0.95, 0.999])
@pytest.mark.parametrize("kind", ["constant", "normal", "smaller", "gone"])
def test_moments_and_parameters_follow(kind, beta2):
    steps = 2000
    g = torch.Generator(device=DEV).manual_seed(5)
    spread = [torch.exp(torch.randn(n, generator=g, device=DEV)) * 1e-3 for n in SIZES]
    grads = [torch.randn(n, generator=g, device=DEV) * s for n, s in zip(SIZES, spread)]
    opts = [MoEAdamW([torch.zeros(n, device=DEV) for n in SIZES], grads, lr=1e-4, betas=(0.9, beta2), weight_decay=0.0,
                     state=state) for state in ("f32", "q8")]
    for t in range(steps):
        if kind != "constant":
            for x, s in zip(grads, spread):
                x.normal_(generator=g).mul_(s)
                if t >= steps // 2:
                    if kind == "smaller":
                        x.mul_(0.1)
                    elif kind == "gone":
                        x[::2] = 0
        for o in opts:
            o.step_()
    torch.cuda.synchronize()
    true, held = opts
    odd = [torch.arange(n, device=DEV) % 2 == 1 for n in SIZES]
    on = torch.cat(odd if kind == "gone" else [torch.ones_like(x) for x in odd])
    s = torch.cat(spread).double()[on]
    v = torch.cat([true.moment_values(i)[1] for i in range(3)]).double()[on]
    root = torch.cat([held.moment_values(i)[1] for i in range(3)]).double()[on]
    ratio = (root / v.sqrt()).median().item()
    mean = ((root / s).square().mean() / (v / s.square()).mean()).item()
    move = [torch.cat([p.double().abs() for p in o.params]).mean().item() for o in opts]
    say(f"  {kind}, beta2 {beta2}: median root {ratio:.3f}, mean of v {mean:.4f}, movement {move[1] / move[0]:.3f}")
    assert true.step.item() == held.step.item() == steps
    assert abs(ratio - 1) < 0.05 and abs(mean - 1) < 0.01 and abs(move[1] / move[0] - 1) < 0.05
