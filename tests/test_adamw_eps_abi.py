"""AdamW refuses an eps that float32 holds as a subnormal number, which the
kernel's division would take for 0.  No device work: every call is refused."""

import pytest
import torch

import mixture_experts_expert_amd as moe
from test_abi import ALIGNED as A, INVALID, NUL, UNSUPPORTED
from test_block_abi import BIG, table

TINY = 2.0 ** -126


@pytest.mark.parametrize("stochastic", [False, True])
def test_the_calls(stochastic):
    t = table(m_scales=4097, v_scales=4099)

    def step(eps, lr=A):
        args = (t, 1, A, BIG, lr, 0.9, 0.95, eps, NUL, 0.0, A)
        if stochastic:
            return moe.lib.moe_adamw_step_stochastic(*args, 0, NUL)
        return moe.lib.moe_adamw_step(*args, NUL)
    for eps in (1e-39, 1e-60, 5e-324, TINY * (1 - 2.0 ** -20)):
        assert step(eps) == UNSUPPORTED, eps
    for eps in (0.0, TINY, 1e-8):                       # taken: the missing rate is what is refused
        assert step(eps, lr=NUL) == INVALID, eps


def test_the_optimizer():
    z = torch.zeros(8)
    with pytest.raises(ValueError, match="eps must be"):
        moe.MoEAdamW([z], [z], eps=1e-39)
