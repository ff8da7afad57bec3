"""The entry point of include/moe_moments.h: exported with its arguments, and
what it and its Python side refuse.  No device work."""

import ctypes
import re

import pytest
import torch

import mixture_experts_expert_amd as moe
from mixture_experts_expert_amd import _native as nat
from test_abi import ALIGNED as A, INVALID, MIS, MISALIGNED, NUL
from test_block_abi import BIG, table


def test_the_declared_symbol_is_exported_with_its_arguments():
    assert moe.header_functions(moe.MOMENTS_HEADER_PATH) == ["moe_adamw_step_stochastic"]
    text = re.sub(r"/\*.*?\*/", "", open(moe.MOMENTS_HEADER_PATH).read(), flags=re.S)
    args = re.search(r"moe_adamw_step_stochastic\s*\((.*?)\)\s*;", text, flags=re.S).group(1)
    assert len(args.split(",")) == len(nat._SIGNATURES["moe_adamw_step_stochastic"][1])


def test_validation():
    f = moe.lib.moe_adamw_step_stochastic
    t = table(m_scales=4097, v_scales=4099)

    def step(t=t, count=1, p=A, size=BIG, lr=A, b1=0.9, b2=0.95, eps=1e-8, norm=NUL, most=0.0, at=A):
        return f(t, count, p, size, lr, b1, b2, eps, norm, most, at, 0, NUL)
    assert step(t=table()) == INVALID                             # moments in 32 bits
    assert step(t=None) == INVALID and step(count=-1) == INVALID and step(p=NUL) == INVALID and step(p=MIS) == MISALIGNED
    assert step(size=ctypes.c_size_t(8)) == INVALID and step(b1=1.0) == INVALID and step(b2=-0.1) == INVALID
    assert step(eps=-1.0) == INVALID and step(norm=A, most=0.0) == INVALID and step(lr=NUL) == INVALID
    assert step(at=NUL) == INVALID and step(at=ctypes.c_void_p(4098)) == MISALIGNED


def test_the_optimizer_refuses():
    z = torch.zeros
    for kw in (dict(state="f32", rounding="stochastic"), dict(state="f32", rounding="nearest"),
               dict(state="q8", rounding="up"), dict(rounding="stochastic")):
        with pytest.raises(ValueError, match="rounding"):
            moe.MoEAdamW([z(8)], [z(8)], **kw)
    for seed in (-1, 1 << 32):
        with pytest.raises(ValueError, match="seed"):
            moe.MoEAdamW([z(8)], [z(8)], state="q8", seed=seed)
    with pytest.raises(ValueError, match="seed"):
        moe.moe_adamw_step_stochastic(None, None, (0.9, 0.95), 1e-8, None, -1)
