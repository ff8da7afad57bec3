"""AdamW's list holds the memory that its plan names, also of tensors that are
given other memory later."""

import gc

import pytest
import torch

from mixture_experts_expert_amd import MoEAdamW

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("which", ["param", "grad", "master", "moment"])
def test_memory_that_a_tensor_gave_up_is_not_handed_out(which):
    n = 3 << 20                                  # a block of its own in the allocator
    p, g = torch.ones(n, dtype=torch.bfloat16, device=DEV), torch.ones(n, device=DEV)
    opt = MoEAdamW([p], [g], lr=1e-3, masters="make")
    t = dict(param=p, grad=g, master=opt.masters[0], moment=opt.moments["m"][0])[which]
    old = t.data_ptr()
    t.data = torch.zeros_like(t)                 # what module.to() and the like do
    gc.collect()
    others = [torch.full((n,), 7, dtype=t.dtype, device=DEV) for _ in range(4)]
    assert all(o.data_ptr() != old for o in others)
    opt.step_()
    torch.cuda.synchronize()
    assert all((o == 7).all() for o in others)
