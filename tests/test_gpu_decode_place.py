"""moe_ffn_decode with y in the place of an input that it may be."""

import pytest
import torch

from mixture_experts_expert_amd import DecodeBuffers, forward_decode, moe_ffn_decode

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16


@pytest.mark.parametrize("N,H,I,E,K", [(1, 512, 256, 8, 2), (10, 448, 256, 8, 2), (64, 256, 128, 32, 4)])
@pytest.mark.parametrize("place", ["x", "residual", "both"])
def test_y_in_an_inputs_place(N, H, I, E, K, place):
    g = torch.Generator(device=DEV).manual_seed(N)
    w1 = torch.empty((E, 2 * I, H), dtype=BF16, device=DEV).normal_(0, 0.05, generator=g)
    w2 = torch.empty((E, H, I), dtype=BF16, device=DEV).normal_(0, 0.05, generator=g)
    x, r = (torch.randn((N, H), generator=g, device=DEV).to(BF16) for _ in range(2))
    if place == "both":
        r = x
    logits = torch.randn((N, E), generator=g, device=DEV)
    buf = DecodeBuffers(N, H, I, E, K)
    want = forward_decode(buf, logits, x, w1, w2, residual=r).clone()
    cx, cr = x.clone(), r.clone()
    if place == "both":
        cr = cx
    y = cr if place == "residual" else cx
    moe_ffn_decode(logits, cx, w1, w2, buf.topk_ids, buf.topk_probs, buf.workspace, y, residual=cr)
    assert torch.equal(y, want)
