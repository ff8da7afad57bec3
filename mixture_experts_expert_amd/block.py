"""A transformer block's feed-forward half around the MoE layer, from residual
stream to residual stream:

    total = x + residual;  u = norm(total);  logits = u router^T
    stream = total + MoE(u, logits)

MoEBlock holds the weights and runs it for the few tokens of a decode step;
MoEBlockStep holds the buffers of a training step and runs it forward and
backward, leaving gradients for MoEAdamW.  A stream is handed on as its two
parts, (y, total): the next block's norm adds them.  The norm, the layer and
their backward run in libmoe_native's kernels; the router's product is a plain
float32 matrix product of torch's.
"""

from __future__ import annotations

import torch

from . import _native as nat
from .forward import DecodeBuffers, MoEBackwardBuffers, MoEBuffers, forward_decode


class MoEBlock:
    """norm_weight float32 [H] (norm_bias likewise, or None), router float32
    [E, H], w1 bf16 [E, 2I, H], w2 bf16 [E, H, I], K experts a token.  rms: RMS
    norm, else layer norm."""

    def __init__(self, norm_weight, router, w1, w2, K: int, norm_bias=None, rms: bool = True, eps: float = 1e-6):
        self.E, I2, self.H = w1.shape
        self.I, self.K = I2 // 2, K
        if router.shape != (self.E, self.H) or w2.shape != (self.E, self.H, self.I) or norm_weight.shape != (self.H,):
            raise ValueError("need norm_weight [H], router [E, H], w1 [E, 2I, H] and w2 [E, H, I]")
        self.norm_weight, self.norm_bias, self.router, self.w1, self.w2 = norm_weight, norm_bias, router, w1, w2
        self.rms, self.eps = bool(rms), float(eps)

    def params(self):
        """The weights, in the order of MoEBlockStep.grads()."""
        return [self.norm_weight] + ([self.norm_bias] if self.norm_bias is not None else []) + [
            self.router, self.w1, self.w2]

    def decode_buffers(self, N: int) -> "BlockDecodeBuffers":
        return BlockDecodeBuffers(self, N)

    def decode(self, buf: "BlockDecodeBuffers", x, residual, n_live=None):
        """The stream of n <= buf.layer.N tokens (bf16 [n, H]) behind the block,
        whole: three launches of the library and the router's product.  Valid
        until the next call with the same buffers."""
        n = x.shape[0]
        if n > buf.layer.N:
            raise ValueError(f"{n} tokens, the buffers hold {buf.layer.N}")
        total, u = buf.total[:n], buf.u[:n]
        nat.moe_layer_norm_fwd(x, self.norm_weight, self.norm_bias, self.eps, u, buf.mean[:n] if buf.mean is not None else None,
                               buf.rstd[:n], residual=residual, total=total)
        logits = torch.mm(u.float(), self.router.t())
        return forward_decode(buf.layer, logits, u, self.w1, self.w2, residual=total, n_live=n_live)


class BlockDecodeBuffers:
    """Device buffers for MoEBlock.decode of up to N tokens."""

    def __init__(self, block: MoEBlock, N: int):
        dev, bf16 = block.w1.device, torch.bfloat16
        self.layer = DecodeBuffers(N, block.H, block.I, block.E, block.K, dev)
        self.total = torch.zeros((N, block.H), dtype=bf16, device=dev)
        self.u = torch.zeros((N, block.H), dtype=bf16, device=dev)
        self.mean = None if block.rms else torch.zeros(N, device=dev)
        self.rstd = torch.zeros(N, device=dev)


class MoEBlockStep:
    """Device buffers of one training step of a block over N tokens, capacity
    factor F.  Weight gradients are added into float32 buffers (grads(), zeroed
    by zero_grad()); checkpoint as in MoEBackwardBuffers."""

    def __init__(self, block: MoEBlock, N: int, F: float, checkpoint: str = "bf16"):
        self.block, self.N = block, N
        H, dev, bf16 = block.H, block.w1.device, torch.bfloat16
        self.layer = MoEBuffers(N, H, block.I, block.E, block.K, F, dev)
        self.bwd = MoEBackwardBuffers(self.layer, main_grad=True, checkpoint=checkpoint)
        self.total = torch.zeros((N, H), dtype=bf16, device=dev)
        self.u = torch.zeros((N, H), dtype=bf16, device=dev)
        self.mean = None if block.rms else torch.zeros(N, device=dev)
        self.rstd = torch.zeros(N, device=dev)
        self.dx = torch.zeros((N, H), dtype=bf16, device=dev)
        self.d_norm_weight = torch.zeros(H, device=dev)
        self.d_norm_bias = None if block.norm_bias is None else torch.zeros(H, device=dev)
        self.d_router = torch.zeros((block.E, H), device=dev)
        self.workspace = nat.layer_norm_workspace(N, H, dev)

    def grads(self):
        """The weights' gradients, in the order of MoEBlock.params()."""
        return [self.d_norm_weight] + ([self.d_norm_bias] if self.d_norm_bias is not None else []) + [
            self.d_router, self.bwd.main_dw1, self.bwd.main_dw2]

    def zero_grad(self):
        for g in self.grads():
            g.zero_()

    def forward(self, x, residual):
        """(y, total): the two parts of the stream behind the block (bf16 [N, H])."""
        b = self.block
        nat.moe_layer_norm_fwd(x, b.norm_weight, b.norm_bias, b.eps, self.u, self.mean, self.rstd, residual=residual,
                               total=self.total)
        logits = torch.mm(self.u.float(), b.router.t())
        return self.bwd.forward(logits, self.u, b.w1, b.w2), self.total

    def backward(self, d):
        """From the gradient d of the stream (bf16 [N, H], the same for both parts)
        to dx, the gradient of x and of residual; the weights' are added."""
        b = self.block
        self.bwd.backward(d, self.u, b.w1, b.w2)
        self.d_router.addmm_(self.bwd.d_logits.t(), self.u.float())
        # the router's part is added in float32 to the experts' (bwd.dx, rounded to bf16 by the layer's backward), and
        # their sum rounded to u's type
        du = torch.addmm(self.bwd.dx.float(), self.bwd.d_logits, b.router).to(torch.bfloat16)
        nat.moe_layer_norm_bwd(du, self.total, b.norm_weight, self.mean, self.rstd, self.dx, self.d_norm_weight,
                               self.d_norm_bias, self.workspace, dtotal=d, accumulate=True)
        return self.dx
