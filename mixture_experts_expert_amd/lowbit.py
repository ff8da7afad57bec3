"""Expert weights in 4 bits, for the dropless forward and the serving ladder.

W4Weights holds one weight tensor [E, rows, cols] as 4-bit codes and one scale
byte for every 32 columns (layout: include/moe_lowbit.h).  A pair of them goes
where the bf16 weights go: forward_dropless(buf, logits, x, w1, w2) and
ServingLadder(w1, w2, ...).
"""

from __future__ import annotations

import torch

from . import _native as nat


def _hand_over(stream, *tensors: torch.Tensor):
    """Order `stream` (None: the current one) behind the current stream, where
    the fresh outputs among `tensors` were allocated: work pending there may
    still write their blocks.  The allocator learns that `stream` uses them
    all, so that none is handed out again too early."""
    if stream is None:
        return
    t = tensors[0]
    nat._here_of(t, "the tensor", stream)             # refusals come first
    if not hasattr(stream, "wait_stream"):            # a raw handle
        stream = torch.cuda.ExternalStream(int(stream), device=t.device)
    stream.wait_stream(torch.cuda.current_stream(t.device))
    for t in tensors:
        t.record_stream(stream)


class W4Weights:
    """codes uint8 [E, rows, cols/2] and scales uint8 [E, rows, cols/32]."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales must be uint8")
        self.shape = nat._w4_shape(codes, scales, "W4Weights")
        self.codes, self.scales = codes, scales

    @classmethod
    def quantize(cls, w: torch.Tensor, stream=None) -> "W4Weights":
        """From bf16 weights [E, rows, cols] on the device.  With a stream, the
        conversion runs there, behind the current stream's work so far."""
        if w.dim() != 3 or w.shape[2] % 32:
            raise ValueError("w must be [E, rows, cols] with cols a multiple of 32")
        E, rows, cols = w.shape
        codes = torch.empty((E, rows, cols // 2), dtype=torch.uint8, device=w.device)
        scales = torch.empty((E, rows, cols // 32), dtype=torch.uint8, device=w.device)
        _hand_over(stream, w, codes, scales)
        nat.moe_w4_quantize(w, codes, scales, stream)
        return cls(codes, scales)

    def dequantize(self, stream=None) -> torch.Tensor:
        """The bf16 weights the codes stand for (exact).  With a stream, as quantize."""
        w = torch.empty(self.shape, dtype=torch.bfloat16, device=self.codes.device)
        _hand_over(stream, w, self.codes, self.scales)
        nat.moe_w4_dequantize(self.codes, self.scales, w, stream)
        return w


def is_w4(w1, w2) -> bool:
    """Whether a layer's weights are 4-bit: both or neither."""
    a, b = isinstance(w1, W4Weights), isinstance(w2, W4Weights)
    if a != b:
        raise TypeError("w1 and w2 must both be W4Weights, or neither")
    return a
