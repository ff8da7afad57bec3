"""AdamW over many tensors at once, clipped by the gradients' global norm.

The gradients are buffers that the backward writes (a MoEBackwardBuffers'
main_dw1 and main_dw2, a norm's dweight), so a step is two launches for any
number of tensors, reads nothing back and can be captured into a hipGraph with
the backward: the learning rate and the number of the step are device scalars.
All arithmetic runs in libmoe_native's kernels.
"""

from __future__ import annotations

import warnings

import torch

from . import _native as nat


class MoEAdamW:
    """The optimizer's state for parameters `params` (bf16 or float32 device
    tensors) with gradients `grads` (bf16 or float32, the same buffers every
    step).

    masters      None; "make": a float32 copy of each bf16 parameter, which the
                 step updates and the parameter is rounded from; or the copies
    state        "f32": moments in 32 bits; "q8": in 8 (include/moe_block.h)
    max_norm     gradients are scaled down to this global norm where theirs is
                 larger, and a step whose norm is not finite is not taken
                 (None: neither)
    weight_decay one number, or one for each parameter
    moments      None (zeros), or dict(m=, v=[, m_scales=, v_scales=]) of lists:
                 another run's state, used as it is
    rounding     of 8-bit moments after a step: "stochastic" (a hash of `seed`, the
                 step and the element's place; the moments follow the gradients),
                 or "nearest" (for a step or a few: over many the moments stay
                 behind, see include/moe_moments.h).  None: stochastic for moments
                 made here; moments handed in are rounded to nearest, with a
                 warning, so a program that goes on with a run says "stochastic"
    seed         0 to 2^32 - 1; a run that goes on takes its own again
    lr           a number, or a float32 [1] device tensor to be written between steps
    step         a number of steps taken, or an int32 [1] device tensor

    norm (float32 [1]) holds the last step's global norm, step the steps taken.
    Parameters, gradients and state stay where they are from here on.  What is
    made here is made on the current stream; no parameter may be given twice.
    """

    def __init__(self, params, grads, lr=1e-3, betas=(0.9, 0.95), eps: float = 1e-8, weight_decay=0.1,
                 max_norm=None, state: str = "f32", masters=None, moments=None, step=0, rounding=None, seed: int = 0):
        params, grads = list(params), list(grads)
        if state not in ("f32", "q8"):
            raise ValueError('state must be "f32" or "q8"')
        if not params:
            raise ValueError("no parameters")
        for p in params:
            if not isinstance(p, torch.Tensor):
                raise TypeError("a parameter must be a torch.Tensor")
        if max_norm is not None and not max_norm > 0:
            raise ValueError("max_norm must be above 0")
        b1, b2 = betas
        if not (0 <= b1 < 1 and 0 <= b2 < 1) or not eps >= 0:
            raise ValueError("need 0 <= beta < 1 and eps >= 0")
        if 0 < eps < 2.0 ** -126:
            raise ValueError("eps must be 0 or a normal float32 number, 2^-126 or more")
        if rounding not in (None, "stochastic", "nearest") or (rounding and state != "q8"):
            raise ValueError('rounding must be "stochastic" or "nearest", and goes with state "q8"')
        if not 0 <= seed < 1 << 32:
            raise ValueError("seed must be 0 to 2^32 - 1")
        dev = params[0].device
        self.betas, self.eps, self.max_norm, self.state = (float(b1), float(b2)), float(eps), max_norm, state
        if masters == "make":
            masters = [p.float() if p.dtype == torch.bfloat16 else None for p in params]
        given = moments is not None
        if moments is None:
            kind = torch.float32 if state == "f32" else torch.uint8
            moments = {k: [torch.zeros(p.numel(), dtype=kind, device=dev) for p in params] for k in ("m", "v")}
            if state == "q8":
                for k in ("m_scales", "v_scales"):
                    moments[k] = [torch.ones(-(-p.numel() // 32), dtype=torch.uint8, device=dev) for p in params]
        if (state == "q8") != ("m_scales" in moments):
            raise ValueError("8-bit moments come with scales, 32-bit ones without")
        if state == "q8" and rounding is None:
            rounding = "nearest" if given else "stochastic"
            if given:
                warnings.warn('8-bit moments rounded to nearest do not follow their gradients over many steps; rounding="stochastic" '
                              'goes on with a run, rounding="nearest" says that this is meant', stacklevel=2)
        self.rounding, self.seed = rounding, int(seed)
        self.params, self.grads, self.masters, self.moments = params, grads, masters, moments
        self.table = nat.AdamWTable(params, grads, moments["m"], moments["v"], moments.get("m_scales"),
                                    moments.get("v_scales"), masters, weight_decay)
        self.lr = lr if isinstance(lr, torch.Tensor) else torch.full((1,), float(lr), device=dev)
        self.step = step if isinstance(step, torch.Tensor) else torch.full((1,), int(step), dtype=torch.int32, device=dev)
        self.norm = torch.zeros(1, device=dev)

    def step_(self, stream=None):
        """Clip and step: every parameter, moment and master copy, in place."""
        clip = {}
        if self.max_norm is not None:
            nat.moe_grad_norm(self.table, self.norm, stream)
            clip = dict(grad_norm=self.norm, max_norm=self.max_norm)
        if self.rounding == "stochastic":
            nat.moe_adamw_step_stochastic(self.table, self.lr, self.betas, self.eps, self.step, self.seed, stream=stream, **clip)
        else:
            nat.moe_adamw_step(self.table, self.lr, self.betas, self.eps, self.step, stream=stream, **clip)

    def moment_values(self, i: int, stream=None):
        """What parameter i's moments stand for: (m, root of v) in bf16 for 8-bit
        moments, (m, v) themselves for 32-bit ones."""
        if self.state == "f32":
            return self.moments["m"][i], self.moments["v"][i]
        k = self.moments
        out = [torch.empty(self.params[i].numel(), dtype=torch.bfloat16, device=self.params[i].device) for _ in range(2)]
        nat.moe_moment_values(k["m"][i], k["m_scales"][i], k["v"][i], k["v_scales"][i], *out, stream=stream)
        return tuple(out)
