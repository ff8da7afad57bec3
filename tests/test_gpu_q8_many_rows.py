"""moe_swiglu_bwd_q8 with more rows than one launch's threads can cover: rows
wider than 1024 columns take a workgroup of 256 threads each, and a grid holds
fewer than 2^32 threads, 2^24 such rows."""

import pytest
import torch

from gpu_support import say
from mixture_experts_expert_amd import moe_swiglu_bwd_q8

pytestmark = pytest.mark.gpu

DEV = "cuda"


def test_rows_past_one_grid():
    I, R = 1088, (1 << 24) + 37
    need = R * (2 * I + 2 * I // 32 + 4 + 2 * I + 4 * I + 4)
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < need + (16 << 30):
        pytest.skip(f"needs {need >> 30} GiB of device memory")
    say(f"[q8] swiglu_bwd R {R} I {I}")
    g = torch.Generator(device=DEV).manual_seed(3)
    codes = torch.empty((R, 2 * I), dtype=torch.int8, device=DEV)
    for lo in range(0, R, 1 << 21):
        codes[lo:lo + (1 << 21)].random_(0, 64, generator=g)
    # the incoming gradient is the codes' own bytes (both are only read): every
    # pair of bytes below 64 is a bf16 in [0, 1)
    d_act = codes.view(torch.bfloat16)
    scales = torch.empty((R, 2 * I // 32), dtype=torch.uint8, device=DEV).random_(118, 122, generator=g)
    probs = torch.rand((R,), generator=g, device=DEV)
    act = torch.empty((R, I), dtype=torch.bfloat16, device=DEV)
    d_pre = torch.empty((R, 2 * I), dtype=torch.bfloat16, device=DEV)
    d_prob = torch.empty((R,), device=DEV)
    edges = [0, (1 << 22) - 40, 1 << 23, (1 << 24) - 64, R - 37]      # first rows, about the powers of two, last rows
    for lo in edges:
        for t in (act, d_pre, d_prob):
            t[max(lo - 64, 0):lo + 64].fill_(7.0)
    moe_swiglu_bwd_q8(codes, scales, d_act, probs, act, d_pre, d_prob)
    torch.cuda.synchronize()
    for lo in edges:
        rows = slice(max(lo - 64, 0), min(lo + 64, R))
        n = rows.stop - rows.start
        a, p, q = (torch.empty((n, *t.shape[1:]), dtype=t.dtype, device=DEV) for t in (act, d_pre, d_prob))
        moe_swiglu_bwd_q8(codes[rows].clone(), scales[rows].clone(), d_act[rows].clone(), probs[rows].clone(), a, p, q)
        for name, got, want in (("act", act, a), ("d_preact", d_pre, p), ("d_prob", d_prob, q)):
            assert torch.equal(got[rows], want), f"{name}, rows from {rows.start}"
    del codes, d_act, scales, probs, act, d_pre, d_prob
    torch.cuda.empty_cache()
