"""moe_swiglu_bwd and moe_dispatch_rows with more rows than one launch's
threads can cover (a grid holds fewer than 2^32 threads): a wave a row, 2^26
rows, and a thread a 16-byte piece, 2^29 rows of 64 columns."""

import pytest
import torch

from gpu_support import say
from mixture_experts_expert_amd import moe_dispatch_rows, moe_swiglu_bwd

pytestmark = pytest.mark.gpu

DEV = "cuda"


def room(need):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < need + (16 << 30):
        pytest.skip(f"needs {need >> 30} GiB of device memory")


def around(row, R):
    return slice(max(row - 64, 0), min(row + 64, R))


def test_swiglu_bwd_rows_past_one_grid():
    I, R = 64, (1 << 26) + 37
    room(R * (4 * I + 2 * I + 4 + 2 * I + 4 * I + 4))
    say(f"[bwd] swiglu_bwd R {R} I {I}")
    g = torch.Generator(device=DEV).manual_seed(3)
    bf16 = torch.bfloat16
    pre, d_act = (torch.empty((R, n), dtype=bf16, device=DEV) for n in (2 * I, I))
    for lo in range(0, R, 1 << 24):
        pre[lo:lo + (1 << 24)].normal_(generator=g)
        d_act[lo:lo + (1 << 24)].normal_(generator=g)
    probs = torch.rand((R,), generator=g, device=DEV)
    act, d_pre, d_prob = torch.empty((R, I), dtype=bf16, device=DEV), torch.empty_like(pre), torch.empty((R,), device=DEV)
    edges = [0, 1 << 24, 1 << 25, (1 << 26) - 64, R]
    for row in edges:
        for t in (act, d_pre, d_prob):
            t[around(row, R)] = 7.0
    moe_swiglu_bwd(pre, d_act, probs, act, d_pre, d_prob)
    torch.cuda.synchronize()
    for row in edges:
        s = around(row, R)
        want = [torch.empty_like(t[s]) for t in (act, d_pre, d_prob)]
        moe_swiglu_bwd(pre[s].clone(), d_act[s].clone(), probs[s].clone(), *want)
        for name, t, w in zip(("act", "d_preact", "d_prob"), (act, d_pre, d_prob), want):
            assert torch.equal(t[s], w), f"{name}, rows from {s.start}"
    del pre, d_act, probs, act, d_pre, d_prob, t
    torch.cuda.empty_cache()


def test_dispatch_rows_past_one_grid():
    N, H, R = 1000, 64, (1 << 29) + 37
    room(R * (2 * H + 4))
    say(f"[dispatch] R {R} H {H}")
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn((N, H), generator=g, device=DEV).to(torch.bfloat16)
    ids = torch.empty((R,), dtype=torch.int32, device=DEV).random_(0, N + 1, generator=g)     # N: a zero row
    rows = torch.empty((R, H), dtype=torch.bfloat16, device=DEV)
    edges = [0, 1 << 27, 1 << 28, (1 << 29) - 64, R]
    for row in edges:
        rows[around(row, R)] = 7.0
    moe_dispatch_rows(x, ids, rows)
    torch.cuda.synchronize()
    full = torch.cat([x, torch.zeros_like(x[:1])])
    for row in edges:
        s = around(row, R)
        assert torch.equal(rows[s], full[ids[s].to(torch.int64)]), f"rows from {s.start}"
    del ids, rows
    torch.cuda.empty_cache()
