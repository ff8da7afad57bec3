"""The 4-bit FFN in the forms that few sizes take: the streaming kernel's second
pass over its weights (an expert with more than 16 rows where the average is
small) with several steps, panels of scales and both alignments of their rows;
the bounds of early streaming; the other kernels' less usual alignments; and
the float32 combine of 9 to 16 routes a token.  Bars as in test_gpu_w4.py, and
every token alone equals the token in the batch, bit for bit."""

import numpy as np
import pytest
import torch

import moe_inputs
from gpu_support import host, say
from mixture_experts_expert_amd import DroplessBuffers
from test_gpu_w4 import DEV, case, check, live_slots, run

pytestmark = pytest.mark.gpu


def pads_as_set(buf):
    rest = torch.ones(buf.R, dtype=torch.bool, device=DEV)
    rest[torch.from_numpy(live_slots(buf)[0]).to(DEV)] = False
    return bool((buf.act[rest] == 7).all()) and bool((buf.route_out[rest] == 7).all())


def alone(buf, logits, x, w1, w2, y, tokens):
    """Tokens one at a time (few tiles: other kernels) against the batch's rows."""
    for t in tokens:
        b = DroplessBuffers(1, buf.H, buf.I, buf.E, buf.K, DEV, w4=True)
        b.route(logits[t:t + 1].clone())             # rows of 9 floats are not 16-byte aligned
        assert torch.equal(run(b, x[t:t + 1].contiguous(), w1, w2)[0], y[t]), f"token {t} alone differs"


@pytest.mark.parametrize("H,I", [(2304, 2304), (2240, 2240), (2304, 2240), (2240, 2304)])
@pytest.mark.parametrize("N", [17, 32, 40])
def test_streaming_in_two_passes(N, H, I):
    # FC1 and FC2 stream 9 steps, two panels of scales; one expert has every
    # token: blocks of 17, of 32, and of 32 and 8 rows
    E, K = 36, 2
    say(f"[w4] two passes N {N} H {H} I {I}")
    logits = torch.zeros((N, E), device=DEV)
    t = torch.arange(N, device=DEV)
    logits[t, torch.where(t % (E - 1) < 3, t % (E - 1), t % (E - 1) + 1)] = 1.0     # any expert but 3
    logits[:, 3] = 2.0
    buf, x, w1, w2 = case(N, H, I, E, K, logits=logits)
    counts = host(buf.route_counts)
    assert counts[3] == N and counts.sum() == 2 * N
    buf.act.fill_(7.0)
    buf.route_out.fill_(7.0)
    y = run(buf, x, w1, w2).clone()
    assert pads_as_set(buf)
    check(buf, x, w1, w2, buf.act, buf.route_out, y, experts=[3, 0, E - 1])
    alone(buf, logits, x, w1, w2, y, (0, 15, 16, N - 1))


SHAPES = {
    # N, H, I, E, K
    "fc1_early": (24, 2048, 1472, 16, 4),
    "fc1_just_below_early": (24, 2048, 1408, 16, 4),
    "fc2_early": (24, 2880, 2048, 16, 4),
    "fc2_just_below_early": (24, 2816, 2048, 16, 4),
    "fc1_64_rows_two_route_tiles": (60, 1024, 640, 4, 3),
    "fc2_64_rows_two_route_tiles_odd": (60, 1216, 832, 4, 3),
    "fc1_64_rows": (12, 1024, 1024, 20, 4),
    "fc2_64_rows_long_odd": (12, 1664, 2112, 20, 4),
    "fc2_streams_two_route_tiles": (64, 3264, 256, 8, 2),
    # steps that the contraction ends inside of: split for few tiles, streaming
    # for many, in FC1 and in FC2 with whole words of scales
    "fc1_ends_inside_split": (64, 576, 576, 64, 4),
    "fc1_ends_inside_streams": (64, 576, 960, 64, 4),
    "fc1_ends_inside_streams_aligned": (64, 640, 960, 64, 4),
    "fc1_ends_inside_streams_few_rows": (16, 832, 1088, 64, 4),
    "fc2_ends_inside_split": (64, 5376, 640, 64, 4),
    "fc2_ends_inside_streams": (64, 5632, 640, 64, 4),
    "fc2_ends_inside_split_odd": (64, 5632, 576, 64, 4),
    # workgroups of 32 or 64 rows with one row an expert
    "split_32_rows_few_rows": (8, 512, 576, 32, 4),
    "split_64_rows_few_rows": (8, 512, 640, 32, 4),
    # codes straight to registers or through LDS
    "five_and_six_steps": (4, 1280, 1536, 32, 4),
    "six_and_five_steps": (4, 1536, 1280, 32, 4),
    "seven_steps_odd_scales": (4, 1600, 1728, 32, 4),
    "nine_steps_odd_scales": (9, 2112, 2240, 16, 2),
    # FC2 with the token's sum or without
    "tokens_in_one_launch": (24, 512, 512, 16, 2),
    "tokens_in_two_launches": (25, 512, 512, 16, 2),
    "twelve_routes_a_token": (33, 256, 128, 24, 12),
    "nine_routes_a_token": (5, 192, 64, 9, 9),
    "sixteen_routes_a_token": (70, 64, 192, 40, 16),
    "seventeen_routes_a_token": (40, 64, 64, 17, 17),
}


@pytest.mark.parametrize("name", SHAPES)
def test_form(name):
    say(f"[w4] {name} {SHAPES[name]}")
    buf, x, w1, w2 = case(*SHAPES[name])
    buf.act.fill_(7.0)
    buf.route_out.fill_(7.0)
    y = run(buf, x, w1, w2).clone()
    assert pads_as_set(buf)
    check(buf, x, w1, w2, buf.act, buf.route_out, y, experts=[0, 3, SHAPES[name][3] - 1] if buf.E > 48 else None)
    N, E = SHAPES[name][0], SHAPES[name][3]
    logits = torch.from_numpy(np.ascontiguousarray(moe_inputs.make_logits(N, E, 1), dtype=np.float32)).to(DEV)
    alone(buf, logits, x, w1, w2, y, (0, N // 2, N - 1))


@pytest.mark.parametrize("shape", [
    # one route tile: 4 routes an expert, 840 and 910 tiles; one, 1088 and 1152
    (32, 512, 768, 32, 4), (32, 512, 832, 32, 4), (8, 512, 1088, 32, 4), (8, 512, 1152, 32, 4),
    # two: 32 or 64 weight rows, with 2 steps and with 4
    (64, 512, 960, 8, 2), (64, 512, 1024, 8, 2), (64, 1024, 576, 8, 2), (64, 1024, 640, 8, 2),
    # streaming with 16, 32 and 64 routes an expert
    (64, 512, 1344, 8, 2), (64, 512, 1408, 8, 2), (128, 512, 704, 8, 2), (128, 512, 768, 8, 2),
    (256, 512, 384, 8, 2), (256, 512, 448, 8, 2),
    # and where the contraction ends inside a step
    (64, 1088, 1856, 8, 2), (64, 1088, 1920, 8, 2), (64, 576, 2560, 8, 2), (64, 576, 2624, 8, 2),
    (128, 576, 1344, 8, 2), (128, 576, 1408, 8, 2), (256, 1152, 448, 8, 2),
], ids=str)
def test_either_side_of_the_bounds(shape):
    say(f"[w4] {shape}")
    buf, x, w1, w2 = case(*shape)
    buf.act.fill_(7.0)
    buf.route_out.fill_(7.0)
    y = run(buf, x, w1, w2).clone()
    assert pads_as_set(buf)
    check(buf, x, w1, w2, buf.act, buf.route_out, y, experts=[0, buf.E - 1])
    logits = torch.from_numpy(np.ascontiguousarray(moe_inputs.make_logits(buf.N, buf.E, 1), dtype=np.float32)).to(DEV)
    alone(buf, logits, x, w1, w2, y, (0, buf.N - 1))
