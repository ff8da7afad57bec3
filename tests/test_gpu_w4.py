"""The dropless expert FFN on 4-bit weights on the GPU (moe_grouped_fc1_swiglu_w4,
moe_grouped_fc2_w4, moe_gather_combine_f32, moe_grouped_ffn_w4), against the
oracle in float64 on the same codes.

Bars, from the arithmetic (u = 2^-24, half a float32 step).  The weights'
values and their products with bf16 rows are exact; a contraction of length L
is a float32 sum of L products, at most L additions of at most one step (2u)
of the sum of magnitudes S each: dh = 2 L u S.

* act = bf16(silu(g) u p): |silu'| <= 1.1 and |silu(g)| <= |g|, so before the
  rounding it is off by p (1.1 dg (|u| + du) + (|g| + dg) du) and, for exp2,
  the reciprocal and three products, 16 * 2u of its magnitude; the rounding
  adds 2^-8 of the result.
* route_out (float32), from the kernel's own act: 2 I u S.
* y, from the kernel's own route_out: the same float32 additions in the same
  order and one rounding: bit for bit.
"""

import numpy as np
import pytest
import torch

import moe_inputs
import oracle
from gpu_support import assert_bf16_close, host, say
from mixture_experts_expert_amd import (DroplessBuffers, MoEError, ServingLadder, W4Weights, forward_dropless,
                                        moe_grouped_fc1_swiglu_w4,
                                        moe_grouped_fc2_w4, moe_grouped_ffn_w4, moe_route_dropless_live)

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24


def weights(E, H, I, seed, wide_scales=False):
    """Random codes; scales near those of N(0, 0.02) weights, or far apart."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    lo, hi = (100, 130) if wide_scales else (118, 121)

    def one(rows, cols):
        return W4Weights(torch.randint(0, 256, (E, rows, cols // 2), generator=g, device=DEV, dtype=torch.uint8),
                         torch.randint(lo, hi, (E, rows, cols // 32), generator=g, device=DEV, dtype=torch.uint8))
    return one(2 * I, H), one(H, I)


def case(N, H, I, E, K, seed=1, logits=None, wide_scales=False):
    w1, w2 = weights(E, H, I, seed, wide_scales)
    g = torch.Generator(device=DEV).manual_seed(seed + 50)
    x = torch.randn(N, H, generator=g, device=DEV).to(torch.bfloat16)
    if logits is None:
        logits = torch.from_numpy(np.ascontiguousarray(moe_inputs.make_logits(N, E, seed), dtype=np.float32)).to(DEV)
    buf = DroplessBuffers(N, H, I, E, K, DEV, w4=True)
    buf.route(logits)
    return buf, x, w1, w2


def run(buf, x, w1, w2, well_formed=True):
    """y by the one call, and by the three, which also leave act and route_out
    in the buffers: equal bit for bit if the route list is well formed."""
    buf.ffn_w4(x, w1, w2)
    y = buf.y.clone()
    lst = (buf.expert_ids, buf.block_start, buf.route_counts)
    moe_grouped_fc1_swiglu_w4(x, w1.codes, w1.scales, buf.sorted_slot_ids, buf.slot_probs, *lst, buf.K, buf.act)
    moe_grouped_fc2_w4(buf.act, w2.codes, w2.scales, *lst, buf.N, buf.K, buf.route_out)
    buf.combine()
    torch.cuda.synchronize()
    if well_formed:
        assert torch.equal(y.view(torch.int16), buf.y.view(torch.int16)), "one call and three calls differ"
    return buf.y


def live_slots(buf):
    """Slot, token and expert of every route of the list."""
    ssi = host(buf.sorted_slot_ids)
    counts, start = host(buf.route_counts), host(buf.block_start)
    slots = np.concatenate([start[e] * 32 + np.arange(counts[e]) for e in range(buf.E)]).astype(np.int64)
    return slots, ssi[slots], np.repeat(np.arange(buf.E), counts)


def check(buf, x, w1, w2, act, route_out, y, experts=None):
    xf = oracle.bf16_bits_to_f64(host(x))
    probs = host(buf.slot_probs).astype(np.float64)
    slots, toks, own = live_slots(buf)
    actf = oracle.bf16_bits_to_f64(host(act))
    ro = host(route_out).astype(np.float64)
    H, I = buf.H, buf.I
    for e in np.unique(own) if experts is None else experts:
        s, t = slots[own == e], toks[own == e]
        if not len(s):
            continue
        v1 = oracle.w4_values(host(w1.codes[e]), host(w1.scales[e])).T
        h, S = xf[t] @ v1, np.abs(xf[t]) @ np.abs(v1)
        g, u, dg, du = h[:, :I], h[:, I:], 2 * H * U * S[:, :I], 2 * H * U * S[:, I:]
        p = probs[s][:, None]
        with np.errstate(over="ignore"):
            want = g / (1 + np.exp(-g)) * u * p
        before = p * (1.1 * dg * (np.abs(u) + du) + (np.abs(g) + dg) * du) + 32 * U * np.abs(want)
        bar = before + 2.0 ** -8 * (np.abs(want) + before) + 2.0 ** -133
        err = np.abs(actf[s] - want)
        assert np.all(err <= bar), f"expert {e}: act {np.max(err / bar)} of its bar"
        v2 = oracle.w4_values(host(w2.codes[e]), host(w2.scales[e])).T
        r, S = actf[s] @ v2, np.abs(actf[s]) @ np.abs(v2)
        err = np.abs(ro[s] - r)
        assert np.all(err <= 2 * I * U * S + 1e-38), f"expert {e}: route_out"
    # y: float32 sums in k order of the kernel's own rows
    tr, r32 = host(buf.token_routes), host(route_out)
    acc = np.zeros((tr.shape[0], H), dtype=np.float32)
    for k in range(tr.shape[1]):
        has = tr[:, k] >= 0
        acc[has] += r32[tr[has, k]]
    assert np.array_equal(host(y), oracle.f64_to_bf16_bits(acc)), "y"


SHAPES = {
    # N, H, I, E, K
    "one_token": (1, 64, 64, 1, 1),
    "one_token_of_8_experts": (1, 256, 192, 8, 3),
    "two_tokens": (2, 128, 128, 4, 4),
    "columns_end_in_a_step": (7, 192, 320, 6, 2),
    "long_contraction": (5, 2048, 768, 16, 8),
    "odd_steps": (19, 1088, 448, 5, 3),
    "seventeen_rows": (17, 128, 256, 2, 2),
    "thirty_three_rows": (33, 256, 64, 1, 1),
    "three_blocks_an_expert": (90, 128, 192, 3, 3),
    "many_rows": (300, 192, 128, 4, 2),
    "all_to_few": (64, 64, 64, 1000, 32),
    # enough tiles for the streaming kernel: few and many rows an expert, steps
    # that end inside the row, more than one panel of scales
    "stream_few_rows": (70, 512, 1280, 64, 4),
    "stream_many_rows": (260, 320, 704, 64, 8),
    "stream_odd_scales": (60, 1088, 1344, 48, 8),
    "stream_long": (40, 4160, 1536, 48, 4),
    "split_long": (3, 4160, 2112, 4, 2),
    # either side of the sizes that choose the kernel: FC2 with the sum or
    # without, workgroups of 32 or 64 rows, streaming early or late
    "many_tokens_of_a_small_layer": (257, 64, 64, 12, 1),
    "tokens_at_the_bound": (256, 64, 64, 12, 1),
    "split_64_rows_many_rows": (60, 832, 640, 4, 3),
    "split_64_rows_long": (12, 2176, 1024, 20, 4),
    "split_64_rows_long_odd": (12, 2112, 1024, 20, 4),
    "stream_early_many_rows": (120, 768, 1280, 12, 3),
    "stream_early_few_rows": (42, 512, 1216, 32, 6),
    "split_steps_end_inside": (64, 1088, 576, 64, 6),
    # the longest contraction, in whole steps and ending inside one: two panels
    # of scales a wave of the split kernel
    "longest": (2, 16384, 64, 2, 1),
    "longest_odd": (2, 16320, 64, 2, 1),
    "longest_fc2": (2, 64, 16384, 2, 1),
}


@pytest.mark.parametrize("name", SHAPES)
def test_ffn_w4(name):
    say(f"[w4] {name} {SHAPES[name]}")
    buf, x, w1, w2 = case(*SHAPES[name])
    buf.act.fill_(7.0)
    buf.route_out.fill_(7.0)
    y = run(buf, x, w1, w2)
    assert bool((buf.act != 7).any())
    check(buf, x, w1, w2, buf.act, buf.route_out, y)
    # rows that are no route's stay as they were
    slots, _, _ = live_slots(buf)
    rest = torch.ones(buf.R, dtype=torch.bool, device=DEV)
    rest[torch.from_numpy(slots).to(DEV)] = False
    assert bool((buf.act[rest] == 7).all()) and bool((buf.route_out[rest] == 7).all())


def test_scales_far_apart():
    buf, x, w1, w2 = case(9, 320, 192, 4, 2, seed=8, wide_scales=True)
    y = run(buf, x, w1, w2)
    check(buf, x, w1, w2, buf.act, buf.route_out, y)


def test_every_route_to_one_expert_and_none_to_the_others():
    N, E, K = 131, 7, 1
    logits = torch.zeros((N, E), device=DEV)
    logits[:, 5] = 1.0
    buf, x, w1, w2 = case(N, 128, 192, E, K, logits=logits)
    assert host(buf.route_counts).tolist() == [0, 0, 0, 0, 0, N, 0]
    y = run(buf, x, w1, w2)
    check(buf, x, w1, w2, buf.act, buf.route_out, y)


@pytest.mark.parametrize("H,I", [(192, 128), (2112, 192), (192, 2112), (2304, 64), (256, 2304)])
def test_more_rows_than_the_average_promises(H, I):
    # 24 rows for each of two experts, 3 an expert on average: the kernels made
    # for 16 rows go over the weights twice (straight, staged and streaming)
    N, E, K = 24, 16, 2
    logits = torch.zeros((N, E), device=DEV)
    logits[:, 3], logits[:, 11] = 2.0, 1.0
    buf, x, w1, w2 = case(N, H, I, E, K, logits=logits)
    assert max(host(buf.route_counts)) == N
    y = run(buf, x, w1, w2)
    check(buf, x, w1, w2, buf.act, buf.route_out, y)


@pytest.mark.parametrize("H,I,E,K", [(1088, 448, 8, 3), (256, 2048, 4, 4), (1088, 832, 48, 8), (2304, 1280, 64, 2)])
def test_a_token_alone_equals_the_token_in_any_batch(H, I, E, K):
    N = 260                                   # up to 260 rows an expert
    buf, x, w1, w2 = case(N, H, I, E, K)
    logits = torch.from_numpy(np.ascontiguousarray(moe_inputs.make_logits(N, E, 1), dtype=np.float32)).to(DEV)
    y = run(buf, x, w1, w2).clone()
    for n in (1, 2, 16, 40, 130):
        for lo in (0, N - n):
            b = DroplessBuffers(n, H, I, E, K, DEV, w4=True)
            got = forward_dropless(b, logits[lo:lo + n].contiguous(), x[lo:lo + n].contiguous(), w1, w2)
            assert torch.equal(got, y[lo:lo + n]), f"tokens {lo}..{lo + n - 1} alone differ"


def test_nan_infinity_and_garbage_stay_where_they_belong():
    buf, x, w1, w2 = case(40, 192, 192, 4, 2)
    clean = run(buf, x, w1, w2).clone()
    # what the kernels must not read: act and route_out of pad slots
    buf.act.fill_(float("nan"))
    buf.route_out.fill_(float("nan"))
    assert torch.equal(run(buf, x, w1, w2), clean)
    # a token with NaN and one with infinity leave the others alone
    x2 = x.clone()
    x2[3, 100], x2[9, 0] = float("nan"), float("inf")
    y = run(buf, x2, w1, w2)
    keep = torch.ones(40, dtype=torch.bool, device=DEV)
    keep[3] = keep[9] = False
    assert torch.equal(y[keep], clean[keep])
    assert bool(torch.isnan(y[3]).all())
    # a group that stands for NaN: every token of that expert, no other
    s2 = w2.scales.clone()
    s2[1, 7, 0] = 255
    y = run(buf, x, w1, W4Weights(w2.codes, s2))
    uses = (buf.topk_ids == 1).any(dim=1)
    assert bool(torch.isnan(y[uses, 7]).all()) and not bool(torch.isnan(y[~uses]).any())
    cols = torch.ones(192, dtype=torch.bool, device=DEV)
    cols[7] = False
    assert torch.equal(y[:, cols], clean[:, cols])


@pytest.mark.parametrize("name", ["stream_early_few_rows", "stream_early_many_rows", "split_64_rows_long_odd", "odd_steps"])
def test_every_kernel_leaves_pads_and_other_tokens_alone(name):
    buf, x, w1, w2 = case(*SHAPES[name])
    clean = run(buf, x, w1, w2).clone()
    buf.act.fill_(5.0)
    buf.route_out.fill_(5.0)
    x2 = x.clone()
    x2[2, 1::7] = float("nan")
    y = run(buf, x2, w1, w2)
    keep = torch.ones(x.shape[0], dtype=torch.bool, device=DEV)
    keep[2] = False
    assert torch.equal(y[keep], clean[keep]) and bool(torch.isnan(y[2]).all())
    pads = torch.ones(buf.R, dtype=torch.bool, device=DEV)
    pads[torch.from_numpy(live_slots(buf)[0]).to(DEV)] = False
    assert bool((buf.act[pads] == 5).all()) and bool((buf.route_out[pads] == 5).all())


def test_list_entries_out_of_range_are_dropped():
    """Device data is range-checked: experts, blocks, counts and tokens that
    name nothing read and write nothing (codes past the routes stay as set)."""
    N, H, I, E, K = 20, 64, 64, 4, 2
    buf, x, w1, w2 = case(N, H, I, E, K)
    run(buf, x, w1, w2)
    good = buf.route_out.clone()
    buf.expert_ids[-1] = 4
    buf.expert_ids[-2] = -7
    y = run(buf, x, w1, w2).clone()
    slots = torch.from_numpy(live_slots(buf)[0]).to(DEV)
    assert torch.equal(buf.route_out[slots], good[slots])
    e0 = buf.route_counts.clone()
    buf.route_counts[0] = -5                  # no rows
    buf.route_out.fill_(7.0)
    run(buf, x, w1, w2, well_formed=False)
    first = int(buf.block_start[0]) * 32
    assert bool((buf.route_out[first:first + int(e0[0])] == 7).all())
    buf.route_counts.copy_(e0)
    buf.sorted_slot_ids[first] = N + 3        # a token that is none: a row of zeros
    buf.token_routes[0, 0] = buf.R + 5        # a slot that is none
    y2 = run(buf, x, w1, w2, well_formed=False)
    assert bool((buf.act[first] == 0).all()) and bool(torch.isfinite(y2.float()).all())
    assert y.shape == y2.shape


@pytest.mark.parametrize("live", [0, 1, 13, 48])
def test_live_count_on_the_device(live):
    N, H, I, E, K = 48, 192, 128, 6, 2
    buf, x, w1, w2 = case(N, H, I, E, K)
    logits = torch.from_numpy(np.ascontiguousarray(moe_inputs.make_logits(N, E, 1), dtype=np.float32)).to(DEV)
    full = run(buf, x, w1, w2).clone()
    n = torch.tensor([live], dtype=torch.int32, device=DEV)
    moe_route_dropless_live(logits, K, n, buf.topk_ids, buf.topk_probs, buf.route_within, buf.route_counts,
                            buf.sorted_slot_ids, buf.slot_probs, buf.expert_ids, buf.block_start,
                            buf.token_routes, buf.token_route_count, buf.num_tokens_post_padded, buf.workspace)
    y = run(buf, x, w1, w2)
    assert torch.equal(y[:live], full[:live]) and not bool(y[live:].any())


def test_no_tokens():
    _, _, w1, w2 = case(4, 64, 64, 4, 2)
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device=DEV)      # noqa: E731
    R = 4 * 32
    y = z(0, 64, dt=torch.bfloat16)
    moe_grouped_ffn_w4(z(0, 64, dt=torch.bfloat16), w1.codes, w1.scales, w2.codes, w2.scales, z(R),
                       z(R, dt=torch.float32), z(R // 32), z(4), z(4), z(0, 2), z(R, 64, dt=torch.bfloat16),
                       z(R, 64, dt=torch.float32), y)
    torch.cuda.synchronize()


def test_refusals():
    buf, x, w1, w2 = case(8, 64, 128, 4, 2)
    with pytest.raises(ValueError, match="w4=True"):
        forward_dropless(DroplessBuffers(8, 64, 128, 4, 2, DEV), torch.zeros((8, 4), device=DEV), x, w1, w2)
    with pytest.raises(TypeError, match="both"):
        forward_dropless(buf, torch.zeros((8, 4), device=DEV), x, w1, w2.dequantize())
    with pytest.raises(ValueError, match="weights must be"):
        buf.ffn_w4(x, w2, w1)
    with pytest.raises(ValueError, match="contiguous"):
        buf.ffn_w4(torch.zeros((64, 8), dtype=torch.bfloat16, device=DEV).t(), w1, w2)
    with pytest.raises(TypeError, match="bfloat16"):
        buf.ffn_w4(x.float(), w1, w2)
    with pytest.raises(ValueError, match="token_routes"):
        buf.ffn_w4(x[:4], w1, w2)
    with pytest.raises(ValueError, match="at least"):
        b2 = DroplessBuffers(8, 64, 128, 4, 2, DEV, w4=True)
        b2.act = b2.act[:32]
        b2.ffn_w4(x, w1, w2)
    with pytest.raises(ValueError, match="W4Weights must be codes|cols"):
        W4Weights.quantize(torch.zeros((2, 4, 40), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(MoEError):
        W4Weights.quantize(torch.zeros((2, 4, 96), dtype=torch.bfloat16, device=DEV))


def test_another_stream_and_graph_replays():
    buf, x, w1, w2 = case(33, 320, 192, 6, 3)
    logits = torch.from_numpy(np.ascontiguousarray(moe_inputs.make_logits(33, 6, 1), dtype=np.float32)).to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        forward_dropless(buf, logits, x, w1, w2)
    torch.cuda.synchronize()
    other = torch.empty_like(buf.y)
    buf.ffn_w4(x, w1, w2, stream=side)                       # a stream given by hand
    side.synchronize()
    other.copy_(buf.y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward_dropless(buf, logits, x, w1, w2)
    for i in range(3):
        g = torch.Generator(device=DEV).manual_seed(i)
        x.copy_(torch.randn(x.shape, generator=g, device=DEV).to(torch.bfloat16))
        logits.copy_(torch.randn(logits.shape, generator=g, device=DEV))
        want = forward_dropless(buf, logits, x, w1, w2).clone()
        torch.cuda.synchronize()
        buf.y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf.y, want), f"replay {i} differs from eager"


def test_serving_ladder_on_4_bit_weights():
    """Replays equal eager runs bit for bit (whatever the bucket), and both the
    bf16 layer's oracle on the 4-bit values within the forward's bars."""
    w = moe_inputs.WORKLOADS["small_qwen3moe_n1024_h512_e8_k2"]
    T = moe_inputs.make_tensors(w, DEV)
    q1, q2 = W4Weights.quantize(T["w1"]), W4Weights.quantize(T["w2"])
    lad = ServingLadder(q1, q2, w.K, expected=32, max_tokens=80, device=DEV, reserve_bytes=0)
    assert lad.capture() == lad.ladder.sizes
    eager = ServingLadder(q1, q2, w.K, expected=32, max_tokens=80, device=DEV, reserve_bytes=0)
    v1, v2 = host(q1.dequantize()), host(q2.dequantize())
    lg, x = T["logits"], T["x"]
    for n in (1, 14, 16, 17, 30, 40, 64, 80):
        y, ye = lad.run(lg[:n], x[:n]).clone(), eager.run(lg[:n], x[:n]).clone()
        torch.cuda.synchronize()
        assert torch.equal(y, ye), f"n={n}: replay differs from eager"
        if n in (1, 17, 80):
            o = oracle.dropless_forward(host(lg[:n]), host(x[:n]), v1, v2, w.K)
            assert_bf16_close(host(y), o["y"], f"y (n={n}) vs oracle")
    assert sum(v for k, v in lad.counts.items() if k != "eager") >= 6


def test_weights_past_32_bit_offsets():
    # codes of 80 experts are over 2^31 bytes; the last expert as in a layer of its own
    N, H, I, E = 5, 7168, 4096, 80
    g = torch.Generator(device=DEV).manual_seed(9)

    def big(rows, cols):
        w = W4Weights(torch.zeros(E, rows, cols // 2, dtype=torch.uint8, device=DEV),
                      torch.full((E, rows, cols // 32), 119, dtype=torch.uint8, device=DEV))
        w.codes[-1] = torch.randint(0, 256, (rows, cols // 2), generator=g, device=DEV, dtype=torch.uint8)
        return w
    w1, w2 = big(2 * I, H), big(H, I)
    assert w1.codes.numel() > 2 ** 31
    x = torch.randn(N, H, generator=g, device=DEV).to(torch.bfloat16)
    logits = torch.zeros((N, E), device=DEV)
    logits[:, -1] = 100.0                      # a probability of 1
    got = forward_dropless(DroplessBuffers(N, H, I, E, 1, DEV, w4=True), logits, x, w1, w2)
    one = [W4Weights(w.codes[-1:], w.scales[-1:]) for w in (w1, w2)]
    alone = forward_dropless(DroplessBuffers(N, H, I, 1, 1, DEV, w4=True), logits[:, -1:].contiguous(), x, *one)
    assert torch.equal(got, alone) and bool((got != 0).any())
