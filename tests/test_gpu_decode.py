"""The layer for a few tokens on the GPU (moe_ffn_decode): routing against
moe_route_dropless bit for bit, the products against float64.

Bars, from the arithmetic (u = 2^-24, half a float32 step).  Products of bf16
values are exact in float32; a contraction of length L is a float32 sum of L
products, at most L additions of at most one step (2u) of the sum of magnitudes
S each: dh = 2 L u S.

* act = bf16(silu(g) u p): |silu'| <= 1.1 and |silu(g)| <= |g|, so before the
  rounding it is off by p (1.1 dg (|u| + du) + (|g| + dg) du) and, for exp2, the
  reciprocal and three products, 16 * 2u of its magnitude; the rounding adds
  2^-8 of the result.
* y, from the kernel's own act (the workspace): K contractions of length I and
  the residual, 2 (K I + 1) u S, and one rounding, 2^-8 of the result.
"""

import numpy as np
import pytest
import torch

import moe_inputs
from gpu_support import say
from mixture_experts_expert_amd import (DecodeBuffers, DroplessBuffers, MoEError, ServingLadder, forward_decode,
                                        forward_dropless, moe_ffn_decode, moe_ffn_decode_max_tokens, moe_ffn_decode_workspace_bytes)

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
BF16 = torch.bfloat16


def layer(H, I, E, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w1 = torch.empty((E, 2 * I, H), dtype=BF16, device=DEV).normal_(0, 0.05, generator=g)
    w2 = torch.empty((E, H, I), dtype=BF16, device=DEV).normal_(0, 0.05, generator=g)
    return w1, w2


def tokens(N, H, E, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed + 50)
    x = torch.randn((N, H), generator=g, device=DEV).to(BF16)
    residual = torch.randn((N, H), generator=g, device=DEV).to(BF16)
    logits = torch.from_numpy(np.ascontiguousarray(moe_inputs.make_logits(N, E, seed), dtype=np.float32)).to(DEV)
    return logits, x, residual


def check(buf, logits, x, w1, w2, residual, y, live=None):
    """The buffers' contents and y against float64."""
    n, H = x.shape
    E, K, I = buf.E, buf.K, buf.I
    live = n if live is None else live
    ids, probs = buf.topk_ids[:n], buf.topk_probs[:n]
    ref = DroplessBuffers(max(live, 1), H, I, E, K, DEV)
    if live:
        ref.route(logits[:live].contiguous())
        assert torch.equal(ids[:live], ref.topk_ids), "ids differ from moe_route_dropless's"
        assert torch.equal(probs[:live].view(torch.int32), ref.topk_probs.view(torch.int32)), "probabilities differ"
    assert (ids[live:] == -1).all() and (probs[live:] == 0).all()
    act = buf.workspace[:n * K * I * 2].view(BF16).reshape(n, K, I)
    worst = [0.0, 0.0]
    sums = torch.zeros((n, H), dtype=torch.float64, device=DEV)
    mags = torch.zeros_like(sums)
    for e in torch.unique(ids[:live]).tolist():
        t, k = torch.where(ids[:live] == e)
        xs, w = x[t].double(), w1[e].double()
        h = xs @ w.t()
        dh = 2 * H * U * (xs.abs() @ w.abs().t())
        g, u, dg, du = h[:, :I], h[:, I:], dh[:, :I], dh[:, I:]
        p = probs[t, k].double()[:, None]
        a = g * torch.sigmoid(g) * u * p
        bar = p * (1.1 * dg * (u.abs() + du) + (g.abs() + dg) * du) + 32 * U * a.abs()
        bar = bar + 2.0 ** -8 * (a.abs() + bar)
        got = act[t, k].double()
        assert torch.isfinite(got).all(), "act"
        over = ((got - a).abs() / bar.clamp(min=1e-300)).max().item()
        worst[0] = max(worst[0], over)
        sums.index_add_(0, t, got @ w2[e].double().t())
        mags.index_add_(0, t, got.abs() @ w2[e].double().abs().t())
    if residual is not None:
        sums, mags = sums + residual.double(), mags + residual.double().abs()
    bar = 2 * (K * I + 1) * U * mags
    bar = bar + 2.0 ** -8 * (sums.abs() + bar)
    assert torch.isfinite(y[:live]).all(), "y"
    if live:
        worst[1] = ((y[:live].double() - sums[:live]).abs() / bar[:live].clamp(min=1e-300)).max().item()
    say(f"  {n} tokens, H {H}, I {I}, E {E}, K {K}: act {worst[0]:.3f}, y {worst[1]:.3f} of the bars")
    assert worst[0] <= 1.0 and worst[1] <= 1.0, worst


SIZES = [
    # N, H, I, E, K
    (1, 64, 64, 1, 1),
    (1, 2048, 768, 128, 8),
    (3, 512, 1024, 8, 2),
    (16, 2048, 768, 128, 8),
    (61, 1088, 448, 12, 5),
    (64, 64, 64, 4, 4),
    (64, 192, 320, 1, 1),           # every route in one expert
    (64, 128, 192, 1024, 32),       # the most routes and experts
    (17, 320, 64, 129, 17),
    (5, 704, 128, 300, 1),
    (33, 16384, 64, 3, 2),
    (2, 64, 16384, 5, 3),
    (40, 576, 576, 16, 3),
    (64, 960, 704, 128, 8),
    (8, 128, 64, 64, 20),           # a wave a token, more picks than a row of lanes
    (9, 128, 64, 64, 32),           # 16 lanes a token, all their picks
    (9, 192, 64, 200, 31),
    (3, 64, 128, 256, 32),
    (2, 64, 64, 257, 32),
    (64, 64, 64, 16, 16),
    (61, 256, 704, 61, 6),          # up to 8 routes an expert on average, 4-column tiles
    (9, 512, 1088, 22, 8),
    (20, 1024, 192, 8, 2),
    (20, 1088, 192, 8, 2),          # more tiles than compute units: 8 columns
]


@pytest.mark.parametrize("N,H,I,E,K", SIZES)
def test_against_float64(N, H, I, E, K):
    w1, w2 = layer(H, I, E)
    logits, x, residual = tokens(N, H, E)
    buf = DecodeBuffers(N, H, I, E, K)
    buf.workspace.fill_(255)                    # bf16 NaN: nothing unwritten is read
    buf.y.fill_(float("nan"))
    y = forward_decode(buf, logits, x, w1, w2, residual=residual)
    torch.cuda.synchronize()
    check(buf, logits, x, w1, w2, residual, y)
    first = y.clone()
    for _ in range(3):
        assert torch.equal(forward_decode(buf, logits, x, w1, w2, residual=residual), first), "not the same bits twice"


@pytest.mark.parametrize("N,H,I,E,K", [(1, 2048, 768, 128, 8), (9, 256, 192, 6, 3), (64, 64, 64, 4, 4)])
def test_without_a_residual_and_close_to_the_dropless_form(N, H, I, E, K):
    w1, w2 = layer(H, I, E, 3)
    logits, x, _ = tokens(N, H, E, 3)
    buf = DecodeBuffers(N, H, I, E, K)
    y = forward_decode(buf, logits, x, w1, w2)
    check(buf, logits, x, w1, w2, None, y)
    ref = DroplessBuffers(N, H, I, E, K, DEV)
    z = forward_dropless(ref, logits, x, w1, w2)
    # the dropless form rounds each of the K routes to bf16 as well: 2^-8 of each, K rounded rows of about y / sqrt(K)
    rms = z.double().square().mean().sqrt()
    assert ((y.double() - z.double()).abs() <= 2.0 ** -8 * (2 * z.double().abs() + 8 * rms)).all()


@pytest.mark.parametrize("live", [0, 1, 7, 12, 99, -3])
def test_rows_past_the_live_ones_stay_as_they_were(live):
    N, H, I, E, K = 12, 320, 128, 10, 4
    w1, w2 = layer(H, I, E, 5)
    logits, x, residual = tokens(N, H, E, 5)
    logits[max(min(live, N), 0):] = float("nan")     # not read
    x[max(min(live, N), 0):] = float("nan")
    buf = DecodeBuffers(N, H, I, E, K)
    buf.y.fill_(7.0)
    n_live = torch.full((1,), live, dtype=torch.int32, device=DEV)
    y = forward_decode(buf, logits, x, w1, w2, residual=residual, n_live=n_live)
    n = max(min(live, N), 0)
    check(buf, logits, x, w1, w2, residual, y, live=n)
    assert (y[n:] == 7.0).all()


def test_fewer_tokens_than_the_buffers_hold():
    N, H, I, E, K = 20, 256, 192, 9, 3
    w1, w2 = layer(H, I, E, 6)
    logits, x, residual = tokens(N, H, E, 6)
    buf = DecodeBuffers(N, H, I, E, K)
    buf.y.fill_(5.0)
    y = forward_decode(buf, logits[:6].contiguous(), x[:6].contiguous(), w1, w2, residual=residual[:6].contiguous())
    assert y.shape == (6, H)
    check(buf, logits[:6].contiguous(), x[:6].contiguous(), w1, w2, residual[:6], y)
    assert (buf.y[6:] == 5.0).all()


def test_the_residual_may_be_the_output():
    N, H, I, E, K = 10, 448, 256, 8, 2
    w1, w2 = layer(H, I, E, 7)
    logits, x, residual = tokens(N, H, E, 7)
    buf = DecodeBuffers(N, H, I, E, K)
    want = forward_decode(buf, logits, x, w1, w2, residual=residual).clone()
    buf.y.copy_(residual)
    assert torch.equal(forward_decode(buf, logits, x, w1, w2, residual=buf.y), want)


@pytest.mark.parametrize("kind", ["tied", "minus_inf", "plus_inf", "nan", "one_expert", "zeros"])
def test_unusual_logits(kind):
    N, H, I, E, K = 13, 192, 128, 40, 6
    w1, w2 = layer(H, I, E, 8)
    logits, x, residual = tokens(N, H, E, 8)
    if kind == "tied":
        logits = torch.round(logits)                # many equal logits: the lower expert first
    elif kind == "minus_inf":
        logits[:, 2:] = float("-inf")               # fewer experts than K left
    elif kind == "plus_inf":
        logits[3, 5] = float("inf")                 # inf - inf: a NaN probability for that token alone
    elif kind == "nan":
        logits[4, 7] = float("nan")
    elif kind == "one_expert":
        logits[:, 17] = 50.0
    else:
        logits.zero_()
    buf = DecodeBuffers(N, H, I, E, K)
    y = forward_decode(buf, logits, x, w1, w2, residual=residual)
    ref = DroplessBuffers(N, H, I, E, K, DEV)
    ref.route(logits)
    assert torch.equal(buf.topk_ids, ref.topk_ids)
    a, b = buf.topk_probs, ref.topk_probs
    assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a[~torch.isnan(a)], b[~torch.isnan(b)])
    bad = torch.isnan(b).any(1)
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()
    if kind in ("plus_inf", "nan"):
        assert bad.sum() == 1
    if not bad.any():
        check(buf, logits, x, w1, w2, residual, y)


def test_weights_past_32_bit_offsets():
    H, I, E, K = 4096, 1792, 160, 1                  # w1 4.7 GB, w2 2.3 GB
    w1 = torch.zeros((E, 2 * I, H), dtype=BF16, device=DEV)
    w2 = torch.zeros((E, H, I), dtype=BF16, device=DEV)
    a, b = layer(H, I, 1, 9)
    w1[E - 1], w2[E - 1] = a[0], b[0]
    _, x, residual = tokens(2, H, 4, 9)
    logits = torch.zeros((2, E), device=DEV)
    logits[:, E - 1] = 3.0
    buf = DecodeBuffers(2, H, I, E, K)
    y = forward_decode(buf, logits, x, w1, w2, residual=residual)
    assert (buf.topk_ids == E - 1).all()
    check(buf, logits, x, w1, w2, residual, y)       # (a layer of that expert alone shares its sums out otherwise)


def test_captured_and_replayed():
    N, H, I, E, K = 8, 512, 384, 32, 4
    w1, w2 = layer(H, I, E, 11)
    sets = [tokens(N, H, E, s) for s in (11, 12, 13)]
    buf, eager = DecodeBuffers(N, H, I, E, K), DecodeBuffers(N, H, I, E, K)
    logits, x, residual = [t.clone() for t in sets[0]]
    n_live = torch.full((1,), N, dtype=torch.int32, device=DEV)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        forward_decode(buf, logits, x, w1, w2, residual=residual, n_live=n_live)
    torch.cuda.current_stream().wait_stream(stream)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        forward_decode(buf, logits, x, w1, w2, residual=residual, n_live=n_live)
    for i, live in enumerate((N, 3, N, 1, N)):
        lg, xx, rr = sets[i % 3]
        logits.copy_(lg), x.copy_(xx), residual.copy_(rr), n_live.fill_(live)
        buf.y.fill_(1.0)
        g.replay()
        eager.y.fill_(1.0)
        want = forward_decode(eager, lg, xx, w1, w2, residual=rr, n_live=n_live)
        torch.cuda.synchronize()
        assert torch.equal(buf.y, want) and torch.equal(buf.topk_ids, eager.topk_ids), i


def test_two_streams_at_once():
    N, H, I, E, K = 16, 1024, 512, 32, 4
    w1, w2 = layer(H, I, E, 14)
    sets = [tokens(N, H, E, s) for s in (14, 15)]
    bufs = [DecodeBuffers(N, H, I, E, K) for _ in sets]
    want = [forward_decode(b, lg, x, w1, w2, residual=r).clone() for b, (lg, x, r) in zip(bufs, sets)]
    for b in bufs:
        b.y.zero_()
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for s, b, (lg, x, r) in zip(streams, bufs, sets):
            forward_decode(b, lg, x, w1, w2, residual=r, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(b.y, w) for b, w in zip(bufs, want))


def test_nothing_beside_the_outputs_is_written():
    N, H, I, E, K = 5, 192, 64, 7, 3
    w1, w2 = layer(H, I, E, 16)
    logits, x, residual = tokens(N, H, E, 16)
    pad = 64

    def band(shape, dtype):
        n = int(np.prod(shape))
        t = torch.full((n + 2 * pad,), 77, dtype=dtype, device=DEV)
        return t, t[pad:pad + n].view(shape)
    ids, vids = band((N, K), torch.int32)
    probs, vprobs = band((N, K), torch.float32)
    y, vy = band((N, H), BF16)
    need = moe_ffn_decode_workspace_bytes(N, H, I, E, K)
    ws, vws = band((need,), torch.uint8)
    moe_ffn_decode(logits, x, w1, w2, vids, vprobs, vws, vy, residual=residual)
    torch.cuda.synchronize()
    for t in (ids, probs, y, ws):
        assert (t[:pad] == 77).all() and (t[-pad:] == 77).all()
    buf = DecodeBuffers(N, H, I, E, K)
    assert torch.equal(vy, forward_decode(buf, logits, x, w1, w2, residual=residual))


def test_refusals():
    H, I, E, K = 128, 64, 4, 2
    w1, w2 = layer(H, I, E)
    most = moe_ffn_decode_max_tokens()
    logits, x, residual = tokens(most + 1, H, E)
    with pytest.raises(MoEError):
        DecodeBuffers(most + 1, H, I, E, K)
    buf = DecodeBuffers(4, H, I, E, K)
    with pytest.raises(ValueError, match="5 tokens"):
        forward_decode(buf, logits[:5].contiguous(), x[:5].contiguous(), w1, w2)
    lg, xx, rr = logits[:4].contiguous(), x[:4].contiguous(), residual[:4].contiguous()
    with pytest.raises(ValueError, match="agree in N"):
        forward_decode(buf, logits[:3].contiguous(), xx, w1, w2)
    with pytest.raises(ValueError, match="residual must be"):
        forward_decode(buf, lg, xx, w1, w2, residual=rr[:3])
    with pytest.raises(ValueError, match="contiguous"):
        forward_decode(buf, lg, x[:8:2], w1, w2)
    with pytest.raises(TypeError, match="bfloat16"):
        forward_decode(buf, lg, xx.float(), w1, w2)
    with pytest.raises(ValueError, match="weights must be"):
        forward_decode(buf, lg, xx, w1, w2[:, :, :32])
    with pytest.raises(ValueError, match="workspace: needs"):
        moe_ffn_decode(lg, xx, w1, w2, buf.topk_ids, buf.topk_probs, buf.workspace[:16], buf.y)
    with pytest.raises(MoEError):                    # rows that do not begin on 16 bytes
        flat = torch.zeros(4 * H + 1, dtype=BF16, device=DEV)
        forward_decode(buf, lg, flat[1:].view(4, H), w1, w2)
