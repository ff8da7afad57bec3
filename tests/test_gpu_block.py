"""The operators around the layer in a run, as a block uses them: the block's
forward and backward against float64, its decode step, the training step with
the optimizer, and the serving ladder's items of a few tokens.

Bars: u = 2^-8 is half a step of bf16.  The float64 side takes the kernels'
picks, total and u (each checked by itself), so what is left are the roundings
of the pre-activation, of d_act, of the products' results and of the sums, each
at most u of a term.  A result's bar is their number times u times the sum of its
terms' magnitudes (`magnitudes`), where silu' and x silu'' / silu' count 1.1 and
0.4 at most: act 1.1 + 1 + 1, d_pre 0.4 + 1.1 * 3, so 4; a route's d_a one more,
the routes' sum one, du one, dx one: 8.  A pre-activation in 8 bits is off by
2^-4 of the value: 2.1 * 2^-4 more.  Normwise the roundings add as squares: one of
bf16 is u / sqrt(3) / 1.53 = 0.15% (1.53: the root mean square of a significand),
so 8 in phase make 1.2%; of e4m3 2.4%, two of them in silu(g) u' 3.4% (5% in phase).
"""

import numpy as np
import pytest
import torch

import moe_inputs
from gpu_support import say
from mixture_experts_expert_amd import (DecodeBuffers, MoEAdamW, MoEBlock, MoEBlockStep, ServingLadder, forward_decode,
                                        moe_ffn_decode_max_tokens)

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16


def block(H, I, E, K, rms, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    return MoEBlock(1 + 0.1 * r(H), 0.1 * r(E, H), (0.05 * r(E, 2 * I, H)).to(BF16), (0.05 * r(E, H, I)).to(BF16), K,
                    norm_bias=None if rms else 0.1 * r(H), rms=rms)


def stream(N, H, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn((N, H), generator=g, device=DEV).to(BF16) for _ in range(3)]


def reference(b, x, residual, d, ids, total_k, u_k):
    """The block in float64 on the CPU with the kernels' picks, total and u: y,
    total, u, the gradients of x, residual and the weights, and the terms'
    magnitudes of y and of the gradients of x and of the weights."""
    f = lambda t: t.detach().double().cpu()  # noqa: E731
    leaves = [f(x), f(residual)] + [f(p) for p in b.params()]
    for t in leaves:
        t.requires_grad_(True)
    xx, rr, w = leaves[0], leaves[1], leaves[2]
    bias = leaves[3] if b.norm_bias is not None else None
    router, w1, w2 = leaves[-3:]
    exact_total = xx + rr
    total = exact_total + (f(total_k) - exact_total).detach()
    m = 0.0 if b.rms else total.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((total - m).square().mean(1, keepdim=True) + b.eps)
    xhat = (total - m) * rstd
    exact_u = xhat * w + bias if bias is not None else xhat * w
    u = exact_u + (f(u_k) - exact_u).detach()
    ids = ids.long().cpu()
    p = torch.softmax(torch.gather(u @ router.t(), 1, ids), 1)
    y = torch.zeros_like(total)
    routes = []
    for e in range(b.E):
        t, k = torch.where(ids == e)
        h = u[t] @ w1[e].t()
        act = torch.nn.functional.silu(h[:, :b.I]) * h[:, b.I:]
        a = act * p[t, k][:, None]
        a.retain_grad()
        y = y.index_add(0, t, a @ w2[e].t())
        routes.append((t, k, h, act, a))
    ((total + y) * f(d)).sum().backward()
    with torch.no_grad():
        my, du, dp = torch.zeros_like(y), torch.zeros_like(y), torch.zeros_like(p)
        mw1, mw2 = torch.zeros_like(w1), torch.zeros_like(w2)
        for e, (t, k, h, act, a) in enumerate(routes):
            da = a.grad.abs() * p[t, k][:, None]
            pre = torch.cat([da * h[:, b.I:].abs(), da * h[:, :b.I].abs()], 1)
            my.index_add_(0, t, a.abs() @ w2[e].abs().t())
            du.index_add_(0, t, pre @ w1[e].abs())
            dp[t, k] = (a.grad * act).abs().sum(1)
            mw1[e], mw2[e] = pre.t() @ u[t].abs(), f(d)[t].abs().t() @ a.abs()
        dl = torch.zeros((len(ids), b.E), dtype=torch.float64)
        dl.scatter_(1, ids, p * (dp + (p * dp).sum(1, keepdim=True)))
        du += dl @ router.abs()
        dh = du * w.abs()
        mx = f(d).abs() + rstd * (dh + dh.mean(1, keepdim=True) + xhat.abs() * (dh * xhat.abs()).mean(1, keepdim=True))
        terms = [my, mx, (du * xhat.abs()).sum(0)] + ([du.sum(0)] if bias is not None else [])
        terms += [dl.t() @ u.abs(), mw1, mw2]
    return y.detach(), exact_total.detach(), exact_u.detach(), [t.grad for t in leaves], terms


def check(got, want, terms, count, name, norm_tol):
    err = (got.double().cpu() - want).abs()
    norm = (err.norm() / want.norm()).item()
    say(f"  {name}: normwise {norm:.2e}, of the terms {(err / terms.clamp_min(1e-30)).max():.2e}, bar {count:.2e}")
    assert (err <= count * terms).all() and norm <= norm_tol, name


@pytest.mark.parametrize("rms", [True, False])
@pytest.mark.parametrize("checkpoint", ["bf16", "q8"])
def test_forward_and_backward_of_a_block(rms, checkpoint):
    N, H, I, E, K = 96, 128, 64, 6, 2
    b = block(H, I, E, K, rms)
    x, residual, d = stream(N, H, 3)
    step = MoEBlockStep(b, N, float(E) / K, checkpoint=checkpoint)     # capacity N: nothing is dropped
    y, total = step.forward(x, residual)
    dx = step.backward(d)
    torch.cuda.synchronize()
    ry, rtotal, ru, grads, terms = reference(b, x, residual, d, step.layer.topk_ids, total, step.u)
    check(total, rtotal, rtotal.abs(), 2.0 ** -8, "total", 1e-2)
    # beside its own rounding u has that of total: of a row's largest, through the norm
    check(step.u, ru, ru.abs() + 4 * ru.abs().amax(1, keepdim=True), 2.0 ** -8, "u", 1e-2)
    check(y, ry, terms[0], 3 * 2.0 ** -8, "y", 1e-2)
    q8 = checkpoint == "q8"
    count, tol = (8 * 2.0 ** -8 + 2.1 * 2.0 ** -4, 5e-2) if q8 else (8 * 2.0 ** -8, 1.2e-2)
    assert torch.equal(grads[0], grads[1])
    names = ["dx", "norm weight"] + (["norm bias"] if not rms else []) + ["router", "w1", "w2"]
    for name, got, want, t in zip(names, [dx] + step.grads(), grads[1:], terms[1:], strict=True):
        check(got, want, t, count, name, tol)
    # a second micro-batch adds to them, and they can be cleared
    first = [g.clone() for g in step.grads()]
    step.forward(x, residual)
    step.backward(d)
    for g, f in zip(step.grads(), first):
        assert (g - 2 * f).abs().max() <= 1e-5 * (1 + f.abs().max())
    step.zero_grad()
    assert all(not g.any() for g in step.grads())


@pytest.mark.parametrize("rms", [True, False])
def test_decode_agrees_with_the_training_forward(rms):
    N, H, I, E, K = 24, 256, 128, 8, 2
    b = block(H, I, E, K, rms, 5)
    x, residual, _ = stream(N, H, 6)
    step = MoEBlockStep(b, N, float(E) / K)
    y, total = step.forward(x, residual)
    buf = b.decode_buffers(N)
    out = b.decode(buf, x, residual)
    assert torch.equal(buf.layer.topk_ids, step.layer.topk_ids) and torch.equal(buf.total, total)
    want = total.double() + y.double()
    # y is rounded once as a sum of K rounded routes there, with the stream here: 2^-8 of each
    rms_y = y.double().square().mean().sqrt()
    assert ((out.double() - want).abs() <= 2.0 ** -8 * (2 * want.abs() + 4 * y.double().abs() + 4 * rms_y)).all()
    part = b.decode(buf, x[:5].contiguous(), residual[:5].contiguous())
    assert part.shape == (5, H)


def test_training_steps_run_captured_and_eager_alike():
    N, H, I, E, K = 64, 128, 64, 4, 2

    def build():
        b = block(H, I, E, K, True, 7)
        s = MoEBlockStep(b, N, 2.0)
        return b, s, MoEAdamW(b.params(), s.grads(), lr=1e-3, weight_decay=[0.0, 0.1, 0.1, 0.1], max_norm=1.0, masters="make")

    def step(s, opt, x, residual, d):
        s.zero_grad()
        s.forward(x, residual)
        s.backward(d)
        opt.step_()
    (b1, s1, o1), (b2, s2, o2) = build(), build()
    x, residual, d = stream(N, H, 8)
    ins = [t.clone() for t in (x, residual, d)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(s1, o1, *ins)
    torch.cuda.current_stream().wait_stream(side)
    step(s2, o2, x, residual, d)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(s1, o1, *ins)
    for i in range(4):
        new = stream(N, H, 20 + i)
        for a, t in zip(ins, new):
            a.copy_(t)
        g.replay()
        step(s2, o2, *new)
        torch.cuda.synchronize()
        assert o1.step.item() == o2.step.item() == i + 2 and torch.equal(o1.norm, o2.norm)
        for p, q in zip(b1.params(), b2.params()):
            assert torch.equal(p, q), i
    say("  norm", o1.norm.item())
    for p, q in zip(b1.params(), block(H, I, E, K, True, 7).params()):
        assert not torch.equal(p, q)


def ladder_case():
    w = moe_inputs.WORKLOADS["small_qwen3moe_n1024_h512_e8_k2"]
    T = moe_inputs.make_tensors(w, DEV)
    lg = torch.from_numpy(np.ascontiguousarray(moe_inputs.make_logits(96, w.E, 23), dtype=np.float32)).to(DEV)
    x = torch.randn(96, w.H, generator=torch.Generator(device=DEV).manual_seed(23), device=DEV).to(BF16)
    return w, T, lg, x


def test_ladder_items_of_a_few_tokens():
    w, T, lg, x = ladder_case()
    ladder = ServingLadder(T["w1"], T["w2"], w.K, expected=32, max_tokens=96, reserve_bytes=0, decode_tokens=48)
    plain = ServingLadder(T["w1"], T["w2"], w.K, expected=32, max_tokens=96, reserve_bytes=0)
    sizes = ladder.capture()
    assert plain.capture() == sizes and min(sizes) <= 48 < max(sizes)
    buf = DecodeBuffers(48, w.H, w.I, w.E, w.K)
    for n in (1, 7, 16, 30, 32, 45, 48, 49, 64, 96, 3):
        y = ladder.run(lg[:n], x[:n]).clone()
        torch.cuda.synchronize()
        if n <= 48 and (ladder.ladder.pick(n) or n) <= 48:
            # a bucket's graph has the bucket's N, and with it another order of sums than the item alone
            want = forward_decode(buf, lg[:n].contiguous(), x[:n].contiguous(), T["w1"], T["w2"])
            scale = want.double().square().mean().sqrt()
            assert ((y.double() - want.double()).abs() <= 2.0 ** -7 * (want.double().abs() + 1e-2 * scale)).all(), n
        else:
            assert torch.equal(y, plain.run(lg[:n], x[:n])), n
    eager = ServingLadder(T["w1"], T["w2"], w.K, expected=32, max_tokens=96, decode_tokens=48)     # nothing captured
    for n in (1, 16, 48):
        want = forward_decode(buf, lg[:n].contiguous(), x[:n].contiguous(), T["w1"], T["w2"]).clone()
        assert torch.equal(eager.run(lg[:n], x[:n]), want)


def test_ladder_refusals():
    w, T, _, _ = ladder_case()
    for n in (-1, moe_ffn_decode_max_tokens() + 1):
        with pytest.raises(ValueError, match="decode_tokens"):
            ServingLadder(T["w1"], T["w2"], w.K, expected=32, max_tokens=96, decode_tokens=n)
    b = block(64, 64, 4, 2, True)
    with pytest.raises(ValueError, match="need norm_weight"):
        MoEBlock(b.norm_weight, b.router[:, :32], b.w1, b.w2, 2)
    with pytest.raises(ValueError, match="5 tokens"):
        b.decode(b.decode_buffers(4), *stream(5, 64, 1)[:2])
