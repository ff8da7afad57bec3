"""The gradients' global norm and the AdamW step on the GPU (moe_grad_norm,
moe_adamw_step, MoEAdamW) against float64, and the 8-bit moments' codes.

Bars, from the arithmetic (u = 2^-24; inputs are taken as they are, the scalars
beta, 1 - beta, eps and max_norm rounded to float32, u relative each):
* norm: float64 sums, one rounding: 2u.  The clip is off by 4u (two rounded
  operands, a division), the clipped gradient by 5u
* m: 8u (|b1 m| + |(1 - b1) g|);  v: 16u (b2 v + (1 - b2) g^2)
* root v: half of v's relative error and u;  the denominator 16u relative;  the
  quotient's absolute error: that of m over the denominator, and 20u of it;  the
  rate lr / bc1 4u, keep = 1 - lr wd 2u:
  p: 6u |p| + rate (dm / den + 30u |m| / den), and its rounding
* 8-bit moments: the values come within half a step of a code of what is
  rounded, dm and droot beside it
"""

import math

import pytest
import torch

from gpu_support import say
from mixture_experts_expert_amd import (AdamWTable, MoEAdamW, MoEError, moe_grad_norm, moe_moment_codes,
                                        moe_moment_values)

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
B1, B2, EPS = 0.9, 0.95, 1e-8


def rnd(n, g, std=1.0):
    return torch.randn(n, generator=g, device=DEV) * std


def two_to(k):
    """2^k in float64 by its exponent field: the device's pow(), and ldexp through it, is off in its last bit."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def first_codes_ref(m):
    """The documented codes of float64 values [groups, 32]: (values, scale bytes)."""
    amax = m.abs().amax(1)
    _, e = torch.frexp(amax.clamp(min=1e-300))
    b = e - 1 - 8
    b = b + (amax / two_to(b) >= 464).int()
    b = torch.where(amax > 0, (b + 127).clamp(min=1), torch.ones_like(b))
    s = two_to(b - 127)[:, None]
    a = m / s
    _, ea = torch.frexp(a.abs().clamp(min=2.0 ** -6))
    step = two_to(ea - 1 - 3)
    return torch.round(a / step) * step * s, b, step * s


def root_codes_ref(r):
    amax = r.amax(1)
    _, e = torch.frexp(amax.clamp(min=1e-300))
    b = e - 1
    b = b + (amax / two_to(b) >= 63 / 32).int()
    b = torch.where(amax > 0, (b + 127).clamp(min=1), torch.ones_like(b))
    s = two_to(b - 127)[:, None]
    a = r / s
    _, ea = torch.frexp(a.clamp(min=2.0 ** -15))
    step = two_to(ea - 1 - 4)
    q = torch.where(r > 0, (torch.round(a / step) * step).clamp(min=17 / 16 * 2.0 ** -15), torch.zeros_like(a))
    return q * s, b, step * s


def grouped(t):
    n = t.numel()
    p = torch.zeros(-(-n // 32) * 32, dtype=torch.float64, device=DEV)
    p[:n] = t.double()
    return p.view(-1, 32)


def make(sizes, pt, gt, state, masters, seed=1, **kw):
    g = torch.Generator(device=DEV).manual_seed(seed)
    params = [rnd(n, g, 0.05).to(BF16 if pt == "bf16" else F32) for n in sizes]
    grads = [(rnd(n, g) * torch.exp(rnd(n, g)) * 1e-3).to(BF16 if gt == "bf16" else F32) for n in sizes]
    m = [rnd(n, g, 3e-4) for n in sizes]
    v = [rnd(n, g, 1e-3).square() for n in sizes]
    if state == "q8":
        mom = dict(m=[], v=[], m_scales=[], v_scales=[])
        for a, b in zip(m, v):
            n = a.numel()
            c = [torch.zeros(n, dtype=torch.uint8, device=DEV), torch.zeros(-(-n // 32), dtype=torch.uint8, device=DEV),
                 torch.zeros(n, dtype=torch.uint8, device=DEV), torch.zeros(-(-n // 32), dtype=torch.uint8, device=DEV)]
            moe_moment_codes(a, b, *c)
            for k, t in zip(("m", "m_scales", "v", "v_scales"), c):
                mom[k].append(t)
    else:
        mom = dict(m=m, v=v)
    mast = None
    if masters:
        mast = [p.float() + rnd(p.numel(), g, 1e-5) if p.dtype == BF16 else None for p in params]
    return MoEAdamW(params, grads, betas=(B1, B2), eps=EPS, state=state, masters=mast, moments=mom, **kw)


def decay_of(opt, i):
    return float(opt.table.array[i].weight_decay)


def snapshot(opt):
    out = []
    for i, p in enumerate(opt.params):
        m, v = opt.moment_values(i)
        v = v.double().square() if opt.state == "q8" else v.double()
        start = opt.masters[i] if opt.masters and opt.masters[i] is not None else p
        out.append((start.double().clone(), opt.grads[i].double().clone(), m.double().clone(), v.clone()))
    return out


def check_step(opt, before, lr, t):
    """Everything a step writes, against `before`."""
    worst = {}
    norm = math.sqrt(sum(float(g.square().sum()) for _, g, _, _ in before))
    clip, dclip = 1.0, 0.0
    if opt.max_norm is not None:
        assert abs(opt.norm.item() - norm) <= 2 * U * norm, (opt.norm.item(), norm)
        if norm > opt.max_norm:
            clip, dclip = opt.max_norm / norm, 5 * U
    bc1, bc2 = 1 - B1 ** t, 1 - B2 ** t
    rate = lr / bc1

    def note(name, got, want, bar):
        if got.numel():
            assert torch.isfinite(got).all(), name
            worst[name] = max(worst.get(name, 0.0), ((got.double() - want).abs() / bar.clamp(min=1e-300)).max().item())
    for i, (p, g, m, v) in enumerate(before):
        if p.numel() == 0:
            continue
        g = g * clip
        m1 = B1 * m + (1 - B1) * g
        dm = (8 * U + dclip) * ((B1 * m).abs() + ((1 - B1) * g).abs())
        v1 = B2 * v + (1 - B2) * g * g
        dv = (16 * U + 2 * dclip) * v1
        root = torch.sqrt(v1)
        den = root / math.sqrt(bc2) + EPS
        p1 = p * (1 - lr * decay_of(opt, i)) - rate * m1 / den
        dp = 6 * U * p.abs() + rate * (dm / den + 30 * U * m1.abs() / den)
        master = opt.masters[i] if opt.masters else None
        if master is not None:
            note("master", master, p1, dp + U * p1.abs())
            assert torch.equal(opt.params[i], master.to(opt.params[i].dtype)), "the parameter is not its master's rounding"
        else:
            half = U if opt.params[i].dtype == F32 else 2.0 ** -8
            note("param", opt.params[i], p1, dp + half * (p1.abs() + dp))
        got_m, got_v = opt.moment_values(i)
        if opt.state == "f32":
            note("m", got_m, m1, dm)
            note("v", got_v, v1, dv)
            continue
        n = p.numel()
        for name, got, want, d, ref in (("m codes", got_m, m1, dm, first_codes_ref),
                                        ("root codes", got_v, root, (10 * U + dclip) * root, root_codes_ref)):
            _, b, step = ref(grouped(want))
            scales = opt.moments["m_scales" if ref is first_codes_ref else "v_scales"][i].int()
            bar = step.reshape(-1)[:n] / 2 + d
            # a group within the error of the next scale's border may take that scale, whose steps are twice as long
            near = torch.zeros(b.shape, dtype=torch.bool, device=DEV)
            for f in (1 - 1e-5, 1 + 1e-5):
                near |= ref(grouped(want) * f)[1] != b
            assert (scales[~near] == b[~near]).all(), "scale bytes"
            ok = ~near.repeat_interleave(32)[:n]
            low = got.double() == torch.where(want > 0, 17 / 16 * 2.0 ** -15, 0.0) * two_to(b - 127).repeat_interleave(32)[:n]
            note(name, got[ok & ~low], want[ok & ~low], bar[ok & ~low])
            if ref is root_codes_ref:
                assert (got[want > 0] > 0).all(), "a root vanished"
    say("  " + ", ".join(f"{k} {x:.3f}" for k, x in worst.items()) + " of the bars")
    assert max(worst.values()) <= 1.0, worst


SIZES = [[1], [31, 32, 33], [4095, 4096, 4097, 0, 5], [100000, 7, 65536 + 3]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("pt,masters", [("bf16", False), ("f32", False), ("bf16", True)])
@pytest.mark.parametrize("gt", ["bf16", "f32"])
@pytest.mark.parametrize("state", ["f32", "q8"])
def test_steps(sizes, pt, masters, gt, state):
    opt = make(sizes, pt, gt, state, masters, seed=len(sizes), lr=1e-3, weight_decay=0.1, max_norm=0.01, step=7)
    for t in (8, 9, 10):
        before = snapshot(opt)
        opt.step_()
        torch.cuda.synchronize()
        check_step(opt, before, float(opt.lr.item()), t)
        assert opt.step.item() == t


def test_the_first_step_without_clipping_and_with_a_decay_for_each():
    opt = make([1000, 77, 4096], "f32", "f32", "f32", False, seed=3, lr=2e-3, weight_decay=[0.0, 0.5, 0.1])
    for m, v in zip(opt.moments["m"], opt.moments["v"]):
        m.zero_(), v.zero_()
    before = snapshot(opt)
    opt.step_()
    check_step(opt, before, float(opt.lr.item()), 1)
    assert opt.step.item() == 1 and opt.norm.item() == 0.0


@pytest.mark.parametrize("state", ["f32", "q8"])
def test_more_tensors_than_a_launch_takes(state):
    sizes = [(i * 37) % 5000 for i in range(150)]
    opt = make(sizes, "bf16", "f32", state, True, seed=4, lr=1e-3, max_norm=1.0, step=3)
    for t in (4, 5):
        before = snapshot(opt)
        opt.step_()
        check_step(opt, before, float(opt.lr.item()), t)
        assert opt.step.item() == t


def test_types_mixed_in_one_call():
    g = torch.Generator(device=DEV).manual_seed(5)
    params = [rnd(999, g).to(BF16), rnd(321, g), rnd(4100, g).to(BF16)]
    grads = [rnd(999, g, 1e-2), rnd(321, g, 1e-2).to(BF16), rnd(4100, g, 1e-2).to(BF16)]
    opt = MoEAdamW(params, grads, lr=1e-3, betas=(B1, B2), eps=EPS, masters="make", max_norm=0.1)
    assert opt.masters[1] is None and opt.masters[0].dtype == F32
    for t in (1, 2):
        before = snapshot(opt)
        opt.step_()
        check_step(opt, before, float(opt.lr.item()), t)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("state", ["f32", "q8"])
def test_a_step_whose_norm_is_not_finite_is_not_taken(bad, state):
    opt = make([5000, 33], "bf16", "f32", state, True, seed=6, lr=1e-3, max_norm=1.0, step=11)
    opt.grads[1][20] = bad
    held = [t.clone() for t in opt.params + opt.masters + sum(opt.moments.values(), [])]
    opt.step_()
    assert not math.isfinite(opt.norm.item()) and opt.step.item() == 11
    assert all(torch.equal(a, b) for a, b in zip(held, opt.params + opt.masters + sum(opt.moments.values(), [])))
    opt.grads[1][20] = 1e-3
    before = snapshot(opt)
    opt.step_()
    check_step(opt, before, float(opt.lr.item()), 12)


def test_gradients_whose_squares_leave_float32():
    big = torch.full((3000,), 1e25, device=DEV)
    small = torch.full((70,), 1e-30, device=DEV)
    for grads, want in (([big], 1e25 * math.sqrt(3000)), ([small], 1e-30 * math.sqrt(70))):
        p = [torch.zeros_like(g) for g in grads]
        opt = MoEAdamW(p, grads, lr=1e-3, max_norm=1.0)
        moe_grad_norm(opt.table, opt.norm)
        assert abs(opt.norm.item() - want) <= 4 * U * want
    opt = MoEAdamW([torch.ones(3000, device=DEV)], [big], lr=1e-3, max_norm=1.0, weight_decay=0.0)
    opt.step_()                                  # clipped to a norm of 1: every element 1 / sqrt(3000)
    assert (opt.params[0] - (1 - 1e-3)).abs().max() < 1e-6
    # an element without a gradient yet does not move, and is not divided by nothing
    opt = MoEAdamW([torch.ones(64, device=DEV)], [torch.zeros(64, device=DEV)], lr=1e-3, weight_decay=0.0, state="q8")
    opt.step_()
    assert (opt.params[0] == 1).all()


def test_gradient_norm_at_many_sizes():
    g = torch.Generator(device=DEV).manual_seed(7)
    for n in (1, 3, 4, 1023, 16383, 16384, 16385, 1 << 20, (1 << 20) + 1):
        for dt in (BF16, F32):
            x = rnd(n, g).to(dt)
            opt = MoEAdamW([torch.zeros(n, device=DEV)], [x], max_norm=1.0)
            moe_grad_norm(opt.table, opt.norm)
            want = x.double().square().sum().sqrt().item()
            assert abs(opt.norm.item() - want) <= 2 * U * want, (n, dt)


def test_every_code_of_8_bit_moments():
    # The lowest bit of an m code is worth 2^(b - 127 - 9), that of a root's 2^(b - 127 - 19): bf16, whose lowest
    # subnormal bit is 2^-133, holds every value from b = 3 and b = 13 on; below, values are rounded to it.
    codes = torch.arange(256, dtype=torch.uint8, device=DEV)
    for b in (1, 2, 64, 119, 127, 200, 246, 255):
        sc = torch.full((8,), b, dtype=torch.uint8, device=DEV)
        m, r = torch.empty(256, dtype=BF16, device=DEV), torch.empty(256, dtype=BF16, device=DEV)
        moe_moment_values(codes, sc, codes, torch.full_like(sc, min(b, 253) if b != 255 else 255), m, r)
        if b == 255:
            assert torch.isnan(m).all() and torch.isnan(r).all()
            continue
        want = codes.view(torch.float8_e4m3fn).double() * 2.0 ** (b - 127)
        if b < 3:
            want = want.to(BF16).double()
        assert torch.equal(torch.isnan(m), torch.isnan(want)) and torch.equal(
            m.double()[~torch.isnan(want)], want[~torch.isnan(want)])
        c = codes.int()
        want = torch.where(c > 0, (1 + c.double() % 16 / 16) * two_to(c // 16 - 15 + min(b, 253) - 127), 0.0)
        if b < 13:
            want = want.to(BF16).double()
        assert torch.equal(r.double(), want)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 1000, 4096, 5001])
def test_moments_to_codes_and_back(n):
    g = torch.Generator(device=DEV).manual_seed(n)
    m = rnd(n, g) * torch.exp(6 * rnd(n, g))
    v = (rnd(n, g) * torch.exp(6 * rnd(n, g))).square()
    m[n // 2], v[n // 2] = 0.0, 0.0
    edge = torch.tensor([464.0, 463.9, 448.0, 2.0 ** -9, 2.0 ** -10, -464.0, 1.5 * 2.0 ** -9], device=DEV)
    if n >= 64:
        m[32:64] = 0.0
        m[32:39] = edge
        v[32:64] = 0.0
        v[32:36] = torch.tensor([1.96875 ** 2, 1.9 ** 2, 1e-30, 1e-12], device=DEV)
    c = [torch.zeros(n, dtype=torch.uint8, device=DEV), torch.zeros(-(-n // 32), dtype=torch.uint8, device=DEV),
         torch.zeros(n, dtype=torch.uint8, device=DEV), torch.zeros(-(-n // 32), dtype=torch.uint8, device=DEV)]
    moe_moment_codes(m, v, *c)
    a, r = torch.empty(n, dtype=BF16, device=DEV), torch.empty(n, dtype=BF16, device=DEV)
    moe_moment_values(*c, a, r)
    want, b, _ = first_codes_ref(grouped(m))
    assert torch.equal(c[1].int(), b.int()) and torch.equal(a.double(), want.reshape(-1)[:n])
    root = torch.sqrt(v.double())
    want, b, step = root_codes_ref(grouped(root))
    assert torch.equal(c[3].int(), b.int())
    # the root is rounded to float32 first: at a middle between codes it may fall to either
    off = (r.double() - root).abs() <= (step.reshape(-1)[:n] / 2) * (1 + 1e-5) + 0 * root
    low = (root > 0) & (r.double() == (17 / 16 * 2.0 ** -15 * two_to(b - 127)).repeat_interleave(32)[:n])
    assert (off | low).all() and torch.equal(r > 0, v > 0)


def test_groups_with_what_is_not_a_number():
    m, v = torch.ones(96, device=DEV), torch.ones(96, device=DEV)
    m[5], v[70] = float("inf"), float("nan")
    c = [torch.zeros(96, dtype=torch.uint8, device=DEV), torch.zeros(3, dtype=torch.uint8, device=DEV),
         torch.zeros(96, dtype=torch.uint8, device=DEV), torch.zeros(3, dtype=torch.uint8, device=DEV)]
    moe_moment_codes(m, v, *c)
    a, r = torch.empty(96, dtype=BF16, device=DEV), torch.empty(96, dtype=BF16, device=DEV)
    moe_moment_values(*c, a, r)
    assert torch.isnan(a[:32]).all() and (a[32:] == 1).all()
    assert (r[:64] == 1).all() and torch.isnan(r[64:]).all()


def test_captured_and_replayed():
    def build():
        return make([70000, 513, 64], "bf16", "f32", "q8", True, seed=8, lr=1e-3, max_norm=0.02, step=2)
    opt, eager = build(), build()
    for o in (opt, eager):
        o.step_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        opt.step_()
    for i in range(5):
        for o in (opt, eager):
            gen = torch.Generator(device=DEV).manual_seed(90 + i)
            for t in o.grads:
                t.copy_(rnd(t.numel(), gen, 1e-3))
            o.lr.fill_(1e-3 / (i + 1))
        g.replay()
        eager.step_()
        torch.cuda.synchronize()
        assert opt.step.item() == eager.step.item() == 4 + i
        for a, b in zip(opt.params + opt.masters + sum(opt.moments.values(), []),
                        eager.params + eager.masters + sum(eager.moments.values(), [])):
            assert torch.equal(a, b), i
        assert torch.equal(opt.norm, eager.norm)


def test_two_graphs_that_share_a_plan_replayed_in_turn():
    def build():
        return make([9000, 4097, 5], "bf16", "f32", "f32", True, seed=12, lr=1e-3, max_norm=0.02)
    opt, eager = build(), build()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            opt.step_()
    for i in range(6):
        graphs[i % 2].replay()
        eager.step_()
        torch.cuda.synchronize()
        assert opt.step.item() == eager.step.item() and torch.equal(opt.norm, eager.norm)
        assert all(torch.equal(a, b) for a, b in zip(opt.params + opt.masters, eager.params + eager.masters)), i


def test_another_stream_and_nothing_beside_the_tensors():
    n, pad = 4099, 32
    bufs = [torch.full((n + 2 * pad,), 3.0, device=DEV) for _ in range(4)]
    p, g, m, v = [b[pad:pad + n] for b in bufs]
    g.fill_(0.5), m.zero_(), v.zero_()
    s = torch.cuda.Stream()
    opt = MoEAdamW([p], [g], lr=0.25, weight_decay=0.0, moments=dict(m=[m], v=[v]))
    s.wait_stream(torch.cuda.current_stream())
    opt.step_(s)
    torch.cuda.synchronize()
    assert all((b[:pad] == 3.0).all() and (b[pad + n:] == 3.0).all() for b in bufs)
    assert (p - 2.75).abs().max() < 1e-5


def test_a_tensor_past_32_bit_offsets():
    n = (1 << 32) + 12345
    p, g = torch.zeros(n, dtype=BF16, device=DEV), torch.zeros(n, dtype=BF16, device=DEV)
    at = torch.tensor([0, (1 << 31) + 1, n - 1], device=DEV)
    g[at] = 1.0
    mom = dict(m=[torch.zeros(n, dtype=torch.uint8, device=DEV)], v=[torch.zeros(n, dtype=torch.uint8, device=DEV)],
               m_scales=[torch.ones(-(-n // 32), dtype=torch.uint8, device=DEV)],
               v_scales=[torch.ones(-(-n // 32), dtype=torch.uint8, device=DEV)])
    opt = MoEAdamW([p], [g], lr=0.5, betas=(B1, B2), weight_decay=0.0, max_norm=100.0, state="q8", moments=mom)
    opt.step_()
    assert abs(opt.norm.item() - math.sqrt(3)) < 1e-6 and opt.step.item() == 1
    assert (p[at] == -0.5).all() and (mom["m"][0][at] != 0).all() and (mom["v"][0][at] != 0).all()
    p[at] = 0
    mom["m"][0][at] = 0
    mom["v"][0][at] = 0
    for t in (p, mom["m"][0], mom["v"][0]):
        for i in range(0, n, 1 << 30):
            assert not t[i:i + (1 << 30)].any()


def test_refusals():
    z = lambda n, dt=F32: torch.zeros(n, dtype=dt, device=DEV)  # noqa: E731
    with pytest.raises(ValueError, match="no parameters"):
        MoEAdamW([], [])
    with pytest.raises(ValueError, match="state"):
        MoEAdamW([z(8)], [z(8)], state="q4")
    with pytest.raises(ValueError, match="beta"):
        MoEAdamW([z(8)], [z(8)], betas=(0.9, 1.0))
    with pytest.raises(ValueError, match="max_norm"):
        MoEAdamW([z(8)], [z(8)], max_norm=0.0)
    with pytest.raises(ValueError, match="needs 8 elements"):
        MoEAdamW([z(8)], [z(9)])
    with pytest.raises(TypeError, match="bfloat16 or torch.float32"):
        MoEAdamW([z(8, torch.float16)], [z(8)])
    with pytest.raises(TypeError, match="expected torch.float32"):
        AdamWTable([z(8)], [z(8)], [z(8, BF16)], [z(8)])
    with pytest.raises(ValueError, match="weight_decay: 2 values"):
        MoEAdamW([z(8)], [z(8)], weight_decay=[0.1, 0.2])
    with pytest.raises(ValueError, match="scales"):
        MoEAdamW([z(8)], [z(8)], state="q8", moments=dict(m=[z(8)], v=[z(8)]))
    p = z(64)
    for params, grads in (([p, p], [z(64), z(64)]), ([p, p[32:]], [z(64), z(32)]), ([p], [p])):
        with pytest.raises(MoEError):                # a buffer that is written twice, or is a gradient too
            MoEAdamW(params, grads)
    g = z(64)
    MoEAdamW([p[:32], p[32:]], [g[:32], g[:32]])     # neighbours, and a gradient for two
    with pytest.raises(MoEError):                    # off by 4 bytes
        MoEAdamW([z(12)[1:9]], [z(8)])
