"""The AdamW step that rounds 8-bit moments stochastically, on the GPU: every
code against the documented rule's, from float64.

The kernel's moments are float32 (u = 2^-24): m off by dm = (8u + 5u for the clip)
(|b1 m| + |(1 - b1) g|), the root by droot = (11 + 5)u of itself.  A decision
compares a fraction of the way between two codes with a random one; the fraction
is off by dm over the codes' distance and 2^-19 (20 random bits, and the sum that
brings small magnitudes to a common step), a root's by 2.1 droot over the
distance and 2^-20.  Elements whose two fractions are nearer than that, or are
that near to 0 and 1, may go either way; so may groups whose largest
magnitude is that near to a scale's border.
"""

import warnings

import numpy as np
import pytest
import torch

from gpu_support import say
from mixture_experts_expert_amd import MoEAdamW, moe_moment_codes
from oracle import moments as M

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
BF16 = torch.bfloat16
B1, B2 = 0.9, 0.999


def make(sizes, inputs=1, spread=1.0, pt=torch.float32, masters=None, **kw):
    g = torch.Generator(device=DEV).manual_seed(inputs)
    rnd = lambda n: torch.randn(n, generator=g, device=DEV)  # noqa: E731
    params = [(0.05 * rnd(n)).to(pt) for n in sizes]
    grads = [1e-3 * rnd(n) * torch.exp(spread * rnd(n)) for n in sizes]
    mom = dict(m=[], v=[], m_scales=[], v_scales=[])
    for n in sizes:
        c = [torch.zeros(k, dtype=torch.uint8, device=DEV) for k in (n, -(-n // 32), n, -(-n // 32))]
        if n:
            moe_moment_codes(3e-4 * rnd(n) * torch.exp(spread * rnd(n)), (1e-3 * rnd(n) * torch.exp(spread * rnd(n))).square(), *c)
        for k, t in zip(("m", "m_scales", "v", "v_scales"), c):
            mom[k].append(t)
    kw.setdefault("rounding", "stochastic")
    return MoEAdamW(params, grads, betas=(B1, B2), state="q8", moments=mom, masters=masters, **kw)


def padded(t):
    a = t.double().cpu().numpy()
    return np.concatenate([a, np.zeros(-len(a) % 32)])


def undecided(f, u, x, d, lo, hi, slack, top, scale):
    """Where float32 may round the other way: f the fraction that is compared with u; x is off by up to d."""
    step = np.where(hi > lo, hi - lo, np.inf)
    err = np.where((d > 0) & (hi > lo), d / step + slack, 0.0)      # one code, no decision
    amax = np.abs(x).max(1) / scale
    border = (np.abs(amax - top) <= 1e-5 * top) | (np.abs(amax - top / 2) <= 1e-5 * top)
    # x next to a code may be on its other side: it comes to that code all the same, unless u is as near to 0 or 1
    # (2 err: codes below a power of two are half as far apart)
    ends = ((f <= err) | (f >= 1 - err)) & ((u <= 2 * err) | (u >= 1 - 2 * err))
    return ((np.abs(f - u) <= err) | ends) & (err > 0), border[:, None]


def check(opt, before, t):
    """The moments after step t against the rule; the share of decisions that are too near to call."""
    first, worst, clip = 0, 0.0, 1.0
    if opt.max_norm is not None:
        clip = min(1.0, opt.max_norm / float(np.sqrt(sum((g ** 2).sum() for g, _, _ in before))))
    for i, (g, m, r) in enumerate(before):
        if not len(g):
            continue
        g = g * clip
        h = M.dice(opt.seed, t, first + np.arange(len(g)))
        first += -(-opt.params[i].numel() // 4096) * 4096
        m1, root = B1 * m + (1 - B1) * g, np.sqrt(B2 * r * r + (1 - B2) * g * g)
        got_m, got_r = (padded(x).reshape(-1, 32) for x in opt.moment_values(i))

        x = m1.reshape(-1, 32)
        lo, hi, f, s = M.first_neighbours(m1)
        d = 13 * U * (np.abs(B1 * m) + np.abs((1 - B1) * g)).reshape(x.shape)
        free, border = undecided(f, 1 - M.fractions(h)[0].reshape(x.shape), x, d, lo, hi, 2.0 ** -19, 448.0, s)
        want = M.first_stochastic(m1, h).reshape(x.shape)
        assert ((got_m == want) | free | border).all(), "first moments"
        assert ((np.abs(np.abs(got_m) - np.abs(x)) <= hi - lo + d) | border).all(), "first moments, too near to call"
        worst = max(worst, (free | border).mean())

        x = root.reshape(-1, 32)
        lo, hi, f, s = M.root_neighbours(root)
        free, border = undecided(f, M.fractions(h)[1].reshape(x.shape), x, 2.1 * 16 * U * x, lo, hi, 2.0 ** -20, 1.9375, s)
        want = M.root_stochastic(root, h).reshape(x.shape)
        assert ((got_r == want) | free | border).all(), "roots"
        assert ((np.abs(got_r - x) <= hi - lo + 16 * U * x) | (hi == lo) | border).all(), "roots, too near to call"
        assert (got_r[x > 0] > 0).all(), "a root vanished"
        worst = max(worst, (free | border).mean())
    say(f"  {100 * worst:.3f}% of the decisions are too near to call")
    return worst


def snapshot(opt):
    return [(padded(g), *(padded(x) for x in opt.moment_values(i))) for i, g in enumerate(opt.grads)]


@pytest.mark.parametrize("sizes", [[1], [31, 32, 33], [4095, 4096, 4097, 0, 5], [20000, 7, 8192]])
@pytest.mark.parametrize("seed", [0, 1, (1 << 32) - 1])
@pytest.mark.parametrize("spread", [1.0, 6.0])           # 6: groups that reach down to the smallest codes
def test_codes_are_the_rules(sizes, seed, spread):
    opt = make(sizes, len(sizes), spread, lr=1e-3, max_norm=0.02, step=7, seed=seed)
    for t in (8, 9, 10):
        before = snapshot(opt)
        opt.step_()
        torch.cuda.synchronize()
        near = check(opt, before, t)
        assert sum(sizes) < 1000 or near < 0.02          # a group of 32 at a scale's border is 0.4% of the smaller lists
        assert opt.step.item() == t


def test_parameters_move_as_with_the_other_rounding():
    """By the moments before they are rounded: the same bits from the same moments."""
    a, b = (make([5000, 33], 3, lr=1e-3, max_norm=0.02, step=4, rounding=k) for k in ("stochastic", "nearest"))
    for o in (a, b):
        o.step_()
    assert all(torch.equal(p, q) for p, q in zip(a.params, b.params)) and torch.equal(a.norm, b.norm)
    assert not torch.equal(a.moments["m"][0], b.moments["m"][0])


def test_one_seed_gives_the_same_bits_another_gives_others():
    def after(seed):
        o = make([9000, 4097], 4, lr=1e-3, seed=seed)
        for _ in range(3):
            o.step_()
        return o.params + sum(o.moments.values(), [])
    a, b, c = after(5), after(5), after(6)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert not all(torch.equal(x, y) for x, y in zip(a, c))


def test_captured_and_replayed():
    def build():
        return make([70000, 513, 64], 8, pt=BF16, masters="make", lr=1e-3, max_norm=0.02, step=2, seed=9)
    opt, eager = build(), build()
    for o in (opt, eager):
        o.step_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        opt.step_()
    for i in range(5):
        g.replay()
        eager.step_()
        torch.cuda.synchronize()
        assert opt.step.item() == eager.step.item() == 4 + i
        for a, b in zip(opt.params + opt.masters + sum(opt.moments.values(), []),
                        eager.params + eager.masters + sum(eager.moments.values(), [])):
            assert torch.equal(a, b), i


def test_what_is_not_a_number_and_what_is_nothing():
    n = 96
    opt = MoEAdamW([torch.ones(n, device=DEV)], [torch.zeros(n, device=DEV)], lr=1e-3, weight_decay=0.0, state="q8")
    opt.step_()                                          # no gradient yet: nothing moves
    assert opt.rounding == "stochastic" and (opt.params[0] == 1).all()
    assert not opt.moments["m"][0].any() and not opt.moments["v"][0].any()
    opt.grads[0][:] = 1.0
    opt.grads[0][5], opt.grads[0][70] = float("inf"), float("nan")
    opt.step_()                                          # without a norm the step is taken: their groups are NaN
    m, r = opt.moment_values(0)
    assert torch.isnan(m[:32]).all() and torch.isnan(m[64:]).all() and torch.isfinite(m[32:64]).all()
    assert torch.isnan(r[:32]).all() and torch.isnan(r[64:]).all() and torch.isfinite(r[32:64]).all()
    held = [t.clone() for t in opt.params + sum(opt.moments.values(), [])]
    opt.max_norm = 1.0                                   # with one it is not
    opt.step_()
    assert opt.step.item() == 2
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(held, opt.params + sum(opt.moments.values(), [])))


def test_the_largest_codes():
    """Magnitudes between the largest code and where nearest rounding would leave it go to the next scale."""
    n = 64
    m, v = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    g = torch.zeros(n, device=DEV)
    g[0], g[32] = 4600.0, 4480.0                         # m 460 and 448 at beta1 0.9
    c = [torch.zeros(k, dtype=torch.uint8, device=DEV) for k in (n, 2, n, 2)]
    moe_moment_codes(m, v, *c)
    opt = MoEAdamW([torch.zeros(n, device=DEV)], [g], betas=(0.9, 0.999), state="q8", rounding="stochastic",
                   moments=dict(m=[c[0]], m_scales=[c[1]], v=[c[2]], v_scales=[c[3]]))
    opt.step_()
    got = opt.moment_values(0)[0]
    assert c[1][0].item() == 128 and got[0].item() in (448.0, 480.0)
    assert got[32].item() in (416.0, 448.0)              # float32's 448 may lie a step below it


def test_how_moments_are_rounded_is_said():
    p, g = torch.zeros(64, device=DEV), torch.zeros(64, device=DEV)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert MoEAdamW([p], [g]).rounding is None
        fresh = MoEAdamW([p], [g], state="q8")
        assert fresh.rounding == "stochastic"
        assert MoEAdamW([p], [g], state="q8", rounding="nearest").rounding == "nearest"
        for k in ("stochastic", "nearest"):
            assert MoEAdamW([p], [g], state="q8", moments=fresh.moments, rounding=k).rounding == k
    with pytest.warns(UserWarning, match="do not follow"):
        assert MoEAdamW([p], [g], state="q8", moments=fresh.moments).rounding == "nearest"


def test_a_run_that_goes_on():
    """Another optimizer with the state, the step and the seed takes the same steps."""
    a = make([5000, 33], 6, pt=BF16, masters="make", lr=1e-3, max_norm=0.02, seed=11)
    for _ in range(2):
        a.step_()
    copy = {k: [t.clone() for t in v] for k, v in a.moments.items()}
    b = MoEAdamW([p.clone() for p in a.params], a.grads, lr=1e-3, betas=(B1, B2), max_norm=0.02, state="q8", moments=copy,
                 masters=[m.clone() for m in a.masters], step=a.step.clone(), rounding="stochastic", seed=11)
    for _ in range(3):
        a.step_(), b.step_()
    assert a.step.item() == b.step.item() == 5
    assert all(torch.equal(x, y) for x, y in zip(a.params + a.masters + sum(a.moments.values(), []),
                                                 b.params + b.masters + sum(b.moments.values(), [])))
