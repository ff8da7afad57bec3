"""Layer norm and RMS norm on the GPU (moe_layer_norm_fwd, moe_layer_norm_bwd)
against float64.

Bars, from the arithmetic (u = 2^-24).  A row's sum is a tree: a lane adds at
most 32 columns, six exchanges join a wave, at most 8 waves are added: under 64
additions deep, so a sum of magnitude-sum S is off by at most 64 u S.

forward (h, the stored total, is compared bit for bit):
* mean: dm = 64 u mean|h| + 2u|mean|
* the variance about the computed mean exceeds the variance by dm^2; each
  difference is rounded (u relative), squared and summed: 68 u of it.  rstd is
  off by half the relative error of var + eps, and 4u for the root and division
* y: |rstd w| (dm + u|h - mean|) + (rel(rstd) + 4u) |xhat w| + 2u |y|, and the
  rounding, half a step of the type (2^-8 or u, relative)

backward, from the given mean and rstd: xhat is off by 3u of itself, so
* c1, the mean of g xhat, by 70 u mean|g xhat|, c2 by 70 u mean|g|
* dx: rstd (6u |g| + dc2 + 4u |c2| + |xhat| (dc1 + 8u |c1|)) + 4u (|dx| + |dtotal|)
  and the rounding
* dweight, dbias: a lane adds its rows in turn (up to four of one workgroup's, one,
  or rows / 256 with 256 workgroups at work), then come up to 64 teams of a
  workgroup, 4 workgroups, 8 and 8 of their sums: (rows / 256 + 84 + 8) u of the sum
  of magnitudes (one workgroup's: 4 + 64)
"""

import pytest
import torch

from gpu_support import say
from mixture_experts_expert_amd import (MoEError, layer_norm_workspace, moe_layer_norm_bwd, moe_layer_norm_fwd)

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: U}
EPS = 1e-6


def draw(shape, dtype, seed, spread=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(shape, generator=g, device=DEV)
    if spread:
        x = x * torch.exp(torch.randn(shape[-1], generator=g, device=DEV)) + torch.randn(shape[-1], generator=g, device=DEV)
    return x.to(dtype)


def params(D, seed, bias=True):
    g = torch.Generator(device=DEV).manual_seed(seed + 1000)
    w = 1 + 0.3 * torch.randn(D, generator=g, device=DEV)
    return w, 0.2 * torch.randn(D, generator=g, device=DEV) if bias else None


def run_fwd(x, w, b, ty, centre, residual=None):
    rows = x.shape[:-1]
    y = torch.full(x.shape, float("nan"), dtype=ty, device=DEV)
    mean = torch.full(rows, float("nan"), device=DEV) if centre else None
    rstd = torch.full(rows, float("nan"), device=DEV)
    total = torch.full_like(x, float("nan")) if residual is not None else None
    moe_layer_norm_fwd(x, w, b, EPS, y, mean, rstd, residual=residual, total=total)
    return y, mean, rstd, total


def check_fwd(x, w, b, y, mean, rstd, residual=None, total=None, eps=EPS):
    if residual is not None:
        assert torch.equal(total, (x.float() + residual.float()).to(x.dtype)), "the total differs"
        x = total
    h = x.double()
    m = h.mean(-1, keepdim=True) if mean is not None else torch.zeros_like(h[..., :1])
    dm = 64 * U * h.abs().mean(-1, keepdim=True) + 2 * U * m.abs() if mean is not None else 0 * m
    var = (h - m).square().mean(-1, keepdim=True)
    r = 1 / torch.sqrt(var + eps)
    rel = 0.5 * (68 * U * var + dm ** 2) / (var + eps) + 4 * U
    xhat = (h - m) * r
    want = xhat * w.double() + (b.double() if b is not None else 0)
    bar = (r * w.double()).abs() * (dm + U * (h - m).abs()) + (rel + 4 * U) * (xhat * w.double()).abs() + 2 * U * want.abs()
    bar = bar + HALF[y.dtype] * (want.abs() + bar)
    over = [0.0]
    if mean is not None:
        over.append(((mean.double() - m[..., 0]).abs() / dm[..., 0].clamp(min=1e-300)).max().item())
    over.append(((rstd.double() - r[..., 0]).abs() / (rel * r)[..., 0]).max().item())
    over.append(((y.double() - want).abs() / bar.clamp(min=1e-300)).max().item())
    say(f"  {tuple(x.shape)} {x.dtype} -> {y.dtype}: " + ", ".join(f"{o:.3f}" for o in over[1:]) + " of the bars")
    assert all(o <= 1.0 for o in over), over      # NaN is not


def check_bwd(dy, h, w, mean, rstd, dx, dw, db, dtotal=None, old=None):
    D, rows = h.shape[-1], h.numel() // h.shape[-1]
    dy, h = dy.double().reshape(rows, D), h.double().reshape(rows, D)
    m = mean.double().reshape(rows, 1) if mean is not None else 0.0
    r = rstd.double().reshape(rows, 1)
    xhat, g = (h - m) * r, dy * w.double()
    c1 = (g * xhat).mean(1, keepdim=True)
    c2 = g.mean(1, keepdim=True) if mean is not None else torch.zeros_like(c1)
    want = r * (g - c2 - xhat * c1)
    dc1, dc2 = 70 * U * (g * xhat).abs().mean(1, keepdim=True), 70 * U * g.abs().mean(1, keepdim=True)
    bar = r * (6 * U * g.abs() + dc2 + 4 * U * c2.abs() + xhat.abs() * (dc1 + 8 * U * c1.abs()))
    if dtotal is not None:
        d = dtotal.double().reshape(rows, D)
        bar, want = bar + 4 * U * d.abs(), want + d
    bar = bar + 4 * U * want.abs()
    bar = bar + HALF[dx.dtype] * (want.abs() + bar)
    over = [((dx.double().reshape(rows, D) - want).abs() / bar.clamp(min=1e-300)).max().item() if rows else 0.0]
    deep = rows / 256 + 84
    for got, terms, k in ((dw, dy * xhat, 0), (db, dy, 1)):
        if got is None:
            continue
        want, mag = terms.sum(0), terms.abs().sum(0)
        bar = (deep + 8) * U * mag + 1e-300
        if old is not None:
            want, bar = want + old[k].double(), bar + 2 * U * (want + old[k].double()).abs()
        over.append(((got.double() - want).abs() / bar).max().item())
    say(f"  backward {rows} x {D}: " + ", ".join(f"{o:.3f}" for o in over) + " of the bars")
    assert all(o <= 1.0 for o in over), over      # NaN is not


SHAPES = [(1, 1), (3, 7), (5, 64), (2, 512), (7, 513), (9, 1024), (4, 1111), (130, 2048), (3, 2049), (6, 4096),
          (2, 5003), (11, 7168), (3, 8192), (2, 8193), (5, 16384), (2, 16383), (2500, 192), (700, 2048),
          # rows that begin anywhere in 16 bytes, one and several of them to a team, each lanes-and-pieces form
          (70000, 9), (20000, 13), (9000, 100), (5000, 250), (5000, 300), (3000, 513), (1, 777), (1500, 1111), (1030, 2047),
          (700, 2049), (300, 4097), (260, 5002), (16, 2048), (17, 2048), (256, 64), (9, 7168), (2, 4097), (3, 5003), (300, 8193), (300, 12292), (40, 16380)]
TYPES = [(BF16, BF16), (F32, BF16), (F32, F32)]


@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("tx,ty", TYPES)
@pytest.mark.parametrize("centre", [True, False])
def test_forward_and_backward(rows, D, tx, ty, centre):
    seed = rows * 31 + D
    x, w = draw((rows, D), tx, seed), params(D, seed)[0]
    b = params(D, seed)[1] if centre else None
    residual = draw((rows, D), tx, seed + 1) if (rows + D) % 2 else None
    y, mean, rstd, total = run_fwd(x, w, b, ty, centre, residual)
    check_fwd(x, w, b, y, mean, rstd, residual, total)
    h = x if residual is None else total
    dy, dtotal = draw((rows, D), ty, seed + 2, False), draw((rows, D), tx, seed + 3, False) if residual is not None else None
    dx = torch.full_like(h, float("nan"))
    dw = torch.full((D,), float("nan"), device=DEV)
    db = torch.full((D,), float("nan"), device=DEV) if centre else None
    ws = layer_norm_workspace(rows, D)
    ws.fill_(255)
    moe_layer_norm_bwd(dy, h, w, mean, rstd, dx, dw, db, ws, dtotal=dtotal)
    check_bwd(dy, h, w, mean, rstd, dx, dw, db, dtotal)
    again = [torch.empty_like(dx), torch.empty_like(dw), torch.empty_like(db) if db is not None else None]
    moe_layer_norm_bwd(dy, h, w, mean, rstd, *again, ws, dtotal=dtotal)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw) and (db is None or torch.equal(again[2], db))


def test_bias_without_a_mean_and_a_mean_without_a_bias():
    x, (w, b) = draw((33, 320), F32, 5), params(320, 5)
    y, mean, rstd, _ = run_fwd(x, w, b, F32, False)
    check_fwd(x, w, b, y, None, rstd)
    y, mean, rstd, _ = run_fwd(x, w, None, F32, True)
    check_fwd(x, w, None, y, mean, rstd)
    dy, ws = draw((33, 320), F32, 6), layer_norm_workspace(33, 320)
    dx, dw, db = torch.empty_like(x), torch.empty(320, device=DEV), torch.empty(320, device=DEV)
    moe_layer_norm_bwd(dy, x, w, None, rstd, dx, dw, db, ws)
    check_bwd(dy, x, w, None, rstd, dx, dw, db)
    moe_layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, None, ws)
    check_bwd(dy, x, w, mean, rstd, dx, dw, None)


@pytest.mark.parametrize("centre", [True, False])
def test_gradients_against_differences(centre):
    rows, D = 3, 70
    x, (w, b) = draw((rows, D), F32, 21), params(D, 21)
    if not centre:
        b = None
    y, mean, rstd, _ = run_fwd(x, w, b, F32, centre)
    dy, ws = draw((rows, D), F32, 22), layer_norm_workspace(rows, D)
    dx, dw = torch.empty_like(x), torch.empty(D, device=DEV)
    db = torch.empty(D, device=DEV) if centre else None
    moe_layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db, ws)

    def loss(x, w, b):
        m = x.mean(1, keepdim=True) if centre else 0.0
        xc = x - m
        z = xc / torch.sqrt(xc.square().mean(1, keepdim=True) + EPS) * w
        return ((z + b if b is not None else z) * dy.double().cpu()).sum()
    args = [x.double().cpu(), w.double().cpu(), b.double().cpu() if centre else None]
    step = 2.0 ** -16                       # truncation about step^2, rounding about 2^-52 / step
    for k, got in enumerate((dx, dw, db)):
        if got is None:
            continue
        flat = args[k].reshape(-1)
        for i in range(0, flat.numel(), 3):
            old = flat[i].item()
            flat[i] = old + step
            up = loss(*args)
            flat[i] = old - step
            down = loss(*args)
            flat[i] = old
            want = ((up - down) / (2 * step)).item()
            assert abs(got.reshape(-1)[i].item() - want) <= 1e-4 * (1 + abs(want)), (k, i)


@pytest.mark.parametrize("rows,D", [(300, 640), (40, 777), (9, 1111), (20, 5001), (5, 10001), (6, 5), (2, 4097), (4, 4104), (16, 1536)])
def test_accumulated_weight_gradients_and_in_place_outputs(rows, D):
    x, (w, b) = draw((rows, D), BF16, 31), params(D, 31)
    residual = draw((rows, D), BF16, 32)
    y, mean, rstd, total = run_fwd(x, w, b, BF16, True, residual)
    dy, dtotal = draw((rows, D), BF16, 33), draw((rows, D), BF16, 34)
    ws = layer_norm_workspace(rows, D)
    dx, dw, db = torch.empty_like(x), torch.empty(D, device=DEV), torch.empty(D, device=DEV)
    moe_layer_norm_bwd(dy, total, w, mean, rstd, dx, dw, db, ws, dtotal=dtotal)
    old = [torch.randn(D, device=DEV), torch.randn(D, device=DEV)]
    aw, ab = old[0].clone(), old[1].clone()
    d2 = dtotal.clone()
    moe_layer_norm_bwd(dy, total, w, mean, rstd, d2, aw, ab, ws, dtotal=d2, accumulate=True)   # dx in dtotal's place
    assert torch.equal(d2, dx) and torch.equal(aw, old[0] + dw) and torch.equal(ab, old[1] + db)
    d3 = dy.clone()
    moe_layer_norm_bwd(d3, total, w, mean, rstd, d3, dw, db, ws, dtotal=dtotal)                 # in dy's
    assert torch.equal(d3, dx)
    d4 = total.clone()
    moe_layer_norm_bwd(dy, d4, w, mean, rstd, d4, dw, db, ws, dtotal=dtotal)                    # in h's
    assert torch.equal(d4, dx)
    # the total in the place of x, and in the residual's; y in x's
    for place in (0, 1):
        a, r = x.clone(), residual.clone()
        y2, m2, s2 = torch.empty_like(y), torch.empty_like(mean), torch.empty_like(rstd)
        moe_layer_norm_fwd(a, w, b, EPS, y2, m2, s2, residual=r, total=(a, r)[place])
        assert torch.equal(y2, y) and torch.equal((a, r)[place], total) and torch.equal(m2, mean)
    a = total.clone()
    moe_layer_norm_fwd(a, w, b, EPS, a, m2, s2)
    assert torch.equal(a, y)


def test_a_stack_of_rows_and_no_rows():
    x, (w, b) = draw((4, 5, 96), BF16, 41), params(96, 41)
    y, mean, rstd, _ = run_fwd(x, w, b, BF16, True)
    check_fwd(x, w, b, y, mean, rstd)
    z, mean0, rstd0, _ = run_fwd(x[:0], w, b, BF16, True)
    assert z.shape == (0, 5, 96)
    dw, db, ws = torch.ones(96, device=DEV), torch.ones(96, device=DEV), layer_norm_workspace(0, 96)
    moe_layer_norm_bwd(x[:0], x[:0], w, mean0, rstd0, torch.empty_like(x[:0]), dw, db, ws, accumulate=True)
    assert (dw == 1).all() and (db == 1).all()
    moe_layer_norm_bwd(x[:0], x[:0], w, mean0, rstd0, torch.empty_like(x[:0]), dw, db, ws)
    assert (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("centre", [True, False])
def test_rows_far_from_zero_rows_of_one_value_and_rows_that_are_not_numbers(centre):
    D = 1000
    x = torch.randn((6, D), device=DEV, generator=torch.Generator(device=DEV).manual_seed(51))
    x[0] += 1000.0                          # the variance is the second pass's
    x[1] = 3.0                              # no variance: eps alone
    x[2] = 0.0
    x[3, 17] = float("inf")
    x[4, 18] = float("nan")
    w, b = params(D, 51)
    y, mean, rstd, _ = run_fwd(x, w, b, F32, centre)
    ok = [0, 1, 2, 5]
    check_fwd(x[ok], w, b, y[ok], mean[ok] if centre else None, rstd[ok])
    assert torch.isnan(y[4]).all() and not torch.isfinite(y[3, 17])
    assert torch.isfinite(y[ok]).all()


@pytest.mark.parametrize("rows,D", [(9, 9), (70, 33), (40, 515), (20, 1111), (11, 2049), (9, 8197), (5, 16383), (8, 5)])
@pytest.mark.parametrize("tx,ty", TYPES)
def test_rows_that_share_16_bytes_keep_to_themselves(rows, D, tx, ty):
    """Every second row holds what is not a number: the others come out as without
    them, bit for bit, and nothing before, behind or between is written twice."""
    x, residual, dy, dtotal = (draw((rows, D), t, 91 + i) for i, t in enumerate((tx, tx, ty, tx)))
    w, b = params(D, 91)
    guard = 24                                             # elements: 16-byte aligned in either type

    def between(t):
        buf = torch.full((t.numel() + 2 * guard,), 7.25, dtype=t.dtype, device=DEV)
        return buf, buf[guard:-guard].view(t.shape)

    def run(x, dy):
        keep, out = [], []
        for like in (x, x.to(ty), x):
            buf, view = between(like)
            keep.append(buf), out.append(view)
        total, y, dx = out
        mean, rstd = torch.zeros(rows, device=DEV), torch.zeros(rows, device=DEV)
        dw, db = torch.zeros(D, device=DEV), torch.zeros(D, device=DEV)
        moe_layer_norm_fwd(x, w, b, EPS, y, mean, rstd, residual=residual, total=total)
        moe_layer_norm_bwd(dy, total, w, mean, rstd, dx, dw, db, layer_norm_workspace(rows, D), dtotal=dtotal)
        for buf in keep:
            assert (buf[:guard] == 7.25).all() and (buf[-guard:] == 7.25).all()
        return total, y, dx
    clean = run(x, dy)
    bad_x, bad_dy = x.clone(), dy.clone()
    for i, v in enumerate((float("nan"), float("inf"), float("-inf"))):
        bad_x[1 + 2 * i::6] = v
        bad_dy[1 + 2 * i::6] = v
    dirty = run(bad_x, bad_dy)
    for c, d in zip(clean, dirty):
        assert torch.equal(c[::2], d[::2])
    assert torch.isnan(dirty[1][1]).all() and torch.isnan(dirty[2][1]).all()


def test_two_streams_at_once():
    cases = []
    for i, (rows, D) in enumerate([(3000, 1111), (2000, 2048)]):
        x, dy, (w, b) = draw((rows, D), BF16, 95 + i), draw((rows, D), BF16, 97 + i), params(D, 95 + i)
        cases.append((x, dy, w, b, layer_norm_workspace(rows, D)))

    def run(c, stream=None):
        x, dy, w, b, ws = c
        rows, D = x.shape
        out = [torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV), torch.empty_like(x),
               torch.empty(D, device=DEV), torch.empty(D, device=DEV)]
        torch.cuda.synchronize()
        for _ in range(3):
            moe_layer_norm_fwd(x, w, b, EPS, out[0], out[1], out[2], stream=stream)
            moe_layer_norm_bwd(dy, x, w, out[1], out[2], out[3], out[4], out[5], ws, stream=stream)
        return out
    alone = [run(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    both = [run(c, s) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for a, t in zip(alone, both):
        assert all(torch.equal(p, q) for p, q in zip(a, t))


def test_rows_past_32_bit_offsets():
    rows, D = (1 << 31) // 2048 + 3, 2048
    x = torch.zeros((rows, D), dtype=BF16, device=DEV)
    tail = draw((5, D), BF16, 61)
    x[-5:] = tail
    w, b = params(D, 61)
    y = torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    moe_layer_norm_fwd(x, w, b, EPS, y, mean, rstd)
    want = run_fwd(tail, w, b, BF16, True)
    assert torch.equal(y[-5:], want[0]) and torch.equal(rstd[-5:], want[2])
    assert torch.equal(y[rows // 2], b.to(BF16))
    dx, dw, db = y, torch.empty(D, device=DEV), torch.empty(D, device=DEV)
    dy = torch.zeros_like(x)
    dy[-5:] = draw((5, D), BF16, 62)
    moe_layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db, layer_norm_workspace(rows, D))
    check_bwd(dy[-5:], tail, w, mean[-5:], rstd[-5:], dx[-5:], None, None)
    xh = (tail.double() - mean[-5:].double()[:, None]) * rstd[-5:].double()[:, None]
    d = dy[-5:].double()
    assert ((dw.double() - (d * xh).sum(0)).abs() <= 100 * U * (d * xh).abs().sum(0)).all()
    assert ((db.double() - d.sum(0)).abs() <= 100 * U * d.abs().sum(0)).all()


def test_captured_and_replayed():
    rows, D = 96, 768
    x, (w, b) = draw((rows, D), BF16, 71), params(D, 71)
    dy, ws = draw((rows, D), BF16, 72), layer_norm_workspace(rows, D)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    dx, dw, db = torch.empty_like(x), torch.zeros(D, device=DEV), torch.zeros(D, device=DEV)

    def step(stream=None):
        moe_layer_norm_fwd(x, w, b, EPS, y, mean, rstd, stream=stream)
        moe_layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db, ws, accumulate=True, stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        x.copy_(draw((rows, D), BF16, 80 + i))
        dw.zero_(), db.zero_()
        g.replay()
        got = [t.clone() for t in (y, mean, rstd, dx, dw, db)]
        dw.zero_(), db.zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, (y, mean, rstd, dx, dw, db))), i


def test_refusals():
    x, (w, b) = draw((4, 64), BF16, 91), params(64, 91)
    y, mean, rstd = torch.empty_like(x), torch.empty(4, device=DEV), torch.empty(4, device=DEV)
    with pytest.raises(ValueError, match="together"):
        moe_layer_norm_fwd(x, w, b, EPS, y, mean, rstd, residual=x)
    with pytest.raises(ValueError, match="weight must have"):
        moe_layer_norm_fwd(x, w[:32], b, EPS, y, mean, rstd)
    with pytest.raises(ValueError, match="contiguous"):
        moe_layer_norm_fwd(draw((4, 128), BF16, 1)[:, :64], w, b, EPS, y, mean, rstd)
    with pytest.raises(TypeError, match="bfloat16 or torch.float32"):
        moe_layer_norm_fwd(x.half(), w, b, EPS, y, mean, rstd)
    with pytest.raises(MoEError):                    # bf16 in, float32 out
        moe_layer_norm_fwd(x, w, b, EPS, y.float(), mean, rstd)
    with pytest.raises(MoEError):
        moe_layer_norm_fwd(x, w, b, -1.0, y, mean, rstd)
    with pytest.raises(MoEError):                    # the total would be lost
        moe_layer_norm_fwd(x, w, b, EPS, y, mean, rstd, residual=x, total=y)
    dw = torch.empty(64, device=DEV)
    with pytest.raises(ValueError, match="workspace: needs"):
        moe_layer_norm_bwd(x, x, w, mean, rstd, y, dw, None, torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="dy must be"):
        moe_layer_norm_bwd(x[:3], x, w, mean, rstd, y, dw, None, layer_norm_workspace(4, 64))
