"""Norms: what one row holds stays out of what it has no part in; outputs in the
place of inputs."""

import pytest
import torch

from mixture_experts_expert_amd import layer_norm_workspace, moe_layer_norm_bwd, moe_layer_norm_fwd

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("rows,D", [(65, 33), (1, 33), (300, 65), (130, 33), (9, 1111), (5, 64), (517, 100), (3, 7), (40, 777)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("row", [0, -1])
@pytest.mark.parametrize("col", [1, -1, -2])
def test_an_infinite_element_reaches_its_own_column_alone(rows, D, dtype, row, col):
    """RMS norm, where the row's other xhat are 0: the weight gradient is NaN (inf * 0) in its column and finite in the
    others, also where teams without a row of their own keep the last row's company."""
    g = torch.Generator(device=DEV).manual_seed(rows + D)
    h = torch.randn((rows, D), generator=g, device=DEV).to(dtype)
    dy = torch.randn((rows, D), generator=g, device=DEV).to(dtype)
    h[row, col] = float("inf")
    w = torch.ones(D, device=DEV)
    rstd = torch.ones(rows, device=DEV)
    rstd[row] = 0.0                                      # 1 / sqrt(inf)
    dx, dw = torch.empty_like(h), torch.empty(D, device=DEV)
    moe_layer_norm_bwd(dy, h, w, None, rstd, dx, dw, None, layer_norm_workspace(rows, D))
    want = (dy.double() * (h.double() * rstd.double()[:, None])).sum(0)
    assert torch.equal(torch.isnan(dw), torch.isnan(want)) and torch.isnan(want).sum() == 1
    others = torch.arange(rows, device=DEV) != row % rows
    assert torch.isfinite(dx[others]).all() and torch.isnan(dx[row % rows, col % D])
    fine = ~torch.isnan(want)
    mag = (dy.double() * h.double() * rstd.double()[:, None]).abs().sum(0)
    # rows / 256 + 92 additions deep at most, and xhat's rounding
    assert ((dw.double() - want).abs()[fine] <= (rows / 256 + 95) * 2.0 ** -24 * mag[fine]).all()


@pytest.mark.parametrize("rows,D", [(9, 1111), (70, 33), (5, 64), (3, 7), (200, 2048)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_outputs_in_the_place_of_inputs(rows, D, dtype):
    """Each that the calls allow, against outputs of their own."""
    g = torch.Generator(device=DEV).manual_seed(rows + D)
    x, r, dy, dt = (torch.randn((rows, D), generator=g, device=DEV).to(dtype) for _ in range(4))
    w, b = torch.randn(D, generator=g, device=DEV), torch.randn(D, generator=g, device=DEV)
    f = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device=DEV)  # noqa: E731

    def fwd(x, r, total, y):
        mean, rstd = f(rows), f(rows)
        moe_layer_norm_fwd(x, w, b, 1e-6, y, mean, rstd, residual=r, total=total)
        return total, y, mean, rstd
    want = fwd(x, r, f(rows, D, t=dtype), f(rows, D, t=dtype))
    for total, y in (("x", None), ("r", None), (None, "x"), (None, "r"), ("x", "r"), ("r", "x")):
        c = dict(x=x.clone(), r=r.clone())
        got = fwd(c["x"], c["r"], c[total] if total else f(rows, D, t=dtype), c[y] if y else f(rows, D, t=dtype))
        assert all(torch.equal(p, q) for p, q in zip(got, want)), (total, y)
    h, _, mean, rstd = want

    def bwd(dy, h, dt, dx):
        dw, db = f(D), f(D)
        moe_layer_norm_bwd(dy, h, w, mean, rstd, dx, dw, db, layer_norm_workspace(rows, D), dtotal=dt)
        return dx, dw, db
    want = bwd(dy, h, dt, f(rows, D, t=dtype))
    for place in ("dy", "h", "dt"):
        c = dict(dy=dy.clone(), h=h.clone(), dt=dt.clone())
        assert all(torch.equal(p, q) for p, q in zip(bwd(c["dy"], c["h"], c["dt"], c[place]), want)), place
