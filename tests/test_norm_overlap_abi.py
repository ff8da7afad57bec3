"""moe_layer_norm_fwd and moe_layer_norm_bwd refuse outputs that share memory
with another buffer, but for those that they may be.  No device work: every
call here is refused (or has no rows)."""

import ctypes

import pytest

import mixture_experts_expert_amd as moe

lib = moe.lib
INVALID = -1
ROWS, D, BF16, F32 = 16, 64, 0, 1
ROOM = 1 << 16                                   # bytes between buffers


def place(names, **at):
    """Addresses a room apart, except those given: (name, offset) of another buffer."""
    p = {k: (i + 1) * ROOM for i, k in enumerate(names)}
    for k, (other, off) in at.items():
        p[k] = p[other] + off
    return p


def fwd(xt=F32, yt=F32, residual=True, **at):
    p = place(("x", "residual", "weight", "bias", "total", "y", "mean", "rstd"), **at)
    if not residual:
        p["residual"] = p["total"] = None
    v = {k: ctypes.c_void_p(a) for k, a in p.items()}
    return lib.moe_layer_norm_fwd(v["x"], v["residual"], v["weight"], v["bias"], ROWS, D, 1e-6, xt, yt, v["total"], v["y"],
                                  v["mean"], v["rstd"], None)


def bwd(xt=F32, yt=F32, **at):
    p = place(("dy", "h", "weight", "mean", "rstd", "dtotal", "dx", "dweight", "dbias", "workspace"), **at)
    v = {k: ctypes.c_void_p(a) for k, a in p.items()}
    return lib.moe_layer_norm_bwd(v["dy"], v["h"], v["weight"], v["mean"], v["rstd"], v["dtotal"], ROWS, D, xt, yt, 0, v["dx"],
                                  v["dweight"], v["dbias"], v["workspace"], ROOM, None)


def test_forward():
    assert fwd(xt=F32, yt=BF16, y=("x", 0), residual=False) == INVALID           # rows of two lengths
    assert fwd(xt=F32, yt=BF16, y=("residual", 0)) == INVALID
    assert fwd(y=("total", 0)) == INVALID
    assert fwd(total=("x", 0), y=("x", 0)) == INVALID                            # the total and y in x's place
    assert fwd(total=("residual", 0), y=("residual", 0)) == INVALID
    for out in ("total", "y"):
        for other in ("x", "residual", "weight", "bias", "mean", "rstd"):
            assert fwd(**{out: (other, 16)}) == INVALID, (out, other)
    for out in ("mean", "rstd"):
        for other in ("x", "residual", "weight", "bias"):
            assert fwd(**{out: (other, 0)}) == INVALID, (out, other)
    assert fwd(mean=("rstd", 0)) == INVALID and fwd(mean=("y", 256)) == INVALID and fwd(rstd=("total", 256)) == INVALID


def test_backward():
    assert bwd(xt=F32, yt=BF16, dx=("dy", 0)) == INVALID                         # rows of two lengths
    for other in ("dy", "h", "dtotal", "weight", "mean", "rstd"):
        assert bwd(dx=(other, 32)) == INVALID, other
    for out in ("dweight", "dbias", "workspace"):
        for other in ("dy", "h", "dtotal", "weight", "mean", "rstd", "dx"):
            assert bwd(**{out: (other, 0)}) == INVALID, (out, other)
    assert bwd(dweight=("dbias", 0)) == INVALID and bwd(dweight=("workspace", 64)) == INVALID
    assert bwd(dbias=("workspace", 0)) == INVALID


@pytest.mark.parametrize("rows", [0])
def test_nothing_to_write_shares_nothing(rows):
    a = ctypes.c_void_p(ROOM)
    assert lib.moe_layer_norm_fwd(a, None, a, None, rows, D, 1e-6, F32, F32, None, a, a, a, None) == 0
