"""The entry points of include/moe_block.h: every declared symbol is exported,
and what the C calls and their Python wrappers refuse.  No device work."""

import ctypes
import re

import pytest
import torch

import mixture_experts_expert_amd as moe
from mixture_experts_expert_amd import _native as nat
from test_abi import ALIGNED as A, INVALID, MIS, MISALIGNED, NUL, OK, UNSUPPORTED

lib = moe.lib
BIG = ctypes.c_size_t(1 << 40)


def test_every_declared_symbol_is_exported_with_its_arguments():
    names = moe.header_functions(moe.BLOCK_HEADER_PATH)
    assert set(names) == {"moe_ffn_decode_max_tokens", "moe_ffn_decode_workspace_bytes", "moe_ffn_decode",
                          "moe_layer_norm_fwd", "moe_layer_norm_bwd_workspace_bytes", "moe_layer_norm_bwd",
                          "moe_adamw_plan_bytes", "moe_adamw_plan", "moe_grad_norm", "moe_adamw_step",
                          "moe_moment_values", "moe_moment_codes"}
    text = re.sub(r"/\*.*?\*/", "", open(moe.BLOCK_HEADER_PATH).read(), flags=re.S)
    for n in names:
        assert hasattr(lib, n) and n in nat._SIGNATURES, n
        args = re.search(r"\b%s\s*\((.*?)\)\s*;" % n, text, flags=re.S).group(1)
        declared = 0 if args.strip() == "void" else len(args.split(","))
        assert declared == len(nat._SIGNATURES[n][1]), n


def test_decode_validation():
    f = lib.moe_ffn_decode
    most = moe.moe_ffn_decode_max_tokens()
    assert most == 64

    def call(N=4, H=64, I=64, E=4, K=2, size=BIG, at=None, ptr=NUL, n_live=NUL, residual=NUL, y=A):
        p = [A, A, A, A, residual, n_live]
        o = [A, A, A]
        if at is not None:
            (p if at < 4 else o)[at if at < 4 else at - 4] = ptr
        return f(*p, N, H, I, E, K, *o, size, y, NUL)
    assert call(N=-1) == INVALID and call(E=0) == INVALID and call(K=0) == INVALID and call(K=5) == INVALID
    assert call(N=most + 1) == UNSUPPORTED and call(H=96) == UNSUPPORTED and call(I=16448) == UNSUPPORTED
    assert call(E=2048) == UNSUPPORTED and call(E=64, K=33) == UNSUPPORTED and call(H=0) == INVALID
    for i in range(7):
        assert call(at=i) == INVALID, i
        assert call(at=i, ptr=MIS) == MISALIGNED, i
    assert call(y=NUL) == INVALID and call(y=MIS) == MISALIGNED and call(residual=MIS) == MISALIGNED
    assert call(n_live=ctypes.c_void_p(4098)) == MISALIGNED
    assert call(size=ctypes.c_size_t(4 * 2 * 64 * 2 + 63)) == INVALID
    assert f(*[NUL] * 6, 0, 64, 64, 4, 2, NUL, NUL, NUL, 0, NUL, NUL) == OK
    g = lib.moe_ffn_decode_workspace_bytes
    assert g(4, 64, 64, 4, 2) == 4 * 2 * 64 * 2 + 64 and g(65, 64, 64, 4, 2) == 0 and g(4, 65, 64, 4, 2) == 0
    with pytest.raises(moe.MoEError):
        moe.moe_ffn_decode_workspace_bytes(4, 64, 64, 2, 3)


def test_norm_validation():
    f, g = lib.moe_layer_norm_fwd, lib.moe_layer_norm_bwd
    ok = dict(x=A, r=NUL, w=A, b=NUL, rows=4, D=64, eps=1e-6, xt=0, yt=0, t=NUL, y=ctypes.c_void_p(8192), m=NUL, s=A)

    def fwd(**kw):
        v = {**ok, **kw}
        return f(v["x"], v["r"], v["w"], v["b"], v["rows"], v["D"], v["eps"], v["xt"], v["yt"], v["t"], v["y"], v["m"],
                 v["s"], NUL)
    assert fwd(rows=-1) == INVALID and fwd(D=0) == INVALID and fwd(D=16385) == UNSUPPORTED
    assert fwd(xt=2) == INVALID and fwd(yt=-1) == INVALID and fwd(xt=0, yt=1) == UNSUPPORTED
    assert fwd(rows=1 << 40, D=2) == UNSUPPORTED and fwd(eps=-1.0) == INVALID and fwd(eps=float("nan")) == INVALID
    assert fwd(r=A) == INVALID and fwd(t=A) == INVALID            # a residual without a total, and the reverse
    assert fwd(r=A, t=ctypes.c_void_p(8192)) == INVALID           # the total in y's place
    for k in ("x", "w", "y", "s"):
        assert fwd(**{k: NUL}) == INVALID, k
        assert fwd(**{k: MIS}) == MISALIGNED, k
    assert fwd(b=MIS) == MISALIGNED and fwd(m=MIS) == MISALIGNED and fwd(r=MIS, t=A) == MISALIGNED
    assert fwd(rows=0, x=NUL, y=NUL, s=NUL) == OK

    def bwd(dy=A, h=A, w=A, m=NUL, s=A, t=NUL, rows=4, D=64, xt=0, yt=0, acc=0, dx=A, dw=A, db=NUL, ws=A, size=BIG):
        return g(dy, h, w, m, s, t, rows, D, xt, yt, acc, dx, dw, db, ws, size, NUL)
    assert bwd(rows=-1) == INVALID and bwd(D=16385) == UNSUPPORTED and bwd(acc=2) == INVALID and bwd(yt=1) == UNSUPPORTED
    for k in ("dy", "h", "w", "s", "dx", "dw", "ws"):
        assert bwd(**{k: NUL}) == INVALID, k
        assert bwd(**{k: MIS}) == MISALIGNED, k
    for k in ("m", "t", "db"):
        assert bwd(**{k: MIS}) == MISALIGNED, k
    need = lib.moe_layer_norm_bwd_workspace_bytes(4, 64)
    assert need >= 2 * 64 * 4 and bwd(size=ctypes.c_size_t(need - 1)) == INVALID
    assert lib.moe_layer_norm_bwd_workspace_bytes(4, 0) == 0 and lib.moe_layer_norm_bwd_workspace_bytes(-1, 4) == 0


def table(n=8, **kw):
    t = (nat.AdamWTensor * 1)()
    a = A.value
    v = dict(param=a, grad=a, m=a, v=a, n=n, weight_decay=0.1, param_type=1, grad_type=1)
    v.update(kw)
    for k, x in v.items():
        setattr(t[0], k, x)
    return t


def test_adamw_validation():
    f, g, w, h = lib.moe_adamw_step, lib.moe_grad_norm, lib.moe_adamw_plan_bytes, lib.moe_adamw_plan

    def plan(t, count=1, p=A, size=BIG):
        return h(t, count, p, size, NUL)

    def step(t, count=1, p=A, size=BIG, lr=A, b1=0.9, b2=0.95, eps=1e-8, norm=NUL, most=0.0, at=A):
        return f(t, count, p, size, lr, b1, b2, eps, norm, most, at, NUL)
    for kw, want in ((dict(n=-1), INVALID), (dict(n=(1 << 34) + 1), UNSUPPORTED), (dict(param_type=2), INVALID),
                     (dict(grad_type=-1), INVALID), (dict(reserved=1), INVALID), (dict(param=0), INVALID),
                     (dict(grad=0), INVALID), (dict(m=0), INVALID), (dict(v=0), INVALID), (dict(param=4104), MISALIGNED),
                     (dict(grad=4104), MISALIGNED), (dict(m=4104), MISALIGNED), (dict(v=4104), MISALIGNED),
                     (dict(master=4104), MISALIGNED), (dict(m_scales=4096), INVALID), (dict(v_scales=4096), INVALID),
                     (dict(weight_decay=float("nan")), INVALID)):
        assert plan(table(**kw)) == want, kw
    t = table()
    two = (nat.AdamWTensor * 2)(t[0], table(m_scales=4097, v_scales=4099)[0])
    assert plan(two, count=2) == INVALID                          # moments of two kinds
    for call in (plan, step):
        assert call(None, count=1) == INVALID and call(t, count=-1) == INVALID
        assert call(t, p=NUL) == INVALID and call(t, p=MIS) == MISALIGNED
        assert call(t, size=ctypes.c_size_t(w(t, 1) - 1)) == INVALID
    assert step(t, b1=1.0) == INVALID and step(t, b2=-0.1) == INVALID and step(t, eps=-1.0) == INVALID
    assert step(t, eps=float("inf")) == INVALID and step(t, b1=float("nan")) == INVALID
    assert step(t, norm=A, most=0.0) == INVALID and step(t, norm=A, most=float("nan")) == INVALID
    assert step(t, lr=NUL) == INVALID and step(t, at=NUL) == INVALID
    assert step(t, lr=ctypes.c_void_p(4098)) == MISALIGNED
    assert w(t, 1) > 0 and w(t, -1) == 0 and w(table(n=-1), 1) == 0 and w(two, 2) == 0
    many = (nat.AdamWTensor * 65)(*[table(n=1 << 34)[0]] * 65)
    assert w(many, 64) > 0 and w(many, 65) == 0                   # 2^40 elements in all
    assert g(t, 1, NUL, BIG, A, NUL) == INVALID and g(t, 1, A, BIG, NUL, NUL) == INVALID
    assert g(t, 1, MIS, BIG, A, NUL) == MISALIGNED and g(t, 1, A, ctypes.c_size_t(4), A, NUL) == INVALID
    assert g(t, 1, A, BIG, ctypes.c_void_p(4098), NUL) == MISALIGNED


def test_adamw_refuses_tensors_that_share_memory():
    """Buffers of 64 elements 512 bytes apart, but for one of a pair that begins inside another."""
    def apart():
        return [dict(n=64, param=base, master=base + 512, grad=base + 1024, m=base + 1536, v=base + 2048, m_scales=0,
                     v_scales=0, param_type=0, grad_type=1) for base in (1 << 20, 1 << 21)]
    for a, b in ((("param", 0), ("param", 1)), (("param", 0), ("master", 0)), (("m", 0), ("v", 0)), (("m", 1), ("m", 0)),
                 (("grad", 0), ("param", 1)), (("param", 1), ("grad", 0)), (("grad", 1), ("v", 1))):
        t = apart()
        t[a[1]][a[0]] = t[b[1]][b[0]] + 16                        # 16 bytes in, so that both overlap
        two = (nat.AdamWTensor * 2)(*[table(**x)[0] for x in t])
        assert lib.moe_adamw_plan(two, 2, A, BIG, NUL) == INVALID, (a, b)


def test_moment_conversion_validation():
    for f, n_in in ((lib.moe_moment_values, 4), (lib.moe_moment_codes, 2)):
        n_out = 6 - n_in
        for n, want in ((-1, INVALID), ((1 << 34) + 1, UNSUPPORTED), (0, OK)):
            assert f(*[A] * n_in, n, *[A] * n_out, NUL) == want
        for i in range(6):
            p = [A] * 6
            p[i] = NUL
            assert f(*p[:n_in], 8, *p[n_in:], NUL) == INVALID, i
    assert ctypes.sizeof(nat.AdamWTensor) == 80


def test_wrappers_refuse_host_tensors():
    z = torch.zeros
    b = torch.bfloat16
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_layer_norm_fwd(z(4, 64), z(64), None, 1e-6, z(4, 64), None, z(4))
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_ffn_decode(z(4, 4), z(4, 64, dtype=b), z(4, 128, 64, dtype=b), z(4, 64, 64, dtype=b),
                           z(4, 2, dtype=torch.int32), z(4, 2), z(64, dtype=torch.uint8), z(4, 64, dtype=b))
    with pytest.raises(ValueError, match="device tensor"):
        moe.MoEAdamW([z(8)], [z(8)])
    with pytest.raises(TypeError, match="torch.Tensor"):
        moe.MoEAdamW([[1.0]], [z(8)])
