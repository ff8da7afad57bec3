"""Cases for the operators around the MoE FFN layer: the norm in front of it, its
forward for a few tokens, and the update of its weights; and their plain forms.

    decode  the whole layer for the few tokens of a decode step on bf16 weights:
            top-K softmax routing of the logits, FC1 -> SwiGLU * probability ->
            FC2 of the chosen experts, each token's sum and the residual stream.
            The activation between the products is stored as bf16, as
            everywhere in the layer.
    norm    layer norm (or, without the mean, RMS norm) of the residual stream,
            with the addition in front of it.
    dnorm   its backward: the stream's gradient and the two weights'.
    adamw   gradient clipping by the global norm and the AdamW step over many
            tensors, with moments in 32 bits, or in 8: the first as e4m3 codes,
            the second by its root as unsigned e4m4 codes, 32 elements to a
            scale byte, a power of two.  The tensors are pieces of flat buffers
            that begin at multiples of 32; what lies between them is zeros.

``own`` false: elementary torch operations in float32, rounded once at the end
of each operator.  ``own`` true: the library's calls.
"""

import math
import random

import torch

own = False

GROUP = 32
DEV = "cuda"
EPS_NORM = 1e-6
LR, BETA1, BETA2, EPS, DECAY = 1e-4, 0.9, 0.95, 1e-8, 0.1
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# ---------------------------------------------------------------- cases


def listed():
    return [
        # a layer of 8 small experts serving three sequences: launch latency is most of it
        dict(name="decode_small_3", kind="decode", N=3, E=8, K=2, H=512, I=1024),
        # one sequence decoding: every one of its 8 experts is read for one row
        dict(name="decode_1", kind="decode", N=1, E=128, K=8, H=2048, I=768),
        # a small decode batch: most experts in use, one or two rows each
        dict(name="decode_16", kind="decode", N=16, E=128, K=8, H=2048, I=768),
        # odd sizes, and experts with more rows than a matrix tile
        dict(name="decode_ragged_61", kind="decode", N=61, E=12, K=5, H=1088, I=448),
        # one rank's experts of a wide layer, most of them in use
        dict(name="decode_wide_8", kind="decode", N=8, E=64, K=8, H=7168, I=2048),
        # the norm of a decode step, with the addition in front of it
        dict(name="norm_token_8", kind="norm", rows=8, D=2048, x="bf16", y="bf16", centre=True, add=True),
        # a wide layer's tokens, a residual stream in float32
        dict(name="norm_8192", kind="norm", rows=8192, D=7168, x="f32", y="bf16", centre=False, add=True),
        # the backward at the benchmark's shape
        dict(name="dnorm_4096", kind="dnorm", rows=4096, D=2048, x="bf16", y="bf16", centre=True, add=True),
        # rows of an odd length, whose starts no wide load is aligned to
        dict(name="dnorm_odd_777", kind="dnorm", rows=777, D=1111, x="bf16", y="bf16", centre=True, add=False),
        # norm weights, biases and small routers: hundreds of odd little tensors
        dict(name="adamw_small_300", kind="adamw", count=300, least=1, most=70000, param="f32", grad="f32", state="f32"),
        # the experts of one rank at the benchmark's shape, gradients accumulated in float32
        dict(name="adamw_experts_f32", kind="adamw", count=2, least=16 * 2048 * 768, most=16 * 2048 * 1536, param="master",
             grad="f32", state="f32"),
        # the same with moments in 8 bits and bf16 gradients
        dict(name="adamw_experts_q8", kind="adamw", count=2, least=16 * 2048 * 768, most=16 * 2048 * 1536, param="master",
             grad="bf16", state="q8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult64(rng, lo, hi):
    return max(1, int(round(_log(rng, lo, hi) / 64))) * 64


def draw(rng):
    kind = rng.choice(["decode", "decode", "norm", "dnorm", "adamw", "adamw"])
    while True:
        if kind == "decode":
            E = _log(rng, 4, 128)
            c = dict(kind=kind, N=_log(rng, 1, 64), E=E, K=rng.randint(1, min(8, E)), H=_mult64(rng, 256, 7168),
                     I=_mult64(rng, 128, 2048))
            # at most the wide layer's weights; the plain form multiplies every token by every expert
            if E * c["H"] * c["I"] <= 64 * 7168 * 2048 and c["N"] * E * c["H"] * c["I"] <= 24 * 64 * 7168 * 2048:
                return c
        elif kind in ("norm", "dnorm"):
            x, y = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
            D = _mult64(rng, 64, 16384) if rng.random() < 0.6 else _log(rng, 33, 16384)
            c = dict(kind=kind, rows=_log(rng, 1, 32768), D=D, x=x, y=y, centre=rng.random() < 0.5, add=rng.random() < 0.5)
            if c["rows"] * D <= 8192 * 7168:
                return c
        else:
            count = _log(rng, 1, 400)
            most = _log(rng, 64, 16 * 2048 * 1536)
            c = dict(kind=kind, count=count, least=_log(rng, 1, most), most=most, param=rng.choice(["bf16", "f32", "master"]),
                     grad=rng.choice(["bf16", "f32"]), state=rng.choice(["f32", "q8"]))
            if sum(_sizes(c)) <= 16 * 2048 * 2304:
                return c


def _sizes(c):
    """The tensors' lengths: the smallest, the largest, and others between them."""
    rng = random.Random(c["count"])
    more = [_log(rng, c["least"], c["most"]) for _ in range(c["count"] - 2)]
    return ([c["most"], c["least"]] + more)[:c["count"]]


def _up(n, m):
    return -(-n // m) * m


# ---------------------------------------------------------------- moments in 8 bits, plain


def _scale(byte):
    """2^(b - 127) in float32."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _power(amax, steps, bump):
    """Scale bytes of groups with largest magnitude amax = m * 2^e, m in [0.5, 1): `steps` powers below it, one more
    where m reaches `bump` (the code past the largest would be as near)."""
    m, e = torch.frexp(amax)
    return torch.clamp(e.to(torch.int32) - 1 - steps + (m >= bump).to(torch.int32) + 127, min=1)


def _first_codes(m):
    """float32 [n] -> e4m3 codes (uint8 [n]) and scale bytes [n/32]."""
    g = m.reshape(-1, GROUP)
    byte = _power(g.abs().amax(1), 8, 464.0 / 512.0)
    return (g / _scale(byte)[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1), byte.to(torch.uint8)


def _first_values(codes, byte):
    return (codes.view(torch.float8_e4m3fn).float().reshape(-1, GROUP) * _scale(byte)[:, None]).reshape(-1)


def _root_codes(r):
    """float32 [n] of roots of second moments -> codes c (uint8 [n]) for (1 + c%16/16) * 2^(c/16 - 15) (0 for 0, and
    nothing else) and scale bytes [n/32]."""
    g = r.reshape(-1, GROUP)
    byte = _power(g.amax(1), 0, 31.5 / 32.0)
    bits = (g / _scale(byte)[:, None]).view(torch.int32)
    c = torch.clamp(((bits + 0x3FFFF + ((bits >> 19) & 1)) >> 19) - 112 * 16, min=1)
    return torch.where(g > 0, c, torch.zeros_like(c)).to(torch.uint8).reshape(-1), byte.to(torch.uint8)


def _root_values(codes, byte):
    c = codes.to(torch.int32)
    v = torch.where(c > 0, ((c << 19) + (112 << 23)).view(torch.float32), torch.zeros((), device=codes.device))
    return (v.reshape(-1, GROUP) * _scale(byte)[:, None]).reshape(-1)


# ---------------------------------------------------------------- inputs


def _prepare_adamw(c, g):
    sizes = _sizes(c)
    starts, n = [], 0
    for k in sizes:
        starts.append(n)
        n += _up(k, GROUP)
    # 1 where a tensor is, 0 in the gaps behind it
    edge = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    at = torch.tensor(starts, device=DEV)
    edge[at] += 1
    edge.index_add_(0, at + torch.tensor(sizes, device=DEV), torch.full((len(sizes),), -1, dtype=torch.int32, device=DEV))
    inside = torch.cumsum(edge[:n], 0, dtype=torch.int32).to(torch.float32)
    rand = lambda: torch.randn(n, generator=g, device=DEV)  # noqa: E731
    # elements of different spread, as the gradients of rarely used rows are
    spread = torch.exp(rand()).mul_(1e-4).mul_(inside)
    grad = (rand() * spread).to(TYPES[c["grad"]])
    m = rand().mul_(0.3).mul_(spread)
    r = (0.5 + torch.rand(n, generator=g, device=DEV)).mul_(spread)
    master = rand().mul_(0.02).mul_(inside)
    s = dict(c, sizes=sizes, starts=starts, grad=grad, lr=torch.full((1,), LR, device=DEV),
             step=torch.full((1,), 100, dtype=torch.int32, device=DEV),
             # half the norm that the gradients come to: the step clips
             max_norm=0.5 * math.sqrt(sum(sizes)) * 1e-4 * math.e)
    s["param"] = master if c["param"] == "f32" else master.to(torch.bfloat16)
    s["master"] = master if c["param"] == "master" else None
    if c["state"] == "q8":
        s["m"], s["m_scales"] = _first_codes(m)
        s["v"], s["v_scales"] = _root_codes(r)
    else:
        s["m"], s["v"] = m, r * r
    s["kind"], s["param_kind"] = "adamw", c["param"]
    return s


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    bf16 = torch.bfloat16
    if c["kind"] == "decode":
        N, E, K, H, I = (c[k] for k in ("N", "E", "K", "H", "I"))
        rand = lambda *shape: torch.randn(shape, generator=g, device=DEV)  # noqa: E731
        return dict(c, logits=rand(N, E), x=rand(N, H).to(bf16), residual=rand(N, H).to(bf16),
                    w1=torch.empty((E, 2 * I, H), dtype=bf16, device=DEV).normal_(0, 0.02, generator=g),
                    w2=torch.empty((E, H, I), dtype=bf16, device=DEV).normal_(0, 0.02, generator=g))
    if c["kind"] == "adamw":
        return _prepare_adamw(c, g)
    rows, D, tx, ty = c["rows"], c["D"], TYPES[c["x"]], TYPES[c["y"]]
    rand = lambda *shape: torch.randn(shape, generator=g, device=DEV)  # noqa: E731
    # a residual stream: channels of different spread, some of them away from zero
    spread, shift = torch.exp(0.5 * rand(D)), 0.3 * rand(D)
    s = dict(c, x=(rand(rows, D) * spread + shift).to(tx), weight=1.0 + 0.1 * rand(D),
             bias=0.1 * rand(D) if c["centre"] else None, types=(tx, ty))
    if c["kind"] == "norm":
        return dict(s, residual=rand(rows, D).to(tx) if c["add"] else None,
                    total=torch.empty((rows, D), dtype=tx, device=DEV) if c["add"] else None,
                    y=torch.empty((rows, D), dtype=ty, device=DEV),
                    mean=torch.empty(rows, device=DEV) if c["centre"] else None, rstd=torch.empty(rows, device=DEV))
    h = s["x"].double()
    mean = h.mean(1) if c["centre"] else torch.zeros(rows, dtype=torch.float64, device=DEV)
    rstd = ((h - mean[:, None]).square().mean(1) + EPS_NORM).rsqrt().float()
    return dict(s, dy=rand(rows, D).to(ty), mean=mean.float() if c["centre"] else None, rstd=rstd,
                dtotal=rand(rows, D).to(tx) if c["add"] else None,
                dx=torch.empty((rows, D), dtype=tx, device=DEV), dweight=torch.empty(D, device=DEV),
                dbias=torch.empty(D, device=DEV) if c["centre"] else None)


# ---------------------------------------------------------------- one pass, plain


def _plain_decode(s):
    N, K, E, H, I = s["N"], s["K"], s["E"], s["H"], s["I"]
    top, ids = torch.sort(s["logits"], dim=1, descending=True, stable=True)
    top, ids = top[:, :K], ids[:, :K]
    e = torch.exp((top - top[:, :1]).double())
    probs = (e / e.sum(1, keepdim=True)).float()
    flat = ids.reshape(-1)
    tok = torch.arange(N, device=flat.device).repeat_interleave(K)
    x = s["x"].float()
    if N * K <= E:      # few routes: each reads its own expert
        h = torch.bmm(s["w1"][flat].float(), x[tok][:, :, None])[:, :, 0]
    else:               # every expert for every token, then the routes' rows
        h = (s["w1"].float().reshape(E * 2 * I, H) @ x.t()).reshape(E, 2 * I, N)[flat, :, tok]
    gate = h[:, :I]
    act = (gate / (1.0 + torch.exp(-gate)) * h[:, I:] * probs.reshape(-1, 1)).to(torch.bfloat16).float()
    if N * K <= E:
        r = torch.bmm(s["w2"][flat].float(), act[:, :, None])[:, :, 0]
    else:
        a = torch.zeros((E, I, N), device=x.device)
        a[flat, :, tok] = act
        r = torch.bmm(s["w2"].float(), a)[flat, :, tok]
    y = (r.reshape(N, K, H).sum(1) + s["residual"].float()).to(torch.bfloat16)
    return {"ids": ids.to(torch.int32), "probs": probs, "y": y}


def _plain_norm(s):
    tx, ty = s["types"]
    out = {}
    h = s["x"].float()
    if s["add"]:
        out["total"] = (h + s["residual"].float()).to(tx)
        h = out["total"].float()
    if s["centre"]:
        out["mean"] = h.mean(1)
        h = h - out["mean"][:, None]
    out["rstd"] = torch.rsqrt(h.square().mean(1) + EPS_NORM)
    y = h * out["rstd"][:, None] * s["weight"]
    out["y"] = (y + s["bias"] if s["centre"] else y).to(ty)
    return out


def _plain_dnorm(s):
    tx, _ = s["types"]
    h, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    if s["centre"]:
        h = h - s["mean"][:, None]
    xhat = h * rstd
    g = dy * s["weight"]
    d = g - xhat * (g * xhat).mean(1, keepdim=True)
    if s["centre"]:
        d = d - g.mean(1, keepdim=True)
    d = d * rstd
    if s["add"]:
        d = d + s["dtotal"].float()
    out = {"dx": d.to(tx), "dweight": (dy * xhat).sum(0)}
    if s["centre"]:
        out["dbias"] = dy.sum(0)
    return out


def _plain_adamw(s):
    g = s["grad"].float()
    norm = torch.sqrt(g.double().square().sum()).float()
    g = g * torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm))
    t = s["step"].add_(1).double()
    lr = s["lr"]
    bc1, root_bc2 = (1 - BETA1 ** t).float(), torch.sqrt(1 - BETA2 ** t).float()
    q8 = s["state"] == "q8"
    m = _first_values(s["m"], s["m_scales"]) if q8 else s["m"]
    v = _root_values(s["v"], s["v_scales"]).square() if q8 else s["v"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g.square() * (1 - BETA2)
    root = torch.sqrt(v)
    p = (s["master"] if s["param_kind"] == "master" else s["param"]).float()
    p = p * (1 - lr * DECAY) - lr / bc1 * (m / (root / root_bc2 + EPS))
    s["param"].copy_(p)
    if s["param_kind"] == "master":
        s["master"].copy_(p)
    out = {"norm": norm.reshape(1), "param": s["param"], "master": s["master"], "step": s["step"]}
    if q8:
        (mc, mb), (vc, vb) = _first_codes(m), _root_codes(root)
        s["m"].copy_(mc), s["m_scales"].copy_(mb), s["v"].copy_(vc), s["v_scales"].copy_(vb)
        return dict(out, m=_first_values(mc, mb).to(torch.bfloat16), root=_root_values(vc, vb).to(torch.bfloat16))
    s["m"].copy_(m), s["v"].copy_(v)
    return dict(out, m=s["m"], v=s["v"])


# ---------------------------------------------------------------- one pass, the library's


def _kept(s, key, make):
    """Buffers and handles that a program makes once and keeps."""
    if key not in s:
        s[key] = make()
    return s[key]


def _optimizer(moe, s):
    def pieces(flat, per=1):
        return [flat[a // per:a // per + -(-n // per)] for a, n in zip(s["starts"], s["sizes"])]

    q8 = s["state"] == "q8"
    moments = dict(m=pieces(s["m"]), v=pieces(s["v"]))
    if q8:
        moments.update(m_scales=pieces(s["m_scales"], GROUP), v_scales=pieces(s["v_scales"], GROUP))
    return moe.MoEAdamW(pieces(s["param"]), pieces(s["grad"]), lr=s["lr"], betas=(BETA1, BETA2), eps=EPS,
                        weight_decay=DECAY, max_norm=s["max_norm"], state=s["state"],
                        masters=pieces(s["master"]) if s["param_kind"] == "master" else None, moments=moments,
                        step=s["step"])


def _own(s):
    import mixture_experts_expert_amd as moe
    if s["kind"] == "decode":
        buf = _kept(s, "buf", lambda: moe.DecodeBuffers(s["N"], s["H"], s["I"], s["E"], s["K"]))
        y = moe.forward_decode(buf, s["logits"], s["x"], s["w1"], s["w2"], residual=s["residual"])
        return {"ids": buf.topk_ids, "probs": buf.topk_probs, "y": y}
    if s["kind"] == "norm":
        moe.moe_layer_norm_fwd(s["x"], s["weight"], s["bias"], EPS_NORM, s["y"], s["mean"], s["rstd"],
                               residual=s["residual"], total=s["total"])
        return {k: s[k] for k in ("total", "mean", "rstd", "y") if s[k] is not None}
    if s["kind"] == "dnorm":
        ws = _kept(s, "ws", lambda: moe.layer_norm_workspace(s["rows"], s["D"]))
        moe.moe_layer_norm_bwd(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"],
                               ws, dtotal=s["dtotal"])
        return {k: s[k] for k in ("dx", "dweight", "dbias") if s[k] is not None}
    opt = _kept(s, "opt", lambda: _optimizer(moe, s))
    opt.step_()
    out = {"norm": opt.norm, "param": s["param"], "master": s["master"], "step": s["step"]}
    if s["state"] != "q8":
        return dict(out, m=s["m"], v=s["v"])
    m, root = _kept(s, "values", lambda: (torch.empty(s["m"].shape, dtype=torch.bfloat16, device=DEV),
                                          torch.empty(s["v"].shape, dtype=torch.bfloat16, device=DEV)))
    moe.moe_moment_values(s["m"], s["m_scales"], s["v"], s["v_scales"], m, root)
    return dict(out, m=m, root=root)


def run(state):
    if own:
        return _own(state)
    if state["kind"] == "decode":
        return _plain_decode(state)
    if state["kind"] == "norm":
        return _plain_norm(state)
    if state["kind"] == "dnorm":
        return _plain_dnorm(state)
    return _plain_adamw(state)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    c = case
    if c["kind"] == "decode":
        N, E, K, H, I = (c[k] for k in ("N", "E", "K", "H", "I"))
        used = E * (1.0 - (1.0 - K / E) ** N)       # experts that some token picks, on average
        return {"bytes": used * 6 * H * I + 4 * N * E + 6 * N * H + 8 * N * K, "flops": 6.0 * N * K * H * I}
    if c["kind"] in ("norm", "dnorm"):
        n, bx, by = c["rows"] * c["D"], 2 if c["x"] == "bf16" else 4, 2 if c["y"] == "bf16" else 4
        both = 2 if c["centre"] else 1
        if c["kind"] == "norm":     # x (and what is added) in, y (and the sum) out
            return {"bytes": n * (bx * (3 if c["add"] else 1) + by) + 4 * both * (c["rows"] + c["D"]), "flops": 8.0 * n}
        return {"bytes": n * (by + bx * (3 if c["add"] else 2)) + 4 * both * (c["rows"] + c["D"]) + 4 * c["D"],
                "flops": 14.0 * n}
    n = sum(_sizes(c))
    grad = 2 if c["grad"] == "bf16" else 4
    param = {"bf16": 4, "f32": 8, "master": 10}[c["param"]]
    # both moments in and out; in 8 bits, the values they stand for as well
    moments = 16 if c["state"] == "f32" else 4 * (1 + 1 / GROUP) + 4
    return {"bytes": n * (grad + param + moments), "flops": 20.0 * n}


# ---------------------------------------------------------------- the definitions in 64 bits


def _two_to(k):
    """2^k in float64 for whole k in [-1022, 1023], from the format's own exponent field."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _floor_log2(a):
    """floor(log2 a) of positive float64 numbers, from their own exponent field; 0 for 0."""
    return torch.where(a > 0, ((a.view(torch.int64) >> 52) & 2047) - 1023, torch.zeros_like(a, dtype=torch.int64))


def _exact_moment(v, top, past, mantissa, least):
    """Magnitudes of float64 groups [n/32, 32] to the nearest code: the scale is the power of two with which the largest
    comes to at most 2^top and `past`; codes have `mantissa` bits, those below 2^least keep the step there."""
    amax = v.abs().amax(1)
    k = _floor_log2(amax) - top
    k = torch.clamp(k + (amax / _two_to(k) >= past).to(torch.int64), min=-126)
    a = v / _two_to(k)[:, None]
    step = _two_to(torch.clamp(_floor_log2(a.abs()), min=least) - mantissa)
    return torch.round(a / step) * step, _two_to(k)[:, None]


def _exact_adamw(case, seed):
    s = prepare(case, seed)
    g = s["grad"].double()
    norm = torch.sqrt((g * g).sum())
    g = g * min(1.0, s["max_norm"] / float(norm))
    t = 101
    q8 = s["state"] == "q8"
    m = _first_values(s["m"], s["m_scales"]).double() if q8 else s["m"].double()
    v = _root_values(s["v"], s["v_scales"]).double().square() if q8 else s["v"].double()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    lr = float(s["lr"])
    p = (s["master"] if case["param"] == "master" else s["param"]).double()
    p = p - lr * DECAY * p - lr * (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
    out = {"norm": norm.reshape(1), "param": p, "master": p if case["param"] == "master" else None, "step": None}
    if not q8:
        return dict(out, m=m, v=v)
    a, scale = _exact_moment(m.reshape(-1, GROUP), 8, 464.0, 3, -6)
    root = torch.sqrt(v).reshape(-1, GROUP)
    b, rscale = _exact_moment(root, 0, 63 / 32, 4, -15)
    b = torch.where(root > 0, torch.clamp(b, min=17 / 16 * 2.0 ** -15), b)
    return dict(out, m=(a * scale).reshape(-1), root=(b * rscale).reshape(-1))


def exact(case, seed):
    if case["kind"] == "adamw":
        return _exact_adamw(case, seed)
    s = prepare(case, seed)
    if s["kind"] == "decode":
        N, K, H, I = s["N"], s["K"], s["H"], s["I"]
        # larger logits first, among equals the lower expert
        order = sorted(range(s["E"]), key=lambda e: e)
        rows = s["logits"].tolist()
        ids = torch.tensor([sorted(order, key=lambda e, r=r: (-r[e], e))[:K] for r in rows], device=DEV)
        top = torch.gather(s["logits"].double(), 1, ids)
        probs = torch.softmax(top, 1)
        p32 = probs.float().double()
        x = s["x"].double()
        y = s["residual"].double()
        for e in sorted(set(ids.reshape(-1).tolist())):
            t, k = torch.where(ids == e)
            h = x[t] @ s["w1"][e].double().t()
            a = h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:] * p32[t, k][:, None]
            y.index_add_(0, t, a.to(torch.bfloat16).double() @ s["w2"][e].double().t())
        return {"ids": None, "probs": probs, "y": y}
    h = s["x"].double()
    w = s["weight"].double()
    if s["kind"] == "norm":
        out = {}
        if s["add"]:
            h = h + s["residual"].double()
            out["total"] = h
            h = h.to(s["types"][0]).double()        # what is stored is what is normalised
        mean = h.mean(1, keepdim=True) if s["centre"] else 0.0
        if s["centre"]:
            out["mean"] = mean[:, 0]
        var = (h - mean).square().mean(1, keepdim=True)
        out["rstd"] = 1.0 / torch.sqrt(var[:, 0] + EPS_NORM)
        y = (h - mean) / torch.sqrt(var + EPS_NORM) * w
        out["y"] = y + s["bias"].double() if s["centre"] else y
        return out
    D, dy, rstd = s["D"], s["dy"].double(), s["rstd"].double()[:, None]
    xhat = (h - (s["mean"].double()[:, None] if s["centre"] else 0.0)) * rstd
    g = dy * w
    d = D * g - xhat * (g * xhat).sum(1, keepdim=True)
    if s["centre"]:
        d = d - g.sum(1, keepdim=True)
    d = d * rstd / D
    out = {"dx": d + s["dtotal"].double() if s["add"] else d, "dweight": (dy * xhat).sum(0)}
    if s["centre"]:
        out["dbias"] = dy.sum(0)
    return out
