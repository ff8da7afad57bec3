"""Cases for the block-scaled operators of the MoE FFN layer, and their plain forms.

Four operators.  Groups of 32 consecutive columns share one byte of scale, a
power of two 2^(b - 127):

    w4    the expert FFN of the dropless route list on 4-bit weights (e2m1
          codes, two a byte, low half first), for the few tokens of a decode
          step: FC1 -> SwiGLU * probability -> FC2 -> each token's sum.  The
          activation between the two products is stored as bf16, as
          everywhere in the layer.
    save  the training forward's FC1 + SwiGLU, keeping its pre-activation
          [gate | up] as 8-bit codes; the kept codes come back as the values
          they stand for.
    bwd   the SwiGLU recompute and backward from those codes.
    pack  a bf16 tensor to 8-bit codes and back.

``own`` false: elementary torch operations in float32, rounded once at the
end of each operator.  ``own`` true: the library's calls.
"""

import math
from fractions import Fraction

import torch

own = False

GROUP = 32
DEV = "cuda"

# ---------------------------------------------------------------- cases


def listed():
    return [
        # a layer of 8 small experts serving three sequences: launch latency is most of it
        dict(name="w4_small_3", kind="w4", N=3, E=8, K=2, H=512, I=1024),
        # one sequence decoding: every one of its 8 experts is read for one row
        dict(name="w4_decode_1", kind="w4", N=1, E=128, K=8, H=2048, I=768),
        # a small decode batch: most experts in use, one or two rows each
        dict(name="w4_decode_16", kind="w4", N=16, E=128, K=8, H=2048, I=768),
        # a full decode batch: every expert in use, about 8 rows each
        dict(name="w4_decode_128", kind="w4", N=128, E=128, K=8, H=2048, I=768),
        # odd sizes: contractions that end inside a 128-wide step, experts with over 16 rows
        dict(name="w4_ragged_93", kind="w4", N=93, E=24, K=5, H=1088, I=448),
        # one rank's experts of a wide layer: 1.4 GB of 4-bit weights a step
        dict(name="w4_wide_24", kind="w4", N=24, E=64, K=8, H=7168, I=2048),
        # the training forward at the benchmark's shape
        dict(name="save_4096", kind="save", N=4096, E=128, K=8, F=1.0, H=2048, I=768),
        # a small layer with a ragged capacity, pads and dropped routes
        dict(name="save_odd_777", kind="save", N=777, E=12, K=3, F=1.1, H=960, I=320),
        # the backward over the benchmark's slots, and over few odd-sized rows
        dict(name="bwd_32768", kind="bwd", R=32768, I=768),
        dict(name="bwd_odd_1184", kind="bwd", R=1184, I=1088),
        # a layer's input kept in 8 bits, and a short odd one
        dict(name="pack_8192", kind="pack", rows=8192, D=7168),
        dict(name="pack_odd_333", kind="pack", rows=333, D=1088),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult64(rng, lo, hi):
    return max(1, int(round(_log(rng, lo, hi) / 64))) * 64


def draw(rng):
    kind = rng.choice(["w4", "w4", "save", "bwd", "pack"])
    while True:
        if kind == "w4":
            E = _log(rng, 4, 128)
            c = dict(kind=kind, N=_log(rng, 1, 256), E=E, K=rng.randint(1, min(8, E)),
                     H=_mult64(rng, 256, 7168), I=_mult64(rng, 128, 2048))
            # at most the widest layer's weights; the plain form multiplies every token by every expert
            if E * c["H"] * c["I"] <= 64 * 7168 * 2048 and c["N"] * E * c["H"] * c["I"] <= 24 * 64 * 7168 * 2048:
                return c
        elif kind == "save":
            E = _log(rng, 4, 128)
            c = dict(kind=kind, N=_log(rng, 64, 8192), E=E, K=rng.randint(1, min(8, E)),
                     F=rng.choice([1.0, 1.0, 1.1, 1.25, 1.5]), H=_mult64(rng, 256, 4096), I=_mult64(rng, 128, 2048))
            slots = c["N"] * c["K"] * c["F"] + 32 * E
            if slots * c["H"] * c["I"] <= 32768 * 2048 * 768 and E * c["H"] * c["I"] <= 128 * 2048 * 768:
                return c
        elif kind == "bwd":
            c = dict(kind=kind, R=_log(rng, 32, 65536), I=_mult64(rng, 64, 4096))
            if c["R"] * c["I"] <= 32768 * 768:
                return c
        else:
            c = dict(kind=kind, rows=_log(rng, 16, 32768), D=_mult64(rng, 64, 14336))
            if c["rows"] * c["D"] <= 8192 * 7168:
                return c


def _capacity(c):
    return math.ceil(Fraction(c["N"] * c["K"]) * Fraction(c["F"]) / c["E"])


def _padded(n):
    return -(-n // 32) * 32


# ---------------------------------------------------------------- storage formats, plain


def _scale(byte):
    """2^(b - 127) in float32."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _power(amax, steps, bump):
    """Scale bytes of groups with largest magnitude amax = m * 2^e, m in [0.5, 1):
    `steps` powers below it, one more where m reaches `bump` (the code past the
    largest would be nearer)."""
    m, e = torch.frexp(amax)
    return torch.clamp(e.to(torch.int32) - 1 - steps + (m >= bump).to(torch.int32) + 127, min=1)


def _q8_codes(v):
    """float32 [..., D] -> whole numbers in [-127, 127] (as float32), scale bytes."""
    g = v.reshape(*v.shape[:-1], -1, GROUP)
    byte = _power(g.abs().amax(-1), 6, 255.0 / 256.0)
    return torch.round(g / _scale(byte)[..., None]).reshape(v.shape), byte


def _q8_values(codes, byte):
    g = codes.to(torch.float32).reshape(*codes.shape[:-1], -1, GROUP)
    return (g * _scale(byte)[..., None]).reshape(codes.shape)


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _w4_codes(v):
    """float32 [..., K] -> codes uint8 [..., K/2], scale bytes uint8 [..., K/32]."""
    g = v.reshape(*v.shape[:-1], -1, GROUP)
    byte = _power(g.abs().amax(-1), 2, 7.0 / 8.0)
    a = (g / _scale(byte)[..., None]).reshape(v.shape)
    m = a.abs()
    # nearest; the middle between two codes goes to the one of even mantissa
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = code.to(torch.uint8) | ((a < 0).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte.to(torch.uint8)


def _w4_values(codes, byte):
    """codes uint8 [..., K/2], scale bytes [..., K/32] -> float32 [..., K]."""
    one = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    pair = torch.stack([one.repeat(16), one.repeat_interleave(16)], 1)          # [256, 2]
    v = pair.index_select(0, codes.reshape(-1).to(torch.int32))
    v = v.reshape(*byte.shape, GROUP) * _scale(byte)[..., None]
    return v.reshape(*codes.shape[:-1], codes.shape[-1] * 2)


# ---------------------------------------------------------------- inputs


def _routing(N, E, K, g):
    logits = torch.randn((N, E), generator=g, device=DEV)
    top, ids = torch.topk(logits, K, dim=1)
    return ids.to(torch.int32), torch.softmax(top, 1)


def _w4_random(E, rows, K, std, g):
    """Quantized N(0, std) weights, some experts at a time."""
    codes = torch.empty((E, rows, K // 2), dtype=torch.uint8, device=DEV)
    byte = torch.empty((E, rows, K // GROUP), dtype=torch.uint8, device=DEV)
    per = max(1, (1 << 26) // (rows * K))
    for e in range(0, E, per):
        n = min(per, E - e)
        w = torch.randn((n, rows, K), generator=g, device=DEV).mul_(std).to(torch.bfloat16)
        codes[e:e + n], byte[e:e + n] = _w4_codes(w.float())
    return codes, byte


def _dropless_list(ids, probs, E):
    """The dropless route list: each expert's routes in token order, segments padded to 32 slots."""
    N, K = ids.shape
    R = _padded(N * min(K, E) + E * 31)
    flat = ids.reshape(-1).to(torch.int64)
    counts = torch.bincount(flat, minlength=E)
    seg = (counts + 31) // 32 * 32
    start = torch.cumsum(seg, 0) - seg
    order = torch.argsort(flat, stable=True)
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(N * K, device=DEV) - (torch.cumsum(counts, 0) - counts)[flat[order]]
    slot = start[flat] + rank
    ssi = torch.full((R,), N, dtype=torch.int32, device=DEV)
    ssi[slot] = torch.arange(N * K, device=DEV, dtype=torch.int32) // K
    sp = torch.zeros(R, device=DEV)
    sp[slot] = probs.reshape(-1)
    blk = torch.arange(R // 32, device=DEV) * 32
    owner = (torch.searchsorted(start + seg, blk, right=True)).to(torch.int32)
    owner[blk >= seg.sum()] = -1
    return dict(sorted_slot_ids=ssi, slot_probs=sp, expert_ids=owner, block_start=(start // 32).to(torch.int32),
                route_counts=counts.to(torch.int32), token_routes=slot.to(torch.int32).reshape(N, K)), R


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    bf16 = torch.bfloat16
    if c["kind"] == "w4":
        N, E, K, H, I = (c[k] for k in ("N", "E", "K", "H", "I"))
        ids, probs = _routing(N, E, K, g)
        lst, R = _dropless_list(ids, probs, E)
        w1c, w1s = _w4_random(E, 2 * I, H, 0.02, g)
        w2c, w2s = _w4_random(E, H, I, 0.02, g)
        x = torch.randn((N, H), generator=g, device=DEV).to(bf16)
        return dict(c, x=x, ids=ids, probs=probs, w1c=w1c, w1s=w1s, w2c=w2c, w2s=w2s, **lst,
                    act=torch.empty((R, I), dtype=bf16, device=DEV), route_out=torch.empty((R, H), device=DEV),
                    y=torch.empty((N, H), dtype=bf16, device=DEV))
    if c["kind"] == "save":
        N, E, K, H, I = (c[k] for k in ("N", "E", "K", "H", "I"))
        C = _capacity(c)
        Cp = _padded(C)
        R = E * Cp
        ids, probs = _routing(N, E, K, g)
        lst, _ = _dropless_list(ids, probs, E)
        # the same ranks, cut at the capacity: expert e owns slots e*Cp ..
        flat = ids.reshape(-1).to(torch.int64)
        rank = lst["token_routes"].reshape(-1).to(torch.int64) - lst["block_start"].to(torch.int64)[flat] * 32
        slot = torch.where(rank < C, flat * Cp + rank, R)
        ssi = torch.full((R + 1,), N, dtype=torch.int32, device=DEV)
        ssi[slot] = torch.arange(N * K, device=DEV, dtype=torch.int32) // K
        sp = torch.zeros(R + 1, device=DEV)
        sp[slot] = probs.reshape(-1)
        return dict(c, C=C, Cp=Cp, sorted_slot_ids=ssi[:R].clone(), slot_probs=sp[:R].clone(),
                    x=torch.randn((N, H), generator=g, device=DEV).to(bf16),
                    w1=torch.randn((E, 2 * I, H), generator=g, device=DEV).mul_(0.02).to(bf16),
                    act=torch.empty((R, I), dtype=bf16, device=DEV),
                    codes=torch.empty((R, 2 * I), dtype=torch.int8, device=DEV),
                    scales=torch.empty((R, 2 * I // GROUP), dtype=torch.uint8, device=DEV),
                    preact=torch.empty((R, 2 * I), dtype=bf16, device=DEV))
    if c["kind"] == "bwd":
        R, I = c["R"], c["I"]
        codes, byte = _q8_codes(torch.randn((R, 2 * I), generator=g, device=DEV).mul_(0.9))
        return dict(c, codes=codes.to(torch.int8), scales=byte.to(torch.uint8),
                    d_act=torch.randn((R, I), generator=g, device=DEV).to(bf16),
                    probs=torch.rand((R,), generator=g, device=DEV),
                    act=torch.empty((R, I), dtype=bf16, device=DEV),
                    d_preact=torch.empty((R, 2 * I), dtype=bf16, device=DEV), d_prob=torch.empty((R,), device=DEV))
    rows, D = c["rows"], c["D"]
    # hidden states: channels of different spread, a few of them large
    spread = torch.exp(torch.randn((D,), generator=g, device=DEV))
    v = (torch.randn((rows, D), generator=g, device=DEV) * spread).to(bf16)
    return dict(c, v=v, codes=torch.empty((rows, D), dtype=torch.int8, device=DEV),
                scales=torch.empty((rows, D // GROUP), dtype=torch.uint8, device=DEV), back=torch.empty_like(v))


# ---------------------------------------------------------------- one pass


def _swiglu(g, u):
    return g / (1.0 + torch.exp(-g)) * u


def _plain_w4(s):
    N, K, E, H, I = s["N"], s["K"], s["E"], s["H"], s["I"]
    ids = s["ids"].reshape(-1).to(torch.int64)
    tok = torch.arange(N, device=ids.device).repeat_interleave(K)
    p = s["probs"].reshape(-1, 1)
    x = s["x"].float()
    if N * K <= E:      # few routes: each reads its own expert
        h = torch.bmm(_w4_values(s["w1c"][ids], s["w1s"][ids]), x[tok][:, :, None])[:, :, 0]
    else:               # every expert for every token, then the routes' rows
        h = (_w4_values(s["w1c"], s["w1s"]).reshape(E * 2 * I, H) @ x.t()).reshape(E, 2 * I, N)[ids, :, tok]
    act = (_swiglu(h[:, :I], h[:, I:]) * p).to(torch.bfloat16).float()
    if N * K <= E:
        r = torch.bmm(_w4_values(s["w2c"][ids], s["w2s"][ids]), act[:, :, None])[:, :, 0]
    else:
        a = torch.zeros((E, I, N), device=x.device)
        a[ids, :, tok] = act
        r = torch.bmm(_w4_values(s["w2c"], s["w2s"]), a)[ids, :, tok]
    return r.reshape(N, K, H).sum(1).to(torch.bfloat16)


def _plain_save(s):
    E, Cp, H, I = s["E"], s["Cp"], s["H"], s["I"]
    x = torch.cat([s["x"].float(), torch.zeros((1, H), device=s["x"].device)])
    h = torch.bmm(x[s["sorted_slot_ids"].to(torch.int64)].reshape(E, Cp, H),
                  s["w1"].float().transpose(1, 2).contiguous()).reshape(E * Cp, 2 * I)
    act = (_swiglu(h[:, :I], h[:, I:]) * s["slot_probs"][:, None]).to(torch.bfloat16)
    return act, _q8_values(*_q8_codes(h)).to(torch.bfloat16)


def _plain_bwd(s):
    I = s["I"]
    h = _q8_values(s["codes"], s["scales"])
    g, u, d, p = h[:, :I], h[:, I:], s["d_act"].float(), s["probs"][:, None]
    sig = 1.0 / (1.0 + torch.exp(-g))
    silu = g * sig
    act = (silu * u * p).to(torch.bfloat16)
    d_preact = torch.cat([d * p * u * sig * (1.0 + g * (1.0 - sig)), d * p * silu], 1).to(torch.bfloat16)
    return act, d_preact, (d * silu * u).sum(1)


def run(state):
    s = state
    if own:
        import mixture_experts_expert_amd as moe
    if s["kind"] == "w4":
        if not own:
            return {"y": _plain_w4(s)}
        moe.moe_grouped_ffn_w4(s["x"], s["w1c"], s["w1s"], s["w2c"], s["w2s"], s["sorted_slot_ids"], s["slot_probs"],
                               s["expert_ids"], s["block_start"], s["route_counts"], s["token_routes"], s["act"],
                               s["route_out"], s["y"])
        return {"y": s["y"]}
    if s["kind"] == "save":
        if not own:
            act, preact = _plain_save(s)
            return {"act": act, "preact": preact}
        moe.moe_grouped_fc1_swiglu_save_q8(s["x"], s["w1"], s["sorted_slot_ids"], s["slot_probs"], s["C"], s["act"],
                                           s["codes"], s["scales"])
        moe.moe_q8_dequantize(s["codes"], s["scales"], s["preact"])
        return {"act": s["act"], "preact": s["preact"]}
    if s["kind"] == "bwd":
        if not own:
            act, d_preact, d_prob = _plain_bwd(s)
            return {"act": act, "d_preact": d_preact, "d_prob": d_prob}
        moe.moe_swiglu_bwd_q8(s["codes"], s["scales"], s["d_act"], s["probs"], s["act"], s["d_preact"], s["d_prob"])
        return {"act": s["act"], "d_preact": s["d_preact"], "d_prob": s["d_prob"]}
    if not own:
        return {"values": _q8_values(*_q8_codes(s["v"].float())).to(torch.bfloat16)}
    moe.moe_q8_quantize(s["v"], s["codes"], s["scales"])
    moe.moe_q8_dequantize(s["codes"], s["scales"], s["back"])
    return {"values": s["back"]}


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    c = case
    if c["kind"] == "w4":
        N, E, K, H, I = (c[k] for k in ("N", "E", "K", "H", "I"))
        used = E * (1.0 - (1.0 - K / E) ** N)       # experts that some token picks, on average
        weights = used * 3 * H * I * (1 / 2 + 1 / GROUP)
        return {"bytes": weights + 4 * N * H + 12 * N * K, "flops": 6.0 * N * K * H * I}
    if c["kind"] == "save":
        N, E, K, H, I = (c[k] for k in ("N", "E", "K", "H", "I"))
        R = E * _padded(_capacity(c))
        return {"bytes": 2.0 * N * H + 4.0 * E * I * H + 8 * R + 2.0 * R * I + 4.0 * R * I,
                "flops": 4.0 * min(N * K, E * _capacity(c)) * I * H}
    if c["kind"] == "bwd":
        R, I = c["R"], c["I"]
        return {"bytes": R * (2 * I * (1 + 1 / GROUP) + 2 * I + 4) + R * (2 * I + 4 * I + 4), "flops": 20.0 * R * I}
    n = c["rows"] * c["D"]
    return {"bytes": 4.0 * n, "flops": 6.0 * n}


# ---------------------------------------------------------------- the definitions in 64 bits


def _two_to(k):
    """2^k in float64 for whole k in [-1022, 1023], from the format's own exponent field (a device's pow() may be off)."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_scale(amax):
    """(amax float64) -> the power of two below which no 7-bit code is off by over half a step."""
    safe = torch.where(amax > 0, amax, torch.ones_like(amax))
    k = torch.floor(torch.log2(safe))
    k = torch.where(_two_to(k) > safe, k - 1, torch.where(_two_to(k + 1) <= safe, k + 1, k))
    k = torch.where(safe / _two_to(k - 6) >= 127.5, k - 5, k - 6)
    return _two_to(torch.clamp(k, min=-126))


def _exact_q8(v):
    g = v.reshape(v.shape[0], -1, GROUP)
    s = _exact_scale(g.abs().amax(2))[:, :, None]
    return (torch.round(g / s) * s).reshape(v.shape)


def _exact_w4(codes, byte):
    """One expert's [rows, K/2] codes in float64, from the fields of a code: sign, 2-bit exponent, 1-bit mantissa."""
    c = torch.stack([codes & 15, codes >> 4], 2).reshape(codes.shape[0], -1).to(torch.int64)
    e, m = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * _two_to(e - 1))
    v = torch.where(c >= 8, -mag, mag)
    return v * _two_to(byte.to(torch.int64) - 127).repeat_interleave(GROUP, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    if s["kind"] == "w4":
        N, K, H, I = s["N"], s["K"], s["H"], s["I"]
        x = s["x"].double()
        y = torch.zeros((N, H), dtype=torch.float64, device=x.device)
        for e in sorted(set(s["ids"].reshape(-1).tolist())):
            t, k = torch.where(s["ids"] == e)
            h = x[t] @ _exact_w4(s["w1c"][e], s["w1s"][e]).t()
            a = h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:] * s["probs"][t, k].double()[:, None]
            y.index_add_(0, t, a.to(torch.bfloat16).double() @ _exact_w4(s["w2c"][e], s["w2s"][e]).t())
        return {"y": y}
    if s["kind"] == "save":
        E, Cp, I, N = s["E"], s["Cp"], s["I"], s["N"]
        acts, pres = [], []
        for e in range(E):
            rows = s["sorted_slot_ids"][e * Cp:(e + 1) * Cp].to(torch.int64)
            live = (rows < N).double()[:, None]
            h = (s["x"][torch.clamp(rows, max=N - 1)].double() * live) @ s["w1"][e].double().t()
            p = s["slot_probs"][e * Cp:(e + 1) * Cp].double()[:, None]
            acts.append(h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:] * p)
            pres.append(_exact_q8(h))
        return {"act": torch.cat(acts), "preact": torch.cat(pres)}
    if s["kind"] == "bwd":
        I = s["I"]
        h = s["codes"].double() * _two_to(s["scales"].to(torch.int64) - 127).repeat_interleave(GROUP, dim=1)
        g, u, d, p = h[:, :I], h[:, I:], s["d_act"].double(), s["probs"].double()[:, None]
        sig = torch.sigmoid(g)
        slope = sig + g * sig * (1 - sig)
        return {"act": g * sig * u * p, "d_preact": torch.cat([d * p * u * slope, d * p * g * sig], 1),
                "d_prob": (d * g * sig * u).sum(1)}
    return {"values": _exact_q8(s["v"].double())}
