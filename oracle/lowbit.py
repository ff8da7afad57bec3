"""Plain CPU definition of the block-scaled storage forms and of the expert
FFN on 4-bit weights.

TEST INFRASTRUCTURE ONLY (see the package docstring).  numpy, float64.

Groups of 32 consecutive columns share a scale byte b, the value 2^(b - 127).
With M the largest code (127 in q8, 6 in w4) and T the magnitude from which a
value would round past it (127.5 and 7), b is the smallest byte >= 1 with
amax / 2^(b-127) < T; codes are the nearest ones, ties to the even one.  A
group with a NaN, an infinity or a magnitude that would round to 2^128 has
b = 255 and codes 0, and stands for NaN.

================  ==============================================  =========================
function          what it computes                                pinned by
================  ==============================================  =========================
q8_quantize       int8 codes and scale bytes                      brute force over b and codes,
w4_quantize       4-bit codes (values' indices) and scale bytes   hand-worked groups
q8_values         the values of codes, float64                    hand-worked groups
w4_values                                                         every code at every scale
w4_pack/unpack    two codes a byte, the even column low           hand-worked bytes
w4_ffn_rows       act and the unrounded FC2 row of given rows     = oracle.expert_ffn on the
                  of one expert                                   same values
================  ==============================================  =========================
"""

from __future__ import annotations

import numpy as np

from .moe import bf16_bits_to_f64, f64_to_bf16_bits, silu

GROUP = 32
NAN_BYTE = 255
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _groups(v):
    v = np.asarray(v, dtype=np.float64)
    return v.reshape(*v.shape[:-1], v.shape[-1] // GROUP, GROUP)


def _scale_bytes(v, top: float, too_big: float):
    """Smallest byte >= 1 whose power of two keeps every magnitude below
    top steps; 255 where a value is not finite or reaches too_big."""
    with np.errstate(invalid="ignore"):
        a = np.abs(_groups(v)).max(axis=-1)              # NaN propagates
        bad = ~(a < too_big)
    a = np.where(bad, 0.0, a)
    m, e = np.frexp(a)                                   # a = m * 2^e, 0.5 <= m < 1
    mt, et = np.frexp(top)
    # a < top * 2^k  <=>  e - et < k, or e - et == k and m < mt
    k = e - et + (m >= mt)
    b = np.maximum(np.where(a > 0, k + 127, 1), 1)
    return np.where(bad, NAN_BYTE, b).astype(np.uint8)


def scale_of(b):
    b = np.asarray(b)
    s = np.ldexp(1.0, b.astype(np.int64) - 127)
    return np.where(b == NAN_BYTE, np.nan, s)


def _scaled(v, b):
    """v / scale, group by group; 0 for a group that stands for NaN."""
    s = np.where(np.asarray(b) == NAN_BYTE, np.inf, scale_of(b))[..., None]
    with np.errstate(invalid="ignore"):
        return np.nan_to_num(_groups(v) / s, nan=0.0, posinf=0.0, neginf=0.0).reshape(np.shape(v))


def q8_quantize(v):
    """float values [..., D] -> int8 codes [..., D], scale bytes [..., D/32]."""
    b = _scale_bytes(v, 127.5, 127.5 * 2.0 ** 121)
    return np.rint(_scaled(v, b)).astype(np.int8), b


def q8_values(codes, b):
    return (_groups(codes) * scale_of(b)[..., None]).reshape(np.shape(codes))


def w4_quantize(v):
    """float values [..., K] -> codes 0..15 [..., K], scale bytes [..., K/32]."""
    b = _scale_bytes(v, 7.0, 7.0 * 2.0 ** 125)
    s = _scaled(v, b)
    d = np.abs(np.abs(s)[..., None] - E2M1)              # distance to every magnitude
    near = d == d.min(axis=-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(axis=-1), even.argmax(axis=-1), near.argmax(axis=-1))
    return (code + 8 * (s < 0)).astype(np.uint8), b


def w4_pack(codes):
    codes = np.asarray(codes, dtype=np.uint8)
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def w4_unpack(packed):
    packed = np.asarray(packed, dtype=np.uint8)
    return np.stack([packed & 15, packed >> 4], axis=-1).reshape(*packed.shape[:-1], -1)


def w4_values(packed, b):
    """float64 values of packed codes [..., K/2] with scale bytes [..., K/32]."""
    c = w4_unpack(packed)
    v = E2M1[c & 7] * np.where(c >= 8, -1.0, 1.0)
    return (_groups(v) * scale_of(b)[..., None]).reshape(c.shape)


def w4_ffn_rows(a_bits, w1, w2, p):
    """One expert on gathered rows a [M, H] (bf16 bits), w1 [2I, H] and
    w2 [H, I] float64 values, p [M]: act as bf16 bits and FC2's rows,
    unrounded, from that act."""
    h = bf16_bits_to_f64(a_bits) @ w1.T
    I = h.shape[1] // 2
    act = f64_to_bf16_bits(silu(h[:, :I]) * h[:, I:] * np.asarray(p, dtype=np.float64)[:, None])
    return act, bf16_bits_to_f64(act) @ w2.T
