"""Pins of the block-scaled storage oracle: hand-worked groups, brute force
over every scale byte and code, and the 4-bit FFN rows against the bf16
layer's expert FFN on the same values."""

import numpy as np
import pytest

import oracle
from oracle.lowbit import E2M1, NAN_BYTE


def group(*first):
    v = np.zeros(32)
    v[:len(first)] = first
    return v


def test_q8_hand_worked_groups():
    # amax 1.0: 1.0 / 2^-6 = 64 < 127.5 and 1.0 / 2^-7 = 128 is not, so b = 127 - 6
    c, b = oracle.q8_quantize(group(1.0, -0.5, 0.0078125, 0.0234375))
    assert b.tolist() == [121] and c[:4].tolist() == [64, -32, 0, 2]     # 0.5 and 1.5 go to the even code
    # 127.49 steps of 2^0 still fit, 127.5 do not (they would round to 128)
    assert oracle.q8_quantize(group(127.49))[1].tolist() == [127]
    c, b = oracle.q8_quantize(group(127.5, 1.0, 3.0))
    assert b.tolist() == [128] and c[:3].tolist() == [64, 0, 2]
    # zeros, and magnitudes below the smallest scale
    c, b = oracle.q8_quantize(np.zeros(64))
    assert b.tolist() == [1, 1] and not c.any()
    c, b = oracle.q8_quantize(group(2.0 ** -126, 2.0 ** -127, 3 * 2.0 ** -127))
    assert b.tolist() == [1] and c[:3].tolist() == [1, 0, 2]


def test_w4_hand_worked_groups():
    c, b = oracle.w4_quantize(group(6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.001, -0.25))
    assert b.tolist() == [127]
    # 6; the middles go to even codes: 0, 1 (code 2), 1 (2), 2 (4), 2 (4), 4 (6), 4 (6); -6; 0
    assert c[:10].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 15, 8]
    assert oracle.w4_quantize(group(6.99))[1].tolist() == [127]          # 7 is the first to move on
    c, b = oracle.w4_quantize(group(7.0, 1.0))
    assert b.tolist() == [128] and c[:2].tolist() == [6, 1]              # 3.5 -> 4, 0.5
    packed = oracle.w4_pack(np.arange(16, dtype=np.uint8))
    assert packed.tolist() == [0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE]
    assert oracle.w4_unpack(packed).tolist() == list(range(16))


@pytest.mark.parametrize("quantize,values,top,big", [
    (oracle.q8_quantize, oracle.q8_values, 127, 127.5 * 2.0 ** 121),
    (oracle.w4_quantize, lambda c, b: oracle.w4_values(oracle.w4_pack(c), b), 6, 7 * 2.0 ** 125)])
def test_smallest_scale_and_nearest_code_brute_force(quantize, values, top, big):
    rng = np.random.default_rng(5)
    grid = np.arange(-127, 128.0) if top == 127 else np.concatenate([-E2M1[::-1], E2M1])
    step_top = 1.0 if top == 127 else 2.0      # the step the codes would go on with past the top
    for i in range(60):
        v = rng.standard_normal(32) * 2.0 ** rng.integers(-140, 126)
        v *= np.exp(rng.standard_normal(32) * rng.integers(0, 3))
        v = np.clip(v.astype(np.float32).astype(np.float64), -0.9 * big, 0.9 * big)
        c, b = quantize(v[None])
        b = int(b[0, 0])
        s = 2.0 ** (b - 127)
        fits = lambda sc: np.abs(v).max() / sc < top + step_top / 2      # noqa: E731
        assert fits(s) and (b == 1 or not fits(s / 2))
        got = values(c, np.array([[b]], np.uint8))[0]
        best = np.abs(v[:, None] / s - grid).min(axis=1)
        assert np.array_equal(np.abs(v / s - got / s), best)


def test_not_finite_and_too_large_groups_stand_for_nan():
    for q, vals, big in ((oracle.q8_quantize, oracle.q8_values, 127.5 * 2.0 ** 121),
                         (oracle.w4_quantize, lambda c, b: oracle.w4_values(oracle.w4_pack(c), b), 7 * 2.0 ** 125)):
        for bad in (np.nan, np.inf, -np.inf, big, -big):
            v = np.zeros((1, 64))
            v[0, 3] = bad
            v[0, 40] = 1.0
            c, b = q(v)
            assert b[0, 0] == NAN_BYTE and b[0, 1] != NAN_BYTE and not c[0, :32].any()
            out = vals(c, b)
            assert np.isnan(out[0, :32]).all() and out[0, 40] == 1.0
        c, b = q(np.full((1, 32), np.nextafter(big, 0)))
        assert b[0, 0] != NAN_BYTE and np.isfinite(vals(c, b)).all()


def test_values_are_bf16_exactly():
    for b in range(1, 253):
        byte = np.array([[b]], np.uint8)
        v4 = oracle.w4_values(oracle.w4_pack(np.tile(np.arange(16, dtype=np.uint8), 2)[None]), byte)
        assert np.array_equal(oracle.bf16_bits_to_f64(oracle.f64_to_bf16_bits(v4)), v4)
        if b <= 248:
            for lo in range(-127, 128, 32):
                c = np.clip(np.arange(lo, lo + 32), -127, 127).astype(np.int8)[None]
                v8 = oracle.q8_values(c, byte)
                assert np.array_equal(oracle.bf16_bits_to_f64(oracle.f64_to_bf16_bits(v8)), v8)


def test_w4_ffn_rows_equal_the_bf16_layer_on_the_same_values():
    rng = np.random.default_rng(9)
    M, H, I = 5, 64, 96
    a = oracle.f64_to_bf16_bits(rng.standard_normal((M, H)))
    w1 = oracle.w4_values(*_packed(rng.standard_normal((2 * I, H)) * 0.1))
    w2 = oracle.w4_values(*_packed(rng.standard_normal((H, I)) * 0.1))
    p = rng.random(M).astype(np.float32)
    act, rows = oracle.w4_ffn_rows(a, w1, w2, p)
    act_ref, out_ref = oracle.expert_ffn(a, oracle.f64_to_bf16_bits(w1), oracle.f64_to_bf16_bits(w2), p)
    assert np.array_equal(act, act_ref) and np.array_equal(oracle.f64_to_bf16_bits(rows), out_ref)


def _packed(w):
    c, b = oracle.w4_quantize(w)
    return oracle.w4_pack(c), b
