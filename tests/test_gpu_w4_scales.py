"""Scale bytes over their whole range, through the conversion and every kernel
of the 4-bit FFN: a weight c * 2^(b-127) counts as that number, exactly, for
every b from 0 to 254 (as far as it is a float32 at all), and as NaN for 255."""

import numpy as np
import pytest
import torch

from gpu_support import say
from mixture_experts_expert_amd import DroplessBuffers, W4Weights, moe_grouped_fc2_w4
from test_gpu_w4 import DEV, case, check, run

pytestmark = pytest.mark.gpu

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def every_byte(rows, cols, codes):
    """Row r has the scale byte r % 256; column j of every row the code codes[j % len]."""
    nib = np.resize(np.array(codes, dtype=np.uint8), cols)
    packed = torch.from_numpy(nib[0::2] | nib[1::2] << 4).to(DEV)
    byte = torch.arange(rows, device=DEV).remainder(256).to(torch.uint8)
    w = W4Weights(packed.expand(1, rows, cols // 2).contiguous(),
                  byte[None, :, None].expand(1, rows, cols // 32).contiguous())
    mag = np.array([E2M1[c & 7] * (-1.0 if c & 8 else 1.0) for c in nib])
    value = mag[None] * np.exp2(np.arange(rows) % 256 - 127.0)[:, None]          # exact in float64
    value[np.arange(rows) % 256 == 255] = np.nan
    return w, value


@pytest.mark.parametrize("codes", [range(16), (0, 1, 2, 3, 8, 9, 10, 11)], ids=["every_code", "up_to_1.5"])
def test_conversion(codes):
    w, value = every_byte(512, 128, codes)
    got = w.dequantize()[0].double().cpu().numpy()
    with np.errstate(over="ignore"):
        want = value.astype(np.float32).astype(np.float64)        # 2^128 and more: infinity
    assert np.array_equal(got, want, equal_nan=True)


# FC2 of 20 experts, whose first alone has routes: H, I, N
FORMS = {
    "split": (256, 64, 16),
    "split_odd_scales": (256, 192, 16),
    "split_through_lds": (256, 2048, 16),
    "split_64_rows": (2560, 256, 16),
    "two_route_tiles": (256, 256, 160),
    "streaming": (4864, 256, 16),
    "streaming_two_route_tiles": (3584, 256, 168),
}


@pytest.mark.parametrize("name", FORMS)
def test_products(name):
    """An activation with a single 1 a route picks one column of the weights."""
    H, I, N = FORMS[name]
    E = 1 if name == "two_route_tiles" else 20
    say(f"[w4] scales {name} H {H} I {I} N {N}")
    # bytes 253 and 254 with codes whose values are float32 numbers: infinity times the other columns' zeros is NaN
    for codes, top in ((range(16), 252), ((0, 1, 2, 3, 8, 9, 10, 11), 254)):
        one, value = every_byte(H, I, codes)
        w = W4Weights(one.codes.expand(E, -1, -1).contiguous(), one.scales.expand(E, -1, -1).contiguous())
        buf = DroplessBuffers(N, H, I, E, 1, DEV, w4=True)
        logits = torch.zeros((N, E), device=DEV)
        logits[:, 0] = 1.0
        buf.route(logits)
        slots = buf.token_routes[:, 0].long()
        cols = torch.arange(N, device=DEV) * 13 % I
        buf.act.zero_()
        for power in (0, -20):
            buf.act[slots, cols] = 2.0 ** power
            moe_grouped_fc2_w4(buf.act, w.codes, w.scales, buf.expert_ids, buf.block_start, buf.route_counts, N, 1,
                               buf.route_out)
            got = buf.route_out[slots].double().cpu().numpy()
            want = value[:, cols.cpu().numpy()].T * 2.0 ** power
            byte = np.arange(H) % 256
            known = (byte <= top) | (byte == 255)
            assert np.array_equal(got[:, known], want[:, known], equal_nan=True), f"act 2^{power}"


@pytest.mark.parametrize("shape", [(1, 320, 192, 4, 2), (9, 320, 192, 4, 2), (40, 192, 2112, 4, 2),
                                   (70, 512, 1280, 64, 4)])
def test_bytes_of_the_whole_range_in_sums(shape):
    """Groups 2^100 apart and more in one row: bars as in test_gpu_w4.py."""
    buf, x, w1, w2 = case(*shape, seed=11)
    g = torch.Generator(device=DEV).manual_seed(12)
    s1 = torch.randint(0, 150, w1.scales.shape, generator=g, device=DEV, dtype=torch.uint8)
    s2 = torch.randint(0, 190, w2.scales.shape, generator=g, device=DEV, dtype=torch.uint8)
    w1, w2 = W4Weights(w1.codes, s1), W4Weights(w2.codes, s2)
    y = run(buf, x, w1, w2)
    check(buf, x, w1, w2, buf.act, buf.route_out, y, experts=None if buf.E < 10 else [0, 17, 63])
