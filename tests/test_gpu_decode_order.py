"""The lists that moe_ffn_decode's first kernel hands on to the second: the
routes of an expert that the second kernel cuts into several blocks are in
ascending order, whatever order the waves came in, so that the same inputs give
the same bits (a block decides which waves sum a route)."""

import pytest
import torch

from mixture_experts_expert_amd import DecodeBuffers, forward_decode

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16


def handed_on(buf, N, size):
    """The workspace behind the activation: [0] blocks, from [4] on the blocks (expert | first << 10 | routes << 22),
    then the routes; blocks hold up to `size` routes."""
    routes = N * buf.K
    raw = buf.workspace[routes * buf.I * 2:].cpu()
    most = min(routes, buf.E + routes // size)
    n = int(raw[:4].view(torch.int32)[0])
    assert 0 < n <= most
    block = raw[16:16 + 4 * n].view(torch.int32).long() & 0xFFFFFFFF
    at = 16 + 4 * most
    return (block & 1023).tolist(), (block >> 10 & 4095).tolist(), (block >> 22).tolist(), \
        raw[at:at + 2 * routes].view(torch.int16).tolist()


CASES = [
    # N, H, I, E, K, routes a block of the second kernel (of the first), experts that the tokens prefer
    (16, 512, 128, 128, 8, 4, 24),          # (8): up to one route an expert on average
    (64, 512, 64, 512, 8, 4, 100),          # (8)
    (64, 256, 192, 64, 3, 8, 24),           # (16): three on average
    (61, 256, 704, 61, 6, 8, 61),           # (16): six, 4-column tiles
    (61, 1088, 448, 12, 5, 16, 12),         # (32): 25
]


@pytest.mark.parametrize("N,H,I,E,K,size,preferred", CASES)
def test_routes_are_handed_on_in_order(N, H, I, E, K, size, preferred):
    g = torch.Generator(device=DEV).manual_seed(N + E)
    w1 = torch.empty((E, 2 * I, H), dtype=BF16, device=DEV).normal_(0, 0.05, generator=g)
    w2 = torch.empty((E, H, I), dtype=BF16, device=DEV).normal_(0, 0.05, generator=g)
    x = torch.randn((N, H), generator=g, device=DEV).to(BF16)
    buf = DecodeBuffers(N, H, I, E, K)
    cut = 0
    for _ in range(12):
        logits = torch.randn((N, E), generator=g, device=DEV)
        logits[:, :preferred] += 4.0
        first = forward_decode(buf, logits, x, w1, w2).clone()
        experts, begin, count, route = handed_on(buf, N, size)
        ids = buf.topk_ids.reshape(-1).tolist()
        of = {}
        for e, b, c in zip(experts, begin, count):
            assert 0 < c <= size
            of.setdefault(e, []).extend(route[b:b + c])
        assert sorted(r for rs in of.values() for r in rs) == list(range(N * K))
        for e, rs in of.items():
            assert all(ids[r] == e for r in rs)
            if len(rs) > size:
                cut += 1
                assert rs == sorted(rs), (e, rs)
        for _ in range(3):
            assert torch.equal(forward_decode(buf, logits, x, w1, w2), first), "not the same bits twice"
    assert cut > 0, "no expert had more routes than a block"
