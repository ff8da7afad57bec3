"""W4Weights.quantize and dequantize on a stream given by hand: they allocate
their outputs on the current stream and write them on the given one, so the
given stream has to wait for the current one's pending work (the allocator may
hand out a block that it still writes), and the allocator has to know of the
given stream before the tensors can be dropped."""

import pytest
import torch

from mixture_experts_expert_amd import W4Weights
from mixture_experts_expert_amd import _native as nat


class Given:
    """A stream that notes what is asked of it."""
    device_index, cuda_stream = 0, 4711

    def __init__(self, log):
        self.log = log

    def wait_stream(self, other):
        self.log.append(("wait", other))


@pytest.fixture
def log(monkeypatch):
    seen = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.append(("record", t.data_ptr(), s)))
    monkeypatch.setattr(nat, "_here_of", lambda t, name, stream: (0, 0))
    for name in ("moe_w4_quantize", "moe_w4_dequantize"):
        monkeypatch.setattr(nat, name, lambda *a: seen.append(("launch", *a)))
    return seen


def expect(log, stream, tensors):
    launch = [i for i, what in enumerate(log) if what[0] == "launch"]
    assert len(launch) == 1 and log[launch[0]][-1] is stream
    assert ("wait", "current") in log[:launch[0]], "the given stream does not wait for the current one"
    for t in tensors:
        assert ("record", t.data_ptr(), stream) in log, "the allocator does not know of the given stream"


def test_quantize_waits_and_records(log):
    s, w = Given(log), torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    q = W4Weights.quantize(w, stream=s)
    expect(log, s, (w, q.codes, q.scales))


def test_dequantize_waits_and_records(log):
    s = Given(log)
    q = W4Weights(torch.zeros((2, 4, 32), dtype=torch.uint8), torch.zeros((2, 4, 2), dtype=torch.uint8))
    w = q.dequantize(stream=s)
    expect(log, s, (w, q.codes, q.scales))


def test_a_handle_is_a_stream(log, monkeypatch):
    made = []

    def external(handle, device=None):
        made.append((handle, device))
        return Given(log)

    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    W4Weights.quantize(torch.zeros((2, 4, 64), dtype=torch.bfloat16), stream=1234)
    assert made == [(1234, torch.device("cpu"))] and ("wait", "current") in log
    assert [what[-1] for what in log if what[0] == "launch"] == [1234]


def test_the_current_stream_needs_neither(log):
    W4Weights.quantize(torch.zeros((2, 4, 64), dtype=torch.bfloat16))
    assert [what[0] for what in log] == ["launch"]


def test_a_host_tensor_is_refused_before_the_stream_is_touched():
    with pytest.raises(ValueError, match="device tensor"):
        W4Weights.quantize(torch.zeros((2, 4, 64), dtype=torch.bfloat16), stream=Given([]))


# ------------------------------------------------------------------ on the GPU


def weights(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((8, 1024, 2048), generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_pending_work_of_the_current_stream_comes_first(handle):
    w = weights(1)
    want = W4Weights.quantize(w)
    back = want.dequantize()
    side = torch.cuda.Stream()
    given = side.cuda_stream if handle else side
    torch.cuda.synchronize()
    for what in ("quantize", "dequantize"):
        # blocks of the outputs' sizes that the current stream has yet to write
        sizes = (want.codes, want.scales) if what == "quantize" else (back,)
        torch.cuda.empty_cache()
        junk = [torch.empty_like(t) for t in sizes]
        torch.cuda._sleep(20_000_000)
        for t in junk:
            t.fill_(77)
        del junk, t
        if what == "quantize":
            q = W4Weights.quantize(w, stream=given)
            side.synchronize()
            assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)
        else:
            v = want.dequantize(stream=given)
            side.synchronize()
            assert torch.equal(v, back)


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_dropped_tensors_outlive_the_given_stream(handle):
    side = torch.cuda.Stream()
    given = side.cuda_stream if handle else side
    w = weights(2)
    keep = W4Weights.quantize(w)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    q = W4Weights.quantize(w, stream=given)
    shape = q.codes.shape
    del q                                                    # the kernel has not run yet
    again = torch.full(shape, 9, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert bool((again == 9).all())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    v = W4Weights(keep.codes.clone(), keep.scales).dequantize(stream=given)   # codes dropped at once
    again = torch.full(shape, 9, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert bool((again == 9).all()) and torch.equal(v, keep.dequantize())


@pytest.mark.gpu
@pytest.mark.parametrize("fork", [False, True])
def test_captured_with_the_stream_given(fork):
    """On the capturing stream by name, and on another that is joined again;
    replays follow the inputs."""
    w = weights(3)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    given = side if fork else main
    W4Weights.quantize(w).dequantize()                       # the kernels are loaded
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        q = W4Weights.quantize(w, stream=given)
        v = q.dequantize(stream=given)
        main.wait_stream(given)
    for seed in (4, 5, 6):
        w.copy_(weights(seed))
        want = W4Weights.quantize(w)
        back = want.dequantize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales) and torch.equal(v, back)
