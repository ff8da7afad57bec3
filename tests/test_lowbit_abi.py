"""The block-scaled entry points: every declared symbol is exported, and what
the C calls and their Python wrappers refuse.  No device work."""

import ctypes

import pytest
import torch

import mixture_experts_expert_amd as moe
from mixture_experts_expert_amd import _native as nat
from test_abi import ALIGNED as A, INVALID, MIS, MISALIGNED, NUL, OK, UNSUPPORTED

lib = moe.lib


def test_every_declared_symbol_is_exported():
    names = moe.header_functions(moe.LOWBIT_HEADER_PATH)
    assert set(names) == {"moe_w4_quantize", "moe_w4_dequantize", "moe_q8_quantize", "moe_q8_dequantize",
                          "moe_grouped_fc1_swiglu_w4", "moe_grouped_fc2_w4", "moe_gather_combine_f32",
                          "moe_grouped_ffn_w4", "moe_grouped_fc1_swiglu_save_q8", "moe_swiglu_bwd_q8"}
    for n in names:
        assert hasattr(lib, n) and n in nat._SIGNATURES and hasattr(moe, n), n


@pytest.mark.parametrize("name", ["moe_w4_quantize", "moe_q8_quantize"])
def test_quantize_validation(name):
    f = getattr(lib, name)
    assert f(A, -1, 64, A, A, NUL) == INVALID
    assert f(A, 4, 0, A, A, NUL) == INVALID
    assert f(A, 4, 96, A, A, NUL) == UNSUPPORTED               # not a multiple of 64
    assert f(A, 4, 32832, A, A, NUL) == UNSUPPORTED
    assert f(NUL, 4, 32768, A, A, NUL) == INVALID              # the widest: a pre-activation's 2I
    assert f(A, (1 << 34) // 64 + 1, 64, A, A, NUL) == UNSUPPORTED
    assert f(NUL, (1 << 34) // 64, 64, A, A, NUL) == INVALID   # the limit itself passes the size check
    assert f(A, 1 << 62, 64, A, A, NUL) == UNSUPPORTED
    assert f(A, 4, 64, NUL, A, NUL) == INVALID
    assert f(A, 4, 64, A, MIS, NUL) == MISALIGNED
    assert f(NUL, 0, 64, NUL, NUL, NUL) == OK                  # no rows


@pytest.mark.parametrize("name", ["moe_w4_dequantize", "moe_q8_dequantize"])
def test_dequantize_validation(name):
    f = getattr(lib, name)
    assert f(A, A, -1, 64, A, NUL) == INVALID
    assert f(A, A, 4, 72, A, NUL) == UNSUPPORTED
    assert f(A, NUL, 4, 64, A, NUL) == INVALID
    assert f(MIS, A, 4, 64, A, NUL) == MISALIGNED
    assert f(NUL, NUL, 0, 64, NUL, NUL) == OK


def test_w4_ffn_validation():
    f1 = lib.moe_grouped_fc1_swiglu_w4
    p8 = [A] * 8
    assert f1(*p8, 16, 100, 64, 4, 2, A, NUL) == UNSUPPORTED   # H % 64
    assert f1(*p8, 16, 64, 96, 4, 2, A, NUL) == UNSUPPORTED    # I % 64
    assert f1(*p8, 16, 64, 64, 4, 5, A, NUL) == INVALID        # K > E
    assert f1(*p8, 16, 64, 64, 4, 0, A, NUL) == INVALID
    assert f1(*p8, -1, 64, 64, 4, 2, A, NUL) == INVALID
    assert f1(*p8, 20000, 64, 64, 4, 2, A, NUL) == UNSUPPORTED
    assert f1(*p8, 16, 64, 64, 2048, 2, A, NUL) == UNSUPPORTED
    assert f1(*p8, 16, 64, 64, 4, 2, MIS, NUL) == MISALIGNED
    for i in range(8):
        q = list(p8)
        q[i] = NUL
        assert f1(*q, 16, 64, 64, 4, 2, A, NUL) == INVALID, i
    assert f1(*([NUL] * 8), 0, 64, 64, 4, 2, NUL, NUL) == OK
    f2 = lib.moe_grouped_fc2_w4
    p6 = [A] * 6
    for i in range(6):
        q = list(p6)
        q[i] = MIS
        assert f2(*q, 16, 64, 64, 4, 2, A, NUL) == MISALIGNED, i
    assert f2(*p6, 16, 64, 72, 4, 2, A, NUL) == UNSUPPORTED
    assert f2(*p6, 16, 64, 64, 4, 2, NUL, NUL) == INVALID
    assert f2(*([NUL] * 6), 0, 64, 64, 4, 2, NUL, NUL) == OK
    g = lib.moe_grouped_ffn_w4
    p11 = [A] * 11
    for i in range(11):
        q = list(p11)
        q[i] = NUL
        assert g(*q, 16, 64, 64, 4, 2, A, A, A, NUL) == INVALID, i
    for i in range(3):
        o = [A] * 3
        o[i] = MIS
        assert g(*p11, 16, 64, 64, 4, 2, *o, NUL) == MISALIGNED, i
    assert g(*p11, 16, 64, 64, 4, 5, A, A, A, NUL) == INVALID
    assert g(*([NUL] * 11), 0, 64, 64, 4, 2, NUL, NUL, NUL, NUL) == OK


def test_combine_f32_validation():
    f = lib.moe_gather_combine_f32
    assert f(A, A, 16, 0, 64, 128, A, NUL) == INVALID
    assert f(A, A, 16, 33, 64, 128, A, NUL) == UNSUPPORTED
    assert f(A, A, 16, 2, 72, 128, A, NUL) == UNSUPPORTED
    assert f(A, MIS, 16, 2, 64, 128, A, NUL) == MISALIGNED
    assert f(A, NUL, 16, 2, 64, 128, A, NUL) == INVALID
    assert f(NUL, NUL, 0, 2, 64, 0, NUL, NUL) == OK


def test_q8_training_validation():
    f = lib.moe_grouped_fc1_swiglu_save_q8
    assert f(A, A, A, A, 16, 100, 64, 4, 8, A, A, A, NUL) == UNSUPPORTED
    assert f(A, A, A, A, -1, 64, 64, 4, 8, A, A, A, NUL) == INVALID
    assert f(A, A, A, A, 16, 64, 64, 4, 8, A, A, MIS, NUL) == MISALIGNED
    assert f(A, A, A, A, 16, 64, 64, 4, 8, A, NUL, A, NUL) == INVALID
    assert f(*([NUL] * 4), 0, 64, 64, 4, 0, NUL, NUL, NUL, NUL) == OK
    h = lib.moe_swiglu_bwd_q8
    assert h(A, A, A, A, 128, 100, A, A, A, NUL) == UNSUPPORTED
    assert h(A, A, A, A, -1, 64, A, A, A, NUL) == INVALID
    assert h(A, A, A, A, 1 << 31, 64, A, A, A, NUL) == UNSUPPORTED
    assert h(A, MIS, A, A, 128, 64, A, A, A, NUL) == MISALIGNED
    assert h(A, A, A, NUL, 128, 64, A, A, A, NUL) == INVALID
    assert h(NUL, NUL, NUL, NUL, 0, 64, NUL, NUL, NUL, NUL) == OK


def test_wrappers_refuse_host_tensors_and_wrong_shapes():
    w = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_w4_quantize(w, torch.zeros((2, 4, 32), dtype=torch.uint8), torch.zeros((2, 4, 2), dtype=torch.uint8))
    with pytest.raises(TypeError, match="torch.Tensor"):
        moe.moe_q8_quantize([1.0], w, w)
    with pytest.raises(ValueError, match="W4Weights must be codes"):
        moe.W4Weights(torch.zeros((2, 4, 32), dtype=torch.uint8), torch.zeros((2, 4, 3), dtype=torch.uint8))
    with pytest.raises(TypeError, match="uint8"):
        moe.W4Weights(torch.zeros((2, 4, 32), dtype=torch.int8), torch.zeros((2, 4, 2), dtype=torch.uint8))
    q = moe.W4Weights(torch.zeros((2, 4, 32), dtype=torch.uint8), torch.zeros((2, 4, 2), dtype=torch.uint8))
    assert q.shape == (2, 4, 64)
    with pytest.raises(TypeError, match="both"):
        moe.ServingLadder(q, w, 1, 8, 16, device="cpu")
    with pytest.raises(ValueError, match="checkpoint"):
        moe.MoEBackwardBuffers(None, checkpoint="fp8")


def test_signatures_take_as_many_arguments_as_declared():
    import re
    text = re.sub(r"/\*.*?\*/", "", open(moe.LOWBIT_HEADER_PATH).read(), flags=re.S)
    for n in moe.header_functions(moe.LOWBIT_HEADER_PATH):
        args = re.search(r"\b%s\s*\((.*?)\)\s*;" % n, text, flags=re.S).group(1)
        assert len(args.split(",")) == len(nat._SIGNATURES[n][1]), n
    assert nat._SIGNATURES["moe_grouped_ffn_w4"][0] is ctypes.c_int


def test_tensors_and_streams_of_another_device_are_refused(monkeypatch):
    class Elsewhere(torch.Tensor):            # a tensor that says it lives on cuda:1
        is_cuda = True
        device = torch.device("cuda:1")

        def get_device(self):
            return 1

    t = torch.zeros(8).as_subclass(Elsewhere)
    assert nat._at(t, torch.float32, 8, "t", 1) == t.data_ptr()
    with pytest.raises(ValueError, match="t is on cuda:1, the current device is cuda:0"):
        nat._at(t, torch.float32, 8, "t", 0)
    with pytest.raises(ValueError, match="at least 9"):
        nat._at(t, torch.float32, 9, "t", 1)
    with pytest.raises(TypeError, match="expected torch.int32"):
        nat._at(t, torch.int32, 8, "t", 1)

    class Stream:
        device_index, cuda_stream = 1, 1234

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="stream is on device 1"):
        nat._here(Stream())
    Stream.device_index = 0
    assert nat._here(Stream()) == (0, 1234)
    assert nat._here(77) == (0, 77)
