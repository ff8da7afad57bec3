"""ctypes binding of libmoe_native (the C ABI in include/moe_native.h,
include/moe_lowbit.h, include/moe_block.h and include/moe_moments.h).

Argument marshalling only: every function takes torch tensors for the
device buffers, checks dtype/device/contiguity/size on the host, passes raw
pointers and the current HIP stream to the C entry point of the same name,
and raises MoEError on a non-zero status.  All arithmetic of the forward runs
in the library's HIP kernels.  There is no fallback: if the library is not
built, importing this module raises.
"""

from __future__ import annotations

import ctypes
import functools
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_native.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "moe_native.h")
LOWBIT_HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "moe_lowbit.h")
BLOCK_HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "moe_block.h")
MOMENTS_HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "moe_moments.h")
PROBE_HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "moe_probe.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it first (python -m mixture_experts_expert_amd.build "
        "or __graft_entry__.build()); there is no non-HIP fallback")

lib = ctypes.CDLL(LIB_PATH)

_i32, _i64, _f64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_double, ctypes.c_void_p


class AdamWTensor(ctypes.Structure):
    """moe_adamw_tensor."""
    _fields_ = [("param", _vp), ("master", _vp), ("grad", _vp), ("m", _vp), ("v", _vp), ("m_scales", _vp),
                ("v_scales", _vp), ("n", _i64), ("weight_decay", ctypes.c_float), ("param_type", _i32),
                ("grad_type", _i32), ("reserved", _i32)]


_SIGNATURES = {
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_source_capacity": (_i64, [_i64, _i32, _i32, _f64]),
    "moe_layout_block_m": (_i32, []),
    "moe_padded_capacity": (_i64, [_i64]),
    "moe_dropless_bound": (_i64, [_i64, _i32, _i32]),
    "moe_route_capacity_workspace_bytes": (ctypes.c_size_t, [_i64, _i32, _i32]),
    "moe_route_dropless": (ctypes.c_int, [_vp, _i64, _i32, _i32] + [_vp] * 11
                           + [_vp, ctypes.c_size_t, _vp]),
    "moe_route_dropless_live": (ctypes.c_int, [_vp, _i64, _i32, _i32] + [_vp] * 12
                                + [_vp, ctypes.c_size_t, _vp]),
    "moe_grouped_ffn_fwd_dropless": (ctypes.c_int, [_vp] * 7 + [_i64, _i32, _i32, _i32, _i32,
                                                                _vp, _vp, _vp]),
    "moe_grouped_fc1_swiglu_dropless": (ctypes.c_int, [_vp] * 6 + [_i64, _i32, _i32, _i32, _i32,
                                                                   _vp, _vp]),
    "moe_grouped_fc2_dropless": (ctypes.c_int, [_vp] * 4 + [_i64, _i32, _i32, _i32, _i32,
                                                            _vp, _vp]),
    "moe_route_capacity": (ctypes.c_int, [_vp, _i64, _i32, _i32, _i64, _vp, _vp, _vp, _vp,
                                          _vp, ctypes.c_size_t, _vp]),
    "moe_route_capacity_align": (ctypes.c_int, [_vp, _i64, _i32, _i32, _i64, _vp, _vp, _vp, _vp,
                                                _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                _vp, ctypes.c_size_t, _vp]),
    "moe_route_capacity_align_noalloc": (ctypes.c_int, [_vp, _i64, _i32, _i32, _i64] + [_vp] * 11
                                         + [_vp]),
    "moe_align": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i32, _i32, _i64,
                                 _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_grouped_ffn_fwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i64,
                                           _vp, _vp, _vp]),
    "moe_grouped_fc1_swiglu": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i64,
                                              _vp, _vp]),
    "moe_grouped_fc2": (ctypes.c_int, [_vp, _vp, _i64, _i32, _i32, _i32, _i64, _vp, _vp]),
    "moe_grouped_fc2_rows": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, _i32, _i32, _i64, _vp, _vp]),
    "moe_gather_combine": (ctypes.c_int, [_vp, _vp, _i64, _i32, _i32, _i64, _vp, _vp]),
    "moe_dispatch_rows": (ctypes.c_int, [_vp, _vp, _i64, _i32, _i64, _vp, _vp]),
    "moe_grouped_fc1_swiglu_save": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32,
                                                   _i64, _vp, _vp, _vp]),
    "moe_grouped_fc2_dgrad": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, _i32, _i32, _i64, _vp,
                                             _vp]),
    "moe_swiglu_bwd": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, _vp, _vp, _vp, _vp]),
    "moe_grouped_fc1_dgrad": (ctypes.c_int, [_vp, _vp, _i64, _i32, _i32, _i32, _i64, _vp, _vp]),
    "moe_grouped_fc2_wgrad": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, _i32, _i32, _i64, _vp,
                                             _vp]),
    "moe_grouped_fc1_wgrad": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, _i32, _i32, _i64, _vp,
                                             _vp]),
    "moe_grouped_fc2_wgrad_accum": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, _i32, _i32, _i64,
                                                   _vp, _vp]),
    "moe_grouped_fc1_wgrad_accum": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, _i32, _i32, _i64,
                                                   _vp, _vp]),
    "moe_route_bwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i32, _i32, _i64, _vp, _vp]),
    "moe_w4_quantize": (ctypes.c_int, [_vp, _i64, _i32, _vp, _vp, _vp]),
    "moe_w4_dequantize": (ctypes.c_int, [_vp, _vp, _i64, _i32, _vp, _vp]),
    "moe_q8_quantize": (ctypes.c_int, [_vp, _i64, _i32, _vp, _vp, _vp]),
    "moe_q8_dequantize": (ctypes.c_int, [_vp, _vp, _i64, _i32, _vp, _vp]),
    "moe_grouped_fc1_swiglu_w4": (ctypes.c_int, [_vp] * 8 + [_i64, _i32, _i32, _i32, _i32, _vp, _vp]),
    "moe_grouped_fc2_w4": (ctypes.c_int, [_vp] * 6 + [_i64, _i32, _i32, _i32, _i32, _vp, _vp]),
    "moe_gather_combine_f32": (ctypes.c_int, [_vp, _vp, _i64, _i32, _i32, _i64, _vp, _vp]),
    "moe_grouped_ffn_w4": (ctypes.c_int, [_vp] * 11 + [_i64, _i32, _i32, _i32, _i32]
                           + [_vp] * 4),
    "moe_grouped_fc1_swiglu_save_q8": (ctypes.c_int, [_vp] * 4 + [_i64, _i32, _i32, _i32, _i64]
                                       + [_vp] * 4),
    "moe_swiglu_bwd_q8": (ctypes.c_int, [_vp] * 4 + [_i64, _i32] + [_vp] * 4),
    "moe_ffn_decode_max_tokens": (_i32, []),
    "moe_ffn_decode_workspace_bytes": (ctypes.c_size_t, [_i64, _i32, _i32, _i32, _i32]),
    "moe_ffn_decode": (ctypes.c_int, [_vp] * 6 + [_i64, _i32, _i32, _i32, _i32]
                       + [_vp] * 3 + [ctypes.c_size_t, _vp, _vp]),
    "moe_layer_norm_fwd": (ctypes.c_int, [_vp] * 4 + [_i64, _i32, _f64, _i32, _i32] + [_vp] * 5),
    "moe_layer_norm_bwd_workspace_bytes": (ctypes.c_size_t, [_i64, _i32]),
    "moe_layer_norm_bwd": (ctypes.c_int, [_vp] * 6 + [_i64, _i32, _i32, _i32, _i32]
                           + [_vp] * 4 + [ctypes.c_size_t, _vp]),
    "moe_adamw_plan_bytes": (ctypes.c_size_t, [_vp, _i32]),
    "moe_adamw_plan": (ctypes.c_int, [_vp, _i32, _vp, ctypes.c_size_t, _vp]),
    "moe_grad_norm": (ctypes.c_int, [_vp, _i32, _vp, ctypes.c_size_t, _vp, _vp]),
    "moe_adamw_step": (ctypes.c_int, [_vp, _i32, _vp, ctypes.c_size_t, _vp, _f64, _f64, _f64, _vp, _f64, _vp, _vp]),
    "moe_adamw_step_stochastic": (ctypes.c_int, [_vp, _i32, _vp, ctypes.c_size_t, _vp, _f64, _f64, _f64, _vp, _f64, _vp,
                                                 ctypes.c_uint32, _vp]),
    "moe_moment_values": (ctypes.c_int, [_vp] * 4 + [_i64] + [_vp] * 3),
    "moe_moment_codes": (ctypes.c_int, [_vp] * 2 + [_i64] + [_vp] * 5),
    "moe_probe_read": (ctypes.c_int, [_vp, ctypes.c_size_t, _vp, _vp]),
    "moe_probe_write": (ctypes.c_int, [_vp, ctypes.c_size_t, _vp]),
    "moe_probe_copy": (ctypes.c_int, [_vp, _vp, ctypes.c_size_t, _vp]),
    "moe_probe_read_pieces": (ctypes.c_int, [_vp, ctypes.c_size_t, _i32, _i32, _i32, _vp, _vp]),
    "moe_probe_write_pieces": (ctypes.c_int, [_vp, ctypes.c_size_t, _i32, _i32, _i32, _i32, _vp]),
    "moe_probe_write_tiles": (ctypes.c_int, [_vp, ctypes.c_size_t, _i32, _i32, _i32, _i32, _vp]),
    "moe_probe_gemm_loop": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp]),
    "moe_probe_lds_ring": (ctypes.c_int, [_vp, ctypes.c_size_t, _i32, _vp, _vp]),
    "moe_probe_mfma_rate": (ctypes.c_int, [_i32, _i32, _vp, _vp]),
    "moe_probe_lds_read": (ctypes.c_int, [_i32, _i32, _vp, _vp]),
}
for _name, (_res, _args) in _SIGNATURES.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def header_functions(path: str = HEADER_PATH):
    """Names of the functions a header (default include/moe_native.h) declares."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))


def _bytes_ptr(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous device tensor")
    return ctypes.c_void_p(t.data_ptr()), t.numel() * t.element_size()


def moe_probe_read(src, sink, stream=None):
    """Stream-read all of src once (an HBM rate probe); sink: int32 device tensor."""
    p, n = _bytes_ptr(src, "src")
    _check("moe_probe_read", lib.moe_probe_read(p, n, _bytes_ptr(sink, "sink")[0], _stream(stream)))


def moe_probe_write(dst, stream=None):
    """Stream-write all of dst once (an HBM rate probe)."""
    p, n = _bytes_ptr(dst, "dst")
    _check("moe_probe_write", lib.moe_probe_write(p, n, _stream(stream)))


def moe_probe_copy(src, dst, stream=None):
    """dst = src, byte for byte (an HBM rate probe); equal sizes."""
    ps, n = _bytes_ptr(src, "src")
    pd, m = _bytes_ptr(dst, "dst")
    if n != m:
        raise ValueError("moe_probe_copy: src and dst differ in size")
    _check("moe_probe_copy", lib.moe_probe_copy(ps, pd, n, _stream(stream)))


def moe_probe_read_pieces(src, row_bytes: int, rows: int, piece_bytes: int, sink, stream=None):
    """Read src as panels of rows x row_bytes, piece column by piece column
    (an access-order probe); sink: int32 device tensor."""
    p, n = _bytes_ptr(src, "src")
    _check("moe_probe_read_pieces", lib.moe_probe_read_pieces(
        p, n, row_bytes, rows, piece_bytes, _bytes_ptr(sink, "sink")[0], _stream(stream)))


def moe_probe_write_pieces(dst, row_bytes: int, rows: int, piece_bytes: int, nontemporal: bool,
                           stream=None):
    """Write dst as panels of rows x row_bytes, piece column by piece column
    (an access-order probe)."""
    p, n = _bytes_ptr(dst, "dst")
    _check("moe_probe_write_pieces", lib.moe_probe_write_pieces(
        p, n, row_bytes, rows, piece_bytes, int(bool(nontemporal)), _stream(stream)))


def moe_probe_write_tiles(dst, row_bytes: int, rows: int, piece_bytes: int, nontemporal: bool,
                          stream=None):
    """Write dst as panels of rows x row_bytes in tiles of rows x piece_bytes,
    neighbouring tiles on one XCD (an access-order probe)."""
    p, n = _bytes_ptr(dst, "dst")
    _check("moe_probe_write_tiles", lib.moe_probe_write_tiles(
        p, n, row_bytes, rows, piece_bytes, int(bool(nontemporal)), _stream(stream)))


def moe_probe_gemm_loop(a, b, E: int, Cp: int, sink, stream=None):
    """The grouped GEMMs' K loop alone over E experts: a bf16 [E*Cp, K],
    b bf16 [E, N, K] (an access-order-style probe); sink: int32 device tensor."""
    K = a.shape[-1]
    N = b.shape[-2]
    if b.shape[-1] != K or a.numel() < E * Cp * K or b.numel() < E * N * K:
        raise ValueError("moe_probe_gemm_loop: a must be [E*Cp, K] and b [E, N, K]")
    _check("moe_probe_gemm_loop", lib.moe_probe_gemm_loop(
        _ptr(a, torch.bfloat16, E * Cp * K, "a"), _ptr(b, torch.bfloat16, E * N * K, "b"), E, Cp, N, K,
        _bytes_ptr(sink, "sink")[0], _stream(stream)))


def moe_probe_lds_ring(src, stages: int, sink, stream=None):
    """Stream src (whole MiB) through an LDS-DMA ring of `stages` 32 KiB
    stages (the GEMMs' load pipeline alone); sink: int32 device tensor."""
    p, n = _bytes_ptr(src, "src")
    _check("moe_probe_lds_ring", lib.moe_probe_lds_ring(p, n, stages, _bytes_ptr(sink, "sink")[0],
                                                        _stream(stream)))


def _clocks(clocks, groups: int, fn: str):
    if (not isinstance(clocks, torch.Tensor) or not clocks.is_cuda or clocks.dtype != torch.int64
            or not clocks.is_contiguous() or clocks.numel() < 2 * groups):
        raise ValueError(f"{fn}: clocks must be a contiguous int64 device tensor of 2 * groups words")
    return ctypes.c_void_p(clocks.data_ptr())


def moe_probe_mfma_rate(groups: int, iters: int, clocks, stream=None):
    """The matrix cores alone: `groups` workgroups (one per compute unit),
    each wave issuing iters x 4 bf16 32x32x16 MFMAs; clocks: int64 device
    tensor of 2 * groups words (engine-clock, constant-clock ticks per
    workgroup)."""
    _check("moe_probe_mfma_rate", lib.moe_probe_mfma_rate(
        groups, iters, _clocks(clocks, groups, "moe_probe_mfma_rate"), _stream(stream)))


def moe_probe_lds_read(groups: int, iters: int, clocks, stream=None):
    """The LDS read path alone: `groups` workgroups (one per compute unit),
    each wave issuing iters x 8 reads of 1 KB; clocks as moe_probe_mfma_rate."""
    _check("moe_probe_lds_read", lib.moe_probe_lds_read(
        groups, iters, _clocks(clocks, groups, "moe_probe_lds_read"), _stream(stream)))


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {moe_status_string(status)} ({status})")
        self.status = status


def moe_status_string(status: int) -> str:
    return lib.moe_status_string(int(status)).decode()


def moe_source_capacity(N: int, K: int, E: int, F: float) -> int:
    c = lib.moe_source_capacity(int(N), int(K), int(E), float(F))
    if c < 0:
        raise MoEError("moe_source_capacity", c)
    return int(c)


def moe_layout_block_m() -> int:
    return int(lib.moe_layout_block_m())


def moe_padded_capacity(C: int) -> int:
    c = lib.moe_padded_capacity(int(C))
    if c < 0:
        raise MoEError("moe_padded_capacity", c)
    return int(c)


def moe_dropless_bound(N: int, K: int, E: int) -> int:
    r = lib.moe_dropless_bound(N, K, E)
    if r < 0:
        raise MoEError("moe_dropless_bound", r)
    return r


def moe_route_capacity_workspace_bytes(N: int, E: int, K: int) -> int:
    b = int(lib.moe_route_capacity_workspace_bytes(int(N), int(E), int(K)))
    if b == 0 and N > 0:
        raise MoEError("moe_route_capacity_workspace_bytes", -2)
    return b


def route_workspace(N: int, E: int, K: int, device="cuda") -> torch.Tensor:
    """A device workspace for the routing calls (uint8, 16-byte aligned)."""
    return torch.empty(max(moe_route_capacity_workspace_bytes(N, E, K), 16), dtype=torch.uint8,
                       device=device)


def _ws(workspace, N: int, E: int, K: int):
    need = moe_route_capacity_workspace_bytes(N, E, K)
    return _ptr(workspace, torch.uint8, need, "workspace"), ctypes.c_size_t(workspace.numel())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t: torch.Tensor, dtype: torch.dtype, numel: int, name: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name}: needs at least {numel} elements, has {t.numel()}")
    return ctypes.c_void_p(t.data_ptr())


def _check(fn: str, status: int):
    if status != 0:
        raise MoEError(fn, status)


def moe_route_capacity(logits, K: int, C: int, topk_ids, topk_probs, route_slot, expert_count,
                       workspace, stream=None):
    N, E = logits.shape
    _check("moe_route_capacity", lib.moe_route_capacity(
        _ptr(logits, torch.float32, N * E, "logits"), N, E, K, C,
        _ptr(topk_ids, torch.int32, N * K, "topk_ids"),
        _ptr(topk_probs, torch.float32, N * K, "topk_probs"),
        _ptr(route_slot, torch.int32, N * K, "route_slot"),
        _ptr(expert_count, torch.int32, E, "expert_count"), *_ws(workspace, N, E, K),
        _stream(stream)))


def moe_route_capacity_align(logits, K: int, C: int, topk_ids, topk_probs, route_slot,
                             expert_count, sorted_slot_ids, slot_probs, expert_ids, block_start,
                             token_routes, token_route_count, num_tokens_post_padded, workspace,
                             stream=None):
    N, E = logits.shape
    R = E * moe_padded_capacity(C)
    BM = moe_layout_block_m()
    _check("moe_route_capacity_align", lib.moe_route_capacity_align(
        _ptr(logits, torch.float32, N * E, "logits"), N, E, K, C,
        _ptr(topk_ids, torch.int32, N * K, "topk_ids"),
        _ptr(topk_probs, torch.float32, N * K, "topk_probs"),
        _ptr(route_slot, torch.int32, N * K, "route_slot"),
        _ptr(expert_count, torch.int32, E, "expert_count"),
        _ptr(sorted_slot_ids, torch.int32, R, "sorted_slot_ids"),
        _ptr(slot_probs, torch.float32, R, "slot_probs"),
        _ptr(expert_ids, torch.int32, R // BM, "expert_ids"),
        _ptr(block_start, torch.int32, E, "block_start"),
        _ptr(token_routes, torch.int32, N * K, "token_routes"),
        _ptr(token_route_count, torch.int32, N, "token_route_count"),
        _ptr(num_tokens_post_padded, torch.int32, 1, "num_tokens_post_padded"),
        *_ws(workspace, N, E, K), _stream(stream)))


def moe_route_capacity_align_noalloc(logits, K: int, C: int, topk_ids, topk_probs, route_slot,
                                     expert_count, sorted_slot_ids, slot_probs, expert_ids,
                                     block_start, token_routes, token_route_count,
                                     num_tokens_post_padded, stream=None):
    """moe_route_capacity_align with the routing map in the library's own
    per-device scratch array (no workspace, nothing allocated)."""
    N, E = logits.shape
    R = E * moe_padded_capacity(C)
    BM = moe_layout_block_m()
    _check("moe_route_capacity_align_noalloc", lib.moe_route_capacity_align_noalloc(
        _ptr(logits, torch.float32, N * E, "logits"), N, E, K, C,
        _ptr(topk_ids, torch.int32, N * K, "topk_ids"),
        _ptr(topk_probs, torch.float32, N * K, "topk_probs"),
        _ptr(route_slot, torch.int32, N * K, "route_slot"),
        _ptr(expert_count, torch.int32, E, "expert_count"),
        _ptr(sorted_slot_ids, torch.int32, R, "sorted_slot_ids"),
        _ptr(slot_probs, torch.float32, R, "slot_probs"),
        _ptr(expert_ids, torch.int32, R // BM, "expert_ids"),
        _ptr(block_start, torch.int32, E, "block_start"),
        _ptr(token_routes, torch.int32, N * K, "token_routes"),
        _ptr(token_route_count, torch.int32, N, "token_route_count"),
        _ptr(num_tokens_post_padded, torch.int32, 1, "num_tokens_post_padded"), _stream(stream)))


def moe_align(topk_ids, topk_probs, route_slot, expert_count, N: int, E: int, K: int, C: int,
              sorted_slot_ids, slot_probs, expert_ids, block_start, token_routes,
              token_route_count, num_tokens_post_padded, stream=None):
    R = E * moe_padded_capacity(C)
    BM = moe_layout_block_m()
    _check("moe_align", lib.moe_align(
        _ptr(topk_ids, torch.int32, N * K, "topk_ids"),
        _ptr(topk_probs, torch.float32, N * K, "topk_probs"),
        _ptr(route_slot, torch.int32, N * K, "route_slot"),
        _ptr(expert_count, torch.int32, E, "expert_count"), N, E, K, C,
        _ptr(sorted_slot_ids, torch.int32, R, "sorted_slot_ids"),
        _ptr(slot_probs, torch.float32, R, "slot_probs"),
        _ptr(expert_ids, torch.int32, R // BM, "expert_ids"),
        _ptr(block_start, torch.int32, E, "block_start"),
        _ptr(token_routes, torch.int32, N * K, "token_routes"),
        _ptr(token_route_count, torch.int32, N, "token_route_count"),
        _ptr(num_tokens_post_padded, torch.int32, 1, "num_tokens_post_padded"), _stream(stream)))


def moe_grouped_ffn_fwd(x, w1, w2, sorted_slot_ids, slot_probs, C: int, act, route_out,
                        stream=None):
    N, H = x.shape
    E, I2, H1 = w1.shape
    I = I2 // 2
    if H1 != H or tuple(w2.shape) != (E, H, I) or I2 != 2 * I:
        raise ValueError("weights must be w1 [E, 2I, H] and w2 [E, H, I]")
    R = E * moe_padded_capacity(C)
    _check("moe_grouped_ffn_fwd", lib.moe_grouped_ffn_fwd(
        _ptr(x, torch.bfloat16, N * H, "x"), _ptr(w1, torch.bfloat16, E * 2 * I * H, "w1"),
        _ptr(w2, torch.bfloat16, E * H * I, "w2"),
        _ptr(sorted_slot_ids, torch.int32, R, "sorted_slot_ids"),
        _ptr(slot_probs, torch.float32, R, "slot_probs"), N, H, I, E, C,
        _ptr(act, torch.bfloat16, R * I, "act"), _ptr(route_out, torch.bfloat16, R * H, "route_out"),
        _stream(stream)))


def moe_grouped_fc1_swiglu(x, w1, sorted_slot_ids, slot_probs, C: int, act, stream=None):
    N, H = x.shape
    E, I2, H1 = w1.shape
    I = I2 // 2
    if H1 != H or I2 != 2 * I:
        raise ValueError("w1 must be [E, 2I, H]")
    R = E * moe_padded_capacity(C)
    _check("moe_grouped_fc1_swiglu", lib.moe_grouped_fc1_swiglu(
        _ptr(x, torch.bfloat16, N * H, "x"), _ptr(w1, torch.bfloat16, E * 2 * I * H, "w1"),
        _ptr(sorted_slot_ids, torch.int32, R, "sorted_slot_ids"),
        _ptr(slot_probs, torch.float32, R, "slot_probs"), N, H, I, E, C,
        _ptr(act, torch.bfloat16, R * I, "act"), _stream(stream)))


def moe_grouped_fc2(act, w2, N: int, C: int, route_out, stream=None):
    E, H, I = w2.shape
    R = E * moe_padded_capacity(C)
    _check("moe_grouped_fc2", lib.moe_grouped_fc2(
        _ptr(act, torch.bfloat16, R * I, "act"), _ptr(w2, torch.bfloat16, E * H * I, "w2"),
        N, H, I, E, C, _ptr(route_out, torch.bfloat16, R * H, "route_out"), _stream(stream)))


def moe_grouped_fc2_rows(act, w2, out_rows, N: int, C: int, route_out, stream=None):
    E, H, I = w2.shape
    R = E * moe_padded_capacity(C)
    _check("moe_grouped_fc2_rows", lib.moe_grouped_fc2_rows(
        _ptr(act, torch.bfloat16, R * I, "act"), _ptr(w2, torch.bfloat16, E * H * I, "w2"),
        _ptr(out_rows, torch.int32, R, "out_rows"), N, H, I, E, C,
        _ptr(route_out, torch.bfloat16, R * H, "route_out"), _stream(stream)))


def moe_gather_combine(route_out, token_routes, y, stream=None):
    N, K = token_routes.shape
    R, H = route_out.shape
    _check("moe_gather_combine", lib.moe_gather_combine(
        _ptr(route_out, torch.bfloat16, R * H, "route_out"),
        _ptr(token_routes, torch.int32, N * K, "token_routes"), N, K, H, R,
        _ptr(y, torch.bfloat16, N * H, "y"), _stream(stream)))


def moe_dispatch_rows(x, sorted_slot_ids, rows, stream=None):
    N, H = x.shape
    R = sorted_slot_ids.shape[0]
    _check("moe_dispatch_rows", lib.moe_dispatch_rows(
        _ptr(x, torch.bfloat16, N * H, "x"), _ptr(sorted_slot_ids, torch.int32, R, "sorted_slot_ids"),
        N, H, R, _ptr(rows, torch.bfloat16, R * H, "rows"), _stream(stream)))


def moe_route_dropless(logits, K: int, topk_ids, topk_probs, route_within, route_counts,
                       sorted_slot_ids, slot_probs, expert_ids, block_start, token_routes,
                       token_route_count, num_tokens_post_padded, workspace, stream=None):
    N, E = logits.shape
    R = moe_dropless_bound(N, K, E)
    BM = moe_layout_block_m()
    _check("moe_route_dropless", lib.moe_route_dropless(
        _ptr(logits, torch.float32, N * E, "logits"), N, E, K,
        _ptr(topk_ids, torch.int32, N * K, "topk_ids"),
        _ptr(topk_probs, torch.float32, N * K, "topk_probs"),
        _ptr(route_within, torch.int32, N * K, "route_within"),
        _ptr(route_counts, torch.int32, E, "route_counts"),
        _ptr(sorted_slot_ids, torch.int32, R, "sorted_slot_ids"),
        _ptr(slot_probs, torch.float32, R, "slot_probs"),
        _ptr(expert_ids, torch.int32, R // BM, "expert_ids"),
        _ptr(block_start, torch.int32, E, "block_start"),
        _ptr(token_routes, torch.int32, N * K, "token_routes"),
        _ptr(token_route_count, torch.int32, N, "token_route_count"),
        _ptr(num_tokens_post_padded, torch.int32, 1, "num_tokens_post_padded"),
        *_ws(workspace, N, E, K), _stream(stream)))


def moe_route_dropless_live(logits, K: int, n_live, topk_ids, topk_probs, route_within,
                            route_counts, sorted_slot_ids, slot_probs, expert_ids, block_start,
                            token_routes, token_route_count, num_tokens_post_padded, workspace,
                            stream=None):
    N, E = logits.shape
    R = moe_dropless_bound(N, K, E)
    BM = moe_layout_block_m()
    _check("moe_route_dropless_live", lib.moe_route_dropless_live(
        _ptr(logits, torch.float32, N * E, "logits"), N, E, K,
        _ptr(n_live, torch.int32, 1, "n_live"),
        _ptr(topk_ids, torch.int32, N * K, "topk_ids"),
        _ptr(topk_probs, torch.float32, N * K, "topk_probs"),
        _ptr(route_within, torch.int32, N * K, "route_within"),
        _ptr(route_counts, torch.int32, E, "route_counts"),
        _ptr(sorted_slot_ids, torch.int32, R, "sorted_slot_ids"),
        _ptr(slot_probs, torch.float32, R, "slot_probs"),
        _ptr(expert_ids, torch.int32, R // BM, "expert_ids"),
        _ptr(block_start, torch.int32, E, "block_start"),
        _ptr(token_routes, torch.int32, N * K, "token_routes"),
        _ptr(token_route_count, torch.int32, N, "token_route_count"),
        _ptr(num_tokens_post_padded, torch.int32, 1, "num_tokens_post_padded"),
        *_ws(workspace, N, E, K), _stream(stream)))


def moe_grouped_ffn_fwd_dropless(x, w1, w2, sorted_slot_ids, slot_probs, block_start,
                                 num_tokens_post_padded, K: int, act, route_out, stream=None):
    N, H = x.shape
    E, I2, _ = w1.shape
    I = I2 // 2
    R = moe_dropless_bound(N, K, E)
    _check("moe_grouped_ffn_fwd_dropless", lib.moe_grouped_ffn_fwd_dropless(
        _ptr(x, torch.bfloat16, N * H, "x"), _ptr(w1, torch.bfloat16, E * 2 * I * H, "w1"),
        _ptr(w2, torch.bfloat16, E * H * I, "w2"),
        _ptr(sorted_slot_ids, torch.int32, R, "sorted_slot_ids"),
        _ptr(slot_probs, torch.float32, R, "slot_probs"),
        _ptr(block_start, torch.int32, E, "block_start"),
        _ptr(num_tokens_post_padded, torch.int32, 1, "num_tokens_post_padded"),
        N, H, I, E, K, _ptr(act, torch.bfloat16, R * I, "act"),
        _ptr(route_out, torch.bfloat16, R * H, "route_out"), _stream(stream)))


def moe_grouped_fc1_swiglu_dropless(x, w1, sorted_slot_ids, slot_probs, block_start,
                                    num_tokens_post_padded, K: int, act, stream=None):
    N, H = x.shape
    E, I2, _ = w1.shape
    I = I2 // 2
    R = moe_dropless_bound(N, K, E)
    _check("moe_grouped_fc1_swiglu_dropless", lib.moe_grouped_fc1_swiglu_dropless(
        _ptr(x, torch.bfloat16, N * H, "x"), _ptr(w1, torch.bfloat16, E * 2 * I * H, "w1"),
        _ptr(sorted_slot_ids, torch.int32, R, "sorted_slot_ids"),
        _ptr(slot_probs, torch.float32, R, "slot_probs"),
        _ptr(block_start, torch.int32, E, "block_start"),
        _ptr(num_tokens_post_padded, torch.int32, 1, "num_tokens_post_padded"),
        N, H, I, E, K, _ptr(act, torch.bfloat16, R * I, "act"), _stream(stream)))


def moe_grouped_fc2_dropless(act, w2, block_start, num_tokens_post_padded, N: int, K: int,
                             route_out, stream=None):
    E, H, I = w2.shape
    R = moe_dropless_bound(N, K, E)
    _check("moe_grouped_fc2_dropless", lib.moe_grouped_fc2_dropless(
        _ptr(act, torch.bfloat16, R * I, "act"), _ptr(w2, torch.bfloat16, E * H * I, "w2"),
        _ptr(block_start, torch.int32, E, "block_start"),
        _ptr(num_tokens_post_padded, torch.int32, 1, "num_tokens_post_padded"),
        N, H, I, E, K, _ptr(route_out, torch.bfloat16, R * H, "route_out"), _stream(stream)))


# ---------------------------------------------------------------- backward

def _ffn_shape(x, w1):
    N, H = x.shape
    E, I2, H1 = w1.shape
    if H1 != H or I2 % 2:
        raise ValueError("w1 must be [E, 2I, H] with x [N, H]")
    return N, H, I2 // 2, E


def moe_grouped_fc1_swiglu_save(x, w1, sorted_slot_ids, slot_probs, C: int, act, preact,
                                stream=None):
    N, H, I, E = _ffn_shape(x, w1)
    R = E * moe_padded_capacity(C)
    _check("moe_grouped_fc1_swiglu_save", lib.moe_grouped_fc1_swiglu_save(
        _ptr(x, torch.bfloat16, N * H, "x"), _ptr(w1, torch.bfloat16, E * 2 * I * H, "w1"),
        _ptr(sorted_slot_ids, torch.int32, R, "sorted_slot_ids"),
        _ptr(slot_probs, torch.float32, R, "slot_probs"), N, H, I, E, C,
        _ptr(act, torch.bfloat16, R * I, "act"), _ptr(preact, torch.bfloat16, R * 2 * I, "preact"),
        _stream(stream)))


def moe_grouped_fc2_dgrad(dy, w2, sorted_slot_ids, C: int, d_act, stream=None):
    N, H = dy.shape
    E, H2, I = w2.shape
    if H2 != H:
        raise ValueError("w2 must be [E, H, I] with dy [N, H]")
    R = E * moe_padded_capacity(C)
    _check("moe_grouped_fc2_dgrad", lib.moe_grouped_fc2_dgrad(
        _ptr(dy, torch.bfloat16, N * H, "dy"), _ptr(w2, torch.bfloat16, E * H * I, "w2"),
        _ptr(sorted_slot_ids, torch.int32, R, "sorted_slot_ids"), N, H, I, E, C,
        _ptr(d_act, torch.bfloat16, R * I, "d_act"), _stream(stream)))


def moe_swiglu_bwd(preact, d_act, slot_probs, act, d_preact, d_prob, stream=None):
    R, I = d_act.shape
    _check("moe_swiglu_bwd", lib.moe_swiglu_bwd(
        _ptr(preact, torch.bfloat16, R * 2 * I, "preact"),
        _ptr(d_act, torch.bfloat16, R * I, "d_act"),
        _ptr(slot_probs, torch.float32, R, "slot_probs"), R, I,
        _ptr(act, torch.bfloat16, R * I, "act"),
        _ptr(d_preact, torch.bfloat16, R * 2 * I, "d_preact"),
        _ptr(d_prob, torch.float32, R, "d_prob"), _stream(stream)))


def moe_grouped_fc1_dgrad(d_preact, w1, N: int, C: int, d_a, stream=None):
    E, I2, H = w1.shape
    I = I2 // 2
    R = E * moe_padded_capacity(C)
    _check("moe_grouped_fc1_dgrad", lib.moe_grouped_fc1_dgrad(
        _ptr(d_preact, torch.bfloat16, R * 2 * I, "d_preact"),
        _ptr(w1, torch.bfloat16, E * 2 * I * H, "w1"), N, H, I, E, C,
        _ptr(d_a, torch.bfloat16, R * H, "d_a"), _stream(stream)))


def moe_grouped_fc2_wgrad(dy, act, sorted_slot_ids, E: int, C: int, dw2, stream=None):
    N, H = dy.shape
    R, I = act.shape
    if R < E * moe_padded_capacity(C):
        raise ValueError("act must hold E*Cp rows")
    R = E * moe_padded_capacity(C)
    _check("moe_grouped_fc2_wgrad", lib.moe_grouped_fc2_wgrad(
        _ptr(dy, torch.bfloat16, N * H, "dy"), _ptr(act, torch.bfloat16, R * I, "act"),
        _ptr(sorted_slot_ids, torch.int32, R, "sorted_slot_ids"), N, H, I, E, C,
        _ptr(dw2, torch.bfloat16, E * H * I, "dw2"), _stream(stream)))


def moe_grouped_fc1_wgrad(d_preact, x, sorted_slot_ids, E: int, C: int, dw1, stream=None):
    N, H = x.shape
    R2, I2 = d_preact.shape
    I = I2 // 2
    R = E * moe_padded_capacity(C)
    if R2 < R:
        raise ValueError("d_preact must hold E*Cp rows")
    _check("moe_grouped_fc1_wgrad", lib.moe_grouped_fc1_wgrad(
        _ptr(d_preact, torch.bfloat16, R * 2 * I, "d_preact"), _ptr(x, torch.bfloat16, N * H, "x"),
        _ptr(sorted_slot_ids, torch.int32, R, "sorted_slot_ids"), N, H, I, E, C,
        _ptr(dw1, torch.bfloat16, E * 2 * I * H, "dw1"), _stream(stream)))


def moe_grouped_fc2_wgrad_accum(dy, act, sorted_slot_ids, E: int, C: int, main_dw2, stream=None):
    """main_dw2 (float32 [E, H, I]) += the FC2 weight gradient."""
    N, H = dy.shape
    R, I = act.shape
    if R < E * moe_padded_capacity(C):
        raise ValueError("act must hold E*Cp rows")
    R = E * moe_padded_capacity(C)
    _check("moe_grouped_fc2_wgrad_accum", lib.moe_grouped_fc2_wgrad_accum(
        _ptr(dy, torch.bfloat16, N * H, "dy"), _ptr(act, torch.bfloat16, R * I, "act"),
        _ptr(sorted_slot_ids, torch.int32, R, "sorted_slot_ids"), N, H, I, E, C,
        _ptr(main_dw2, torch.float32, E * H * I, "main_dw2"), _stream(stream)))


def moe_grouped_fc1_wgrad_accum(d_preact, x, sorted_slot_ids, E: int, C: int, main_dw1, stream=None):
    """main_dw1 (float32 [E, 2I, H]) += the FC1 weight gradient."""
    N, H = x.shape
    R2, I2 = d_preact.shape
    I = I2 // 2
    R = E * moe_padded_capacity(C)
    if R2 < R:
        raise ValueError("d_preact must hold E*Cp rows")
    _check("moe_grouped_fc1_wgrad_accum", lib.moe_grouped_fc1_wgrad_accum(
        _ptr(d_preact, torch.bfloat16, R * 2 * I, "d_preact"), _ptr(x, torch.bfloat16, N * H, "x"),
        _ptr(sorted_slot_ids, torch.int32, R, "sorted_slot_ids"), N, H, I, E, C,
        _ptr(main_dw1, torch.float32, E * 2 * I * H, "main_dw1"), _stream(stream)))


def moe_route_bwd(topk_ids, topk_probs, token_routes, d_prob, d_logits, stream=None):
    N, K = topk_ids.shape
    E = d_logits.shape[1]
    R = d_prob.numel()
    _check("moe_route_bwd", lib.moe_route_bwd(
        _ptr(topk_ids, torch.int32, N * K, "topk_ids"),
        _ptr(topk_probs, torch.float32, N * K, "topk_probs"),
        _ptr(token_routes, torch.int32, N * K, "token_routes"),
        _ptr(d_prob, torch.float32, R, "d_prob"), N, E, K, R,
        _ptr(d_logits, torch.float32, N * E, "d_logits"), _stream(stream)))


# ------------------------------------------------- block-scaled storage forms
#
# These calls take a few microseconds on the device, so their arguments are
# checked in one pass: dtype, device, contiguity and size, then the address.

_BM = int(lib.moe_layout_block_m())
_bound = functools.lru_cache(maxsize=4096)(moe_dropless_bound)
_capacity = functools.lru_cache(maxsize=4096)(moe_padded_capacity)


def _here(stream):
    """The current device and the stream's handle on it.  Kernels are launched
    on the current device: a stream of another one is refused."""
    dev = torch.cuda.current_device()
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    where = getattr(stream, "device_index", None)
    if where is not None and where != dev:
        raise ValueError(f"the stream is on device {where}, the current device is {dev}")
    return dev, stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _here_of(t, name: str, stream):
    """_here, after a look at one tensor: a host tensor is refused without
    touching a device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return _here(stream)


def _at(t, dtype, numel: int, name: str, dev: int) -> int:
    """Address of a contiguous tensor of `dtype` on device `dev` with at least
    `numel` elements; anything else is refused."""
    try:
        if (t.dtype is dtype and t.get_device() == dev and t.is_contiguous()
                and (not numel or t.numel() >= numel)):
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name}: needs at least {numel} elements, has {t.numel()}")


def _pieces(wide, name: str, per_byte: int, codes, scales):
    """Rows and columns of a block-scaled tensor, from its bf16 form."""
    try:                                      # two dimensions, the common case
        rows, cols = wide.shape
        if (codes.shape == (rows, cols // per_byte) and scales.shape == (rows, cols // 32)
                and cols > 0 and not cols % 32):
            return rows, cols
    except (AttributeError, ValueError):
        pass
    for t, what in ((wide, name), (codes, "codes"), (scales, "scales")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what} must be a torch.Tensor")
    v, a, b = list(wide.shape), list(codes.shape), list(scales.shape)
    if not v or v[-1] < 1:
        raise ValueError(f"{name} must have at least one column")
    cols = v.pop()
    if cols % 32 or not a or not b or a.pop() * per_byte != cols or b.pop() * 32 != cols or a != v or b != v:
        raise ValueError(f"codes and scales must be [..., cols/{per_byte}] and [..., cols/32] with "
                         f"{name} [..., cols]: got {tuple(codes.shape)}, {tuple(scales.shape)} and "
                         f"{tuple(wide.shape)}")
    return wide.numel() // cols, cols


def moe_w4_quantize(w, codes, scales, stream=None):
    """bf16 w [..., K] -> 4-bit codes uint8 [..., K/2], scales uint8 [..., K/32]."""
    rows, K = _pieces(w, "w", 2, codes, scales)
    dev, st = _here_of(w, "w", stream)
    _check("moe_w4_quantize", lib.moe_w4_quantize(
        _at(w, torch.bfloat16, 0, "w", dev), rows, K, _at(codes, torch.uint8, 0, "codes", dev),
        _at(scales, torch.uint8, 0, "scales", dev), st))


def moe_w4_dequantize(codes, scales, w, stream=None):
    """The bf16 values w [..., K] that 4-bit codes stand for (exact)."""
    rows, K = _pieces(w, "w", 2, codes, scales)
    dev, st = _here_of(w, "w", stream)
    _check("moe_w4_dequantize", lib.moe_w4_dequantize(
        _at(codes, torch.uint8, 0, "codes", dev), _at(scales, torch.uint8, 0, "scales", dev), rows,
        K, _at(w, torch.bfloat16, 0, "w", dev), st))


def moe_q8_quantize(v, codes, scales, stream=None):
    """bf16 v [..., D] -> codes int8 [..., D], scales uint8 [..., D/32]."""
    rows, D = _pieces(v, "v", 1, codes, scales)
    dev, st = _here_of(v, "v", stream)
    _check("moe_q8_quantize", lib.moe_q8_quantize(
        _at(v, torch.bfloat16, 0, "v", dev), rows, D, _at(codes, torch.int8, 0, "codes", dev),
        _at(scales, torch.uint8, 0, "scales", dev), st))


def moe_q8_dequantize(codes, scales, v, stream=None):
    """The bf16 values v [..., D] that 8-bit codes stand for (exact)."""
    rows, D = _pieces(v, "v", 1, codes, scales)
    dev, st = _here_of(v, "v", stream)
    _check("moe_q8_dequantize", lib.moe_q8_dequantize(
        _at(codes, torch.int8, 0, "codes", dev), _at(scales, torch.uint8, 0, "scales", dev), rows,
        D, _at(v, torch.bfloat16, 0, "v", dev), st))


def _w4_shape(codes, scales, name: str):
    """(E, rows, columns) of 4-bit weights [E, rows, cols/2] with scales [E, rows, cols/32]."""
    a, b = codes.shape, scales.shape
    if len(a) != 3 or len(b) != 3 or a[0] != b[0] or a[1] != b[1] or a[2] != 16 * b[2]:
        raise ValueError(f"{name} must be codes [E, rows, cols/2] with scales [E, rows, cols/32]")
    return a[0], a[1], a[2] * 2


def moe_grouped_fc1_swiglu_w4(x, w1_codes, w1_scales, sorted_slot_ids, slot_probs, expert_ids,
                              block_start, route_counts, K: int, act, stream=None):
    """act [R, I] = silu(gate) * up * prob of the dropless routes, on 4-bit weights
    (codes [E, 2I, H/2], scales [E, 2I, H/32]).  Rows of pad slots are not written."""
    dev, st = _here_of(x, "x", stream)
    N, H = x.shape
    E, I2, H1 = _w4_shape(w1_codes, w1_scales, "w1")
    I = I2 // 2
    if H1 != H or I2 % 2:
        raise ValueError("w1 must be [E, 2I, H] with x [N, H]")
    R = _bound(N, K, E)
    i32, f32, u8, bf16 = torch.int32, torch.float32, torch.uint8, torch.bfloat16
    _check("moe_grouped_fc1_swiglu_w4", lib.moe_grouped_fc1_swiglu_w4(
        _at(x, bf16, 0, "x", dev), _at(w1_codes, u8, 0, "w1_codes", dev),
        _at(w1_scales, u8, 0, "w1_scales", dev),
        _at(sorted_slot_ids, i32, R, "sorted_slot_ids", dev),
        _at(slot_probs, f32, R, "slot_probs", dev),
        _at(expert_ids, i32, R // _BM, "expert_ids", dev),
        _at(block_start, i32, E, "block_start", dev),
        _at(route_counts, i32, E, "route_counts", dev), N, H, I, E, K,
        _at(act, bf16, R * I, "act", dev), st))


def moe_grouped_fc2_w4(act, w2_codes, w2_scales, expert_ids, block_start, route_counts, N: int,
                       K: int, route_out, stream=None):
    """route_out [R, H] (float32) = act W2^T of the dropless routes, on 4-bit weights
    (codes [E, H, I/2], scales [E, H, I/32]).  Rows of pad slots are not written."""
    dev, st = _here_of(act, "act", stream)
    E, H, I = _w4_shape(w2_codes, w2_scales, "w2")
    R = _bound(N, K, E)
    i32, u8 = torch.int32, torch.uint8
    _check("moe_grouped_fc2_w4", lib.moe_grouped_fc2_w4(
        _at(act, torch.bfloat16, R * I, "act", dev), _at(w2_codes, u8, 0, "w2_codes", dev),
        _at(w2_scales, u8, 0, "w2_scales", dev),
        _at(expert_ids, i32, R // _BM, "expert_ids", dev),
        _at(block_start, i32, E, "block_start", dev),
        _at(route_counts, i32, E, "route_counts", dev), N, H, I, E, K,
        _at(route_out, torch.float32, R * H, "route_out", dev), st))


def moe_gather_combine_f32(route_out, token_routes, y, stream=None):
    """moe_gather_combine over float32 rows: y bf16 [N, H], rounded once."""
    dev, st = _here_of(route_out, "route_out", stream)
    N, K = token_routes.shape
    R, H = route_out.shape
    _check("moe_gather_combine_f32", lib.moe_gather_combine_f32(
        _at(route_out, torch.float32, 0, "route_out", dev),
        _at(token_routes, torch.int32, 0, "token_routes", dev), N, K, H, R,
        _at(y, torch.bfloat16, N * H, "y", dev), st))


def moe_grouped_ffn_w4(x, w1_codes, w1_scales, w2_codes, w2_scales, sorted_slot_ids, slot_probs,
                       expert_ids, block_start, route_counts, token_routes, act, route_out, y,
                       stream=None):
    """Steps 4-5 of the dropless form on 4-bit weights: FC1 + SwiGLU * prob, FC2 and each token's
    sum into y.  act [R, I] and route_out [R, H] (float32) are scratch."""
    dev, st = _here_of(x, "x", stream)
    N, H = x.shape
    n, K = token_routes.shape
    E, I2, H1 = _w4_shape(w1_codes, w1_scales, "w1")
    I = I2 // 2
    if H1 != H or I2 % 2 or _w4_shape(w2_codes, w2_scales, "w2") != (E, H, I):
        raise ValueError("weights must be w1 [E, 2I, H] and w2 [E, H, I] with x [N, H]")
    if n != N:
        raise ValueError("token_routes must be [N, K] with x [N, H]")
    R = _bound(N, K, E)
    i32, f32, u8, bf16 = torch.int32, torch.float32, torch.uint8, torch.bfloat16
    _check("moe_grouped_ffn_w4", lib.moe_grouped_ffn_w4(
        _at(x, bf16, 0, "x", dev), _at(w1_codes, u8, 0, "w1_codes", dev),
        _at(w1_scales, u8, 0, "w1_scales", dev), _at(w2_codes, u8, 0, "w2_codes", dev),
        _at(w2_scales, u8, 0, "w2_scales", dev),
        _at(sorted_slot_ids, i32, R, "sorted_slot_ids", dev),
        _at(slot_probs, f32, R, "slot_probs", dev),
        _at(expert_ids, i32, R // _BM, "expert_ids", dev),
        _at(block_start, i32, E, "block_start", dev),
        _at(route_counts, i32, E, "route_counts", dev),
        _at(token_routes, i32, 0, "token_routes", dev), N, H, I, E, K,
        _at(act, bf16, R * I, "act", dev), _at(route_out, f32, R * H, "route_out", dev),
        _at(y, bf16, N * H, "y", dev), st))


def moe_grouped_fc1_swiglu_save_q8(x, w1, sorted_slot_ids, slot_probs, C: int, act, codes, scales,
                                   stream=None):
    """moe_grouped_fc1_swiglu that also keeps the pre-activation in 8 bits:
    codes int8 [R, 2I], scales uint8 [R, 2I/32]."""
    dev, st = _here_of(x, "x", stream)
    N, H, I, E = _ffn_shape(x, w1)
    R = E * _capacity(C)
    bf16, u8 = torch.bfloat16, torch.uint8
    _check("moe_grouped_fc1_swiglu_save_q8", lib.moe_grouped_fc1_swiglu_save_q8(
        _at(x, bf16, 0, "x", dev), _at(w1, bf16, 0, "w1", dev),
        _at(sorted_slot_ids, torch.int32, R, "sorted_slot_ids", dev),
        _at(slot_probs, torch.float32, R, "slot_probs", dev), N, H, I, E, C,
        _at(act, bf16, R * I, "act", dev), _at(codes, torch.int8, R * 2 * I, "codes", dev),
        _at(scales, u8, R * I // 16, "scales", dev), st))


def moe_swiglu_bwd_q8(codes, scales, d_act, slot_probs, act, d_preact, d_prob, stream=None):
    """moe_swiglu_bwd with the pre-activation in 8 bits (codes [R, 2I], scales [R, 2I/32])."""
    dev, st = _here_of(d_act, "d_act", stream)
    R, I = d_act.shape
    bf16, f32 = torch.bfloat16, torch.float32
    _check("moe_swiglu_bwd_q8", lib.moe_swiglu_bwd_q8(
        _at(codes, torch.int8, R * 2 * I, "codes", dev),
        _at(scales, torch.uint8, R * I // 16, "scales", dev), _at(d_act, bf16, 0, "d_act", dev),
        _at(slot_probs, f32, R, "slot_probs", dev), R, I, _at(act, bf16, R * I, "act", dev),
        _at(d_preact, bf16, R * 2 * I, "d_preact", dev), _at(d_prob, f32, R, "d_prob", dev), st))


# ------------------------------------------------- operators around the layer

def moe_ffn_decode_max_tokens() -> int:
    """Most tokens of a moe_ffn_decode call."""
    return int(lib.moe_ffn_decode_max_tokens())


def moe_ffn_decode_workspace_bytes(N: int, H: int, I: int, E: int, K: int) -> int:
    b = int(lib.moe_ffn_decode_workspace_bytes(N, H, I, E, K))
    if b == 0:
        raise MoEError("moe_ffn_decode_workspace_bytes", -2)
    return b


_decode_bytes = functools.lru_cache(maxsize=4096)(moe_ffn_decode_workspace_bytes)


def moe_ffn_decode(logits, x, w1, w2, topk_ids, topk_probs, workspace, y, residual=None, n_live=None, stream=None):
    """The whole layer for up to moe_ffn_decode_max_tokens() tokens, from logits
    [N, E] to y [N, H] (+ residual): ids, probabilities and y are written."""
    dev, st = _here_of(x, "x", stream)
    shape = x.shape
    N, H = shape
    n, E = logits.shape
    ni, K = topk_ids.shape
    e1, I2, h1 = w1.shape
    I = I2 // 2
    if n != N or ni != N or topk_probs.shape != (N, K) or y.shape != shape:
        raise ValueError("logits [N, E], topk_ids and topk_probs [N, K], x and y [N, H] must agree in N")
    if e1 != E or h1 != H or I2 % 2 or w2.shape != (E, H, I):
        raise ValueError("weights must be w1 [E, 2I, H] and w2 [E, H, I] with x [N, H]")
    bf16 = torch.bfloat16
    status = lib.moe_ffn_decode(
        _at(logits, torch.float32, 0, "logits", dev), _at(x, bf16, 0, "x", dev), _at(w1, bf16, 0, "w1", dev),
        _at(w2, bf16, 0, "w2", dev), _like(residual, "residual", shape, bf16, dev),
        0 if n_live is None else _at(n_live, torch.int32, 1, "n_live", dev), N, H, I, E, K,
        _at(topk_ids, torch.int32, 0, "topk_ids", dev), _at(topk_probs, torch.float32, 0, "topk_probs", dev),
        _at(workspace, torch.uint8, _decode_bytes(N, H, I, E, K), "workspace", dev), workspace.numel(),
        _at(y, bf16, 0, "y", dev), st)
    if status:
        raise MoEError("moe_ffn_decode", status)


_TYPE = {torch.bfloat16: 0, torch.float32: 1}


def _type_of(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _TYPE:
        raise TypeError(f"{name}: expected torch.bfloat16 or torch.float32, got {t.dtype}")
    return _TYPE[t.dtype]


def _like(t, name: str, shape, dtype, dev: int) -> int:
    """Address of a tensor of exactly this shape; 0 for None."""
    if t is None:
        return 0
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if isinstance(t, torch.Tensor) and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return _at(t, dtype, 0, name, dev)


def _vector(t, name: str, n: int, dev: int) -> int:
    """Address of a float32 tensor of n elements; 0 for None."""
    if t is None:
        return 0
    try:
        if t.numel() == n and t.dtype is torch.float32 and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if isinstance(t, torch.Tensor) and t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, has {t.numel()}")
    return _at(t, torch.float32, 0, name, dev)


def moe_layer_norm_fwd(x, weight, bias, eps: float, y, mean, rstd, residual=None, total=None, stream=None):
    """y = norm(x + residual) * weight + bias over the last dimension; total, mean and rstd are kept
    for the backward.  mean None: RMS norm.  total is given with residual, and only then."""
    xt, yt = _type_of(x, "x"), _type_of(y, "y")
    if (residual is None) != (total is None):
        raise ValueError("residual and total must be given together")
    dev, st = _here_of(x, "x", stream)
    shape, dt = x.shape, x.dtype
    if not shape:
        raise ValueError("x must be [..., D]")
    D = shape[-1]
    rows = x.numel() // D if D else 0
    status = lib.moe_layer_norm_fwd(
        _at(x, dt, 0, "x", dev), _like(residual, "residual", shape, dt, dev), _vector(weight, "weight", D, dev),
        _vector(bias, "bias", D, dev), rows, D, eps, xt, yt, _like(total, "total", shape, dt, dev),
        _like(y, "y", shape, y.dtype, dev), _vector(mean, "mean", rows, dev), _vector(rstd, "rstd", rows, dev), st)
    if status:
        raise MoEError("moe_layer_norm_fwd", status)


def moe_layer_norm_bwd_workspace_bytes(rows: int, D: int) -> int:
    b = int(lib.moe_layer_norm_bwd_workspace_bytes(rows, D))
    if b == 0:
        raise MoEError("moe_layer_norm_bwd_workspace_bytes", -2)
    return b


_norm_bytes = functools.lru_cache(maxsize=4096)(moe_layer_norm_bwd_workspace_bytes)


def layer_norm_workspace(rows: int, D: int, device="cuda") -> torch.Tensor:
    """A device workspace for moe_layer_norm_bwd (uint8)."""
    return torch.empty(moe_layer_norm_bwd_workspace_bytes(rows, D), dtype=torch.uint8, device=device)


def moe_layer_norm_bwd(dy, h, weight, mean, rstd, dx, dweight, dbias, workspace, dtotal=None, accumulate: bool = False,
                       stream=None):
    """The backward of moe_layer_norm_fwd: h is what was normalised (total, or x), dtotal the gradient
    that reaches h past the norm.  dx is written, dweight and dbias (may be None) written or added to."""
    ht, yt = _type_of(h, "h"), _type_of(dy, "dy")
    dev, st = _here_of(h, "h", stream)
    shape, dt = h.shape, h.dtype
    if not shape:
        raise ValueError("h must be [..., D]")
    D = shape[-1]
    rows = h.numel() // D if D else 0
    status = lib.moe_layer_norm_bwd(
        _like(dy, "dy", shape, dy.dtype, dev), _at(h, dt, 0, "h", dev), _vector(weight, "weight", D, dev),
        _vector(mean, "mean", rows, dev), _vector(rstd, "rstd", rows, dev), _like(dtotal, "dtotal", shape, dt, dev),
        rows, D, ht, yt, 1 if accumulate else 0, _like(dx, "dx", shape, dt, dev), _vector(dweight, "dweight", D, dev),
        _vector(dbias, "dbias", D, dev), _at(workspace, torch.uint8, _norm_bytes(rows, D), "workspace", dev),
        workspace.numel(), st)
    if status:
        raise MoEError("moe_layer_norm_bwd", status)


class AdamWTable:
    """The tensors of moe_grad_norm and moe_adamw_step and their plan: per tensor its parameter,
    gradient, moments (codes with scale bytes: 8 bits), master copy and weight decay.  Holds the
    memory that they have now, and goes on with it if a tensor is given other memory (`.data = `): a
    table is made again then.  The gradients are the buffers the backward writes.  The
    plan is written on `stream` (None: the current one)."""

    def __init__(self, params, grads, m, v, m_scales=None, v_scales=None, masters=None, weight_decay=0.0, stream=None):
        count = len(params)
        lists = dict(grads=grads, m=m, v=v, m_scales=m_scales, v_scales=v_scales, masters=masters)
        for name, ts in lists.items():
            if ts is not None and len(ts) != count:
                raise ValueError(f"{name}: {len(ts)} tensors for {count} parameters")
        if (m_scales is None) != (v_scales is None):
            raise ValueError("m_scales and v_scales must be given together")
        if not count:
            raise ValueError("no parameters")
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * count
        if len(decay) != count:
            raise ValueError(f"weight_decay: {len(decay)} values for {count} parameters")
        self.count, kind = count, torch.float32 if m_scales is None else torch.uint8
        none = [None] * count
        self.tensors = list(zip(params, masters or none, grads, m, v, m_scales or none, v_scales or none))
        for t in self.tensors:
            _type_of(t[0], "a parameter")
            _type_of(t[2], "a gradient")
        self.device, st = _here_of(params[0], "a parameter", stream)
        dev, f32, u8 = self.device, torch.float32, torch.uint8
        self.array = (AdamWTensor * count)()
        for e, (p, master, g, a, b, sa, sb), wd in zip(self.array, self.tensors, decay):
            n = p.numel()
            e.param, e.n, e.weight_decay = _at(p, p.dtype, 0, "a parameter", dev), n, wd
            e.param_type, e.grad_type = _TYPE[p.dtype], _TYPE[g.dtype]
            e.grad = _whole(g, "a gradient", n, g.dtype, dev)
            e.m, e.v = _whole(a, "a first moment", n, kind, dev), _whole(b, "a second moment", n, kind, dev)
            if kind is u8:
                e.m_scales = _whole(sa, "a first moment's scales", -(-n // 32), u8, dev)
                e.v_scales = _whole(sb, "a second moment's scales", -(-n // 32), u8, dev)
            if master is not None:
                e.master = _whole(master, "a master copy", n, f32, dev)
        self.memory = [t.untyped_storage() for ts in self.tensors for t in ts if t is not None]
        self.address = ctypes.addressof(self.array)
        self.bytes = int(lib.moe_adamw_plan_bytes(self.address, count))
        if self.bytes == 0:
            raise MoEError("moe_adamw_plan_bytes", -2)
        self.plan = torch.empty(self.bytes, dtype=torch.uint8, device=params[0].device)
        if stream is not None:
            _hand_over(stream, self.plan)
        self.plan_at = self.plan.data_ptr()
        _check("moe_adamw_plan", lib.moe_adamw_plan(self.address, count, self.plan_at, self.bytes, st))

    def here(self, stream):
        dev, st = _here(stream)
        if dev != self.device:
            raise ValueError(f"the tensors are on cuda:{self.device}, the current device is cuda:{dev}")
        return dev, st


def _whole(t, name, n, dtype, dev):
    p = _at(t, dtype, 0, name, dev)
    if t.numel() != n:
        raise ValueError(f"{name}: needs {n} elements, has {t.numel()}")
    return p


def _hand_over(stream, *tensors: torch.Tensor):
    """Order `stream` (None: the current one) behind the current stream, where
    the fresh outputs among `tensors` were allocated: work pending there may
    still write their blocks.  The allocator learns that `stream` uses them
    all, so that none is handed out again too early."""
    if stream is None:
        return
    t = tensors[0]
    _here_of(t, "the tensor", stream)                 # refusals come first
    if not hasattr(stream, "wait_stream"):            # a raw handle
        stream = torch.cuda.ExternalStream(int(stream), device=t.device)
    stream.wait_stream(torch.cuda.current_stream(t.device))
    for t in tensors:
        t.record_stream(stream)


def moe_grad_norm(table: AdamWTable, norm, stream=None):
    """norm (float32 [1]) = the 2-norm of all gradients of the table."""
    dev, st = table.here(stream)
    _check("moe_grad_norm", lib.moe_grad_norm(
        table.address, table.count, table.plan_at, table.bytes, _at(norm, torch.float32, 1, "norm", dev), st))


def moe_adamw_step(table: AdamWTable, lr, betas, eps: float, step, grad_norm=None, max_norm: float = 0.0,
                   stream=None):
    """One AdamW step of the table's tensors.  lr float32 [1], step int32 [1] (moved on) and grad_norm
    float32 [1] (or None) are device scalars.  8-bit moments are rounded to nearest, and over many steps
    do not follow the gradients: moe_adamw_step_stochastic's do."""
    *args, st = _step_args(table, lr, betas, eps, step, grad_norm, max_norm, stream)
    _check("moe_adamw_step", lib.moe_adamw_step(*args, st))


def moe_adamw_step_stochastic(table: AdamWTable, lr, betas, eps: float, step, seed: int, grad_norm=None,
                              max_norm: float = 0.0, stream=None):
    """The step of a table with 8-bit moments, rounded stochastically by a hash of seed (0 to 2^32 - 1), step
    and place."""
    if not 0 <= seed < 1 << 32:
        raise ValueError("seed must be 0 to 2^32 - 1")
    *args, st = _step_args(table, lr, betas, eps, step, grad_norm, max_norm, stream)
    _check("moe_adamw_step_stochastic", lib.moe_adamw_step_stochastic(*args, seed, st))


def _step_args(table, lr, betas, eps, step, grad_norm, max_norm, stream):
    dev, st = table.here(stream)
    f32 = torch.float32
    return (table.address, table.count, table.plan_at, table.bytes, _at(lr, f32, 1, "lr", dev), betas[0], betas[1], eps,
            0 if grad_norm is None else _at(grad_norm, f32, 1, "grad_norm", dev), max_norm,
            _at(step, torch.int32, 1, "step", dev), st)


def moe_moment_values(m, m_scales, v, v_scales, m_values, root_values, stream=None):
    """What 8-bit moments stand for: m and the root of v, bf16, of a whole tensor's n elements."""
    dev, st = _here_of(m, "m", stream)
    n, u8, bf16 = m.numel(), torch.uint8, torch.bfloat16
    groups = -(-n // 32)
    _check("moe_moment_values", lib.moe_moment_values(
        _at(m, u8, n, "m", dev), _at(m_scales, u8, groups, "m_scales", dev), _at(v, u8, n, "v", dev),
        _at(v_scales, u8, groups, "v_scales", dev), n, _at(m_values, bf16, n, "m_values", dev),
        _at(root_values, bf16, n, "root_values", dev), st))


def moe_moment_codes(m, v, m_codes, m_scales, v_codes, v_scales, stream=None):
    """8-bit moments from float32 ones of a whole tensor."""
    dev, st = _here_of(m, "m", stream)
    n, f32, u8 = m.numel(), torch.float32, torch.uint8
    groups = -(-n // 32)
    _check("moe_moment_codes", lib.moe_moment_codes(
        _at(m, f32, n, "m", dev), _at(v, f32, n, "v", dev), n, _at(m_codes, u8, n, "m_codes", dev),
        _at(m_scales, u8, groups, "m_scales", dev), _at(v_codes, u8, n, "v_codes", dev),
        _at(v_scales, u8, groups, "v_scales", dev), st))
