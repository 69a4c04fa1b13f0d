"""GB300-native FP8 W8A8 rollout linear path: Python binding of ``libfp8rl.so``.

The functions named ``fp8rl_*`` mirror the C ABI in ``include/fp8rl.h`` one
to one: they only marshal arguments (a torch tensor becomes its device
pointer, ``stream=None`` becomes torch's current stream) and raise
``Fp8rlError`` on a non-OK status.  Every step of the path runs in the CUDA
kernels of the library; there is no CPU or PyTorch fallback, and loading fails
loudly when the library has not been built.

The convenience helpers below them (``quant_weight``, ``quant_act``,
``gemm``, ``grouped_gemm``, ``quant_weights_batched``) allocate the outputs
with torch and call the same entry points.  With a ``stream`` given, outputs
still come from torch's current stream (keep them until the other one is done
with them); what a helper makes for the call alone belongs to the given one.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import threading

import torch

from . import _build

__all__ = [
    "Fp8rlError", "SCALE_FP32", "SCALE_UE8M0", "load_library", "library_path",
    "fp8rl_quant_weight_blockwise", "fp8rl_quant_weight_blockwise_batched",
    "fp8rl_host_sync_staging_bytes", "fp8rl_quant_weight_host_batched",
    "fp8rl_quant_act_group", "fp8rl_gemm_blockscaled", "fp8rl_grouped_gemm_blockscaled",
    "fp8rl_gemm_act_quant", "gemm_act_quant",
    "fp8rl_gemm_workspace_size", "fp8rl_gemm_blockscaled_ws", "gemm_workspace",
    "fp8rl_gemm_blockscaled_static", "fp8rl_gemm_swiglu_quant", "fp8rl_grouped_gemm_swiglu_quant",
    "gemm_swiglu_quant", "grouped_gemm_swiglu_quant", "quant_gate_up_interleaved",
    "fp8rl_kv_calibrate", "fp8rl_kv_append", "kv_calibrate", "kv_append",
    "fp8rl_attn_prefill_plan_size", "fp8rl_attn_prefill_plan", "fp8rl_attn_prefill", "attn_prefill_plan", "attn_prefill", "AttnPlan",
    "fp8rl_rmsnorm_quant", "rmsnorm_quant", "fp8rl_attn_decode_workspace_size", "fp8rl_attn_decode",
    "attn_decode_workspace", "attn_decode", "fp8rl_logprob", "fp8rl_logprob_backward", "logprobs", "logprobs_backward",
    "fp8rl_sample", "sample", "fp8rl_rotary", "fp8rl_rotary_kv_append", "rotary_freqs", "RotaryFreqs", "rotary", "rotary_kv_append",
    "fp8rl_kv_reserve_workspace_size", "fp8rl_kv_reserve", "fp8rl_kv_fork", "fp8rl_kv_compact_workspace_size", "fp8rl_kv_compact",
    "KvCaches", "kv_reserve", "kv_fork", "kv_compact",
    "fp8rl_e4m3_encode", "fp8rl_debug_set", "fp8rl_sync_status", "fp8rl_status_string", "fp8rl_version",
    "quant_weight", "quant_weights_batched", "quant_act", "gemm", "grouped_gemm", "HostWeightSync",
    "CanaryError", "canaries_enabled", "check_canaries",
]

SCALE_FP32 = 0
SCALE_UE8M0 = 1

STATUS = {0: "FP8RL_OK", 1: "FP8RL_ERR_INVALID_ARG", 2: "FP8RL_ERR_SHAPE",
          3: "FP8RL_ERR_ALIGNMENT", 4: "FP8RL_ERR_UNSUPPORTED", 5: "FP8RL_ERR_CUDA",
          6: "FP8RL_ERR_TIMEOUT", 7: "FP8RL_ERR_DEVICE_CHECK"}


class Fp8rlError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}")


class WeightDesc(ctypes.Structure):
    """fp8rl_weight_desc"""
    _fields_ = [("w_bf16", ctypes.c_void_p), ("q_e4m3", ctypes.c_void_p),
                ("w_scale", ctypes.c_void_p), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("ldw", ctypes.c_int64), ("ldq", ctypes.c_int64)]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    """``libfp8rl.so``, or ``libfp8rl_debug.so`` when FP8RL_DEBUG=1."""
    return _build.LIB_DEBUG if _build.debug_requested() else _build.LIB


def load_library(build_if_missing: bool = False):
    """Load the library (raises if it is missing and building is not asked for)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if build_if_missing:
            _build.build()
        if not os.path.exists(path):
            raise FileNotFoundError(
                f"{path} is not built; run `python -c \"import __graft_entry__ as g; g.build()\"`")
        lib = ctypes.CDLL(path)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        st = ctypes.c_int
        sig = {
            "fp8rl_quant_weight_blockwise": [vp, i64, i64, i64, vp, i64, vp, st, vp],
            "fp8rl_quant_weight_blockwise_batched": [ctypes.POINTER(WeightDesc), i32, st, vp],
            "fp8rl_host_sync_staging_bytes": [i64, i64, i32, st],
            "fp8rl_quant_weight_host_batched": [ctypes.POINTER(WeightDesc), i32, st, vp, ctypes.c_size_t, i32, vp],
            "fp8rl_quant_act_group": [vp, i64, i64, i64, vp, i64, vp, st, vp],
            "fp8rl_gemm_blockscaled": [vp, vp, vp, vp, vp, i64, i64, i64, st, vp],
            "fp8rl_gemm_act_quant": [vp, i64, vp, vp, vp, i64, i64, i64, st, vp, vp, vp],
            "fp8rl_gemm_workspace_size": [ctypes.POINTER(ctypes.c_size_t)],
            "fp8rl_gemm_blockscaled_ws": [vp, vp, vp, vp, vp, i64, i64, i64, st, vp, ctypes.c_size_t, vp],
            "fp8rl_gemm_blockscaled_static": [vp, vp, vp, vp, vp, i64, i64, i64, st, vp],
            "fp8rl_gemm_swiglu_quant": [vp, vp, vp, vp, i64, i64, i64, vp, vp, st, vp],
            "fp8rl_kv_calibrate": [vp, vp, vp, i64, i64, i64, i64, i64, i64, vp, vp],
            "fp8rl_kv_append": [vp, vp, i64, i64, i64, i64, vp, vp, vp, i64, i64, vp, vp],
            "fp8rl_grouped_gemm_swiglu_quant": [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, vp, st, vp],
            "fp8rl_grouped_gemm_blockscaled": [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, st, vp],
            "fp8rl_e4m3_encode": [vp, i64, vp, vp],
            "fp8rl_moe_plan_workspace_size": [i64, i64, i64],
            "fp8rl_moe_plan": [vp, i64, i64, i64, vp, vp, vp, vp, ctypes.c_size_t, vp],
            "fp8rl_moe_dispatch_quant": [vp, i64, i64, i64, vp, i64, i64, vp, i64, vp, st, vp],
            "fp8rl_moe_combine": [vp, i64, i64, i64, vp, vp, i64, i64, vp, i64, vp],
            "fp8rl_tis_workspace_size": [i64],
            "fp8rl_tis_weights": [vp, vp, vp, i64, ctypes.c_float, vp, vp, vp, ctypes.c_size_t, vp],
            "fp8rl_rmsnorm_quant": [vp, i64, vp, i64, vp, ctypes.c_float, i64, i64, vp, i64, vp, i64, vp, st, vp],
            "fp8rl_attn_prefill_plan_size": [i64, i64, i64, i64],
            "fp8rl_attn_prefill_plan": [vp, i64, i64, i64, i64, vp, ctypes.c_size_t, vp],
            "fp8rl_attn_prefill": [vp, i64, vp, i64, vp, i64, vp, ctypes.c_size_t, i64, i64, i64, i64, i64,
                                   ctypes.c_float, vp, i64, vp, vp],
            "fp8rl_attn_decode_workspace_size": [i64, i64, i64],
            "fp8rl_attn_decode": [vp, i64, i64, i64, i64, i64, vp, vp, i64, i64, vp, i64, i64, i64, vp, vp,
                                  ctypes.c_float, vp, i64, vp, vp, ctypes.c_size_t, vp],
            "fp8rl_logprob": [vp, i32, i64, i64, i64, ctypes.c_float, vp, vp, vp, vp, i64, vp, vp, vp],
            "fp8rl_logprob_backward": [vp, i32, i64, i64, i64, ctypes.c_float, vp, vp, vp, vp, vp, vp, i64, vp],
            "fp8rl_sample": [vp, i32, i64, i64, i64, vp, ctypes.c_float, i64, ctypes.c_float, ctypes.c_float, vp, vp, vp, vp,
                             vp, vp, vp, vp, vp],
            "fp8rl_rotary": [vp, i64, i64, vp, i64, i64, i64, i64, vp, i64, vp, i64, i64, i32, i32, vp, i64, vp, i64, vp],
            "fp8rl_rotary_kv_append": [vp, i64, i64, vp, i64, vp, i64, i64, i64, i64, vp, i64, vp, i64, i64, i32, vp, i64, vp, i64,
                                       vp, vp, vp, i64, i64, vp, vp],
            "fp8rl_kv_reserve_workspace_size": [i64, i64, i64],
            "fp8rl_kv_reserve": [vp, i64, i64, i64, i64, vp, vp, i64, vp, vp, i64, vp, vp, vp, i32, i64, i64, vp,
                                 ctypes.c_size_t, vp],
            "fp8rl_kv_fork": [vp, i64, i64, i64, i64, vp, vp, i64, vp, i64, vp, vp, i64, vp],
            "fp8rl_kv_compact_workspace_size": [i64],
            "fp8rl_kv_compact": [vp, i64, i64, i64, i64, vp, vp, i64, vp, vp, i32, i64, i64, vp, ctypes.c_size_t, vp],
            "fp8rl_debug_set": [i32, i64],
            "fp8rl_sync_status": [vp],
            "fp8rl_status_string": [st],
            "fp8rl_version": [],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = st
        lib.fp8rl_status_string.restype = ctypes.c_char_p
        lib.fp8rl_moe_plan_workspace_size.restype = ctypes.c_size_t
        lib.fp8rl_host_sync_staging_bytes.restype = ctypes.c_size_t
        lib.fp8rl_tis_workspace_size.restype = ctypes.c_size_t
        lib.fp8rl_attn_prefill_plan_size.restype = ctypes.c_size_t
        lib.fp8rl_attn_decode_workspace_size.restype = ctypes.c_size_t
        lib.fp8rl_kv_reserve_workspace_size.restype = ctypes.c_size_t
        lib.fp8rl_kv_compact_workspace_size.restype = ctypes.c_size_t
        lib.fp8rl_version.restype = i32
        _lib = lib
        return lib


# --------------------------------------------------------------------------- marshalling

def _p(x) -> int | None:
    """A device pointer from a tensor, an int, or None."""
    if x is None or type(x) is int:
        return x
    return x.data_ptr() if isinstance(x, torch.Tensor) else int(x)


# the current stream's handle and the current device without torch's wrappers
# around them (a call's host time is most of what a small launch costs); both
# are asked only once CUDA is initialised
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int | None:
    if stream is None:
        if torch.cuda.is_initialized() and _raw_stream is not None:
            return _raw_stream(_current_device())
        if torch.cuda.is_available():
            return torch.cuda.current_stream().cuda_stream
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _on(stream, device):
    """The context in which torch's own allocations and fills belong to the stream
    that a call's kernels take: scratch that a helper makes for one call is cleared
    ahead of them, and reused behind them alone."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        # (ExternalStream takes a null handle for a new stream)
        stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _ok(status: int, what: str) -> None:
    if status != 0:
        raise Fp8rlError(status, what)


# --------------------------------------------------------------------------- C ABI, 1:1

def fp8rl_quant_weight_blockwise(w_bf16, n, k, ldw, q_e4m3, ldq, w_scale, fmt=SCALE_FP32,
                                 stream=None) -> None:
    _ok(load_library().fp8rl_quant_weight_blockwise(_p(w_bf16), n, k, ldw, _p(q_e4m3), ldq,
                                                    _p(w_scale), fmt, _stream(stream)),
        "fp8rl_quant_weight_blockwise")


def fp8rl_quant_weight_blockwise_batched(descs, count, fmt=SCALE_FP32, stream=None) -> None:
    _ok(load_library().fp8rl_quant_weight_blockwise_batched(descs, count, fmt, _stream(stream)),
        "fp8rl_quant_weight_blockwise_batched")


def fp8rl_host_sync_staging_bytes(rows, k, slots, fmt=SCALE_FP32) -> int:
    return int(load_library().fp8rl_host_sync_staging_bytes(rows, k, slots, fmt))


def fp8rl_quant_weight_host_batched(descs, count, fmt, d_staging, staging_bytes, slots, stream=None) -> None:
    _ok(load_library().fp8rl_quant_weight_host_batched(descs, count, fmt, _p(d_staging), int(staging_bytes),
                                                       slots, _stream(stream)),
        "fp8rl_quant_weight_host_batched")


def fp8rl_quant_act_group(x_bf16, m, k, ldx, q_e4m3, ldq, x_scale, fmt=SCALE_FP32,
                          stream=None) -> None:
    _ok(load_library().fp8rl_quant_act_group(_p(x_bf16), m, k, ldx, _p(q_e4m3), ldq, _p(x_scale),
                                             fmt, _stream(stream)),
        "fp8rl_quant_act_group")


def fp8rl_gemm_blockscaled(xq, x_scale, wq, w_scale, y_bf16, m, n, k, fmt=SCALE_FP32,
                           stream=None) -> None:
    _ok(load_library().fp8rl_gemm_blockscaled(_p(xq), _p(x_scale), _p(wq), _p(w_scale),
                                              _p(y_bf16), m, n, k, fmt, _stream(stream)),
        "fp8rl_gemm_blockscaled")


def fp8rl_gemm_act_quant(x_bf16, ldx, wq, w_scale, y_bf16, m, n, k, fmt, xq, x_scale,
                         stream=None) -> None:
    _ok(load_library().fp8rl_gemm_act_quant(_p(x_bf16), ldx, _p(wq), _p(w_scale), _p(y_bf16), m, n, k,
                                            fmt, _p(xq), _p(x_scale), _stream(stream)),
        "fp8rl_gemm_act_quant")


def fp8rl_gemm_workspace_size() -> int:
    n = ctypes.c_size_t(0)
    _ok(load_library().fp8rl_gemm_workspace_size(ctypes.byref(n)), "fp8rl_gemm_workspace_size")
    return int(n.value)


def fp8rl_gemm_blockscaled_ws(xq, x_scale, wq, w_scale, y_bf16, m, n, k, fmt, workspace,
                              workspace_bytes, stream=None) -> None:
    _ok(load_library().fp8rl_gemm_blockscaled_ws(_p(xq), _p(x_scale), _p(wq), _p(w_scale),
                                                 _p(y_bf16), m, n, k, fmt, _p(workspace),
                                                 int(workspace_bytes), _stream(stream)),
        "fp8rl_gemm_blockscaled_ws")


def fp8rl_gemm_blockscaled_static(xq, x_scale, wq, w_scale, y_bf16, m, n, k, fmt=SCALE_FP32,
                                  stream=None) -> None:
    _ok(load_library().fp8rl_gemm_blockscaled_static(_p(xq), _p(x_scale), _p(wq), _p(w_scale),
                                                     _p(y_bf16), m, n, k, fmt, _stream(stream)),
        "fp8rl_gemm_blockscaled_static")


def fp8rl_gemm_swiglu_quant(xq, x_scale, wq_gate_up, w_scale_gate_up, m, inter, k, hq, h_scale,
                            fmt=SCALE_FP32, stream=None) -> None:
    _ok(load_library().fp8rl_gemm_swiglu_quant(_p(xq), _p(x_scale), _p(wq_gate_up), _p(w_scale_gate_up), m,
                                               inter, k, _p(hq), _p(h_scale), fmt, _stream(stream)),
        "fp8rl_gemm_swiglu_quant")


def fp8rl_grouped_gemm_swiglu_quant(xq, x_scale, wq_gate_up, w_scale_gate_up, d_offsets, num_experts, rows,
                                    inter, k, hq, h_scale, fmt=SCALE_FP32, stream=None) -> None:
    _ok(load_library().fp8rl_grouped_gemm_swiglu_quant(_p(xq), _p(x_scale), _p(wq_gate_up),
                                                       _p(w_scale_gate_up), _p(d_offsets), num_experts, rows,
                                                       inter, k, _p(hq), _p(h_scale), fmt, _stream(stream)),
        "fp8rl_grouped_gemm_swiglu_quant")


def fp8rl_kv_calibrate(k_bf16, v_bf16, q_bf16, tokens, kv_dim, ldk, ldv, q_dim, ldq, d_scales,
                       stream=None) -> None:
    _ok(load_library().fp8rl_kv_calibrate(_p(k_bf16), _p(v_bf16), _p(q_bf16), tokens, kv_dim, ldk, ldv, q_dim,
                                          ldq, _p(d_scales), _stream(stream)),
        "fp8rl_kv_calibrate")


def fp8rl_kv_append(k_bf16, v_bf16, tokens, kv_dim, ldk, ldv, d_slot_mapping, k_cache, v_cache, ld_cache,
                    num_slots, d_scales, stream=None) -> None:
    _ok(load_library().fp8rl_kv_append(_p(k_bf16), _p(v_bf16), tokens, kv_dim, ldk, ldv, _p(d_slot_mapping),
                                       _p(k_cache), _p(v_cache), ld_cache, num_slots, _p(d_scales),
                                       _stream(stream)),
        "fp8rl_kv_append")


def fp8rl_moe_plan_workspace_size(tokens, topk, experts) -> int:
    return int(load_library().fp8rl_moe_plan_workspace_size(tokens, topk, experts))


def fp8rl_moe_plan(d_topk, tokens, topk, experts, d_offsets, d_row_of_pair, d_token_of_row, d_workspace,
                   workspace_bytes, stream=None) -> None:
    _ok(load_library().fp8rl_moe_plan(_p(d_topk), tokens, topk, experts, _p(d_offsets), _p(d_row_of_pair),
                                      _p(d_token_of_row), _p(d_workspace), workspace_bytes, _stream(stream)),
        "fp8rl_moe_plan")


def fp8rl_moe_dispatch_quant(x_bf16, tokens, k, ldx, d_row_of_pair, topk, rows, q_e4m3, ldq, x_scale,
                             fmt=SCALE_FP32, stream=None) -> None:
    _ok(load_library().fp8rl_moe_dispatch_quant(_p(x_bf16), tokens, k, ldx, _p(d_row_of_pair), topk, rows,
                                                _p(q_e4m3), ldq, _p(x_scale), fmt, _stream(stream)),
        "fp8rl_moe_dispatch_quant")


def fp8rl_moe_combine(y_bf16, rows, n, ldy, d_row_of_pair, d_gate, tokens, topk, out_bf16, ldo,
                      stream=None) -> None:
    _ok(load_library().fp8rl_moe_combine(_p(y_bf16), rows, n, ldy, _p(d_row_of_pair), _p(d_gate), tokens, topk,
                                         _p(out_bf16), ldo, _stream(stream)),
        "fp8rl_moe_combine")


def fp8rl_tis_workspace_size(n) -> int:
    return int(load_library().fp8rl_tis_workspace_size(n))


def fp8rl_tis_weights(d_lp_train, d_lp_rollout, d_mask, n, clip, d_w, d_kl, d_workspace, workspace_bytes,
                      stream=None) -> None:
    _ok(load_library().fp8rl_tis_weights(_p(d_lp_train), _p(d_lp_rollout), _p(d_mask), n, clip, _p(d_w),
                                         _p(d_kl), _p(d_workspace), workspace_bytes, _stream(stream)),
        "fp8rl_tis_weights")


def fp8rl_rmsnorm_quant(x_bf16, ldx, residual_bf16, ldr, weight_bf16, eps, m, k, h_bf16, ldh, q_e4m3, ldq, x_scale,
                        fmt=SCALE_FP32, stream=None) -> None:
    _ok(load_library().fp8rl_rmsnorm_quant(_p(x_bf16), ldx, _p(residual_bf16), ldr, _p(weight_bf16), eps, m, k,
                                           _p(h_bf16), ldh, _p(q_e4m3), ldq, _p(x_scale), fmt, _stream(stream)),
        "fp8rl_rmsnorm_quant")


def fp8rl_attn_prefill_plan_size(total_tokens, batch, q_heads, kv_heads) -> int:
    return int(load_library().fp8rl_attn_prefill_plan_size(total_tokens, batch, q_heads, kv_heads))


def fp8rl_attn_prefill_plan(d_cu_seqlens, batch, total_tokens, q_heads, kv_heads, d_plan, plan_bytes, stream=None) -> None:
    _ok(load_library().fp8rl_attn_prefill_plan(_p(d_cu_seqlens), batch, total_tokens, q_heads, kv_heads, _p(d_plan),
                                               plan_bytes, _stream(stream)),
        "fp8rl_attn_prefill_plan")


def fp8rl_attn_prefill(q_bf16, ldq, k_bf16, ldk, v_bf16, ldv, d_plan, plan_bytes, batch, total_tokens, q_heads, kv_heads,
                       head_dim, softmax_scale, out_bf16, ldo, d_lse, stream=None) -> None:
    _ok(load_library().fp8rl_attn_prefill(_p(q_bf16), ldq, _p(k_bf16), ldk, _p(v_bf16), ldv, _p(d_plan), plan_bytes,
                                          batch, total_tokens, q_heads, kv_heads, head_dim, softmax_scale, _p(out_bf16),
                                          ldo, _p(d_lse), _stream(stream)),
        "fp8rl_attn_prefill")


def fp8rl_attn_decode_workspace_size(q_heads, kv_heads, head_dim) -> int:
    return int(load_library().fp8rl_attn_decode_workspace_size(q_heads, kv_heads, head_dim))


def fp8rl_attn_decode(q_bf16, ldq, batch, q_heads, kv_heads, head_dim, k_cache, v_cache, ld_cache, num_slots,
                      d_block_table, ldt, max_blocks, block_size, d_lens, d_scales, softmax_scale, out_bf16, ldo, d_lse,
                      d_workspace, workspace_bytes, stream=None) -> None:
    _ok(load_library().fp8rl_attn_decode(_p(q_bf16), ldq, batch, q_heads, kv_heads, head_dim, _p(k_cache), _p(v_cache),
                                         ld_cache, num_slots, _p(d_block_table), ldt, max_blocks, block_size,
                                         _p(d_lens), _p(d_scales), softmax_scale, _p(out_bf16), ldo, _p(d_lse),
                                         _p(d_workspace), workspace_bytes, _stream(stream)),
        "fp8rl_attn_decode")


def fp8rl_logprob(d_logits, logits_fp32, rows, vocab, ld, temperature, d_tokens, d_lp, d_entropy, d_stats, topk,
                  d_top_ids, d_top_lp, stream=None) -> None:
    _ok(load_library().fp8rl_logprob(_p(d_logits), logits_fp32, rows, vocab, ld, temperature, _p(d_tokens), _p(d_lp),
                                     _p(d_entropy), _p(d_stats), topk, _p(d_top_ids), _p(d_top_lp), _stream(stream)),
        "fp8rl_logprob")


def fp8rl_logprob_backward(d_logits, logits_fp32, rows, vocab, ld, temperature, d_tokens, d_stats, d_entropy,
                           d_grad_lp, d_grad_entropy, d_dlogits, ldd, stream=None) -> None:
    _ok(load_library().fp8rl_logprob_backward(_p(d_logits), logits_fp32, rows, vocab, ld, temperature, _p(d_tokens),
                                              _p(d_stats), _p(d_entropy), _p(d_grad_lp), _p(d_grad_entropy),
                                              _p(d_dlogits), ldd, _stream(stream)),
        "fp8rl_logprob_backward")


def fp8rl_sample(d_logits, logits_fp32, rows, vocab, ld, d_uniform, temperature, top_k, top_p, min_p, d_temperature, d_top_k,
                 d_top_p, d_min_p, d_tokens, d_lp, d_lp_kept, d_kept, stream=None) -> None:
    _ok(load_library().fp8rl_sample(_p(d_logits), logits_fp32, rows, vocab, ld, _p(d_uniform), temperature, top_k, top_p, min_p,
                                    _p(d_temperature), _p(d_top_k), _p(d_top_p), _p(d_min_p), _p(d_tokens), _p(d_lp),
                                    _p(d_lp_kept), _p(d_kept), _stream(stream)),
        "fp8rl_sample")


def fp8rl_rotary(q_bf16, ldq, q_heads, k_bf16, ldk, kv_heads, tokens, head_dim, d_freqs, pairs, d_positions, ldp, axes,
                 interleaved, inverse, q_out, ldqo, k_out, ldko, stream=None) -> None:
    _ok(load_library().fp8rl_rotary(_p(q_bf16), ldq, q_heads, _p(k_bf16), ldk, kv_heads, tokens, head_dim, _p(d_freqs), pairs,
                                    _p(d_positions), ldp, axes, interleaved, inverse, _p(q_out), ldqo, _p(k_out), ldko,
                                    _stream(stream)),
        "fp8rl_rotary")


def fp8rl_rotary_kv_append(q_bf16, ldq, q_heads, k_bf16, ldk, v_bf16, ldv, kv_heads, tokens, head_dim, d_freqs, pairs,
                           d_positions, ldp, axes, interleaved, q_out, ldqo, k_out, ldko, d_slot_mapping, k_cache, v_cache,
                           ld_cache, num_slots, d_scales, stream=None) -> None:
    _ok(load_library().fp8rl_rotary_kv_append(_p(q_bf16), ldq, q_heads, _p(k_bf16), ldk, _p(v_bf16), ldv, kv_heads, tokens,
                                              head_dim, _p(d_freqs), pairs, _p(d_positions), ldp, axes, interleaved, _p(q_out),
                                              ldqo, _p(k_out), ldko, _p(d_slot_mapping), _p(k_cache), _p(v_cache), ld_cache,
                                              num_slots, _p(d_scales), _stream(stream)),
        "fp8rl_rotary_kv_append")


def fp8rl_kv_reserve_workspace_size(rows, total_tokens, block_size) -> int:
    return int(load_library().fp8rl_kv_reserve_workspace_size(rows, total_tokens, block_size))


def fp8rl_kv_reserve(d_block_table, ldt, rows, max_blocks, block_size, d_lens, d_refs, pages, d_cu_seqlens, d_count, total_tokens,
                     d_slots, d_info, caches, n_caches, width, ld_cache, d_workspace, workspace_bytes, stream=None) -> None:
    _ok(load_library().fp8rl_kv_reserve(_p(d_block_table), ldt, rows, max_blocks, block_size, _p(d_lens), _p(d_refs), pages,
                                        _p(d_cu_seqlens), _p(d_count), total_tokens, _p(d_slots), _p(d_info), caches, n_caches,
                                        width, ld_cache, _p(d_workspace), workspace_bytes, _stream(stream)),
        "fp8rl_kv_reserve")


def fp8rl_kv_fork(d_block_table, ldt, rows, max_blocks, block_size, d_lens, d_parent, new_rows, d_new_table, ld_new, d_new_lens,
                  d_refs, pages, stream=None) -> None:
    _ok(load_library().fp8rl_kv_fork(_p(d_block_table), ldt, rows, max_blocks, block_size, _p(d_lens), _p(d_parent), new_rows,
                                     _p(d_new_table), ld_new, _p(d_new_lens), _p(d_refs), pages, _stream(stream)),
        "fp8rl_kv_fork")


def fp8rl_kv_compact_workspace_size(pages) -> int:
    return int(load_library().fp8rl_kv_compact_workspace_size(pages))


def fp8rl_kv_compact(d_block_table, ldt, rows, max_blocks, block_size, d_lens, d_refs, pages, d_used, caches, n_caches, width,
                     ld_cache, d_workspace, workspace_bytes, stream=None) -> None:
    _ok(load_library().fp8rl_kv_compact(_p(d_block_table), ldt, rows, max_blocks, block_size, _p(d_lens), _p(d_refs), pages,
                                        _p(d_used), caches, n_caches, width, ld_cache, _p(d_workspace), workspace_bytes,
                                        _stream(stream)),
        "fp8rl_kv_compact")


def fp8rl_grouped_gemm_blockscaled(xq, x_scale, wq, w_scale, d_offsets, num_experts, rows, n, k,
                                   y_bf16, fmt=SCALE_FP32, stream=None) -> None:
    _ok(load_library().fp8rl_grouped_gemm_blockscaled(_p(xq), _p(x_scale), _p(wq), _p(w_scale),
                                                      _p(d_offsets), num_experts, rows, n, k,
                                                      _p(y_bf16), fmt, _stream(stream)),
        "fp8rl_grouped_gemm_blockscaled")


def fp8rl_e4m3_encode(d_in, n, d_out, stream=None) -> None:
    _ok(load_library().fp8rl_e4m3_encode(_p(d_in), n, _p(d_out), _stream(stream)), "fp8rl_e4m3_encode")


DEBUG_RESET, DEBUG_GEMM_BN, DEBUG_FAULT_SKIP_KB, DEBUG_TIMEOUT_NS = 0, 1, 2, 3
DEBUG_WAIT_MODE, DEBUG_L2_PREFETCH, DEBUG_SPLITS, DEBUG_STREAMK, DEBUG_STREAMK_GRID = 4, 5, 6, 7, 8
DEBUG_OUT_STAGE, DEBUG_DECODE, DEBUG_MX, DEBUG_PAIR, DEBUG_PDL = 9, 10, 11, 12, 13


def fp8rl_debug_set(key, value) -> None:
    _ok(load_library().fp8rl_debug_set(int(key), int(value)), "fp8rl_debug_set")


def fp8rl_sync_status(stream=None) -> int:
    """Synchronise and return the status code (0 = OK, 6 = a device wait ran
    out).  With FP8RL_CANARY=1, also checks the guard zones of every output
    allocated since the last call (raises CanaryError)."""
    st = int(load_library().fp8rl_sync_status(_stream(stream)))
    if canaries_enabled():
        check_canaries()
    return st


def fp8rl_status_string(status: int) -> str:
    return load_library().fp8rl_status_string(int(status)).decode()


def fp8rl_version() -> int:
    return int(load_library().fp8rl_version())


# --------------------------------------------------------------------------- helpers

def _scale_dtype(fmt):
    return torch.float32 if fmt == SCALE_FP32 else torch.uint8


# ---------------------------------------------------------------- canary guards
# With FP8RL_CANARY=1 in the environment (a debugging aid, off by default),
# every output the helpers below allocate sits between two guard zones filled
# with a fixed byte; fp8rl_sync_status() checks every guard zone allocated
# since its last call and raises CanaryError if a kernel wrote outside its
# output.  The guarded buffers are kept alive until that check.
CANARY_BYTE = 0xA5
_CANARY_PRE = 4096           # bytes before the output (keeps its 256-byte alignment)
_CANARY_POST = 64 * 1024     # bytes after it (a ragged tile overrun lands here)
_guards = []
_guards_lock = threading.Lock()


class CanaryError(RuntimeError):
    pass


def canaries_enabled() -> bool:
    return os.environ.get("FP8RL_CANARY") == "1"


def _out(shape, dtype, device):
    """An output tensor: plain torch.empty, or guarded when FP8RL_CANARY=1."""
    if not canaries_enabled():
        return torch.empty(shape, dtype=dtype, device=device)
    return _guarded(shape, dtype, device)


def _outs(specs, device):
    """Output tensors of several (shape, dtype): _out of each (None for None),
    with one look at the environment."""
    make = _guarded if canaries_enabled() else _empty
    return [make(*spec, device) if spec else None for spec in specs]


def _empty(shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device)


def _guarded(shape, dtype, device):
    numel = 1
    for d in shape:
        numel *= int(d)
    if numel == 0:
        return torch.empty(shape, dtype=dtype, device=device)
    nbytes = numel * torch.empty((), dtype=dtype).element_size()
    buf = torch.full((_CANARY_PRE + nbytes + _CANARY_POST,), CANARY_BYTE, dtype=torch.uint8, device=device)
    if buf.is_cuda and not torch.cuda.is_current_stream_capturing():
        torch.cuda.current_stream(buf.device).synchronize()  # the call's kernels may go to another stream
    with _guards_lock:
        _guards.append((buf, nbytes))
    return buf[_CANARY_PRE:_CANARY_PRE + nbytes].view(dtype).view(tuple(shape))


def check_canaries() -> int:
    """Check (and forget) every guarded output allocated so far; returns how
    many were checked, raises CanaryError naming the first damaged one."""
    with _guards_lock:
        guards = list(_guards)
        _guards.clear()
    for buf, nbytes in guards:
        pre = buf[:_CANARY_PRE]
        post = buf[_CANARY_PRE + nbytes:]
        if not bool((pre == CANARY_BYTE).all()) or not bool((post == CANARY_BYTE).all()):
            bad_pre = int((pre != CANARY_BYTE).sum())
            bad_post = int((post != CANARY_BYTE).sum())
            raise CanaryError(f"a kernel wrote outside an output of {nbytes} bytes: "
                              f"{bad_pre} guard bytes before it and {bad_post} after it changed")
    return len(guards)


def _check_cuda(*tensors):
    """The kernels dereference device pointers on the current device: every
    tensor argument of a helper must be a CUDA tensor on it (None and
    non-tensor arguments are skipped)."""
    cur = _current_device() if torch.cuda.is_initialized() else None
    for t in tensors:
        if t is None or not isinstance(t, torch.Tensor) or t.get_device() == cur:  # -1 for a host tensor
            continue
        if not t.is_cuda:
            raise ValueError("fp8rl helpers take CUDA tensors; a host tensor's pointer would reach the kernels")
        raise ValueError(f"a tensor on {t.device} while the current device is cuda:{cur}")


def _check_bf16_2d(t: torch.Tensor, name: str):
    if t.dtype != torch.bfloat16 or t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D bf16 tensor with unit column stride")


def quant_weight(w: torch.Tensor, fmt=SCALE_FP32, stream=None):
    """E4M3 codes (uint8 [n,k]) and block scales ([ceil(n/128), ceil(k/128)]) of w."""
    _check_cuda(w)
    _check_bf16_2d(w, "w")
    n, k = w.shape
    q = _out((n, k), torch.uint8, w.device)
    s = _out(((n + 127) // 128, (k + 127) // 128), _scale_dtype(fmt), w.device)
    fp8rl_quant_weight_blockwise(w, n, k, w.stride(0), q, k, s, fmt, stream)
    return q, s


def weight_descs(items):
    """fp8rl_weight_desc array from (w, q, scale) tensor triples."""
    arr = (WeightDesc * max(1, len(items)))()
    for i, (w, q, s) in enumerate(items):
        arr[i] = WeightDesc(w.data_ptr(), q.data_ptr(), s.data_ptr(), w.shape[0], w.shape[1],
                            w.stride(0), q.stride(0))
    return arr


def quant_weights_batched(weights, fmt=SCALE_FP32, stream=None, outputs=None):
    """Quantise a list of bf16 matrices in one pass; returns [(q, scale), ...]."""
    weights = list(weights)
    _check_cuda(*weights, *(t for pair in (outputs or ()) for t in pair))
    if outputs is None:
        outputs = []
        for w in weights:
            _check_bf16_2d(w, "w")
            n, k = w.shape
            outputs.append((_out((n, k), torch.uint8, w.device),
                            _out(((n + 127) // 128, (k + 127) // 128),
                                        dtype=_scale_dtype(fmt), device=w.device)))
    descs = weight_descs([(w, q, s) for w, (q, s) in zip(weights, outputs)])
    fp8rl_quant_weight_blockwise_batched(descs, len(weights), fmt, stream)
    return outputs


def quant_act(x: torch.Tensor, fmt=SCALE_FP32, stream=None):
    """E4M3 codes (uint8 [m,k]) and group scales ([ceil(k/128), m]) of x."""
    _check_cuda(x)
    _check_bf16_2d(x, "x")
    m, k = x.shape
    q = _out((m, k), torch.uint8, x.device)
    s = _out(((k + 127) // 128, m), _scale_dtype(fmt), x.device)
    fp8rl_quant_act_group(x, m, k, x.stride(0), q, k, s, fmt, stream)
    return q, s


def gemm_workspace(device=None) -> torch.Tensor:
    """A zero-filled workspace for fp8rl_gemm_blockscaled_ws on `device`."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        nbytes = fp8rl_gemm_workspace_size()
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def gemm(xq, x_scale, wq, w_scale, fmt=SCALE_FP32, out=None, stream=None, workspace=None):
    """bf16 Y [m, n] = block-scaled X W^T.  With a workspace (gemm_workspace),
    shapes that fill the SMs unevenly run the stream-K schedule."""
    _check_cuda(xq, x_scale, wq, w_scale, out, workspace)
    m, k = xq.shape
    n = wq.shape[0]
    if out is None:
        out = _out((m, n), torch.bfloat16, xq.device)
    if workspace is None:
        fp8rl_gemm_blockscaled(xq, x_scale, wq, w_scale, out, m, n, k, fmt, stream)
    else:
        fp8rl_gemm_blockscaled_ws(xq, x_scale, wq, w_scale, out, m, n, k, fmt, workspace,
                                  workspace.numel() * workspace.element_size(), stream)
    return out


def gemm_act_quant(x, wq, w_scale, fmt=SCALE_FP32, out=None, stream=None):
    """bf16 Y [m, n] = X W^T with X (bf16 [m, k]) quantised 1x128 on the way,
    plus the codes and scales (the results of quant_act(x) then gemm)."""
    _check_cuda(x, wq, w_scale, out)
    _check_bf16_2d(x, "x")
    m, k = x.shape
    n = wq.shape[0]
    if out is None:
        out = _out((m, n), torch.bfloat16, x.device)
    xq = _out((m, k), torch.uint8, x.device)
    sx = _out(((k + 127) // 128, m), _scale_dtype(fmt), x.device)
    fp8rl_gemm_act_quant(x, x.stride(0), wq, w_scale, out, m, n, k, fmt, xq, sx, stream)
    return out, xq, sx


def grouped_gemm(xq, x_scale, wq, w_scale, d_offsets, fmt=SCALE_FP32, out=None, stream=None):
    """bf16 Y [rows, n]: expert e's weights applied to its row segment."""
    _check_cuda(xq, x_scale, wq, w_scale, d_offsets, out)
    rows, k = xq.shape
    e, n, _ = wq.shape
    if out is None:
        out = _out((rows, n), torch.bfloat16, xq.device)
    fp8rl_grouped_gemm_blockscaled(xq, x_scale, wq, w_scale, d_offsets, e, rows, n, k, out, fmt,
                                   stream)
    return out


def quant_gate_up_interleaved(gate: torch.Tensor, up: torch.Tensor, fmt=SCALE_FP32, stream=None,
                              out=None):
    """Quantise a gate and an up weight ([..., inter, k] bf16, optionally with
    leading expert dimensions) straight into the interleaved fused layout that
    fp8rl_gemm_swiglu_quant consumes: 128-row blocks alternate gate, up.  One
    batched quantiser pass (one descriptor per 128-row block); returns
    (q [..., 2 * inter, k] uint8, scale [..., 2 * inter / 128, k / 128])."""
    _check_cuda(gate, up, *(out or ()))
    if gate.shape != up.shape or gate.dtype != torch.bfloat16 or up.dtype != torch.bfloat16:
        raise ValueError("gate and up must be bf16 tensors of one shape")
    *lead, inter, k = gate.shape
    if inter % 128 or k % 128:
        raise ValueError("inter and k must be multiples of 128")
    g2 = gate.reshape(-1, inter, k)
    u2 = up.reshape(-1, inter, k)
    if g2.stride(2) != 1 or u2.stride(2) != 1:
        raise ValueError("weights need unit column stride")
    experts = g2.shape[0]
    if out is None:
        q = _out((experts, 2 * inter, k), torch.uint8, gate.device)
        sc = _out((experts, 2 * inter // 128, k // 128), _scale_dtype(fmt), gate.device)
    else:
        q, sc = (t.view(experts, *t.shape[-2:]) for t in out)
    items = []
    for e in range(experts):
        for b in range(inter // 128):
            for half, src in ((0, g2[e]), (1, u2[e])):
                row = 256 * b + 128 * half
                items.append((src[128 * b:128 * b + 128], q[e, row:row + 128], sc[e, row // 128:row // 128 + 1]))
    for i in range(0, len(items), 256):
        chunk = items[i:i + 256]
        fp8rl_quant_weight_blockwise_batched(weight_descs(chunk), len(chunk), fmt, stream)
    return q.view(*lead, 2 * inter, k), sc.view(*lead, 2 * inter // 128, k // 128)


def gemm_swiglu_quant(xq, x_scale, wq_gate_up, w_scale_gate_up, fmt=SCALE_FP32, out=None, stream=None):
    """(hq [m, inter] uint8, h_scale [inter/128, m]) of SiLU(gate) * up."""
    _check_cuda(xq, x_scale, wq_gate_up, w_scale_gate_up, *(out or ()))
    m, k = xq.shape
    inter = wq_gate_up.shape[0] // 2
    if out is None:
        out = (_out((m, inter), torch.uint8, xq.device),
               _out((inter // 128, m), _scale_dtype(fmt), xq.device))
    fp8rl_gemm_swiglu_quant(xq, x_scale, wq_gate_up, w_scale_gate_up, m, inter, k, out[0], out[1], fmt, stream)
    return out


def grouped_gemm_swiglu_quant(xq, x_scale, wq_gate_up, w_scale_gate_up, d_offsets, fmt=SCALE_FP32, out=None,
                              stream=None):
    """Grouped (MoE) form of gemm_swiglu_quant."""
    _check_cuda(xq, x_scale, wq_gate_up, w_scale_gate_up, d_offsets, *(out or ()))
    rows, k = xq.shape
    e, n2, _ = wq_gate_up.shape
    inter = n2 // 2
    if out is None:
        out = (_out((rows, inter), torch.uint8, xq.device),
               _out((inter // 128, rows), _scale_dtype(fmt), xq.device))
    fp8rl_grouped_gemm_swiglu_quant(xq, x_scale, wq_gate_up, w_scale_gate_up, d_offsets, e, rows, inter, k,
                                    out[0], out[1], fmt, stream)
    return out


def kv_calibrate(k: torch.Tensor, v: torch.Tensor, q: torch.Tensor | None = None, out=None, stream=None):
    """Per-tensor fp32 scales (device float [3]: K, V, Q) of a calibration pass."""
    _check_cuda(k, v, q, out)
    for name, t in (("k", k), ("v", v)) + ((("q", q),) if q is not None else ()):
        _check_bf16_2d(t, name)
    scales = out
    if out is None:
        scales = _out((3,), torch.float32, k.device)
        with _on(stream, k.device):
            scales.zero_()
    tokens, dim = k.shape
    fp8rl_kv_calibrate(k, v, q, tokens, dim, k.stride(0), v.stride(0), 0 if q is None else q.shape[1],
                       0 if q is None else q.stride(0), scales, stream)
    return scales


def kv_append(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
              v_cache: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """Quantise rows of K and V into the E4M3 caches ([num_slots, kv_dim] uint8)."""
    _check_cuda(k, v, slot_mapping, k_cache, v_cache, scales)
    _check_bf16_2d(k, "k")
    _check_bf16_2d(v, "v")
    tokens, dim = k.shape
    fp8rl_kv_append(k, v, tokens, dim, k.stride(0), v.stride(0), slot_mapping, k_cache, v_cache,
                    k_cache.stride(0), k_cache.shape[0], scales, stream)


def moe_plan(topk: torch.Tensor, experts: int, workspace: torch.Tensor | None = None, stream=None):
    """Dispatch plan of replayed top-k indices (device int32 [T, k]): returns
    device int32 (offsets [E+1], row_of_pair [T*k], token_of_row [T*k])."""
    _check_cuda(topk, workspace)
    if topk.dtype != torch.int32 or topk.dim() != 2 or not topk.is_contiguous():
        raise ValueError("topk must be a contiguous int32 [tokens, k] tensor")
    tokens, k = topk.shape
    dev = topk.device
    need = fp8rl_moe_plan_workspace_size(tokens, k, experts)
    if workspace is None:
        with _on(stream, dev):
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    offsets = _out((experts + 1,), torch.int32, dev)
    row_of_pair = _out((tokens * k,), torch.int32, dev)
    token_of_row = _out((tokens * k,), torch.int32, dev)
    fp8rl_moe_plan(topk, tokens, k, experts, offsets, row_of_pair, token_of_row, workspace, workspace.numel(),
                   stream)
    return offsets, row_of_pair, token_of_row


def moe_dispatch_quant(x: torch.Tensor, row_of_pair: torch.Tensor, topk: int, fmt=SCALE_FP32, out=None,
                       stream=None):
    """The grouped activation of the dispatch: token t's 1x128 quantisation in
    rows row_of_pair[t * topk + j], (codes uint8 [R, K], scales [K/128, R]
    fp32 or uint8) with R = tokens * topk."""
    _check_cuda(x, row_of_pair, *(out or ()))
    _check_bf16_2d(x, "x")
    tokens, k = x.shape
    rows = row_of_pair.numel()
    if rows != tokens * topk:
        raise ValueError("row_of_pair must have tokens * topk entries")
    if out is None:
        q = _out((rows, k), torch.uint8, x.device)
        sdt = torch.float32 if fmt == SCALE_FP32 else torch.uint8
        s = _out(((k + 127) // 128, rows), sdt, x.device)
    else:
        q, s = out
    fp8rl_moe_dispatch_quant(x, tokens, k, x.stride(0), row_of_pair, topk, rows, q, q.stride(0), s, fmt, stream)
    return q, s


def moe_combine(y: torch.Tensor, row_of_pair: torch.Tensor, gate: torch.Tensor, out=None, stream=None):
    """bf16 [T, N]: each token's expert output rows weighted by its gates."""
    _check_cuda(y, row_of_pair, gate, out)
    _check_bf16_2d(y, "y")
    if gate.dtype != torch.float32 or gate.dim() != 2 or not gate.is_contiguous():
        raise ValueError("gate must be a contiguous fp32 [tokens, k] tensor")
    tokens, k = gate.shape
    n = y.shape[1]
    o = out if out is not None else _out((tokens, n), torch.bfloat16, y.device)
    fp8rl_moe_combine(y, y.shape[0], n, y.stride(0), row_of_pair, gate, tokens, k, o, o.stride(0), stream)
    return o


def tis_weights(lp_train: torch.Tensor, lp_rollout: torch.Tensor, mask: torch.Tensor | None = None,
                clip: float = 2.0, workspace: torch.Tensor | None = None, out=None, stream=None):
    """(w fp32 [n], kl fp64 [3] = mean, sum, count) on the device."""
    _check_cuda(lp_train, lp_rollout, mask, workspace, *(out or ()))
    for name, t in (("lp_train", lp_train), ("lp_rollout", lp_rollout)):
        if t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 tensor")
    if mask is not None and (mask.dtype != torch.uint8 or not mask.is_contiguous()):
        raise ValueError("mask must be a contiguous uint8 tensor")
    n = lp_train.numel()
    dev = lp_train.device
    need = fp8rl_tis_workspace_size(n)
    if workspace is None:
        with _on(stream, dev):
            workspace = torch.zeros(max(need, 32), dtype=torch.uint8, device=dev)  # header zeroed once
    w, kl = out if out is not None else (_out((n,), torch.float32, dev),
                                         _out((3,), torch.float64, dev))
    fp8rl_tis_weights(lp_train, lp_rollout, mask, n, clip, w, kl, workspace, workspace.numel(), stream)
    return w, kl


class _NoBackward(torch.autograd.Function):
    """Outputs of a call without a backward pass, tied to the inputs that require a
    gradient: a backward pass that reaches them ends in an error instead of in
    gradients that miss the call."""

    @staticmethod
    def forward(ctx, name, outputs, *inputs):
        ctx.name = name
        return tuple(t.detach() for t in outputs)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.name} has no backward pass; call it under torch.no_grad() or on detached tensors")


def rmsnorm_quant(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                  fmt=SCALE_FP32, out=None, stream=None):
    """(q uint8 [m, k], scale [ceil(k/128), m], h bf16 [m, k]): the RMS norm of
    h = x + residual times weight, quantised 1x128; h is None without a
    residual.  `out` is such a triple (its h may be the residual itself).  No
    backward pass: one that reaches h raises."""
    _check_cuda(x, weight, residual, *(out or ()))
    _check_bf16_2d(x, "x")
    m, k = x.shape
    if weight.dtype != torch.bfloat16 or weight.shape != (k,) or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous bf16 [k] tensor")
    if residual is not None:
        _check_bf16_2d(residual, "residual")
        if residual.shape != (m, k):
            raise ValueError("residual must have x's shape")
    if out is None:
        q, s, h = _outs((((m, k), torch.uint8), (((k + 127) // 128, m), _scale_dtype(fmt)),
                         None if residual is None else ((m, k), torch.bfloat16)), x.device)
        ldq = ldh = k
    else:
        q, s, h = out
        _check_out(q, (m, k), torch.uint8, "q", rows=True)
        _check_out(s, ((k + 127) // 128, m), _scale_dtype(fmt), "scale")
        if h is not None:
            _check_out(h, (m, k), torch.bfloat16, "h", rows=True)
        ldq, ldh = _ld(q, m, k), 0 if h is None else _ld(h, m, k)
    fp8rl_rmsnorm_quant(x.data_ptr(), _ld(x, m, k), residual, 0 if residual is None else _ld(residual, m, k),
                        weight.data_ptr(), eps, m, k, h, ldh, q.data_ptr(), ldq, s.data_ptr(), fmt, stream)
    if h is not None and torch.is_grad_enabled() and (x.requires_grad or (residual is not None and residual.requires_grad)):
        h, = _NoBackward.apply("rmsnorm_quant", (h,), x, residual)
    return q, s, h


def _ld(t: torch.Tensor, rows: int, cols: int) -> int:
    """Leading dimension in elements of [rows, cols...]: torch leaves the
    stride of a single row unspecified, so that one counts its columns."""
    return t.stride(0) if rows > 1 else cols


def _check_out(t: torch.Tensor, shape, dtype, name: str, rows=False):
    """A caller's output tensor: its shape and type, contiguous (or, with
    `rows`, of any row stride)."""
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}")
    if not t.is_contiguous() and not (rows and t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= t.shape[1]):
        raise ValueError(f"{name} must be contiguous" + (" in its rows" if rows else ""))


def _check_heads(t: torch.Tensor, name: str):
    """bf16 [tokens, heads, d] whose heads lie side by side (a column range of
    a wider projection output is fine)."""
    if t.dtype != torch.bfloat16 or t.dim() != 3:
        raise ValueError(f"{name} must be a bf16 [tokens, heads, head_dim] tensor")
    _, heads, d = t.shape
    _, by_head, by_column = t.stride()
    if (by_column != 1 and d > 1) or (by_head != d and heads > 1):
        raise ValueError(f"{name}: a token's heads must be contiguous")


class AttnPlan:
    """The work layout of attn_prefill for one set of packed sequences and
    heads (attn_prefill_plan): one per step, used by every layer."""

    def __init__(self, data, batch, total_tokens, q_heads, kv_heads):
        self.data, self.batch, self.total_tokens = data, batch, total_tokens
        self.q_heads, self.kv_heads = q_heads, kv_heads


def attn_prefill_plan(cu_seqlens: torch.Tensor, total_tokens: int, q_heads: int, kv_heads: int, stream=None) -> AttnPlan:
    """The plan of packed sequences: sequence b is tokens [cu_seqlens[b],
    cu_seqlens[b + 1]) (device int32 [batch + 1]) of total_tokens."""
    _check_cuda(cu_seqlens)
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous int32 [batch + 1] tensor")
    batch = cu_seqlens.numel() - 1
    nbytes = fp8rl_attn_prefill_plan_size(total_tokens, batch, q_heads, kv_heads)
    if nbytes == 0:
        raise ValueError("q_heads must be a multiple of kv_heads, at most 2^26 tokens and 2^20 sequences")
    data = _out((nbytes,), torch.uint8, cu_seqlens.device)
    fp8rl_attn_prefill_plan(cu_seqlens, batch, total_tokens, q_heads, kv_heads, data, nbytes, stream)
    return AttnPlan(data, batch, total_tokens, q_heads, kv_heads)


def attn_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, plan: AttnPlan, softmax_scale: float | None = None,
                 out=None, stream=None):
    """(out bf16 [tokens, q_heads, d], lse fp32 [tokens, q_heads]): causal
    attention over packed prompts (q [tokens, q_heads, d], k and v [tokens,
    kv_heads, d]; column ranges of one projection's output are fine).
    softmax_scale defaults to d ** -0.5.  No backward pass: one that reaches the
    outputs raises."""
    _check_cuda(q, k, v, plan.data, *(out or ()))
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_heads(t, name)
    tokens, hq, d = q.shape
    hkv = k.shape[1]
    if k.shape != (tokens, hkv, d) or v.shape != k.shape:
        raise ValueError("k and v must be [tokens, kv_heads, head_dim] with q's tokens and head_dim")
    if (plan.total_tokens, plan.q_heads, plan.kv_heads) != (tokens, hq, hkv):
        raise ValueError("the plan was made for other sizes")
    if out is None:
        out = tuple(_outs((((tokens, hq, d), torch.bfloat16), ((tokens, hq), torch.float32)), q.device))
    else:
        _check_out(out[0], (tokens, hq, d), torch.bfloat16, "out")
        _check_out(out[1], (tokens, hq), torch.float32, "lse")
    fp8rl_attn_prefill(q.data_ptr(), _ld(q, tokens, hq * d), k.data_ptr(), _ld(k, tokens, hkv * d), v.data_ptr(),
                       _ld(v, tokens, hkv * d), plan.data.data_ptr(), plan.data.numel(), plan.batch, tokens, hq, hkv, d,
                       d ** -0.5 if softmax_scale is None else softmax_scale, out[0].data_ptr(), hq * d,
                       out[1].data_ptr(), stream)
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad):
        out = _NoBackward.apply("attn_prefill", out, q, k, v)
    return out


def attn_decode_workspace(q_heads: int, kv_heads: int, head_dim: int, device=None) -> torch.Tensor:
    """A zero-filled workspace for attn_decode with these heads, any batch."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        nbytes = fp8rl_attn_decode_workspace_size(q_heads, kv_heads, head_dim)
    if nbytes == 0:
        raise ValueError("q_heads must be a multiple of kv_heads, head_dim 64 or 128")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def attn_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                lens: torch.Tensor, scales: torch.Tensor, block_size: int, softmax_scale: float | None = None,
                workspace: torch.Tensor | None = None, out=None, stream=None):
    """(out bf16 [batch, q_heads, d], lse fp32 [batch, q_heads]): attention of
    one token per sequence (q [batch, q_heads, d]) over the E4M3 caches
    ([num_slots, kv_heads * d] uint8, as kv_append writes them), the pages of
    sequence b in block_table[b] (int32 [batch, max_blocks]), its number of
    keys in lens[b] (int32).  softmax_scale defaults to d ** -0.5; keep one
    workspace per stream (attn_decode_workspace) rather than one per call.  No
    backward pass: one that reaches the outputs raises."""
    _check_cuda(q, k_cache, v_cache, block_table, lens, scales, workspace, *(out or ()))
    _check_heads(q, "q")
    batch, hq, d = q.shape
    slots, width = k_cache.shape
    ldc = _ld(k_cache, slots, width)
    if k_cache.dtype != torch.uint8 or v_cache.dtype != torch.uint8 or k_cache.stride(1) != 1 or v_cache.stride(1) != 1 or width % d:
        raise ValueError("the caches must be uint8 [num_slots, kv_heads * head_dim] tensors with unit column stride")
    if v_cache.shape != k_cache.shape or _ld(v_cache, slots, width) != ldc:
        raise ValueError("k_cache and v_cache must have one shape and stride")
    rows, blocks = block_table.shape
    if block_table.dtype != torch.int32 or rows != batch or (block_table.stride(1) != 1 and blocks > 1):
        raise ValueError("block_table must be an int32 [batch, max_blocks] tensor with unit column stride")
    if lens.dtype != torch.int32 or lens.shape != (batch,) or not lens.is_contiguous():
        raise ValueError("lens must be a contiguous int32 [batch] tensor")
    if scales.dtype != torch.float32 or scales.numel() < 2 or not scales.is_contiguous():
        raise ValueError("scales must hold the fp32 K and V scales")
    hkv = width // d
    if workspace is None:
        with _on(stream, q.device):
            workspace = attn_decode_workspace(hq, hkv, d, q.device)
    if out is None:
        out = tuple(_outs((((batch, hq, d), torch.bfloat16), ((batch, hq), torch.float32)), q.device))
    else:
        _check_out(out[0], (batch, hq, d), torch.bfloat16, "out")
        _check_out(out[1], (batch, hq), torch.float32, "lse")
    fp8rl_attn_decode(q.data_ptr(), _ld(q, batch, hq * d), batch, hq, hkv, d, k_cache.data_ptr(), v_cache.data_ptr(), ldc,
                      slots, block_table.data_ptr(), _ld(block_table, batch, blocks), blocks, block_size, lens.data_ptr(),
                      scales.data_ptr(), d ** -0.5 if softmax_scale is None else softmax_scale, out[0].data_ptr(), hq * d,
                      out[1].data_ptr(), workspace.data_ptr(), workspace.nbytes, stream)
    if torch.is_grad_enabled() and q.requires_grad:
        out = _NoBackward.apply("attn_decode", out, q)
    return out


def _check_logits(logits: torch.Tensor, tokens: torch.Tensor):
    if logits.dtype not in (torch.bfloat16, torch.float32) or logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be a 2-D bf16 or fp32 tensor with unit column stride")
    if tokens.dtype != torch.int32 or tokens.shape != logits.shape[:1] or not tokens.is_contiguous():
        raise ValueError("tokens must be a contiguous int32 [rows] tensor")


def logprobs(logits: torch.Tensor, tokens: torch.Tensor, temperature: float = 1.0, topk: int = 0, out=None, stream=None):
    """(lp fp32 [rows], entropy fp32 [rows], stats fp32 [rows, 2], top_ids
    int32 [rows, topk], top_lp fp32 [rows, topk]) of logits (bf16 or fp32
    [rows, vocab]) at a temperature; the last two are None with topk = 0.
    Rows whose token is outside the vocabulary (-1: padding) give zeros and
    ids -1.  stats is for logprobs_backward; lp goes to tis_weights.  With logits
    that require a gradient, lp and entropy have theirs (logprobs_backward, on the
    current stream of the backward pass); one that comes from stats or top_lp raises."""
    if torch.is_grad_enabled() and logits.requires_grad:
        return _LogProbs.apply(logits, tokens, temperature, topk, out, stream)
    return _logprobs(logits, tokens, temperature, topk, out, stream)


class _LogProbs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, temperature, topk, out, stream):
        lp, entropy, stats, ids, top_lp = (None if t is None else t.detach()
                                           for t in _logprobs(logits, tokens, temperature, topk, out, stream))
        ctx.save_for_backward(logits, tokens, stats, entropy)
        ctx.temperature = temperature
        ctx.set_materialize_grads(False)
        if ids is not None:
            ctx.mark_non_differentiable(ids)
        return lp, entropy, stats, ids, top_lp

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_lp, grad_entropy, grad_stats, _, grad_top_lp):
        if grad_stats is not None or grad_top_lp is not None:
            raise RuntimeError("logprobs has a backward pass from lp and entropy, not from stats or top_lp")
        if grad_lp is None and grad_entropy is None:
            return (None,) * 6
        logits, tokens, stats, entropy = ctx.saved_tensors
        grad_lp = torch.zeros_like(entropy) if grad_lp is None else grad_lp.contiguous()
        grad_entropy = None if grad_entropy is None else grad_entropy.contiguous()
        return (logprobs_backward(logits, tokens, stats, entropy, grad_lp, grad_entropy, ctx.temperature), *(None,) * 5)


def _logprobs(logits, tokens, temperature, topk, out, stream):
    _check_cuda(logits, tokens, *(out or ()))
    _check_logits(logits, tokens)
    rows, vocab = logits.shape
    specs = [((rows,), torch.float32), ((rows,), torch.float32), ((rows, 2), torch.float32)]
    if topk > 0:
        specs += [((rows, topk), torch.int32), ((rows, topk), torch.float32)]
    if out is None:
        out = _outs(specs, logits.device)
    else:
        if len(out) < len(specs):
            raise ValueError(f"out must hold {len(specs)} tensors")
        for t, (shape, dtype), name in zip(out, specs, ("lp", "entropy", "stats", "top_ids", "top_lp")):
            _check_out(t, shape, dtype, name)
    out = tuple(out) if topk > 0 else (*out[:3], None, None)
    fp8rl_logprob(logits, int(logits.dtype == torch.float32), rows, vocab, _ld(logits, rows, vocab), temperature, tokens, out[0],
                  out[1], out[2], topk, out[3], out[4], stream)
    return out


def logprobs_backward(logits: torch.Tensor, tokens: torch.Tensor, stats: torch.Tensor, entropy: torch.Tensor | None,
                      grad_lp: torch.Tensor, grad_entropy: torch.Tensor | None = None, temperature: float = 1.0,
                      out: torch.Tensor | None = None, stream=None):
    """d logits ([rows, vocab], the logits' type) from the gradients of lp and
    (optionally) entropy; `out` may be the logits tensor itself."""
    _check_cuda(logits, tokens, stats, entropy, grad_lp, grad_entropy, out)
    _check_logits(logits, tokens)
    rows, vocab = logits.shape
    _check_out(stats, (rows, 2), torch.float32, "stats")
    for name, t in (("entropy", entropy), ("grad_lp", grad_lp), ("grad_entropy", grad_entropy)):
        if t is not None:
            _check_out(t, (rows,), torch.float32, name)
    if grad_entropy is not None and entropy is None:
        raise ValueError("grad_entropy needs the forward call's entropy")
    if out is None:
        out = _out((rows, vocab), logits.dtype, logits.device)
    else:
        _check_out(out, (rows, vocab), logits.dtype, "out", rows=True)
    fp8rl_logprob_backward(logits, int(logits.dtype == torch.float32), rows, vocab, _ld(logits, rows, vocab), temperature,
                           tokens, stats, entropy, grad_lp, grad_entropy, out, _ld(out, rows, vocab), stream)
    return out


def sample(logits: torch.Tensor, uniform: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, out=None, stream=None):
    """(tokens int32, lp fp32, lp_kept fp32, kept int32, each [rows]): a token
    drawn from each row of logits (bf16 or fp32 [rows, vocab]) with the random
    numbers uniform (fp64 [rows], in [0, 1); another number, -1 say, marks a row
    without a draw: token -1, zeros).  temperature, top_p, min_p are numbers or fp32
    [rows] tensors, top_k a number or an int32 [rows] tensor; top_k 0, top_p 1 and
    min_p 0 cut nothing off, temperature 0 takes the most likely token.  lp is the
    token's log probability at the temperature (what logprobs gives it), lp_kept its
    log probability among the kept tokens.  No gradient comes from a draw: take lp's
    from logprobs."""
    if logits.dtype not in (torch.bfloat16, torch.float32) or logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be a 2-D bf16 or fp32 tensor with unit column stride")
    rows, vocab = logits.shape
    values, arrays = [temperature, top_k, top_p, min_p], [None] * 4
    for i, v in enumerate(values):
        if isinstance(v, torch.Tensor):
            dtype = torch.int32 if i == 1 else torch.float32
            if v.dtype != dtype or v.shape != (rows,) or not v.is_contiguous():
                raise ValueError(f"{('temperature', 'top_k', 'top_p', 'min_p')[i]} must be a number or a contiguous {dtype} [rows] tensor")
            values[i], arrays[i] = 1, v
    _check_cuda(logits, uniform, *arrays, *(out or ()))
    if uniform.dtype != torch.float64 or uniform.shape != (rows,) or not uniform.is_contiguous():
        raise ValueError("uniform must be a contiguous fp64 [rows] tensor")
    specs = (((rows,), torch.int32), ((rows,), torch.float32), ((rows,), torch.float32), ((rows,), torch.int32))
    if out is None:
        out = tuple(_outs(specs, logits.device))
    else:
        if len(out) != 4:
            raise ValueError("out must hold 4 tensors")
        for t, (shape, dtype), name in zip(out, specs, ("tokens", "lp", "lp_kept", "kept")):
            _check_out(t, shape, dtype, name)
    fp8rl_sample(logits.data_ptr(), int(logits.dtype == torch.float32), rows, vocab, _ld(logits, rows, vocab), uniform.data_ptr(),
                 *values, *arrays, *out, stream)
    if torch.is_grad_enabled() and logits.requires_grad:
        out = (out[0], *_NoBackward.apply("sample", out[1:3], logits), out[3])
    return out


class RotaryFreqs:
    """The frequencies of rotary positions, laid out for the kernels (rotary_freqs):
    one per model."""

    def __init__(self, data, rotary_dim, axes):
        self.data, self.rotary_dim, self.axes = data, rotary_dim, axes


@functools.lru_cache(maxsize=None)
def _pi(bits: int) -> int:
    """pi in units of 2^-bits, off by less than one of them (Machin's formula, in integers)."""
    def arctan_of_one_over(n):
        term = total = (1 << bits + 32) // n
        k = 1
        while term:
            term //= -n * n  # (rounds down: off by a unit a term at most)
            k += 2
            total += term // k
        return total
    return 4 * (4 * arctan_of_one_over(5) - arctan_of_one_over(239)) >> 32


def _turns(f: float) -> int:
    """f / (2 pi) in units of 2^-64, to the nearest: from f's own digits and as many of
    pi (the fp64 quotient is off by 2^-54 of a turn, 2^-23 at position 2^31)."""
    n, d = f.as_integer_ratio()
    bits = 128 + max(0, n.bit_length() - d.bit_length())
    n, d = n << 64 + bits, d * 2 * _pi(bits)
    return (2 * n + d) // (2 * d)


def rotary_freqs(rotary_dim: int, theta: float = 10000.0, sections=None, inv_freq=None, axis=None, device=None) -> RotaryFreqs:
    """Frequencies of rotary_dim // 2 pairs: theta ** (-2 i / rotary_dim) radians a
    position (in fp64), or the given ones (inv_freq: numbers, fp64 where they are exact,
    for scaled positions).  With several axes, sections is how many pairs each takes, one
    after the other ((16, 24, 24): time, height, width), or axis each pair's own
    (any order)."""
    if rotary_dim < 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even")
    pairs = rotary_dim // 2
    if inv_freq is None:
        if not theta > 0:
            raise ValueError("theta must be positive")
        inv_freq = [theta ** (-i / pairs) for i in range(pairs)]
    else:
        inv_freq = [float(f) for f in inv_freq]
    if sections is not None and axis is not None:
        raise ValueError("sections or axis, not both")
    if sections is not None:
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
    axis = [0] * pairs if axis is None else [int(a) for a in axis]
    if len(inv_freq) != pairs or len(axis) != pairs or any(a < 0 for a in axis) or not all(map(math.isfinite, inv_freq)):
        raise ValueError("one finite frequency and one axis for each of the rotary_dim // 2 pairs")
    axes = len(sections) if sections is not None else max(axis, default=0) + 1
    turns = [(_turns(float(f)) + (1 << 63)) % (1 << 64) - (1 << 63) for f in inv_freq]  # as signed words
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return RotaryFreqs(torch.tensor([turns, axis], dtype=torch.int64).to(device), rotary_dim, axes)


def _rotary_args(q, k, positions, freqs):
    """(tokens, q_heads, kv_heads, head_dim, positions [axes, tokens])."""
    _check_heads(q, "q")
    if k is not None:
        _check_heads(k, "k")
        if k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
            raise ValueError("k must be [tokens, kv_heads, head_dim] with q's tokens and head_dim")
    tokens, hq, d = q.shape
    if positions.dim() == 1:
        positions = positions[None]
    if positions.dtype != torch.int32 or positions.shape != (freqs.axes, tokens) or (positions.stride(1) != 1 and tokens > 1):
        raise ValueError("positions must be an int32 [tokens] or [axes, tokens] tensor with the frequencies' axes and unit column stride")
    if freqs.rotary_dim > d:
        raise ValueError("rotary_dim must not exceed head_dim")
    return tokens, hq, 0 if k is None else k.shape[1], d, positions


def _row_ld(t, tokens, width):
    """The row stride of [tokens, heads, d] (a tensor without elements has none that counts)."""
    return t.stride(0) if t is not None and tokens > 1 and width else width


def rotary(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, freqs: RotaryFreqs, interleaved: bool = False,
           inverse: bool = False, out=None, stream=None):
    """(q, k) turned by their positions: q [tokens, q_heads, d] and k [tokens,
    kv_heads, d] (bf16; column ranges of one projection's output are fine; k may be
    None), positions int32 [tokens], or [axes, tokens] for frequencies of several
    axes (one row expanded over them, too).  `out` is such a pair and may be (q, k) itself.  inverse=True turns back,
    which is the backward pass; with q or k that require a gradient it runs under
    autograd (on the current stream of the backward pass)."""
    if torch.is_grad_enabled() and (q.requires_grad or (k is not None and k.requires_grad)):
        if out is not None:
            raise ValueError("rotary with a gradient allocates its outputs")
        return _Rotary.apply(q, k, positions, freqs, interleaved, inverse, stream)
    return _rotary(q, k, positions, freqs, interleaved, inverse, out, stream)


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, freqs, interleaved, inverse, stream):
        ctx.save_for_backward(positions, freqs.data)
        ctx.plan = (freqs.rotary_dim, freqs.axes, interleaved, inverse)
        ctx.set_materialize_grads(False)
        return _rotary(q.detach(), None if k is None else k.detach(), positions, freqs, interleaved, inverse, None, stream)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_q, grad_k):
        positions, data = ctx.saved_tensors
        rotary_dim, axes, interleaved, inverse = ctx.plan
        freqs = RotaryFreqs(data, rotary_dim, axes)
        grads = [None if g is None else _heads_of(g) for g in (grad_q, grad_k)]
        if grads[0] is not None:
            grads = _rotary(grads[0], grads[1], positions, freqs, interleaved, not inverse, None, None)
        elif grads[1] is not None:
            grads = (None, _rotary(grads[1], None, positions, freqs, interleaved, not inverse, None, None)[0])
        return (*grads, None, None, None, None, None)


def _heads_of(g):
    """A gradient as the kernels read heads: as it lies, or copied."""
    _, heads, d = g.shape
    _, by_head, by_column = g.stride()
    return g if (by_column == 1 or d <= 1) and (by_head == d or heads <= 1) and (g.stride(0) >= heads * d or g.shape[0] <= 1) else g.contiguous()


def _rotary(q, k, positions, freqs, interleaved, inverse, out, stream):
    _check_cuda(q, k, positions, freqs.data, *(out or ()))
    tokens, hq, hkv, d, positions = _rotary_args(q, k, positions, freqs)
    if out is None:
        q_out, k_out = _outs((((tokens, hq, d), torch.bfloat16), None if k is None else ((tokens, hkv, d), torch.bfloat16)), q.device)
    else:
        q_out, k_out = out
        for name, t, like in (("out[0]", q_out, q), ("out[1]", k_out, k)):
            if (t is None) != (like is None):
                raise ValueError("out must be a pair like (q, k)")
            if t is not None:
                _check_heads(t, name)
                if t.shape != like.shape:
                    raise ValueError(f"{name} must have its input's shape")
    fp8rl_rotary(q.data_ptr(), _row_ld(q, tokens, hq * d), hq, k, _row_ld(k, tokens, hkv * d), hkv, tokens, d, freqs.data.data_ptr(),
                 freqs.rotary_dim // 2, positions.data_ptr(), _row_ld(positions, freqs.axes, tokens), freqs.axes, int(interleaved),
                 int(inverse), q_out.data_ptr(), _row_ld(q_out, tokens, hq * d), k_out, _row_ld(k_out, tokens, hkv * d), stream)
    return q_out, k_out


def rotary_kv_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, freqs: RotaryFreqs,
                     slot_mapping: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, scales: torch.Tensor,
                     interleaved: bool = False, keys: bool = False, out=None, stream=None):
    """rotary of q and k with kv_append of the turned keys and of v, in one launch:
    (q [tokens, q_heads, d], turned k or None).  The caches ([num_slots, kv_heads *
    d] uint8) get the codes in rows slot_mapping (int32 [tokens]; a slot outside the
    cache, -1 for padding, is skipped).  keys=True gives the turned keys in bf16 as
    well (attention over the prompt itself).  `out` is such a pair and may be (q,
    k).  No backward pass: one that reaches the outputs raises."""
    _check_cuda(q, k, v, positions, freqs.data, slot_mapping, k_cache, v_cache, scales, *(out or ()))
    tokens, hq, hkv, d, positions = _rotary_args(q, k, positions, freqs)
    _check_heads(v, "v")
    if v.shape != k.shape:
        raise ValueError("v must have k's shape")
    slots, width = k_cache.shape
    ldc = _ld(k_cache, slots, width)
    if k_cache.dtype != torch.uint8 or v_cache.dtype != torch.uint8 or k_cache.stride(1) != 1 or v_cache.stride(1) != 1 or width != hkv * d:
        raise ValueError("the caches must be uint8 [num_slots, kv_heads * head_dim] tensors with unit column stride")
    if v_cache.shape != k_cache.shape or _ld(v_cache, slots, width) != ldc:
        raise ValueError("k_cache and v_cache must have one shape and stride")
    if slot_mapping.dtype != torch.int32 or slot_mapping.shape != (tokens,) or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be a contiguous int32 [tokens] tensor")
    if scales.dtype != torch.float32 or scales.numel() < 2 or not scales.is_contiguous():
        raise ValueError("scales must hold the fp32 K and V scales")
    if out is None:
        q_out, k_out = _outs((((tokens, hq, d), torch.bfloat16), ((tokens, hkv, d), torch.bfloat16) if keys else None), q.device)
    else:
        q_out, k_out = out
        for name, t, like in (("out[0]", q_out, q), ("out[1]", k_out, k)):
            if t is None and like is k:
                continue
            _check_heads(t, name)
            if t.shape != like.shape:
                raise ValueError(f"{name} must have its input's shape")
    fp8rl_rotary_kv_append(q.data_ptr(), _row_ld(q, tokens, hq * d), hq, k.data_ptr(), _row_ld(k, tokens, hkv * d), v.data_ptr(),
                           _row_ld(v, tokens, hkv * d), hkv, tokens, d, freqs.data.data_ptr(), freqs.rotary_dim // 2,
                           positions.data_ptr(), _row_ld(positions, freqs.axes, tokens), freqs.axes, int(interleaved),
                           q_out.data_ptr(), _row_ld(q_out, tokens, hq * d), k_out, _row_ld(k_out, tokens, hkv * d),
                           slot_mapping.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), ldc, slots, scales.data_ptr(), stream)
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad):
        if k_out is None:
            q_out, = _NoBackward.apply("rotary_kv_append", (q_out,), q, k, v)
        else:
            q_out, k_out = _NoBackward.apply("rotary_kv_append", (q_out, k_out), q, k, v)
    return q_out, k_out


class KvCaches:
    """The caches that share one table of pages (K and V of every layer, each uint8
    [num_slots, width] of one shape and stride), listed once for kv_reserve and
    kv_compact."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        for t in self.tensors:
            if t.dtype != torch.uint8 or t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
                raise ValueError("the caches must be uint8 [num_slots, width] tensors with unit column stride")
        first = self.tensors[0] if self.tensors else None
        self.slots, self.width = first.shape if self.tensors else (None, 0)
        self.ld = _ld(first, self.slots, self.width) if self.tensors else 0
        if any(t.shape != first.shape or _ld(t, *t.shape) != self.ld or t.device != first.device for t in self.tensors):
            raise ValueError("the caches must have one shape, stride and device")
        self.pointers = (ctypes.c_void_p * max(1, len(self.tensors)))(*(t.data_ptr() for t in self.tensors))


@functools.lru_cache(maxsize=256)
def _page_workspace(rows, total_tokens, block_size, pages):
    """Workspace bytes of kv_reserve (pages None) or kv_compact."""
    return max(64, fp8rl_kv_reserve_workspace_size(rows, total_tokens, block_size) if pages is None else
               fp8rl_kv_compact_workspace_size(pages))


def _workspace(nbytes, device, stream):
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with _on(stream, device):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _page_args(block_table, lens, refs, block_size, caches, *more):
    """The caches' handle and sizes: (caches, rows, max_blocks, ldt, pages)."""
    if not isinstance(caches, KvCaches):
        caches = KvCaches(caches)
    _check_cuda(block_table, lens, refs, *caches.tensors[:1], *more)
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or (block_table.stride(1) != 1 and block_table.shape[1] > 1):
        raise ValueError("block_table must be an int32 [rows, max_blocks] tensor with unit column stride")
    rows, blocks = block_table.shape
    if lens.dtype != torch.int32 or lens.shape != (rows,) or not lens.is_contiguous():
        raise ValueError("lens must be a contiguous int32 [rows] tensor")
    if refs.dtype != torch.int32 or refs.dim() != 1 or not refs.is_contiguous():
        raise ValueError("refs must be a contiguous int32 [pages] tensor")
    pages = refs.numel()
    if caches.slots is not None and pages * block_size > caches.slots:
        raise ValueError("the caches must hold every page: pages * block_size rows")
    return caches, rows, blocks, _ld(block_table, rows, blocks), pages


def kv_reserve(block_table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, block_size: int, caches=(), count=None,
               cu_seqlens=None, total_tokens: int | None = None, workspace: torch.Tensor | None = None, out=None, stream=None):
    """(slots int32, info int32 [2]): room for new tokens in the rows of a paged
    cache; block_table (int32 [rows, max_blocks]), lens (int32 [rows]) and refs (int32
    [pages]: rows that hold each page) are updated.  slots are the cache rows of the
    new tokens, for kv_append or rotary_kv_append.  Decode: a token for each row (slots
    [rows]), with count (int32 [rows], 0 or 1) for some; prompts: row r's new tokens
    are cu_seqlens[r] .. cu_seqlens[r + 1] of total_tokens (slots [total_tokens]).
    Entries that a row does not ask for are -1, and so are those of a row that is
    refused (pages run out, or its table is full; it stays as it was) and, of a padded
    batch, those of no row (in slots of `out` these stay as they were).  info: pages
    free after the call, rows refused.  A last page that other rows hold too is
    copied first, in all `caches` (KvCaches, or a list of tensors)."""
    caches, rows, blocks, ldt, pages = _page_args(block_table, lens, refs, block_size, caches, count, cu_seqlens, workspace, *(out or ()))
    if count is not None and (count.dtype != torch.int32 or count.shape != (rows,) or not count.is_contiguous()):
        raise ValueError("count must be a contiguous int32 [rows] tensor")
    if cu_seqlens is None:
        total_tokens = rows if total_tokens is None else total_tokens
    elif cu_seqlens.dtype != torch.int32 or cu_seqlens.shape != (rows + 1,) or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous int32 [rows + 1] tensor")
    elif total_tokens is None:
        raise ValueError("cu_seqlens needs total_tokens")
    if workspace is None:
        workspace = _workspace(_page_workspace(rows, total_tokens, block_size, None), refs.device, stream)
    if out is None:
        out = tuple(_outs((((total_tokens,), torch.int32), ((2,), torch.int32)), refs.device))
        if cu_seqlens is not None:  # (the kernel leaves entries of no row as they are; no append may take them for slots)
            with _on(stream, refs.device):
                out[0].fill_(-1)
    else:
        _check_out(out[0], (total_tokens,), torch.int32, "slots")
        _check_out(out[1], (2,), torch.int32, "info")
    fp8rl_kv_reserve(block_table.data_ptr(), ldt, rows, blocks, block_size, lens.data_ptr(), refs.data_ptr(), pages, cu_seqlens, count,
                     total_tokens, out[0].data_ptr(), out[1].data_ptr(), caches.pointers, len(caches.tensors), caches.width, caches.ld,
                     workspace.data_ptr(), workspace.nbytes, stream)
    if rows == 0:  # (that launches nothing: info is a row's without a table or tokens, whatever its length)
        workspace = _workspace(_page_workspace(1, 0, block_size, None), refs.device, stream)
        fp8rl_kv_reserve(None, 0, 1, 0, block_size, out[1].data_ptr(), refs.data_ptr(), pages, None, None, 0, None, out[1].data_ptr(),
                         None, 0, 0, 0, workspace.data_ptr(), workspace.nbytes, stream)
    return out


def kv_fork(block_table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, parent: torch.Tensor, block_size: int, out=None,
            stream=None):
    """(block_table int32 [n, max_blocks], lens int32 [n]): row i holds, shared, the
    pages of old row parent[i] (int32 [n]); -1 gives an empty row.  The old rows give
    up theirs (refs is updated): one call forks prompts, frees rows that have ended
    and reorders the others.  `out` may be (block_table, lens) itself; then a row
    with parent[i] != i takes its pages from a row that stays (parent[p] == p), or is
    empty."""
    _, rows, blocks, ldt, pages = _page_args(block_table, lens, refs, block_size, _NO_CACHES, parent, *(out or ()))
    if parent.dtype != torch.int32 or parent.dim() != 1 or not parent.is_contiguous():
        raise ValueError("parent must be a contiguous int32 [rows] tensor")
    n = parent.numel()
    if out is None:
        out = tuple(_outs((((n, blocks), torch.int32), ((n,), torch.int32)), refs.device))
    else:
        _check_out(out[0], (n, blocks), torch.int32, "block_table", rows=True)
        _check_out(out[1], (n,), torch.int32, "lens")
    fp8rl_kv_fork(block_table.data_ptr(), ldt, rows, blocks, block_size, lens.data_ptr(), parent.data_ptr(), n, out[0].data_ptr(),
                  _ld(out[0], n, blocks), out[1].data_ptr(), refs.data_ptr(), pages, stream)
    return out


def kv_compact(block_table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, block_size: int, caches,
               workspace: torch.Tensor | None = None, out=None, stream=None):
    """int32 [1], the number n of pages in use: the used pages move to numbers below
    n, contents (in all `caches`), refs and block_table with them, so that the caches'
    rows from n * block_size on are free for something else."""
    caches, rows, blocks, ldt, pages = _page_args(block_table, lens, refs, block_size, caches, workspace, out)
    if workspace is None:
        workspace = _workspace(_page_workspace(0, 0, block_size, pages), refs.device, stream)
    if out is None:
        out = _out((1,), torch.int32, refs.device)
    else:
        _check_out(out, (1,), torch.int32, "out")
    fp8rl_kv_compact(block_table.data_ptr(), ldt, rows, blocks, block_size, lens.data_ptr(), refs.data_ptr(), pages, out.data_ptr(),
                     caches.pointers, len(caches.tensors), caches.width, caches.ld, workspace.data_ptr(), workspace.nbytes, stream)
    return out


_NO_CACHES = KvCaches(())


class HostWeightSync:
    """Weight sync from host memory: bf16 weights in pinned host buffers are
    quantised (128x128 blocks) into E4M3 codes and scales in pinned host
    buffers.

    Pipelined (default): one call of ``fp8rl_quant_weight_host_batched``, the
    library's copy-in / quantise / copy-out pipeline over chunks of whole
    128-row block rows; the device staging (``slots`` slots of about
    ``chunk_bytes`` of bf16 each) is allocated once, at construction.
    Direct: the quantiser itself reads the pinned bf16 weights and writes the
    codes and scales in host memory over the CPU-GPU link (one batched launch
    of ``fp8rl_quant_weight_blockwise_batched``, no staging).  ``run()`` only
    enqueues work on the current stream; the caller synchronises."""

    def __init__(self, host_weights, host_codes, host_scales, fmt=SCALE_FP32, chunk_bytes=32 << 20,
                 slots=3, device=None, direct=False):
        device = torch.device(device or "cuda")
        self.fmt = fmt
        self.direct = direct
        self.h2d_bytes = sum(w.numel() * 2 for w in host_weights)
        self.d2h_bytes = sum(q.numel() + s.numel() * s.element_size() for q, s in zip(host_codes, host_scales))
        for t in list(host_weights) + list(host_codes) + list(host_scales):
            if t.is_cuda:
                raise ValueError("HostWeightSync takes host tensors")
            if direct and not t.is_pinned():
                raise ValueError("direct mode needs pinned host tensors")
        self._keep = (list(host_weights), list(host_codes), list(host_scales))
        self.descs = weight_descs(list(zip(host_weights, host_codes, host_scales)))
        self.count = len(host_weights)
        if direct:
            return
        self.slots = slots
        need = 0
        for w in host_weights:
            n, k = w.shape
            if n == 0 or k == 0:
                continue
            rows = min(n, max(128, (chunk_bytes // (2 * k)) // 128 * 128))
            need = max(need, fp8rl_host_sync_staging_bytes(rows, k, slots, fmt))
        self.staging = torch.empty(max(need, 256), dtype=torch.uint8, device=device)

    def run(self):
        """Enqueue one full weight sync; returns immediately (the caller syncs)."""
        if self.direct:
            fp8rl_quant_weight_blockwise_batched(self.descs, self.count, self.fmt)
            return
        fp8rl_quant_weight_host_batched(self.descs, self.count, self.fmt, self.staging, self.staging.numel(),
                                        self.slots)
