"""ctypes binding of the C ABI in ``include/qat_attn.h`` (argument marshalling only).

Every function has the C name and argument order.  Tensor arguments may be torch
tensors (their ``data_ptr()`` is passed) or raw integer addresses; ``stream`` may be a
``torch.cuda.Stream``, a raw handle, or ``None`` for torch's current stream on the
current device.  Functions return the ``qat_status_t`` value as a ``Status``.
No computation happens here: the library's kernels do all of it, and a missing
library is an error, never a fallback.
"""

from __future__ import annotations

import ctypes
import enum
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqat_attn.so")

# Every symbol include/qat_attn.h declares (checked by the CPU test suite).
EXPORTED = (
    "qat_attn_fwd",
    "qat_attn_bwd_workspace_bytes",
    "qat_attn_bwd",
    "qat_attn_bwd_noalloc",
    "qat_status_string",
    "qat_attn_device_status",
    "qat_debug_quant_tiles",
    "qat_debug_wait_timeout",
    "qat_channel_mean",
    "qat_fake_quant_tokens",
    "qat_attn_fwd_chunk",
    "qat_attn_merge",
    "qat_attn_bwd_smooth_k",
    "qat_subtract_mean",
    "qat_debug_set_wait_limit_us",
    "qat_qk_norm_rope",
    "qat_qk_norm_rope_bwd_workspace_bytes",
    "qat_qk_norm_rope_bwd",
    "qat_kv_cache_append",
    "qat_kv_cache_read",
    "qat_attn_decode_workspace_bytes",
    "qat_attn_decode",
)


class Status(enum.IntEnum):
    OK = 0
    INVALID_ARG = 1
    UNSUPPORTED = 2
    CUDA = 3
    TIMEOUT = 4
    WORKSPACE = 5
    BAD_PAGE = 6


QUANT_NONE = 0
QUANT_P_FP8E4M3_ROW_TILE64 = 1
QUANT_P_FP8E4M3_ROW_TILE64_PAGE_BWD = 2


_OK = Status.OK


def _status(code: int) -> Status:
    return _OK if code == 0 else Status(code)


class QatError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = Status(status)
        super().__init__(f"{what}: {qat_status_string(status)}" if what else qat_status_string(status))


_lib = None
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_ll = ctypes.c_longlong
_ll3 = _ll * 3


def lib() -> ctypes.CDLL:
    """The loaded library (loaded once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it first "
                "(python -m quantization_aware_attention_gb300.build)")
        L = ctypes.CDLL(LIB_PATH)
        L.qat_attn_fwd.argtypes = [_vp] * 6 + [_i] * 5 + [_f, _i, _i, _vp]
        L.qat_attn_fwd.restype = _i
        L.qat_attn_bwd_workspace_bytes.argtypes = [_i] * 5
        L.qat_attn_bwd_workspace_bytes.restype = _sz
        L.qat_attn_bwd.argtypes = [_vp] * 9 + [_i] * 5 + [_f, _i, _i, _vp, _sz, _vp]
        L.qat_attn_bwd.restype = _i
        L.qat_attn_bwd_noalloc.argtypes = [_vp] * 9 + [_i] * 5 + [_f, _i, _i, _vp]
        L.qat_attn_bwd_noalloc.restype = _i
        L.qat_status_string.argtypes = [_i]
        L.qat_status_string.restype = ctypes.c_char_p
        L.qat_attn_device_status.argtypes = [_vp]
        L.qat_attn_device_status.restype = _i
        L.qat_debug_quant_tiles.argtypes = [_vp, _i, _i, _vp, _vp, _vp, _vp]
        L.qat_debug_quant_tiles.restype = _i
        L.qat_debug_wait_timeout.argtypes = [_i, _vp]
        L.qat_debug_wait_timeout.restype = _i
        L.qat_channel_mean.argtypes = [_vp, _vp] + [_i] * 4 + [_vp]
        L.qat_channel_mean.restype = _i
        L.qat_fake_quant_tokens.argtypes = [_vp] * 4 + [_i] * 4 + [_vp]
        L.qat_fake_quant_tokens.restype = _i
        L.qat_attn_fwd_chunk.argtypes = [_vp] * 6 + [_i] * 7 + [_f, _i, _vp]
        L.qat_attn_fwd_chunk.restype = _i
        L.qat_attn_merge.argtypes = [_vp] * 8 + [_i] * 4 + [_vp]
        L.qat_attn_merge.restype = _i
        L.qat_attn_bwd_smooth_k.argtypes = [_vp] * 10 + [_i] * 5 + [_f, _i, _i, _vp, _sz, _vp]
        L.qat_attn_bwd_smooth_k.restype = _i
        L.qat_subtract_mean.argtypes = [_vp] * 3 + [_i] * 4 + [_vp]
        L.qat_subtract_mean.restype = _i
        L.qat_debug_set_wait_limit_us.argtypes = [_i, _vp]
        L.qat_debug_set_wait_limit_us.restype = _i
        L.qat_qk_norm_rope.argtypes = [_vp] * 7 + [_ll] + [_vp] * 3 + [_i] * 8 + [_f, _f, _vp]
        L.qat_qk_norm_rope.restype = _i
        L.qat_qk_norm_rope_bwd_workspace_bytes.argtypes = [_i]
        L.qat_qk_norm_rope_bwd_workspace_bytes.restype = _sz
        L.qat_qk_norm_rope_bwd.argtypes = ([_vp] * 9 + [_ll] + [_vp] * 3 + [_i] + [_vp] * 6 + [_i] * 7
                                           + [_f, _f, _vp, _sz, _vp])
        L.qat_qk_norm_rope_bwd.restype = _i
        L.qat_kv_cache_append.argtypes = [_vp] * 11 + [_i] * 7 + [_vp]
        L.qat_kv_cache_append.restype = _i
        L.qat_kv_cache_read.argtypes = [_vp] * 8 + [_i] * 8 + [_vp]
        L.qat_kv_cache_read.restype = _i
        L.qat_attn_decode_workspace_bytes.argtypes = [_i] * 4
        L.qat_attn_decode_workspace_bytes.restype = _sz
        L.qat_attn_decode.argtypes = [_vp] * 9 + [_i] * 8 + [_f, _i, _vp, _sz, _vp]
        L.qat_attn_decode.restype = _i
        _lib = L
    return _lib


_ops = None


def torch_ops():
    """The torch extension over the library (loaded once).  Raises if it has not been built."""
    global _ops
    if _ops is None:
        lib()
        try:
            from . import _qat_torch
        except ImportError as e:
            raise RuntimeError("the torch extension is missing or does not load: build it first "
                               f"(python -m quantization_aware_attention_gb300.build): {e}") from e
        _ops = _qat_torch
    return _ops


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_raw_stream = None


def _stream(s) -> int | None:
    if s is None:
        global _raw_stream
        import torch
        if _raw_stream is None:  # the handle without the Stream object around it, where torch has it
            torch.cuda.current_stream()
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda device: torch.cuda.current_stream(device).cuda_stream)
        return _raw_stream(torch.cuda.current_device())
    if isinstance(s, int):
        return s
    return s.cuda_stream


def qat_status_string(status: int) -> str:
    return lib().qat_status_string(int(status)).decode()


def qat_attn_fwd(q, k, v, o_q, o_hp, lse, B, H, Nq, Nkv, D, sm_scale, causal, quant_mode,
                 stream=None) -> Status:
    return Status(lib().qat_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o_q), _ptr(o_hp), _ptr(lse),
                                     B, H, Nq, Nkv, D, float(sm_scale), int(causal),
                                     int(quant_mode), _stream(stream)))


def qat_attn_bwd_workspace_bytes(B, H, Nq, Nkv, D) -> int:
    return int(lib().qat_attn_bwd_workspace_bytes(B, H, Nq, Nkv, D))


def qat_attn_bwd(q, k, v, o_hp, lse, dO, dq, dk, dv, B, H, Nq, Nkv, D, sm_scale, causal,
                 quant_mode, workspace, workspace_bytes, stream=None) -> Status:
    return Status(lib().qat_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o_hp), _ptr(lse), _ptr(dO),
                                     _ptr(dq), _ptr(dk), _ptr(dv), B, H, Nq, Nkv, D,
                                     float(sm_scale), int(causal), int(quant_mode),
                                     _ptr(workspace), int(workspace_bytes), _stream(stream)))


def qat_attn_bwd_noalloc(q, k, v, o_hp, lse, dO, dq, dk, dv, B, H, Nq, Nkv, D, sm_scale, causal,
                         quant_mode, stream=None) -> Status:
    return Status(lib().qat_attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o_hp), _ptr(lse),
                                             _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv), B, H, Nq,
                                             Nkv, D, float(sm_scale), int(causal),
                                             int(quant_mode), _stream(stream)))


def qat_attn_bwd_smooth_k(q, k, v, o_hp, lse, dO, dq, dk, dv, k_mean, B, H, Nq, Nkv, D, sm_scale,
                          causal, quant_mode, workspace, workspace_bytes, stream=None) -> Status:
    return Status(lib().qat_attn_bwd_smooth_k(_ptr(q), _ptr(k), _ptr(v), _ptr(o_hp), _ptr(lse),
                                              _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv),
                                              _ptr(k_mean), B, H, Nq, Nkv, D, float(sm_scale),
                                              int(causal), int(quant_mode), _ptr(workspace),
                                              int(workspace_bytes), _stream(stream)))


def qat_subtract_mean(x, mean, out, B, H, N, D, stream=None) -> Status:
    return Status(lib().qat_subtract_mean(_ptr(x), _ptr(mean), _ptr(out), B, H, N, D,
                                          _stream(stream)))


def qat_debug_set_wait_limit_us(limit_us, stream=None) -> Status:
    return Status(lib().qat_debug_set_wait_limit_us(int(limit_us), _stream(stream)))


def qat_attn_device_status(stream=None) -> Status:
    return Status(lib().qat_attn_device_status(_stream(stream)))


def qat_debug_wait_timeout(limit_ms, stream=None) -> Status:
    return Status(lib().qat_debug_wait_timeout(limit_ms, _stream(stream)))


def qat_debug_quant_tiles(p, rows, cols, deq, scales, codes, stream=None) -> Status:
    return Status(lib().qat_debug_quant_tiles(_ptr(p), rows, cols, _ptr(deq), _ptr(scales),
                                              _ptr(codes), _stream(stream)))


def qat_channel_mean(x, mean, B, H, N, D, stream=None) -> Status:
    return Status(lib().qat_channel_mean(_ptr(x), _ptr(mean), B, H, N, D, _stream(stream)))


def qat_fake_quant_tokens(x, mean, out, scales, B, H, N, D, stream=None) -> Status:
    return Status(lib().qat_fake_quant_tokens(_ptr(x), _ptr(mean), _ptr(out), _ptr(scales), B, H,
                                              N, D, _stream(stream)))


def qat_attn_fwd_chunk(q, k, v, o_q, o_hp, lse, B, H, Nq, Nkv_total, kv_begin, kv_len, D,
                       sm_scale, quant_mode, stream=None) -> Status:
    return Status(lib().qat_attn_fwd_chunk(_ptr(q), _ptr(k), _ptr(v), _ptr(o_q), _ptr(o_hp),
                                           _ptr(lse), B, H, Nq, Nkv_total, kv_begin, kv_len, D,
                                           float(sm_scale), int(quant_mode), _stream(stream)))


def qat_attn_merge(o_q_acc, o_hp_acc, lse_acc, o_q_part, o_hp_part, lse_part, o_q_out, o_hp_out,
                   B, H, Nq, D, stream=None) -> Status:
    return Status(lib().qat_attn_merge(_ptr(o_q_acc), _ptr(o_hp_acc), _ptr(lse_acc),
                                       _ptr(o_q_part), _ptr(o_hp_part), _ptr(lse_part),
                                       _ptr(o_q_out), _ptr(o_hp_out), B, H, Nq, D,
                                       _stream(stream)))


def _s3(strides):
    """Three element strides as a host array, or NULL (contiguous)."""
    return None if strides is None else _ll3(*strides)


def qat_qk_norm_rope(q, q_strides, k, k_strides, q_out, k_out, positions, position_stride, phases,
                     q_weight, k_weight, weight_bf16, B, Hq, Hk, N, D, rotary_dim, interleaved,
                     amplitude, eps, stream=None) -> Status:
    return _status(lib().qat_qk_norm_rope(
        _ptr(q), _s3(q_strides), _ptr(k), _s3(k_strides), _ptr(q_out), _ptr(k_out), _ptr(positions),
        position_stride, _ptr(phases), _ptr(q_weight), _ptr(k_weight), int(weight_bf16), B, Hq, Hk, N,
        D, rotary_dim, interleaved, amplitude, eps, _stream(stream)))


def qat_qk_norm_rope_bwd_workspace_bytes(D) -> int:
    return int(lib().qat_qk_norm_rope_bwd_workspace_bytes(D))


def qat_qk_norm_rope_bwd(q, q_strides, k, k_strides, dq_out, dq_out_strides, dk_out, dk_out_strides,
                         positions, position_stride, phases, q_weight, k_weight, weight_bf16, dq,
                         dq_strides, dk, dk_strides, dq_weight, dk_weight, B, Hq, Hk, N, D, rotary_dim,
                         interleaved, amplitude, eps, workspace, workspace_bytes,
                         stream=None) -> Status:
    return _status(lib().qat_qk_norm_rope_bwd(
        _ptr(q), _s3(q_strides), _ptr(k), _s3(k_strides), _ptr(dq_out), _s3(dq_out_strides),
        _ptr(dk_out), _s3(dk_out_strides), _ptr(positions), position_stride, _ptr(phases),
        _ptr(q_weight), _ptr(k_weight), int(weight_bf16), _ptr(dq), _s3(dq_strides), _ptr(dk),
        _s3(dk_strides), _ptr(dq_weight), _ptr(dk_weight), B, Hq, Hk, N, D, rotary_dim, interleaved,
        amplitude, eps, _ptr(workspace), workspace_bytes, _stream(stream)))


def qat_kv_cache_append(k, k_strides, v, v_strides, k_codes, v_codes, k_scales, v_scales, block_table,
                        seq_lens, new_lens, B, H, N, D, num_pages, page_size, max_pages,
                        stream=None) -> Status:
    return _status(lib().qat_kv_cache_append(
        _ptr(k), _s3(k_strides), _ptr(v), _s3(v_strides), _ptr(k_codes), _ptr(v_codes),
        _ptr(k_scales), _ptr(v_scales), _ptr(block_table), _ptr(seq_lens), _ptr(new_lens), B, H, N, D,
        num_pages, page_size, max_pages, _stream(stream)))


def qat_kv_cache_read(k_codes, v_codes, k_scales, v_scales, block_table, seq_lens, k_out, v_out, B, H,
                      begin, N, D, num_pages, page_size, max_pages, stream=None) -> Status:
    return _status(lib().qat_kv_cache_read(
        _ptr(k_codes), _ptr(v_codes), _ptr(k_scales), _ptr(v_scales), _ptr(block_table),
        _ptr(seq_lens), _ptr(k_out), _ptr(v_out), B, H, begin, N, D, num_pages, page_size, max_pages,
        _stream(stream)))


def qat_attn_decode_workspace_bytes(Hq, Hkv, T, D) -> int:
    return int(lib().qat_attn_decode_workspace_bytes(Hq, Hkv, T, D))


def qat_attn_decode(q, k_codes, v_codes, k_scales, v_scales, block_table, seq_lens, o, lse, B, Hq, Hkv,
                    T, D, num_pages, page_size, max_pages, sm_scale, quant_mode, workspace,
                    workspace_bytes, stream=None) -> Status:
    return _status(lib().qat_attn_decode(
        _ptr(q), _ptr(k_codes), _ptr(v_codes), _ptr(k_scales), _ptr(v_scales), _ptr(block_table),
        _ptr(seq_lens), _ptr(o), _ptr(lse), B, Hq, Hkv, T, D, num_pages, page_size, max_pages,
        float(sm_scale), int(quant_mode), _ptr(workspace), workspace_bytes, _stream(stream)))
