"""CPU tests of the arguments' checks of the norm + rotation, the FP8 cache and decoding: every C call
here is refused, or has no work, before anything reaches a device."""

import math

import pytest
import torch

from quantization_aware_attention_gb300 import (KVCache, RopePlan, qat_attention_decode,
                                                qat_qk_norm_rope)
from quantization_aware_attention_gb300 import build as qbuild
from quantization_aware_attention_gb300 import capi
from quantization_aware_attention_gb300.capi import Status

A = 0x100000  # an aligned fake address: never dereferenced by these tests


@pytest.fixture(scope="module", autouse=True)
def built():
    qbuild.build()


ROPE = dict(q=A, q_strides=None, k=A, k_strides=None, q_out=A, k_out=A, positions=A, position_stride=0,
            phases=A, q_weight=A, k_weight=A, weight_bf16=0, B=1, Hq=2, Hk=1, N=0, D=64, rotary_dim=64,
            interleaved=0, amplitude=1.0, eps=1e-6, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(), Status.OK),  # no tokens
    (dict(B=0, N=5, q=None), Status.OK),
    (dict(D=96), Status.INVALID_ARG),
    (dict(B=-1), Status.INVALID_ARG),
    (dict(rotary_dim=8), Status.INVALID_ARG),
    (dict(rotary_dim=80), Status.INVALID_ARG),
    (dict(rotary_dim=-16), Status.INVALID_ARG),
    (dict(interleaved=2), Status.INVALID_ARG),
    (dict(weight_bf16=2), Status.INVALID_ARG),
    (dict(eps=0.0), Status.INVALID_ARG),
    (dict(eps=math.nan), Status.INVALID_ARG),
    (dict(amplitude=math.inf), Status.INVALID_ARG),
    (dict(N=4, positions=None), Status.INVALID_ARG),
    (dict(N=4, phases=A + 4), Status.INVALID_ARG),
    (dict(N=4, position_stride=-1), Status.INVALID_ARG),
    (dict(N=4, q=A + 8), Status.INVALID_ARG),
    (dict(N=4, k=None), Status.INVALID_ARG),
    (dict(N=4, k_out=None), Status.INVALID_ARG),
    (dict(N=4, k_weight=None), Status.INVALID_ARG),
    (dict(N=4, q_weight=A + 4), Status.INVALID_ARG),
    (dict(N=4, q_strides=(256, 64, 60)), Status.INVALID_ARG),
    (dict(N=4, k_strides=(256, 64, -64)), Status.INVALID_ARG),
    (dict(N=1 << 30, Hq=4), Status.INVALID_ARG),
])
def test_norm_rope_validation(kw, want):
    assert capi.qat_qk_norm_rope(**{**ROPE, **kw}) == want


BWD = dict(q=A, q_strides=None, k=A, k_strides=None, dq_out=A, dq_out_strides=None, dk_out=A,
           dk_out_strides=None, positions=A, position_stride=0, phases=A, q_weight=A, k_weight=A,
           weight_bf16=0, dq=A, dq_strides=None, dk=A, dk_strides=None, dq_weight=A, dk_weight=A, B=1,
           Hq=2, Hk=1, N=4, D=64, rotary_dim=64, interleaved=0, amplitude=1.0, eps=1e-6, workspace=A,
           workspace_bytes=1 << 20, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(dq_out=None), Status.INVALID_ARG),
    (dict(dk=A + 2), Status.INVALID_ARG),
    (dict(dq_out_strides=(0, 0, 4)), Status.INVALID_ARG),
    (dict(dq_strides=(0, 64, 4)), Status.INVALID_ARG),
    (dict(workspace=None), Status.WORKSPACE),
    (dict(workspace_bytes=100), Status.WORKSPACE),
    (dict(workspace=A + 16), Status.INVALID_ARG),
    (dict(Hk=0), Status.INVALID_ARG),                       # a gradient of an absent weight
    (dict(q_weight=None, k_weight=None), Status.INVALID_ARG),
    (dict(D=32), Status.INVALID_ARG),
    (dict(N=0, dq_weight=None, dk_weight=None), Status.OK),
])
def test_norm_rope_bwd_validation(kw, want):
    assert capi.qat_qk_norm_rope_bwd(**{**BWD, **kw}) == want


def test_workspace_sizes():
    assert capi.qat_qk_norm_rope_bwd_workspace_bytes(96) == 0
    assert capi.qat_qk_norm_rope_bwd_workspace_bytes(128) % 256 == 0
    for bad in ((8, 2, 1, 96), (8, 3, 1, 64), (8, 0, 1, 64), (0, 1, 1, 64), (8, 2, -1, 64), (8, 2, 17, 64)):
        assert capi.qat_attn_decode_workspace_bytes(*bad) == 0
    # grows with the rows that share a KV head, up to 16
    sizes = [capi.qat_attn_decode_workspace_bytes(hq, 2, 1, 64) for hq in (2, 8, 16, 32, 64)]
    assert sizes[0] < sizes[1] < sizes[2] < sizes[3] == sizes[4]


APPEND = dict(k=A, k_strides=None, v=A, v_strides=None, k_codes=A, v_codes=A, k_scales=A, v_scales=A,
              block_table=A, seq_lens=A, new_lens=None, B=2, H=1, N=0, D=64, num_pages=4, page_size=16,
              max_pages=2, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(), Status.OK),
    (dict(B=0, N=3, k=None, block_table=None, seq_lens=None), Status.OK),
    (dict(D=80), Status.INVALID_ARG),
    (dict(H=0), Status.INVALID_ARG),
    (dict(num_pages=0), Status.INVALID_ARG),
    (dict(max_pages=0), Status.INVALID_ARG),
    (dict(page_size=24), Status.UNSUPPORTED),
    (dict(page_size=512), Status.UNSUPPORTED),
    (dict(max_pages=1 << 27), Status.UNSUPPORTED),
    (dict(N=-1), Status.INVALID_ARG),
    (dict(N=3, k=None), Status.INVALID_ARG),
    (dict(N=3, v=A + 8), Status.INVALID_ARG),
    (dict(N=3, k_codes=A + 8), Status.INVALID_ARG),
    (dict(N=3, v_scales=A + 4), Status.INVALID_ARG),
    (dict(N=3, block_table=None), Status.INVALID_ARG),
    (dict(N=3, seq_lens=A + 2), Status.INVALID_ARG),
    (dict(N=3, new_lens=A + 1), Status.INVALID_ARG),
    (dict(N=3, v_strides=(4, 64, 64)), Status.INVALID_ARG),
])
def test_append_validation(kw, want):
    assert capi.qat_kv_cache_append(**{**APPEND, **kw}) == want


@pytest.mark.parametrize("kw,want", [
    (dict(), Status.OK),
    (dict(begin=-1), Status.INVALID_ARG),
    (dict(N=3, k_out=None), Status.INVALID_ARG),
    (dict(N=3, v_out=A + 8), Status.INVALID_ARG),
    (dict(N=3, k_scales=None), Status.INVALID_ARG),
    (dict(page_size=8), Status.UNSUPPORTED),
])
def test_read_validation(kw, want):
    args = dict(k_codes=A, v_codes=A, k_scales=A, v_scales=A, block_table=A, seq_lens=A, k_out=A, v_out=A,
                B=2, H=1, begin=0, N=0, D=64, num_pages=4, page_size=16, max_pages=2, stream=0)
    assert capi.qat_kv_cache_read(**{**args, **kw}) == want


@pytest.mark.parametrize("kw,want", [
    (dict(T=0), Status.OK),
    (dict(B=0, q=None, o=None), Status.OK),
    (dict(T=17), Status.UNSUPPORTED),
    (dict(B=4097), Status.UNSUPPORTED),
    (dict(Hq=3), Status.INVALID_ARG),
    (dict(Hq=0), Status.INVALID_ARG),
    (dict(Hkv=0), Status.INVALID_ARG),
    (dict(sm_scale=0.0), Status.INVALID_ARG),
    (dict(sm_scale=math.nan), Status.INVALID_ARG),
    (dict(quant_mode=2), Status.INVALID_ARG),
    (dict(page_size=48), Status.UNSUPPORTED),
    (dict(B=4096, Hkv=64, Hq=64, max_pages=1 << 24, page_size=64), Status.UNSUPPORTED),
    (dict(q=None), Status.INVALID_ARG),
    (dict(o=A + 8), Status.INVALID_ARG),
    (dict(lse=A + 2), Status.INVALID_ARG),
    (dict(k_codes=None), Status.INVALID_ARG),
    (dict(seq_lens=None), Status.INVALID_ARG),
    (dict(workspace=None), Status.WORKSPACE),
    (dict(workspace_bytes=4096), Status.WORKSPACE),
    (dict(workspace=A + 64), Status.INVALID_ARG),
])
def test_decode_validation(kw, want):
    args = dict(q=A, k_codes=A, v_codes=A, k_scales=A, v_scales=A, block_table=A, seq_lens=A, o=A, lse=A,
                B=2, Hq=4, Hkv=2, T=1, D=64, num_pages=4, page_size=16, max_pages=2, sm_scale=0.125,
                quant_mode=1, workspace=A, workspace_bytes=1 << 30, stream=0)
    assert capi.qat_attn_decode(**{**args, **kw}) == want


@pytest.mark.parametrize("args,kw", [
    ((24,), {}), ((0,), {}), ((144,), {}), ((64,), dict(layout="quarter")),
    ((64,), dict(scaling="cubic", factor=2.0)), ((64,), dict(base=1.0)), ((64,), dict(base=math.nan)),
    ((64,), dict(factor=2.0)), ((64,), dict(scaling="linear", factor=0.5)),
    ((64,), dict(scaling="yarn", factor=2.0)),
    ((64,), dict(scaling="yarn", factor=2.0, original_len=4096, beta_fast=1.0, beta_slow=2.0)),
    ((64,), dict(amplitude=math.inf)), ((64,), dict(device="cpu")),
])
def test_rope_plan_refusals(args, kw):
    with pytest.raises(ValueError):
        RopePlan(*args, **{"device": "cpu", **kw})


def test_host_tensors_are_refused():
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        qat_qk_norm_rope(x, x)
    f8 = torch.zeros(2, 1, 16, 64, dtype=torch.float8_e4m3fn)
    s = torch.zeros(2, 1, 16)
    with pytest.raises(ValueError, match="CUDA"):
        KVCache(f8, f8, s, s)
    with pytest.raises(TypeError):
        qat_attention_decode(x, None, None, None)


class _Wrapper(torch.Tensor):
    """Sizes and a device, no memory."""

    @staticmethod
    def __new__(cls, shape, dtype):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device="cuda:0")

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError(str(func))


def test_tensors_without_memory_are_refused():
    x = _Wrapper((2, 3, 5, 64), torch.bfloat16)
    with pytest.raises(ValueError, match="memory"):
        qat_qk_norm_rope(x)
    f8, s = _Wrapper((2, 3, 16, 64), torch.float8_e4m3fn), _Wrapper((2, 3, 16), torch.float32)
    cache = KVCache(f8, f8, s, s)
    table, lens = _Wrapper((2, 1), torch.int32), _Wrapper((2,), torch.int32)
    with pytest.raises(ValueError, match="memory"):
        qat_attention_decode(x, cache, table, lens)
    with pytest.raises(ValueError, match="memory"):
        cache.append(x, x, table, lens)
    with pytest.raises(ValueError, match="memory"):
        cache.read(table, lens)
