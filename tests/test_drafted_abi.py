"""CPU tests of the arguments' checks of windowed attention, trees over the cache, their masks and kept paths: every
C call here is refused, or has no work, before anything reaches a device."""

import pytest
import torch

from quantization_aware_attention_gb300 import (KVCache, attention, qat_attention_backward, qat_attention_decode,
                                                qat_attention_forward, qat_attention_tree, qat_draft_tree)
from quantization_aware_attention_gb300 import build as qbuild
from quantization_aware_attention_gb300 import capi
from quantization_aware_attention_gb300.capi import Status

A = 0x100000  # an aligned fake address: never dereferenced by these tests


@pytest.fixture(scope="module", autouse=True)
def built():
    qbuild.build()


FWD = dict(q=A, k=A, v=A, o_q=A, o_hp=A, lse=A, B=1, H=1, N=8, D=64, sm_scale=0.1, window=4, sinks=1, quant_mode=1,
           stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(window=0), Status.INVALID_ARG),
    (dict(window=-1), Status.INVALID_ARG),
    (dict(sinks=-1), Status.INVALID_ARG),
    (dict(D=96), Status.INVALID_ARG),
    (dict(N=0), Status.INVALID_ARG),
    (dict(N=-1), Status.INVALID_ARG),
    (dict(N=(1 << 30) + 1), Status.UNSUPPORTED),
    (dict(sm_scale=0.0), Status.INVALID_ARG),
    (dict(quant_mode=3), Status.INVALID_ARG),
    (dict(q=None), Status.INVALID_ARG),
    (dict(o_hp=A + 8), Status.INVALID_ARG),
    (dict(H=0, q=None), Status.OK),
])
def test_forward_validation(kw, want):
    assert capi.qat_attn_fwd_window(**{**FWD, **kw}) == want


BWD = dict(q=A, k=A, v=A, o_hp=A, lse=A, dO=A, dq=A, dk=A, dv=A, k_mean=None, B=1, H=1, N=8, D=64, sm_scale=0.1,
           window=4, sinks=1, quant_mode=1, workspace=A, workspace_bytes=0, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(window=0), Status.INVALID_ARG),
    (dict(sinks=-1), Status.INVALID_ARG),
    (dict(N=(1 << 30) + 1), Status.UNSUPPORTED),
    (dict(dk=None), Status.INVALID_ARG),
    (dict(k_mean=A + 4), Status.INVALID_ARG),
    (dict(), Status.WORKSPACE),
    (dict(workspace=None, workspace_bytes=1 << 30), Status.WORKSPACE),
    (dict(workspace=A + 16, workspace_bytes=1 << 30), Status.INVALID_ARG),
    (dict(B=0, q=None), Status.OK),
])
def test_backward_validation(kw, want):
    assert capi.qat_attn_bwd_window(**{**BWD, **kw}) == want


def test_backward_workspace():
    """Sinks' sums are cut into pieces where a head's queries are many against an SM's share of the work; the
    workspace holds 128 rows of fp32 dV and dK for each."""
    f = capi.qat_attn_bwd_window_workspace_bytes
    base = f(1, 8, 65536, 128, 512, 0)
    assert base > 0 and (f(1, 8, 65536, 128, 512, 4) - base) % (8 * 2 * 128 * 128 * 4) == 0
    assert 8 <= (f(1, 8, 65536, 128, 512, 4) - base) // (8 * 2 * 128 * 128 * 4) <= 128
    assert f(20, 32, 8192, 128, 1024, 4) == f(20, 32, 8192, 128, 1024, 0)  # enough heads for all SMs
    for S in (1, 500, 4000, 8191):  # never more than 1216 pieces
        assert f(1, 8, 8192, 64, 64, S) - f(1, 8, 8192, 64, 64, 0) <= 1216 * 2 * 128 * 64 * 4
    assert f(1, 1, 4096, 64, 128, 4096) == f(1, 1, 4096, 64, 128, 1 << 30)
    for bad in ((1, 1, 8, 64, 0, 0), (1, 1, 8, 64, 1, -1), (1, 1, 8, 96, 1, 0), (-1, 1, 8, 64, 1, 0)):
        assert f(*bad) == 0
    short = capi.qat_attn_bwd_window(**{**BWD, "N": 65536, "H": 8, "D": 128, "window": 512, "sinks": 4,
                                        "workspace_bytes": base})
    assert short == Status.WORKSPACE  # the pieces' sums do not fit


TREE = dict(q=A, k_codes=A, v_codes=A, k_scales=A, v_scales=A, block_table=A, seq_lens=A, tree=A, tree_stride=4, o=A,
            lse=None, B=1, Hq=4, Hkv=2, T=4, D=64, num_pages=4, page_size=16, max_pages=2, sm_scale=0.1, window=0,
            sinks=0, quant_mode=1, workspace=A, workspace_bytes=0, stream=0)
BAD_CACHE = [
    (dict(D=96), Status.INVALID_ARG),
    (dict(Hkv=3), Status.INVALID_ARG),
    (dict(page_size=24), Status.UNSUPPORTED),
    (dict(max_pages=0), Status.INVALID_ARG),
    (dict(B=4097), Status.UNSUPPORTED),
    (dict(quant_mode=2), Status.INVALID_ARG),
    (dict(sm_scale=-1.0), Status.INVALID_ARG),
    (dict(q=A + 8), Status.INVALID_ARG),
    (dict(lse=A + 2), Status.INVALID_ARG),
    (dict(), Status.WORKSPACE),
    (dict(workspace=A + 16, workspace_bytes=1 << 30), Status.INVALID_ARG),
    (dict(T=0, q=None), Status.OK),
    (dict(B=0, q=None), Status.OK),
]


@pytest.mark.parametrize("kw,want", BAD_CACHE + [
    (dict(T=65), Status.UNSUPPORTED),
    (dict(tree=None), Status.INVALID_ARG),
    (dict(tree=A + 4), Status.INVALID_ARG),
    (dict(tree_stride=-1), Status.INVALID_ARG),
    (dict(window=-1), Status.INVALID_ARG),
    (dict(window=5, sinks=-1), Status.INVALID_ARG),
    (dict(sinks=1), Status.INVALID_ARG),
])
def test_tree_validation(kw, want):
    assert capi.qat_attn_tree(**{**TREE, **kw}) == want


@pytest.mark.parametrize("kw,want", BAD_CACHE + [
    (dict(T=17), Status.UNSUPPORTED),
    (dict(window=0), Status.INVALID_ARG),
    (dict(sinks=-1), Status.INVALID_ARG),
])
def test_decode_window_validation(kw, want):
    args = {k: v for k, v in TREE.items() if not k.startswith("tree")}
    assert capi.qat_attn_decode_window(**{**args, "window": 5, **kw}) == want


def test_tree_workspace():
    for Hq, Hkv, T, D in ((4, 2, 64, 128), (4, 2, 1, 64), (64, 8, 64, 64)):
        assert capi.qat_attn_tree_workspace_bytes(Hq, Hkv, T, D) > 0
    for bad in ((4, 3, 1, 64), (4, 2, 65, 64), (4, 2, -1, 64), (4, 2, 1, 96), (0, 1, 1, 64)):
        assert capi.qat_attn_tree_workspace_bytes(*bad) == 0
    assert capi.qat_attn_decode_workspace_bytes(4, 2, 17, 64) == 0


def test_tree_workspace_holds_both_kernels_partials():
    """Two partials of a row tile, fp32 sums, maximum and sum a row, for each of 152 blocks of the tensor core's kernel
    (more than 32 rows a KV head at D 128, 64 at D 64); from 16 rows on a larger tree's workspace does for a smaller."""
    for D, rows in ((128, 32), (64, 64)):
        for T in (9, 16, 17, 33, 64):
            for G in (1, 2, 5, 8, 64):
                R, f = G * T, capi.qat_attn_tree_workspace_bytes
                if R > rows:
                    assert f(G, 1, T, D) >= 152 * 2 * min(R, 128) * (D + 2) * 4
                assert f(2 * G, 2, T, D) == f(G, 1, T, D)
                if G * (T - 1) >= 16:
                    assert f(G, 1, T, D) >= f(G, 1, T - 1, D)


DRAFT = dict(parents=A, parents_stride=0, seq_lens=A, tree=A, positions=A, B=2, T=4, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(T=65), Status.UNSUPPORTED),
    (dict(T=-1), Status.INVALID_ARG),
    (dict(B=-1), Status.INVALID_ARG),
    (dict(parents_stride=-4), Status.INVALID_ARG),
    (dict(parents=None), Status.INVALID_ARG),
    (dict(tree=A + 4), Status.INVALID_ARG),
    (dict(positions=A + 2), Status.INVALID_ARG),
    (dict(seq_lens=None), Status.INVALID_ARG),
    (dict(B=0, parents=None), Status.OK),
    (dict(T=0, parents=None), Status.OK),
])
def test_draft_validation(kw, want):
    assert capi.qat_draft_tree(**{**DRAFT, **kw}) == want


KEEP = dict(k_codes=A, v_codes=A, k_scales=A, v_scales=A, block_table=A, seq_lens=A, path=A, path_lens=A, new_lens=2 * A,
            B=2, H=2, T=8, L=4, D=64, num_pages=4, page_size=16, max_pages=2, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(T=65), Status.UNSUPPORTED),
    (dict(L=9), Status.UNSUPPORTED),
    (dict(L=-1), Status.INVALID_ARG),
    (dict(D=32), Status.INVALID_ARG),
    (dict(page_size=8), Status.UNSUPPORTED),
    (dict(path=None), Status.INVALID_ARG),
    (dict(path_lens=A + 2), Status.INVALID_ARG),
    (dict(new_lens=None), Status.INVALID_ARG),
    (dict(k_codes=A + 4), Status.INVALID_ARG),
    (dict(B=0, path=None), Status.OK),
    # blocks of one sequence read what another writes the new length to
    (dict(seq_lens=A + 64, new_lens=A + 64), Status.INVALID_ARG),
    (dict(path_lens=A + 64, new_lens=A + 64), Status.INVALID_ARG),
])
def test_keep_validation(kw, want):
    assert capi.qat_kv_cache_keep(**{**KEEP, **kw}) == want


def test_torch_calls_refuse_before_any_device():
    x = torch.zeros(1, 1, 8, 64, dtype=torch.bfloat16)
    for how in (dict(causal=True, window=0), dict(causal=True, window=4, sinks=-1), dict(causal=False, window=4),
                dict(causal=True, sinks=3), dict(causal=True, window=4)):
        with pytest.raises(ValueError):
            attention(x, x, x, **how)
        with pytest.raises(ValueError):
            qat_attention_forward(x, x, x, **how)
        with pytest.raises(ValueError):
            qat_attention_backward(x, x, x, x, x, x, **how)
    with pytest.raises(TypeError):
        attention(x, x, x, causal=True, window=4.5)
    with pytest.raises(TypeError):
        qat_attention_tree(x, None, None, None, None)
    with pytest.raises(TypeError):
        qat_attention_decode(x, None, None, None, window=3)
    with pytest.raises(ValueError):
        qat_draft_tree(torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        qat_draft_tree([[-1]], torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        KVCache.empty(2, 1, 16, 64, device="cpu")
