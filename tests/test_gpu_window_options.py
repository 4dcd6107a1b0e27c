"""GPU parity of windowed attention's options against the fp64 oracle: what the forward and what the backward run on with
qkv_quant, smooth_k and use_qat_qkv_backward, and rows that see few keys.  The oracle makes its own fake-quantized inputs and
forms P from the forward's lse, as the backward does; tolerances are the training kernels' (gpu_util) where no other is derived."""

import numpy as np
import pytest
import torch

from oracle import drafted_oracle as do_
from oracle import qat_oracle as orc
from quantization_aware_attention_gb300 import QUANT_P_FP8E4M3_ROW_TILE64_PAGE_BWD as PAGE
from quantization_aware_attention_gb300 import attention, check_device_status, qat_attention_backward, qat_attention_forward
from quantization_aware_attention_gb300 import build as qbuild
from quantization_aware_attention_gb300.inputs import custom_inputs

from gpu_util import TOL_Q, dev_bf16, host_f64, oracle_f64, rel_l2

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    qbuild.build()


def _backward(q, k, v, do, o, lse, sm, seen, quant_dv, k_mean):
    """One head's gradients, fp64, with P of the given lse (base 2) and Delta of the given output."""
    p = np.where(seen, np.exp2(sm * (q @ k.T) * do_.LOG2E - lse[:, None]), 0.0)
    ds = p * (do @ v.T - (do * o).sum(-1, keepdims=True))
    dq = sm * (ds @ k)
    if k_mean is not None:
        dq = dq + sm * ds.sum(-1, keepdims=True) * k_mean
    return dq, sm * (ds.T @ q), (orc.quant_rows_exact(p) if quant_dv else p).T @ do


@pytest.mark.parametrize("quant_mode", [0, 1, PAGE])
@pytest.mark.parametrize("use_qat_qkv_backward", [True, False])
@pytest.mark.parametrize("smooth_k", [True, False])
@pytest.mark.parametrize("N,D,window,sinks", [(300, 64, 70, 3), (420, 128, 200, 130)])
def test_quantized_inputs(N, D, window, sinks, smooth_k, use_qat_qkv_backward, quant_mode):
    H, sm = 2, D ** -0.5
    inp = custom_inputs(30 + N, 1, H, N, N, D)
    inp["k"] = (orc.f32_to_bf16_rn((orc.bf16_bits_to_f64(inp["k"]) + np.linspace(-2, 2, D)).astype(np.float32))
                .view(np.uint32) >> 16).astype(np.uint16)
    f = oracle_f64(inp)
    leaves = [dev_bf16(inp[n]).requires_grad_(True) for n in ("q", "k", "v")]
    o = attention(*leaves, causal=True, quant_mode=quant_mode, qkv_quant=True, smooth_k=smooth_k,
                  use_qat_qkv_backward=use_qat_qkv_backward, window=window, sinks=sinks, check=True)
    got = (o.detach(),) + torch.autograd.grad(o, leaves, dev_bf16(inp["do"]))
    check_device_status()
    mean = orc.channel_mean(f["k"]).astype(np.float32) if smooth_k else None
    mean64 = mean.astype(np.float64) if smooth_k else None
    seen = do_.window_seen(range(N), N, window, sinks)
    want = []
    for h in range(H):
        q, k, v = (f[n][0, h].astype(np.float32) for n in ("q", "k", "v"))
        by = [orc.fake_quant_tokens_fp32(x, m)[0].astype(np.float64) for x, m in ((q, None), (k, mean), (v, None))]
        r = do_.head_train(*by, f["do"][0, h], sm, seen, quant=quant_mode != 0)
        back = by if use_qat_qkv_backward else [f["q"][0, h], f["k"][0, h], f["v"][0, h]]
        if smooth_k and not use_qat_qkv_backward:
            back[1] = orc.subtract_mean_bf16(k, mean).astype(np.float64)
        page = quant_mode == PAGE
        want.append((r["o_q"],) + _backward(*back, f["do"][0, h], r["o_q" if page else "o_hp"], r["lse"], sm, seen, page,
                                            mean64))
    for n, g, w in zip(("o", "dq", "dk", "dv"), got, zip(*want)):
        assert rel_l2(host_f64(g[0]), np.stack(w)) <= TOL_Q, n


def _few_keys(N, D, seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    q, v, do = normal(1, 2, N, D) * 1.5, normal(1, 2, N, D), normal(1, 2, N, D)
    return [q, normal(1, 2, N, D) + 0.5 * normal(D), v, do]


def _errors(t, window, sinks, rows=slice(None)):
    """Relative errors of dQ and dK (of the given rows and keys) against fp64."""
    q, k, v, do = t
    _, o_hp, lse = qat_attention_forward(q, k, v, True, window=window, sinks=sinks)
    grads = qat_attention_backward(q, k, v, o_hp, lse, do, True, window=window, sinks=sinks)
    check_device_status()
    N, D = q.shape[2:]
    seen = do_.window_seen(range(N), N, window, sinks)
    want = [do_.head_train(*(host_f64(x[0, h]) for x in t), D ** -0.5, seen) for h in range(q.shape[1])]
    return [rel_l2(host_f64(grads[i][0])[:, rows], np.stack([w[n][rows] for w in want]))
            for i, n in enumerate(("dq", "dk"))]


@pytest.mark.parametrize("N,D,window,sinks", [(900, 64, 32, 0), (900, 128, 31, 1), (900, 64, 33, 0), (900, 128, 31, 2),
                                              (900, 64, 20, 20), (900, 128, 1, 40)])
def test_gradients_about_where_the_running_maximum_is_raised_at_once(N, D, window, sinks):
    """It is for window + sinks of up to 32.  The bound on each side is the few keys' own: roundings to bf16 are off by 1.7e-3
    of a value (rms of half a step over mantissas), in quadrature the output once, dS once, which keys with an offset of half
    their spread make sqrt(1.25) of dQ, and P in O_hp and with it in Delta at most as much: 1.7e-3 sqrt(3.25) = 3.1e-3."""
    assert max(_errors(_few_keys(N, D, N + window), window, sinks)) <= 3.1e-3


@pytest.mark.parametrize("N,D,window,sinks", [(500, 64, 400, 0), (500, 128, 300, 130), (1500, 128, 1000, 4), (300, 64, 1 << 40, 0)])
def test_gradients_of_the_first_rows(N, D, window, sinks):
    """Of whatever window the first rows see few keys: all of them in one block of 128, whose largest score is the row's own
    from the start.  dQ of these rows by the same bound."""
    assert _errors(_few_keys(N, D, N), window, sinks, slice(0, 32))[0] <= 3.1e-3
