"""Pins of the oracle of the norm + rotation, the FP8 cache and decoding (oracle/serving_oracle.py):
closed forms, library routines and finite differences, on the CPU."""

import numpy as np
import pytest
import torch

from oracle import qat_oracle as orc
from oracle import serving_oracle as so


def _rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_is_complex_multiplication(layout):
    rng = _rng(1)
    B, H, N, D, R = 2, 3, 5, 64, 32
    x = rng.standard_normal((B, H, N, D))
    pos = rng.integers(0, 1 << 20, (B, N))
    f = 10000.0 ** (-2.0 * np.arange(R // 2) / R)
    y = so.norm_rope(x, None, pos, f, layout, 1.5)
    turn = 1.5 * np.exp(1j * pos[:, None, :, None] * f)
    if layout == "half":
        c = (x[..., :R // 2] + 1j * x[..., R // 2:R]) * turn
        want = np.concatenate([c.real, c.imag, x[..., R:]], -1)
    else:
        c = (x[..., 0:R:2] + 1j * x[..., 1:R:2]) * turn
        want = x.copy()
        want[..., 0:R:2], want[..., 1:R:2] = c.real, c.imag
    assert np.allclose(y, want, atol=1e-12)
    # scores depend on the distance alone
    same = np.full((B, N), 77)
    u, v = so.norm_rope(x, None, same, f, layout), so.norm_rope(x, None, same + 1000, f, layout)
    assert np.allclose(u @ u.swapaxes(-1, -2), v @ v.swapaxes(-1, -2), atol=1e-10)


def test_norm_is_rms_norm():
    rng = _rng(2)
    x, w = rng.standard_normal((2, 2, 3, 64)), rng.standard_normal(64)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x), (64,), torch.from_numpy(w), 1e-3).numpy()
    assert np.allclose(so.norm_rope(x, w, np.zeros((2, 3)), [], "half", eps=1e-3), want, atol=1e-12)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", [True, False])
def test_backward_against_differences(layout, norm):
    rng = _rng(3)
    B, H, N, D, R = 1, 2, 3, 64, 32
    x, dy = rng.standard_normal((B, H, N, D)), rng.standard_normal((B, H, N, D))
    w = 1 + 0.3 * rng.standard_normal(D) if norm else None
    pos = rng.integers(0, 1000, (B, N))
    f = 100.0 ** (-2.0 * np.arange(R // 2) / R)
    dx, dw = so.norm_rope_backward(x, w, dy, pos, f, layout, 1.2)

    def value(x, w):
        return float((dy * so.norm_rope(x, w, pos, f, layout, 1.2)).sum())

    h = 1e-5
    for _ in range(12):
        d = rng.standard_normal(x.shape)
        num = (value(x + h * d, w) - value(x - h * d, w)) / (2 * h)
        assert abs(num - (dx * d).sum()) <= 1e-7 * max(1.0, abs(num))
        if norm:
            d = rng.standard_normal(D)
            num = (value(x, w + h * d) - value(x, w - h * d)) / (2 * h)
            assert abs(num - (dw * d).sum()) <= 1e-7 * max(1.0, abs(num))


def test_cache_rows():
    x = orc.f32_to_bf16_rn(_rng(4).standard_normal((50, 64)).astype(np.float32)).astype(np.float64)
    x[3] = 0.0
    x[4] *= 2.0 ** -120
    x[5, 7] = np.inf
    x[6, 9] = np.nan
    x[7] *= 1e30
    codes, scales = so.quant_row(x)
    v = so.dequant(codes, scales)
    assert (v[3] == 0).all() and (v[4] == 0).all() and scales[3] == 0 and scales[4] == 0
    assert np.isnan(v[5]).all() and np.isnan(v[6]).all() and (codes[5] == 0).all()
    for i in (0, 1, 7, 20):
        amax = np.abs(x[i]).max()
        # half a step of E4M3 (2^-4 relative), or of its subnormals (2^-10 of a scale)
        assert (np.abs(v[i] - x[i]) <= 1.001 * np.maximum(2.0 ** -4 * np.abs(x[i]), amax / 448 * 2.0 ** -10)).all()
        assert codes[i, np.abs(x[i]).argmax()] & 0x7F == 0x7E  # the largest is 448


@pytest.mark.parametrize("quant", [False, True])
def test_decode_is_the_last_rows_of_causal_attention(quant):
    rng = _rng(5)
    n, T, D = 150, 4, 64
    k, v, q = (rng.standard_normal((n, D)) for _ in range(3))
    r = orc.head_forward(q, k, v, 0.125, True, quant)
    o, lse, tol, lse_tol = so.decode_head(q[n - T:], k, v, np.arange(n - T, n), 0.125, quant)
    assert np.allclose(o, r["o_q" if quant else "o_hp"][n - T:], atol=1e-12)
    assert np.allclose(lse, r["lse"][n - T:], atol=1e-12)
    assert (tol > 0).all() and (tol < 0.1).all() and (lse_tol < 1e-3).all()
    o, lse, _, _ = so.decode_head(q[:2], k[:1], v[:1], np.array([-1, 0]), 0.125, quant)
    assert (o[0] == 0).all() and lse[0] == -np.inf and np.allclose(o[1], v[0])
