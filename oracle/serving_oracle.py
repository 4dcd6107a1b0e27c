"""Plain fp64 oracle of the query/key norm with rotary positions, the FP8 key/value cache and the
attention over it.  TEST INFRASTRUCTURE ONLY, like ``qat_oracle``: it imports nothing from the product
package.

  norm + rotation   z = x w / sqrt(mean x^2 + eps) (no norm without w); channel pairs (a, b) of the first
                    R channels become amplitude (a cos - b sin, a sin + b cos), the angle position * f_i
  cache row         amax = max |x|, code = E4M3(fl32(x fl32(448 / amax))), scale = fl32(amax / 448);
                    zeros below 2^-110; codes 0 and scale NaN with a NaN or infinity
  decode            token t of T is position len - T + t and sees keys up to its own
"""

from __future__ import annotations

import numpy as np

from .qat_oracle import bf16_bits_to_f64, e4m3_decode, e4m3_rne_satfinite, quant_rows_exact  # noqa: F401

LOG2E = 1.4426950408889634
TINY_ROW = 2.0 ** -110


# ------------------------------------------------------------------ norm + rotation

def _split(x, R, layout):
    if layout == "half":
        return x[..., :R // 2], x[..., R // 2:R]
    return x[..., 0:R:2], x[..., 1:R:2]


def _rotate(z, positions, freqs, layout, amplitude, sign):
    """z [B, H, N, D] (fp64), positions [B, N] integers, freqs [R / 2] radians per position."""
    R = 2 * len(freqs)
    if R == 0:
        return z
    ang = sign * np.asarray(positions, np.float64)[:, None, :, None] * np.asarray(freqs, np.float64)
    c, s = amplitude * np.cos(ang), amplitude * np.sin(ang)
    a, b = _split(z, R, layout)
    y = z.copy()
    ya, yb = _split(y, R, layout)
    ya[...], yb[...] = a * c - b * s, a * s + b * c
    return y


def norm_rope(x, w, positions, freqs, layout, amplitude=1.0, eps=1e-6):
    z = x
    if w is not None:
        z = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return _rotate(z, positions, freqs, layout, amplitude, 1.0)


def norm_rope_backward(x, w, dy, positions, freqs, layout, amplitude=1.0, eps=1e-6):
    """(dx, dw) of <dy, norm_rope(x, w)>; dw None without w."""
    dz = _rotate(dy, positions, freqs, layout, amplitude, -1.0)
    if w is None:
        return dz, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    dn = dz * w
    return r * (dn - n * (dn * n).mean(-1, keepdims=True)), (dz * n).sum((0, 1, 2))


# ------------------------------------------------------------------ cache

def quant_row(x):
    """x [..., D] bf16 values (fp64) -> (code bytes, fp32 scales), the rule's fp32 steps literally."""
    x32 = np.asarray(x, np.float32)
    amax = np.abs(x32).max(-1)
    bad = ~np.isfinite(x32).all(-1)
    amax = np.where(bad | (amax < TINY_ROW), np.float32(0), amax).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        inv = np.where(amax > 0, np.float32(448) / amax, np.float32(0)).astype(np.float32)
        y = (np.where(bad[..., None], np.float32(0), x32) * inv[..., None]).astype(np.float32)
    codes, _ = e4m3_rne_satfinite(y.astype(np.float64))
    scale = (amax / np.float32(448)).astype(np.float32)
    return codes.astype(np.uint8), np.where(bad, np.float32(np.nan), scale)


def dequant(codes, scales):
    """Exact value of cached rows (fp64)."""
    return e4m3_decode(codes) * np.asarray(scales, np.float64)[..., None]


# ------------------------------------------------------------------ decode

def decode_head(q, k, v, positions, sm_scale, quant):
    """One query head: q [T, D], k and v [n, D] (fp64), positions [T].  Returns (o [T, D], lse [T],
    tol [T, D], lse_tol [T]): the tolerances are the sum of what each rounding of a kernel with fp32 sums
    and f16 weights of V may add:
      scores    fp32 products and sums: 2^-19 of sum_d |q_d k_d| sm_scale log2 e, plus 2^-20 for exp2
                and the row sum, both relative to p
      codes     one E4M3 step where 448 p / amax lies that near to the middle between two codes
      weights   f16: half a step, 2^-11 relative; below its normal range absolute 2^-38 of the row's own
                largest weight, p times the largest |v| of a key
      output    bf16: half a step, 2^-8 relative; fp32 sum over n keys: 2^-20 of sum p |v|."""
    T, D = q.shape
    n = k.shape[0]
    o, lse = np.zeros((T, D)), np.full(T, -np.inf)
    tol, lse_tol = np.zeros((T, D)), np.zeros(T)
    for t in range(T):
        seen = min(n, int(positions[t]) + 1)
        if seen <= 0:
            continue
        kk, vv = k[:seen], v[:seen]
        s = kk @ q[t] * sm_scale
        m = s.max()
        e = np.exp(s - m)
        l = e.sum()
        lse[t] = (m + np.log(l)) * LOG2E
        eps_p = 2.0 ** -20 + 2.0 ** -19 * LOG2E * sm_scale * float((np.abs(kk) @ np.abs(q[t])).max())
        p, flips = e, np.zeros(seen)
        if quant:
            p = np.zeros(seen)
            for a in range(0, seen, 64):
                x = e[a:a + 64]
                amax = x.max()
                if amax < 2.0 ** -100:
                    continue
                y = x * (448.0 / amax)
                val = e4m3_rne_satfinite(y)[1]
                step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(y, 2.0 ** -20))), -6) - 3)
                frac = np.abs(np.abs(y / step - np.floor(y / step)) - 0.5) * step  # to the middle
                p[a:a + 64] = val * (amax / 448.0)
                flips[a:a + 64] = np.where(frac <= 4 * eps_p * y, step, 0.0) * (amax / 448.0)
        o[t] = p @ vv / l
        mass = p @ np.abs(vv) / l
        tol[t] = (2.0 ** -8 * np.abs(o[t]) + (2.0 ** -11 + 4 * eps_p + 2.0 ** -20) * mass
                  + flips @ np.abs(vv) / l + n * 2.0 ** -38 * (p * np.abs(vv).max(-1, initial=0.0)).max() / l)
        lse_tol[t] = LOG2E * 2 * eps_p + 2.0 ** -22 * abs(lse[t])
    return o, lse, tol, lse_tol
