"""Plain fp64 oracle of attention whose rows see given keys: sliding windows with sinks (training and over the
cache), trees of drafted tokens, and the cache's keeping of accepted ones.  TEST INFRASTRUCTURE ONLY: it imports
nothing from the product package.

  window   query i sees key j if j <= i and (j > i - window or j < sinks)
  tree     token t (slot len - T + t) sees the keys before len - T and drafted token s iff bit s of its mask; with
           a window, keys j before len - T also need j > pos - window or j < sinks, pos = len - T + popcount - 1
  draft    mask(t) = bit t | mask(parent), 0 for padding (a parent outside [-1, t)) and what continues it
"""

from __future__ import annotations

import numpy as np

from .qat_oracle import e4m3_rne_satfinite, quant_rows_exact

LOG2E = 1.4426950408889634
#: the largest error of a weight of V as an operand of the product, relative to itself: half a step
F16, BF16 = 2.0 ** -11, 2.0 ** -8


# ------------------------------------------------------------------ who sees what

def window_seen(rows, n, window, sinks):
    """Truth values [len(rows), n] for queries at the given positions (negative: none)."""
    i, j = np.asarray(rows)[:, None], np.arange(n)[None]
    return (j <= i) & ((j > i - window) | (j < sinks))


def popcount(masks):
    return np.array([bin(int(m) & (2 ** 64 - 1)).count("1") for m in masks])


def tree_seen(length, masks, window=None, sinks=0):
    """Truth values [T, max(length, 0)] for the drafted tokens at the end of a sequence."""
    T, n = len(masks), max(int(length), 0)
    seen = np.zeros((T, n), bool)
    base = int(length) - T
    pos = base + popcount(masks) - 1
    for t, m in enumerate(masks):
        for j in range(n):
            if j >= base:
                seen[t, j] = int(m) >> (j - base) & 1
            else:
                seen[t, j] = window is None or j > pos[t] - window or j < sinks
    return seen


def draft(parents, length):
    """(masks as Python integers, positions) of one sequence's tree."""
    T, masks, pad = len(parents), [], []
    for t, parent in enumerate(int(x) for x in parents):
        bad = parent < -1 or parent >= t or (parent >= 0 and pad[parent])
        pad.append(bad)
        masks.append(0 if bad else (1 << t) | (masks[parent] if parent >= 0 else 0))
    return masks, np.array([length - T + bin(m).count("1") - 1 for m in masks])


# ------------------------------------------------------------------ training

def _head(q, k, sm_scale, seen):
    s = np.where(seen, sm_scale * (q @ k.T), -np.inf)
    m = s.max(-1, keepdims=True)
    e = np.exp(s - m)
    l = e.sum(-1, keepdims=True)
    return e / l, (m + np.log(l))[:, 0] * LOG2E


def head_train(q, k, v, do, sm_scale, seen, quant=True, page=False, k_mean=None):
    """One head, all fp64: o_q, o_hp, lse and the gradients of <do, o_hp> (page: of the page's backward, dV from
    the quantized P and Delta from o_q).  Every row sees a key."""
    p, lse = _head(q, k, sm_scale, seen)
    pq = quant_rows_exact(p) if quant else p
    o_q, o_hp = pq @ v, p @ v
    delta = (do * (o_q if page else o_hp)).sum(-1, keepdims=True)
    ds = p * (do @ v.T - delta)
    dq = sm_scale * (ds @ k)
    if k_mean is not None:
        dq = dq + sm_scale * ds.sum(-1, keepdims=True) * np.asarray(k_mean, np.float64)
    return dict(o_q=o_q, o_hp=o_hp, lse=lse, dq=dq, dk=sm_scale * (ds.T @ q), dv=(pq if page else p).T @ do)


# ------------------------------------------------------------------ over the cache

def attend_rows(q, k, v, seen, sm_scale, quant, weight_eps):
    """Rows q [T, D] over k and v [n, D] (fp64) by truth values seen [T, n].  Returns (o, lse, tol, lse_tol): the
    tolerances are the sum of what each rounding of a kernel with fp32 sums may add, weights of V rounded by
    weight_eps of themselves:
      scores    fp32 products and sums: 2^-19 of sum_d |q_d k_d| sm_scale log2 e, plus 2^-20 for exp2
                and the row sum, both relative to p
      codes     one E4M3 step where 448 p / amax lies that near to the middle between two codes
      weights   weight_eps relative; absolute 2^-38 of the row's largest weight (an f16's range)
      output    bf16: half a step, 2^-8 relative; fp32 sum over n keys: 2^-20 of sum p |v|."""
    T, D = q.shape
    n = k.shape[0]
    o, lse = np.zeros((T, D)), np.full(T, -np.inf)
    tol, lse_tol = np.zeros((T, D)), np.zeros(T)
    for t in range(T):
        if not seen[t].any():
            continue
        s = np.where(seen[t], k @ q[t] * sm_scale, -np.inf)
        m = s.max()
        e = np.exp(s - m)
        l = e.sum()
        lse[t] = (m + np.log(l)) * LOG2E
        eps_p = 2.0 ** -20 + 2.0 ** -19 * LOG2E * sm_scale * float((np.abs(k[seen[t]]) @ np.abs(q[t])).max())
        p, flips = e, np.zeros(n)
        if quant:
            p = np.zeros(n)
            for a in range(0, n, 64):
                x = e[a:a + 64]
                amax = x.max()
                if amax < 2.0 ** -100:
                    continue
                y = x * (448.0 / amax)
                step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(y, 2.0 ** -20))), -6) - 3)
                frac = np.abs(np.abs(y / step - np.floor(y / step)) - 0.5) * step  # to the middle
                p[a:a + 64] = e4m3_rne_satfinite(y)[1] * (amax / 448.0)
                flips[a:a + 64] = np.where(frac <= 4 * eps_p * y, step, 0.0) * (amax / 448.0)
        vv = np.where(seen[t][:, None], v, 0.0)
        o[t] = p @ vv / l
        mass = p @ np.abs(vv) / l
        tol[t] = (2.0 ** -8 * np.abs(o[t]) + (weight_eps + 4 * eps_p + 2.0 ** -20) * mass
                  + flips @ np.abs(vv) / l + n * 2.0 ** -38 * (p * np.abs(vv).max(-1, initial=0.0)).max() / l)
        lse_tol[t] = LOG2E * 2 * eps_p + 2.0 ** -22 * abs(lse[t])
    return o, lse, tol, lse_tol


def keep(lengths, T, path, path_lens):
    """(moves as (sequence, from, to) positions, new lengths) of accepted drafted tokens."""
    moves, new = [], []
    L = np.shape(path)[1]
    for b, n in enumerate(lengths):
        base, kept = int(n) - T, min(max(int(path_lens[b]), 0), L)
        new.append(max(base + kept, 0))
        for i in range(kept):
            p = int(path[b][i])
            if 0 <= p < T and base + p >= 0 and base + i >= 0:
                moves.append((b, base + p, base + i))
    return moves, new
