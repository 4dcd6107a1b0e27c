"""GPU parity of what serves windows and drafted trees over the FP8 cache: decoding with a window, the attention of a
tree, its masks and positions, the keeping of accepted tokens, and all of them in a row, against the fp64 oracle
(oracle/drafted_oracle.py, which also gives the tolerances)."""

import numpy as np
import pytest
import torch

from oracle import drafted_oracle as do_
from oracle import serving_oracle as so
from quantization_aware_attention_gb300 import (KVCache, QatError, RopePlan, check_device_status,
                                                qat_attention_decode, qat_attention_tree, qat_draft_tree,
                                                qat_qk_norm_rope)
from quantization_aware_attention_gb300 import build as qbuild
from quantization_aware_attention_gb300 import capi
from quantization_aware_attention_gb300.capi import Status
from quantization_aware_attention_gb300.inputs import normal_bf16

from gpu_util import dev_bf16, host_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    qbuild.build()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _i64(masks):
    """Python integers below 2^64 as int64."""
    return torch.from_numpy(np.asarray(masks, np.uint64).view(np.int64).copy()).cuda()


def _cache(lens, H, D, page, seed, unseen=None, v_spread=1.0):
    """A cache whose written slots are normal rows of differing magnitudes; what no sequence holds has NaN scales and
    NaN codes.  unseen: positions of each sequence whose rows are NaN rows too."""
    B, per = len(lens), max(1, max((n + page - 1) // page for n in lens))
    pages = B * per + 2
    rng = np.random.default_rng(seed)
    table = rng.permutation(pages)[:B * per].reshape(B, per).astype(np.int32)
    there, clean = np.zeros((pages, page), bool), np.zeros((pages, page), bool)
    for b, n in enumerate(lens):
        for i in range(n):
            at = table[b, i // page], i % page
            there[at] = True
            clean[at] = unseen is None or not unseen(b, i)
    codes, scales = [], []
    for spread in (1.0, v_spread):
        x = rng.standard_normal((pages, H, page, D)).astype(np.float32)
        x *= np.exp(spread * rng.standard_normal((pages, H, page, 1))).astype(np.float32)
        c, s = so.quant_row(x)
        ok = np.broadcast_to(clean[:, None], s.shape)
        c = np.where(np.broadcast_to(there[:, None], s.shape)[..., None], np.where(ok[..., None], c, 0), 0x7f)
        codes.append(c.astype(np.uint8))
        scales.append(np.where(ok, s, np.float32(np.nan)))
    f8 = [torch.from_numpy(c).cuda().view(torch.float8_e4m3fn) for c in codes]
    return KVCache(f8[0], f8[1], *(torch.from_numpy(s).cuda() for s in scales)), table, codes, scales


def _rows(codes, scales, table, b, h, n, page):
    i = np.arange(max(n, 0))
    at = table[b, i // page], h, i % page
    return so.dequant(codes[at], scales[at])


def _compare(o, lse, q, lens, seen_of, cache, page, data, quant, eps, sm=None, heads=None):
    B, Hq, T, D = q.shape
    table, codes, scales = data
    sm = D ** -0.5 if sm is None else sm
    fq, fo, fl = host_f64(q), host_f64(o), host_f64(lse)
    G = Hq // cache.heads
    for b in range(B):
        seen = seen_of(b)
        for h in (range(cache.heads) if heads is None else heads):
            k, v = (_rows(c, s, table, b, h, lens[b], page) for c, s in zip(codes, scales))
            k, v = (np.where(seen.any(0)[:, None], x, 0.0) for x in (k, v))
            for hq in range(h * G, (h + 1) * G):
                w, wl, tol, ltol = do_.attend_rows(fq[b, hq], k, v, seen, sm, quant, eps)
                err = np.abs(fo[b, hq] - w)
                assert (err <= tol).all(), (b, hq, float((err / np.maximum(tol, 1e-300)).max()))
                some = np.isfinite(wl)
                assert np.array_equal(np.isneginf(fl[b, hq]), ~some)
                assert (np.abs(fl[b, hq][some] - wl[some]) <= ltol[some]).all()


# ------------------------------------------------------------------ windows

@pytest.mark.parametrize("quant", [0, 1])
@pytest.mark.parametrize("lens,Hq,Hkv,T,D,page,window,sinks", [
    ([1], 1, 1, 1, 128, 16, 1, 0),
    ([0, 5], 4, 2, 1, 64, 16, 3, 1),
    ([200], 4, 4, 1, 64, 64, 1, 0),
    ([200], 4, 2, 1, 128, 16, 1, 5),
    ([700, 63, 0, 129], 8, 2, 1, 128, 16, 100, 4),
    ([1500], 8, 1, 1, 128, 32, 64, 64),
    ([1500, 65], 8, 1, 1, 64, 32, 65, 63),
    ([1500, 300], 3, 1, 1, 128, 128, 200, 130),
    ([900, 3, 400], 5, 1, 5, 128, 16, 7, 2),           # a window about as long as the new tokens
    ([777, 1, 20], 32, 2, 16, 64, 32, 3, 0),           # shorter than they are
    ([777, 1], 32, 2, 16, 128, 32, 50, 700),
    ([513, 2000], 6, 2, 2, 128, 256, 1 << 40, 0),      # no limit
    ([513, 2000], 6, 2, 2, 128, 256, 9, 1 << 40),
])
def test_decode_window(lens, Hq, Hkv, T, D, page, window, sinks, quant):
    """With the pages that no token sees taken out of the block table, and NaN rows in the unseen places of others."""
    def seen_of(b):
        return do_.window_seen(lens[b] - T + np.arange(T), max(lens[b], 0), window, sinks)

    any_seen = [seen_of(b).any(0) for b in range(len(lens))]
    cache, table, codes, scales = _cache(lens, Hkv, D, page, 17 + Hq, unseen=lambda b, i: not any_seen[b][i])
    given = table.copy()
    for b, n in enumerate(lens):
        for p in range(table.shape[1]):
            if not any_seen[b][p * page:(p + 1) * page].any():
                given[b, p] = -1 if p % 2 else 1 << 30
    q = dev_bf16(normal_bf16(40 + T, (len(lens), Hq, T, D)))
    args = (q, cache, _i32(given), _i32(lens), None, quant)
    o, lse = qat_attention_decode(*args, return_lse=True, check=True, window=window, sinks=sinks)
    _compare(o, lse, q, lens, seen_of, cache, page, (table, codes, scales), quant, do_.F16)
    again = qat_attention_decode(*args, return_lse=True, window=window, sinks=sinks)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_decode_window_many_sequences():
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 400, 300)]
    lens[13], lens[14], lens[299] = 5000, 0, 0
    cache, table, codes, scales = _cache(lens, 1, 64, 16, 3)
    q = dev_bf16(normal_bf16(9, (300, 3, 1, 64)))
    o, lse = qat_attention_decode(q, cache, _i32(table), _i32(lens), return_lse=True, check=True, window=70, sinks=20)
    _compare(o, lse, q, lens, lambda b: do_.window_seen([lens[b] - 1], lens[b], 70, 20), cache, 16,
             (table, codes, scales), 1, do_.F16)


def test_decode_window_bad_pages_and_lengths():
    """A page that a token sees is looked up; lengths beyond the table are reported."""
    lens, page = [400], 16
    cache, table, codes, scales = _cache(lens, 1, 64, page, 9)
    q = dev_bf16(normal_bf16(13, (1, 2, 1, 64)))
    for place, bad in ((0, True), (1, False), (20, False), (21, True), (24, True)):
        given = table.copy()
        given[0, place] = 10 ** 6
        o = qat_attention_decode(q, cache, _i32(given), _i32(lens), window=50, sinks=3)
        assert bool(torch.isnan(o).all()) == bad and bool(torch.isfinite(o).all()) != bad
        assert capi.qat_attn_device_status() == (Status.BAD_PAGE if bad else Status.OK)
    with pytest.raises(QatError):
        qat_attention_decode(q, cache, _i32(table), _i32([10 ** 9]), window=50, check=True)
    o, lse = qat_attention_decode(q, cache, _i32(table), _i32([-3]), window=50, return_lse=True, check=True)
    assert (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("D,page,T,sinks", [(64, 16, 1, 0), (128, 16, 3, 16), (64, 32, 16, 33), (128, 256, 2, 0)])
def test_windows_that_begin_with_a_page(D, page, T, sinks):
    """The first token's window begins where a page does: the page before it is not looked up, the page itself is."""
    first = 3 * page
    window = 2 * page - T + 1
    lens = [first + window + T - 1]
    cache, table, _, _ = _cache(lens, 2, D, page, 9)
    q = dev_bf16(normal_bf16(13, (1, 4, T, D)))
    want = qat_attention_decode(q, cache, _i32(table), _i32(lens), window=window, sinks=sinks, check=True)
    given = table.copy()
    given[0, 2] = -1
    got = qat_attention_decode(q, cache, _i32(given), _i32(lens), window=window, sinks=sinks, check=True)
    assert torch.equal(got, want)
    given[0, 3] = -1
    got = qat_attention_decode(q, cache, _i32(given), _i32(lens), window=window, sinks=sinks)
    assert capi.qat_attn_device_status() == Status.BAD_PAGE and torch.isnan(got[:, :, 0]).all()


# ------------------------------------------------------------------ trees

def _trees(rng, B, T, kind):
    """Masks of B trees as Python integers."""
    out = []
    for _ in range(B):
        if kind == "tree":
            parents = [int(rng.integers(max(-1, t - 8), t)) for t in range(T)]
            out.append(do_.draft(parents, T)[0])
        elif kind == "chain":
            out.append([(2 << t) - 1 for t in range(T)])
        else:  # any bits, those of no token among them, and empty masks
            out.append([2 * int(x) + 1 if i % 7 else 0 for i, x in enumerate(rng.integers(0, (1 << 63) - 1, T))])
    return out


def _eps(Hq, Hkv, T, D):
    return do_.F16 if Hq // Hkv * T <= (64 if D == 64 else 32) else do_.BF16


TREES = [
    ([1], 1, 1, 1, 128, 16, "tree"),
    ([0, 70], 4, 2, 2, 64, 16, "tree"),
    ([64], 8, 1, 2, 128, 64, "any"),                   # 16 rows
    ([130, 3, 0], 2, 1, 9, 64, 16, "any"),             # 18
    ([129, 700], 4, 1, 5, 128, 32, "tree"),
    ([63, 1, 128, 64], 4, 2, 16, 64, 16, "tree"),      # 32 rows
    ([300, 40, 5], 4, 1, 33, 128, 128, "tree"),        # 132: two row tiles
    ([64, 65, 63, 10, 0], 1, 1, 64, 64, 16, "any"),
    ([1000, 127], 8, 1, 64, 128, 64, "tree"),          # 512
    ([1500, 2], 12, 4, 31, 128, 256, "chain"),
    ([2100, 900, 17], 5, 1, 27, 64, 32, "any"),        # 135
    ([130, 3, 0], 4, 1, 9, 128, 16, "any"),            # 36
    ([64, 65, 63, 10, 0], 2, 1, 64, 64, 16, "any"),    # 128
    ([128, 129, 255, 1], 3, 1, 43, 128, 16, "tree"),   # 129: one row in the second tile
    ([5, 1300], 26, 2, 5, 64, 128, "chain"),           # 65
]


@pytest.mark.parametrize("quant", [0, 1])
@pytest.mark.parametrize("lens,Hq,Hkv,T,D,page,kind", TREES)
def test_tree(lens, Hq, Hkv, T, D, page, kind, quant):
    masks = _trees(np.random.default_rng(T), len(lens), T, kind)
    cache, table, codes, scales = _cache(lens, Hkv, D, page, 17 + Hq)
    q = dev_bf16(normal_bf16(40 + T, (len(lens), Hq, T, D)))
    args = (q, cache, _i32(table), _i32(lens), _i64(masks), None, quant)
    o, lse = qat_attention_tree(*args, return_lse=True, check=True)
    _compare(o, lse, q, lens, lambda b: do_.tree_seen(lens[b], masks[b]), cache, page, (table, codes, scales), quant,
             _eps(Hq, Hkv, T, D))
    again = qat_attention_tree(*args, return_lse=True)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 3), (64, 64), (200, 130), (300, 0), (1 << 40, 0)])
@pytest.mark.parametrize("Hq,Hkv,T,D", [(4, 2, 3, 128), (6, 1, 7, 64), (4, 1, 40, 128), (6, 2, 30, 64)])
def test_tree_with_a_window(Hq, Hkv, T, D, window, sinks):
    lens, page = [900, 130, 20, 2], 16
    masks = _trees(np.random.default_rng(T + window % 100), len(lens), T, "tree" if window % 2 else "any")
    if not window % 2:  # bits of no token do not count towards the depth that windows go by
        masks = [[m & ((1 << T) - 1) for m in row] for row in masks]

    def seen_of(b):
        return do_.tree_seen(lens[b], masks[b], window, sinks)

    any_seen = [seen_of(b).any(0) for b in range(len(lens))]
    cache, table, codes, scales = _cache(lens, Hkv, D, page, 21, unseen=lambda b, i: not any_seen[b][i])
    q = dev_bf16(normal_bf16(41, (len(lens), Hq, T, D)))
    o, lse = qat_attention_tree(q, cache, _i32(table), _i32(lens), _i64(masks), return_lse=True, check=True,
                                window=window, sinks=sinks)
    _compare(o, lse, q, lens, seen_of, cache, page, (table, codes, scales), 1, _eps(Hq, Hkv, T, D))


@pytest.mark.parametrize("Hq,T,D", [(2, 5, 64), (4, 40, 128)])
def test_bits_of_no_token(Hq, T, D):
    """Bits from T on are ignored: they name no token, and do not add to the depth that windows go by."""
    lens, page = [300, 60], 16
    masks = _trees(np.random.default_rng(T), 2, T, "tree")
    more = [[m | (2 ** 64 - 2 ** T) for m in row] for row in masks]
    cache, table, _, _ = _cache(lens, 1, D, page, 21)
    q = dev_bf16(normal_bf16(41, (2, Hq, T, D)))
    for how in ({}, dict(window=20, sinks=2)):
        a, b = (qat_attention_tree(q, cache, _i32(table), _i32(lens), _i64(m), return_lse=True, check=True, **how)
                for m in (masks, more))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("lens,Hq,Hkv,T,D", [
    ([40000], 4, 1, 8, 128),                           # one item for all blocks
    ([20000, 5, 0, 300], 8, 1, 16, 64),
    ([1400 + 170 * i for i in range(20)], 4, 2, 12, 128),
    ([3000] + [40 + i % 60 for i in range(199)], 2, 1, 32, 64),
    ([2000] * 6, 16, 4, 64, 128),
    ([40000], 4, 1, 12, 128),                          # the same for the wide kernel
    ([1400 + 170 * i for i in range(20)], 16, 2, 12, 128),
    ([3000] + [40 + i % 60 for i in range(199)], 2, 1, 40, 64),
])
def test_tree_items_cut_by_ranges(lens, Hq, Hkv, T, D):
    """Partials of cut items added up: every row right, the same bits in replays, with a workspace that holds anything,
    and a NaN in one sequence's keys in that sequence's rows alone."""
    page = 64
    masks = _trees(np.random.default_rng(1), len(lens), T, "tree")
    cache, table, codes, scales = _cache(lens, Hkv, D, page, 23)
    q = dev_bf16(normal_bf16(12, (len(lens), Hq, T, D)))
    args = (q, cache, _i32(table), _i32(lens), _i64(masks))
    o, lse = qat_attention_tree(*args, return_lse=True, check=True)
    few = [0, len(lens) // 2, len(lens) - 1]
    for b in sorted(set(few)):
        n = lens[b]
        k, v = (_rows(c, s, table, b, Hkv - 1, n, page) for c, s in zip(codes, scales))
        w, wl, tol, ltol = do_.attend_rows(host_f64(q[b, Hq - 1]), k, v, do_.tree_seen(n, masks[b]), D ** -0.5, True,
                                           _eps(Hq, Hkv, T, D))
        assert (np.abs(host_f64(o[b, Hq - 1]) - w) <= tol).all()
        some = np.isfinite(wl)
        assert (np.abs(host_f64(lse[b, Hq - 1])[some] - wl[some]) <= ltol[some]).all()
    ws = torch.full((capi.qat_attn_tree_workspace_bytes(Hq, Hkv, T, D),), 0xff, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        again = qat_attention_tree(*args, return_lse=True, workspace=ws)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = qat_attention_tree(*args, workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, o)
    at = lens[0] // 3
    cache.k_scale[int(table[0, at // page]), 0, at % page] = float("nan")
    bad, bad_lse = qat_attention_tree(*args, return_lse=True, check=True)
    G = Hq // Hkv
    assert torch.isnan(bad[0, :G]).all() and torch.isnan(bad_lse[0, :G]).all()
    assert torch.equal(bad[1:], o[1:]) and torch.equal(bad[0, G:], o[0, G:]) and torch.equal(bad_lse[1:], lse[1:])


@pytest.mark.parametrize("Hq,T", [(2, 8), (8, 16)])
def test_a_chain_is_decoding(Hq, T):
    """A tree that is a chain is the decoding of its tokens: both within their tolerances of the same values."""
    lens, D, page = [333, 90], 64, 16
    cache, table, codes, scales = _cache(lens, 1, D, page, 4)
    q = dev_bf16(normal_bf16(10, (2, Hq, T, D)))
    chain = _i64([(2 << t) - 1 for t in range(T)])
    for how in ({}, dict(window=40, sinks=2)):
        o, lse = qat_attention_tree(q, cache, _i32(table), _i32(lens), chain, return_lse=True, check=True, **how)
        w, wl = qat_attention_decode(q, cache, _i32(table), _i32(lens), return_lse=True, **how)
        assert torch.allclose(lse, wl, rtol=2.0 ** -18, atol=2.0 ** -16)
        assert float((o.float() - w.float()).norm() / w.float().norm()) <= 2.0 ** -7


def test_one_tree_for_all_and_strided_ones():
    lens, D, page, T = [90, 50, 20], 64, 16, 10
    cache, table, _, _ = _cache(lens, 1, D, page, 4)
    q = dev_bf16(normal_bf16(10, (3, 4, T, D)))
    masks = _trees(np.random.default_rng(3), 1, T, "tree")[0]
    one = qat_attention_tree(q, cache, _i32(table), _i32(lens), _i64(masks), check=True)
    wide = torch.full((3, 2 * T), -1, dtype=torch.int64, device="cuda")
    wide[:, :T] = _i64(masks)
    for tree in (_i64([masks] * 3), _i64(masks).expand(3, T), wide[:, :T]):
        assert torch.equal(one, qat_attention_tree(q, cache, _i32(table), _i32(lens), tree))


@pytest.mark.parametrize("T", [4, 20])
def test_nonfinite_rows_stay_with_who_sees_them(T):
    """A drafted token's NaN row reaches the tokens that see it and no other; a NaN query its own row; a bad page
    the rows that see it."""
    lens, D, page, Hq = [190], 64, 16, 4
    cache, table, _, _ = _cache(lens, 1, D, page, 8)
    masks = do_.draft([-1] + [0 if t % 2 else -1 for t in range(1, T)], T)[0]
    q = dev_bf16(normal_bf16(13, (1, Hq, T, D)))
    args = (q, cache, _i32(table), _i32(lens), _i64(masks))
    clean, clean_lse = qat_attention_tree(*args, return_lse=True)
    at = table[0, (190 - T) // page], 0, (190 - T) % page  # the first drafted token
    with_it = torch.tensor([bool(m & 1) for m in masks], device="cuda")
    for s in (cache.k_scale, cache.v_scale):
        keep = s[at].clone()
        s[at] = float("nan")
        o, lse = qat_attention_tree(*args, return_lse=True)
        assert torch.isnan(o[:, :, with_it]).all() and torch.equal(o[:, :, ~with_it], clean[:, :, ~with_it])
        assert torch.equal(lse[:, :, ~with_it], clean_lse[:, :, ~with_it])
        s[at] = keep
    q[0, 1, 2, 5] = float("nan")
    o = qat_attention_tree(*args)
    assert torch.isnan(o[0, 1, 2]).all()
    o[0, 1, 2] = clean[0, 1, 2]
    assert torch.equal(o, clean)
    q[0, 1, 2, 5] = 0
    table[0, 2] = -1
    bad = qat_attention_tree(q, cache, _i32(table), *args[3:])
    assert torch.isnan(bad).all() and capi.qat_attn_device_status() == Status.BAD_PAGE


@pytest.mark.parametrize("T", [2, 16])
def test_extreme_magnitudes(T):
    """Queries from 2^-126 to 2^100, rows of V that differ by 2^20, and scores hundreds apart."""
    lens, D, page = [200], 128, 16
    cache, table, codes, scales = _cache(lens, 2, D, page, 7, v_spread=3.0)
    masks = [(2 << t) - 1 for t in range(T)]
    q = dev_bf16(normal_bf16(12, (1, 8, T, D))).clone()
    for h, s in enumerate((1.0, 2.0 ** -60, 2.0 ** -126, 0.0, 2.0 ** 60, 2.0 ** 100, 1e-20, 3e4)):
        q[0, h] *= s
    for x, sm, quant in ((q, 2.0 ** -104, 0), (q[:, :1].expand(1, 8, T, D).contiguous(), 2.0, 1)):
        o, lse = qat_attention_tree(x, cache, _i32(table), _i32(lens), _i64(masks), sm, quant, True, check=True)
        _compare(o, lse, x, lens, lambda b: do_.tree_seen(200, masks), cache, page, (table, codes, scales), quant,
                 _eps(8, 2, T, D), sm)


@pytest.mark.parametrize("T", [2, 16, 20])
def test_keys_of_extreme_magnitude(T):
    """Keys near 2^118 and near 2^-105, and queries that bring their scores to about one."""
    lens, D, page = [100], 64, 16
    for power in (118.0, -105.0):
        cache, table, codes, scales = _cache(lens, 1, D, page, 7)
        cache.k_scale.mul_(2.0 ** power * 2.0 ** -8)
        scaled = [scales[0] * np.float32(2.0 ** power * 2.0 ** -8), scales[1]]
        masks = [(2 << t) - 1 for t in range(T)]
        q = dev_bf16(normal_bf16(12, (1, 4, T, D))) * (2.0 ** -power)
        o, lse = qat_attention_tree(q, cache, _i32(table), _i32(lens), _i64(masks), None, 0, True, check=True)
        _compare(o, lse, q, lens, lambda b: do_.tree_seen(100, masks), cache, page, (table, codes, scaled), 0,
                 _eps(4, 1, T, D))


@pytest.mark.parametrize("Hq", [1, 4])
def test_largest_batch(Hq):
    lens = [int(x) for x in np.random.default_rng(8).integers(0, 60, 4096)]
    cache, table, codes, scales = _cache(lens, 1, 64, 16, 3)
    T = 20
    masks = _trees(np.random.default_rng(2), 1, T, "tree")[0]
    q = dev_bf16(normal_bf16(9, (4096, Hq, T, 64)))
    o = qat_attention_tree(q, cache, _i32(table), _i32(lens), _i64(masks), check=True)
    for b in (0, 1, 2047, 4094, 4095):
        k, v = (_rows(c, s, table, b, 0, lens[b], 16) for c, s in zip(codes, scales))
        w, _, tol, _ = do_.attend_rows(host_f64(q[b, 0]), k, v, do_.tree_seen(lens[b], masks), 0.125, True,
                                       _eps(Hq, 1, T, 64))
        assert (np.abs(host_f64(o[b, 0]) - w) <= tol).all()


@pytest.mark.parametrize("change", [
    lambda a: a.update(q=a["q"].float()),
    lambda a: a.update(q=a["q"][:, :3].contiguous()),
    lambda a: a.update(q=a["q"].transpose(1, 2)),
    lambda a: a.update(q=a["q"].repeat(1, 1, 22, 1)),
    lambda a: a.update(tree=a["tree"].int()),
    lambda a: a.update(tree=a["tree"][:, :2]),
    lambda a: a.update(tree=a["tree"].t().contiguous().t()),
    lambda a: a.update(tree=a["tree"].cpu()),
    lambda a: a.update(tree=None),
    lambda a: a.update(block_table=a["block_table"][0]),
    lambda a: a.update(seq_lens=a["seq_lens"].long()),
    lambda a: a.update(window=0),
    lambda a: a.update(window=4, sinks=-1),
    lambda a: a.update(sinks=3),
    lambda a: a.update(sm_scale=-1.0),
    lambda a: a.update(quant_mode=2),
    lambda a: a.update(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
    lambda a: a.update(q=a["q"].clone().requires_grad_(True)),
])
def test_tree_refusals(change):
    cache = KVCache.empty(4, 2, 16, 64)
    args = dict(q=dev_bf16(normal_bf16(5, (2, 4, 3, 64))), cache=cache, block_table=_i32([[0, 1], [2, 3]]),
                seq_lens=_i32([0, 0]), tree=_i64([[1, 3, 5]] * 2))
    assert (qat_attention_tree(**args) == 0).all()
    change(args)
    with pytest.raises((ValueError, TypeError, QatError)):
        qat_attention_tree(**args)
    check_device_status()


# ------------------------------------------------------------------ masks, positions, kept paths

@pytest.mark.parametrize("B,T", [(1, 1), (3, 2), (5, 31), (2, 32), (7, 33), (33, 64), (1000, 17)])
def test_draft_tree(B, T):
    rng = np.random.default_rng(B)
    parents = np.stack([[int(rng.integers(-1, t)) for t in range(T)] for _ in range(B)])
    parents[0] = np.arange(T) - 1                       # the longest path
    if B > 2:
        parents[1] = rng.integers(-3, T + 2, T)         # padding here and there
        parents[2] = np.array([-2 ** 31, 2 ** 31 - 1] * 32)[:T]
    lens = rng.integers(0, 2 ** 31 - 1, B)
    want = [do_.draft(p, n) for p, n in zip(parents, lens)]
    wide = torch.zeros((B, T + 3), dtype=torch.int32, device="cuda")
    wide[:, :T] = _i32(parents)
    for given in (_i32(parents), wide[:, :T]):
        tree, pos = qat_draft_tree(given, _i32(lens))
        assert tree.dtype == torch.int64 and pos.dtype == torch.int32
        assert torch.equal(tree, _i64([m for m, _ in want]))
        assert torch.equal(pos, _i32(np.stack([p for _, p in want])))
    tree, _ = qat_draft_tree(_i32(parents[0]), _i32(lens))
    assert torch.equal(tree, _i64([want[0][0]] * B))


def test_draft_tree_refusals():
    parents, lens = _i32([[-1, 0], [-1, 0]]), _i32([5, 5])
    for p, n in ((parents.long(), lens), (parents, lens.long()), (parents, lens[:1]), (parents.t(), lens),
                 (parents, lens.cpu()), (_i32(np.zeros((2, 65))), lens), (parents[0, 0], lens)):
        with pytest.raises((ValueError, QatError)):
            qat_draft_tree(p, n)
    tree, pos = qat_draft_tree(_i32(np.zeros((0, 4))), _i32(np.zeros(0)))
    assert tree.shape == pos.shape == (0, 4)
    assert qat_draft_tree(_i32(np.zeros((2, 0))), lens)[0].shape == (2, 0)


def _bytes(cache):
    return [t.clone() for t in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale.view(torch.int32),
                                cache.v_scale.view(torch.int32))]


@pytest.mark.parametrize("lens,H,T,L,D,page", [
    ([10], 1, 4, 4, 64, 16),
    ([100, 64, 33], 2, 32, 9, 128, 16),
    ([130, 3, 0, 64, 65], 3, 64, 64, 128, 64),          # shorter than their trees too
    ([300] * 40, 8, 16, 16, 64, 256),
])
@pytest.mark.parametrize("kind", ["ascending", "any"])
def test_keep(lens, H, T, L, D, page, kind):
    """Codes and scales of every slot after the move, bit for bit; any order and repeats; counts out of range."""
    rng = np.random.default_rng(T + L)
    cache, table, _, _ = _cache(lens, H, D, page, 5)
    B = len(lens)
    path = np.stack([np.sort(rng.permutation(T)[:L]) if kind == "ascending" else rng.integers(0, T, L)
                     for _ in range(B)])
    kept = rng.integers(0, L + 1, B)
    kept[0] = L + 3
    if B > 1:
        kept[1] = -2
    moves, new = do_.keep(lens, T, path, kept)
    want = _bytes(cache)
    old = [x.clone() for x in want]
    for b, src, dst in moves:
        for x, y in zip(want, old):
            x[int(table[b, dst // page]), :, dst % page] = y[int(table[b, src // page]), :, src % page]
    got = cache.keep(_i32(table), _i32(lens), T, _i32(path), _i32(kept), check=True)
    assert got.tolist() == new and got.dtype == torch.int32
    assert all(torch.equal(x, y) for x, y in zip(want, _bytes(cache)))


def test_keep_bad_entries():
    """What is outside is not moved, not followed, and reported; the rest moves."""
    lens, T, page = [40, 40], 8, 16
    cache, table, _, _ = _cache(lens, 1, 64, page, 5)
    path = [[1, 8, 3], [2, -1, 7]]
    before = _bytes(cache)
    with pytest.raises(QatError) as e:
        cache.keep(_i32(table), _i32(lens), T, _i32(path), _i32([3, 3]), check=True)
    assert e.value.status == Status.BAD_PAGE
    for x, y in zip(_bytes(cache), before):
        for b, i, p in ((0, 32, 33), (0, 33, 33), (0, 34, 35), (1, 32, 34), (1, 33, 33), (1, 34, 39)):
            assert torch.equal(x[int(table[b, i // page]), :, i % page], y[int(table[b, p // page]), :, p % page])
    given = table.copy()
    given[0, 2], given[1, 2] = -1, 10 ** 6
    before = _bytes(cache)
    cache.keep(_i32(given), _i32(lens), T, _i32([[1, 2], [1, 2]]), _i32([2, 2]))
    assert capi.qat_attn_device_status() == Status.BAD_PAGE
    assert all(torch.equal(x, y) for x, y in zip(_bytes(cache), before))
    new = cache.keep(_i32(table), _i32([10 ** 9, 40]), T, _i32([[1], [1]]), _i32([1, 0]))
    assert capi.qat_attn_device_status() == Status.BAD_PAGE and new.tolist() == [10 ** 9 - 7, 32]
    assert all(torch.equal(x, y) for x, y in zip(_bytes(cache), before))


def test_keep_refusals():
    cache, table, _, _ = _cache([40], 1, 64, 16, 5)
    good = (_i32(table), _i32([40]), 8, _i32([[1, 2]]), _i32([2]))
    for i, bad in ((1, _i32([40, 40])), (2, 65), (2, 1), (2, -1), (3, _i32([1, 2])), (3, good[3].long()),
                   (4, _i32([[2]])), (4, good[4].cpu()), (0, _i32(table[0]))):
        args = list(good)
        args[i] = bad
        with pytest.raises((ValueError, QatError)):
            cache.keep(*args)
    assert cache.keep(_i32(table), _i32([40]), 8, _i32(np.zeros((1, 0))), _i32([0])).tolist() == [32]
    check_device_status()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("T,window", [(3, None), (12, 48), (20, 48)])
def test_drafting_steps(T, window, captured):
    """Prompts, then steps of drafting: masks and positions, norm and rotation, append, the tree's attention, keeping
    a path, and a plain token behind it, which must see the kept rows as if they had been appended one by one."""
    B, Hq, Hkv, D, page, steps = 2, 8, 2, 64, 16, 3
    rng = np.random.default_rng(2)
    rope = RopePlan(D, base=10000.0)
    wq, wk = (torch.ones(D, device="cuda") for _ in range(2))
    lens = [70, 33]
    per = 14
    table = _i32(rng.permutation(B * per).reshape(B, per))
    caches = [KVCache.empty(B * per, Hkv, page, D) for _ in range(2)]  # drafted, and one by one
    prompt = [dev_bf16(normal_bf16(20 + i, (B, Hkv, max(lens), D))) for i in range(2)]
    for c in caches:
        c.append(*prompt, table, _i32(lens), _i32(lens), check=True)
    # P is not quantized here: a drafted token lies in another slot than when it is appended alone, so it may fall into
    # another 64-key tile, whose largest P and with it the rounding of all of its P (2^-4 each) is another
    how = dict(quant_mode=0, **({} if window is None else dict(window=window, sinks=4)))

    seq = _i32([n + T for n in lens])
    bufs = [torch.empty((B, h, T, D), dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv)]
    parents, path, kept = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((B, T), (B, T), (B,)))

    def step():
        tree, positions = qat_draft_tree(parents, seq)
        q, k = qat_qk_norm_rope(bufs[0], bufs[1], positions, rope, wq, wk)
        caches[0].append(k, bufs[2], table, seq)
        o = qat_attention_tree(q, caches[0], table, seq, tree, **how)
        return o, q, k, positions, caches[0].keep(table, seq, T, path, kept)

    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        state = [t.clone() for t in (caches[0].k, caches[0].v, caches[0].k_scale, caches[0].v_scale)]
        for t in (parents, path, kept):
            t.fill_(0)
        parents.fill_(-1)
        for t in bufs:
            t.fill_(1.0)
        with torch.cuda.stream(side):
            step()  # the first call of a kernel loads it
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for t, s in zip((caches[0].k, caches[0].v, caches[0].k_scale, caches[0].v_scale), state):
            t.copy_(s)
    for i in range(steps):
        tree = np.stack([[int(rng.integers(max(-1, t - 3), t)) for t in range(T)] for _ in range(B)])
        parents.copy_(_i32(tree))
        for j, t in enumerate(bufs):
            t.copy_(dev_bf16(normal_bf16(100 * i + j, tuple(t.shape))))
        paths = []
        for b in range(B):  # the path of the last token, or of one before it
            t, p = T - 1 - i % 2, []
            while t >= 0:
                p.insert(0, t)
                t = int(tree[b, t])
            paths.append(p)
        path.copy_(_i32([p + [0] * (T - len(p)) for p in paths]))
        kept.copy_(_i32([len(p) for p in paths]))
        if captured:
            graph.replay()
        else:
            out = step()
        o, q, k, positions, new = out
        check_device_status()
        assert new.tolist() == [n + len(p) for n, p in zip(lens, paths)]
        # one by one: the path's tokens appended to the other cache, the last of them decoded
        for b in range(B):
            rows = slice(b, b + 1)
            for d, t in enumerate(paths[b]):
                n = _i32([lens[b] + d + 1])
                assert int(positions[b, t]) == lens[b] + d
                caches[1].append(k[rows, :, t:t + 1], bufs[2][rows, :, t:t + 1], table[rows], n)
                w = qat_attention_decode(q[rows, :, t:t + 1].contiguous(), caches[1], table[rows], n, **how)
                # both round weights and outputs: bf16's half step each (the tree's weights are bf16's from 65 rows on)
                err = (o[rows, :, t:t + 1].float() - w.float()).norm() / w.float().norm()
                assert float(err) <= 2.0 ** -7, (i, b, t, float(err))
            lens[b] += len(paths[b])
        for x, y in zip(caches[0].read(table, _i32(lens), check=True), caches[1].read(table, _i32(lens), check=True)):
            assert torch.equal(x, y)
        seq.copy_(_i32([n + T for n in lens]))


def test_calls_on_two_streams():
    """Calls with workspaces of their own on two streams at once give what each gives alone."""
    lens, D, page, T = [3000, 700], 128, 64, 16
    cache, table, _, _ = _cache(lens, 2, D, page, 31)
    masks = _i64(_trees(np.random.default_rng(4), 2, T, "tree"))
    qs = [dev_bf16(normal_bf16(60 + i, (2, 8, T, D))) for i in range(2)]
    args = [(q, cache, _i32(table), _i32(lens)) for q in qs]
    want = [(qat_attention_tree(*a, masks), qat_attention_decode(*a, window=300, sinks=4)) for a in args]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((qat_attention_tree(*args[i], masks), qat_attention_decode(*args[i], window=300, sinks=4)))
    torch.cuda.synchronize()
    for i in range(2):
        for x, y in got[i]:
            assert torch.equal(x, want[i][0]) and torch.equal(y, want[i][1])


@pytest.mark.parametrize("Hq,T", [(8, 4), (16, 16)])
def test_offsets_beyond_32_bits(Hq, T):
    """A cache whose codes pass 2^32 bytes, the sequences on its last pages: the bits of a small cache's results."""
    lens, Hkv, D, page, B = [300, 77], 8, 128, 128, 2
    small, table, _, _ = _cache(lens, Hkv, D, page, 5)
    n, pages = small.k.shape[0], (1 << 32) // (Hkv * page * D) + 40
    big = KVCache.empty(pages, Hkv, page, D)
    for x, y in ((big.k, small.k), (big.v, small.v)):
        x.view(torch.uint8)[pages - n:] = y.view(torch.uint8)
    for x, y in ((big.k_scale, small.k_scale), (big.v_scale, small.v_scale)):
        x[pages - n:] = y
    q = dev_bf16(normal_bf16(12, (B, Hq, T, D)))
    tree = _i64(_trees(np.random.default_rng(T), 1, T, "tree")[0])
    path, kept = _i32(np.stack([np.arange(1, T, 2)] * B)), _i32([T // 2] * B)
    got = []
    for cache, at in ((small, 0), (big, pages - n)):
        given = _i32(table + at)
        got.append((qat_attention_tree(q, cache, given, _i32(lens), tree, check=True),
                    qat_attention_decode(q, cache, given, _i32(lens), window=100, sinks=4, check=True),
                    cache.keep(given, _i32(lens), T, path, kept, check=True)))
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert torch.equal(big.k.view(torch.uint8)[pages - n:], small.k.view(torch.uint8))
    assert torch.equal(big.v_scale[pages - n:].view(torch.int32), small.v_scale.view(torch.int32))


def test_expired_waits_of_the_wide_kernel():
    """With the waits' limit at nothing the kernel gives up at a wait, lets its copies and products complete, reports it
    and returns; the next call gives what the first gave."""
    lens, D, page, T, Hq = [20000, 300, 9000], 128, 64, 32, 8
    cache, table, _, _ = _cache(lens, 1, D, page, 4)
    q = dev_bf16(normal_bf16(10, (3, Hq, T, D)))
    args = (q, cache, _i32(table), _i32(lens), _i64(_trees(np.random.default_rng(4), 3, T, "tree")))
    want = qat_attention_tree(*args, check=True)
    assert capi.qat_debug_set_wait_limit_us(0) == Status.OK
    try:
        with pytest.raises(QatError) as e:
            for _ in range(5):
                qat_attention_tree(*args, check=True)
        assert e.value.status == Status.TIMEOUT
    finally:
        assert capi.qat_debug_set_wait_limit_us(4000000) == Status.OK
        capi.qat_attn_device_status()
    assert torch.equal(qat_attention_tree(*args, check=True), want)


def test_nothing_to_do():
    """No sequences, no tokens, no drafted tokens."""
    cache = KVCache.empty(4, 2, 16, 64)
    table, lens = _i32([[0, 1]]), _i32([20])

    def q(B, T):
        return torch.zeros((B, 4, T, 64), dtype=torch.bfloat16, device="cuda")

    tree = torch.zeros((1, 3), dtype=torch.int64, device="cuda")
    assert qat_attention_tree(q(1, 0), cache, table, lens, tree[:, :0]).shape == (1, 4, 0, 64)
    for given in (tree[:0], tree[0]):
        assert qat_attention_tree(q(0, 3), cache, table[:0], lens[:0], given).shape == (0, 4, 3, 64)
    assert qat_attention_decode(q(1, 0), cache, table, lens, window=3).shape == (1, 4, 0, 64)
    assert cache.keep(table[:0], lens[:0], 3, _i32([[0]])[:0], lens[:0]).shape == (0,)
    assert cache.keep(table, lens, 0, _i32(np.zeros((1, 0))), _i32([0])).tolist() == [20]
    check_device_status()


def test_many_rows_of_one_head():
    """64 query heads a KV head and 64 tokens: 4096 rows, 32 row tiles."""
    lens, D, page, T, Hq = [150], 64, 16, 64, 64
    cache, table, codes, scales = _cache(lens, 1, D, page, 6)
    masks = _trees(np.random.default_rng(9), 1, T, "tree")
    q = dev_bf16(normal_bf16(14, (1, Hq, T, D)))
    o, lse = qat_attention_tree(q, cache, _i32(table), _i32(lens), _i64(masks), return_lse=True, check=True)
    _compare(o, lse, q, lens, lambda b: do_.tree_seen(lens[b], masks[b]), cache, page, (table, codes, scales), 1,
             _eps(Hq, 1, T, D))
