"""GPU tests of a drafted tree's attention at its edges, the narrow and the wide kernel alike: codes that are not a number,
and pages that no token's window reaches."""

import numpy as np
import pytest
import torch

from oracle import drafted_oracle as do_
from quantization_aware_attention_gb300 import check_device_status, qat_attention_tree
from quantization_aware_attention_gb300 import build as qbuild
from quantization_aware_attention_gb300 import capi
from quantization_aware_attention_gb300.capi import Status
from quantization_aware_attention_gb300.inputs import normal_bf16

from gpu_util import dev_bf16
from test_gpu_drafted import _cache, _i32, _i64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    qbuild.build()


@pytest.mark.parametrize("Hq,T,D", [(4, 4, 64), (2, 3, 128), (4, 20, 64), (4, 20, 128)])  # 16, 6, 80 and 80 rows
@pytest.mark.parametrize("quant", [0, 1])
def test_codes_that_are_not_a_number(Hq, T, D, quant):
    """An E4M3 NaN, which a cache that others filled may hold, counts as NaN: in a key it is the whole row of every token
    that sees the key and of no other; in a value the channel of every token that sees it (with the kernel of few rows
    possibly of others as well)."""
    lens, page = [190], 16
    cache, table, _, _ = _cache(lens, 1, D, page, 8)
    masks = do_.draft([-1] + [0 if t % 2 else -1 for t in range(1, T)], T)[0]
    q = dev_bf16(normal_bf16(13, (1, Hq, T, D)))
    args = (q, cache, _i32(table), _i32(lens), _i64(masks), None, quant, True)
    clean, clean_lse = qat_attention_tree(*args)
    k, v = cache.k.view(torch.uint8), cache.v.view(torch.uint8)
    every = torch.ones(T, dtype=torch.bool, device="cuda")
    first = torch.tensor([bool(m & 1) for m in masks], device="cuda")
    assert not first.all()
    for pos, rows in ((37, every), (190 - T, first)):  # in the text; the first drafted token
        at = table[0, pos // page], 0, pos % page
        for d in range(D):
            code = 0x7f if d % 3 else 0xff
            keep, k[at][d] = int(k[at][d]), code
            o, lse = qat_attention_tree(*args)
            k[at][d] = keep
            assert torch.isnan(o[:, :, rows]).all() and torch.isnan(lse[:, :, rows]).all(), (pos, d)
            assert torch.equal(o[:, :, ~rows], clean[:, :, ~rows]) and torch.equal(lse[:, :, ~rows], clean_lse[:, :, ~rows])
            keep, v[at][d] = int(v[at][d]), code
            o, lse = qat_attention_tree(*args)
            v[at][d] = keep
            assert torch.isnan(o[:, :, rows, d]).all(), (pos, d)
            if Hq * T > (64 if D == 64 else 32):
                assert torch.equal(o[:, :, ~rows], clean[:, :, ~rows]), (pos, d)
            others = [c for c in range(D) if c != d]
            assert torch.equal(o[..., others], clean[..., others]) and torch.equal(lse, clean_lse), (pos, d)
    assert torch.equal(qat_attention_tree(*args)[0], clean)
    check_device_status()


SHAPES = [(4, 2, 3, 128), (6, 1, 7, 64), (4, 1, 40, 128), (6, 2, 30, 64)]  # 6 and 42 rows, 160 and 90


def _masks(rng, B, T):
    """Trees whose first token's mask is empty, as padding's is."""
    out = [do_.draft([int(rng.integers(max(-1, t - 8), t)) for t in range(T)], T)[0] for _ in range(B)]
    for m in out:
        m[0] = 0
    return out


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 3), (64, 64), (70, 17), (200, 130)])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("Hq,Hkv,T,D", SHAPES)
def test_pages_that_no_token_sees(Hq, Hkv, T, D, page, window, sinks):
    """Pages of keys before seq_lens - T - window that hold no sinks may be anything in the block table."""
    lens = [1500, 700, 130, 20, 2]
    masks = _masks(np.random.default_rng(T), len(lens), T)
    cache, table, _, _ = _cache(lens, Hkv, D, page, 21)
    given, gone = table.copy(), 0
    for b, n in enumerate(lens):
        for p in range(table.shape[1]):
            if (p + 1) * page <= n - T - window and p * page >= sinks:
                given[b, p] = -1 if p % 2 else 1 << 30
                gone += 1
    assert gone > 0
    q = dev_bf16(normal_bf16(41, (len(lens), Hq, T, D)))
    how = dict(return_lse=True, check=True, window=window, sinks=sinks)
    want = qat_attention_tree(q, cache, _i32(table), _i32(lens), _i64(masks), **how)
    got = qat_attention_tree(q, cache, _i32(given), _i32(lens), _i64(masks), **how)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("page,sinks", [(16, 0), (32, 33), (256, 1)])
@pytest.mark.parametrize("Hq,Hkv,T,D", SHAPES)
def test_a_page_that_begins_with_the_first_key_seen(Hq, Hkv, T, D, page, sinks):
    """Key seq_lens - T - window begins a page: a token with an empty mask sees it, and none the page before."""
    window = 2 * page - T % 5
    lens = [3 * page + window + T]
    masks = _masks(np.random.default_rng(T), 1, T)
    cache, table, _, _ = _cache(lens, Hkv, D, page, 9)
    q = dev_bf16(normal_bf16(13, (1, Hq, T, D)))
    how = dict(window=window, sinks=sinks)
    want = qat_attention_tree(q, cache, _i32(table), _i32(lens), _i64(masks), check=True, **how)
    given = table.copy()
    given[0, 2] = -1
    assert torch.equal(qat_attention_tree(q, cache, _i32(given), _i32(lens), _i64(masks), check=True, **how), want)
    given[0, 3] = 1 << 30
    got = qat_attention_tree(q, cache, _i32(given), _i32(lens), _i64(masks), **how)
    assert capi.qat_attn_device_status() == Status.BAD_PAGE
    assert torch.isnan(got[:, :, 0]).all()


@pytest.mark.parametrize("window,sinks", [(None, 0), (300, 20)])
@pytest.mark.parametrize("Hq,T,D", [(8, 16, 128), (4, 40, 64)])  # 128 and 160 rows a KV head
def test_codes_that_are_not_a_number_in_many_steps(Hq, T, D, window, sinks):
    """In some sequences' pages, at several places of many steps, and behind a sequence's end: with the kernel of many rows
    what no token sees changes nothing, and the other sequences keep their bits."""
    lens, page = [5000, 131, 2600, 700], 32
    masks = _masks(np.random.default_rng(T), len(lens), T)
    cache, table, _, _ = _cache(lens, 1, D, page, 25)
    q = dev_bf16(normal_bf16(17, (len(lens), Hq, T, D)))
    how = {} if window is None else dict(window=window, sinks=sinks)
    args = (q, cache, _i32(table), _i32(lens), _i64(masks), None, 1, True)
    clean, clean_lse = qat_attention_tree(*args, **how)
    assert torch.isfinite(clean).all()
    hit = torch.zeros((len(lens), T), dtype=torch.bool, device="cuda")
    for b, places in ((0, (0, 15, 1000, 2047, 4700)), (2, (3, 1100, 2590))):
        seen = do_.tree_seen(lens[b], masks[b], window, sinks)
        for i, pos in enumerate(places):
            at = table[b, pos // page], 0, pos % page
            codes = (cache.k, cache.v)[i % 2].view(torch.uint8)
            codes[at][(37 * i + 5) % D] = 0x7f + 0x80 * (i % 2)
            hit[b] |= torch.from_numpy(seen[:, pos]).cuda()
    assert hit[0].any() and not hit[1].any()
    o, lse = qat_attention_tree(*args, **how, check=True)
    hit = hit[:, None].expand(-1, Hq, -1)
    assert torch.isnan(o[hit]).any(-1).all()
    assert torch.equal(o[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])
