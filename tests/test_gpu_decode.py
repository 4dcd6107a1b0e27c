"""GPU parity of the attention of new tokens over the FP8 cache against the fp64 oracle, which also gives
the tolerances (oracle/serving_oracle.py, decode_head)."""

import numpy as np
import pytest
import torch

from oracle import serving_oracle as so
from quantization_aware_attention_gb300 import KVCache, QatError, check_device_status, qat_attention_decode
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
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache(lens, H, D, page, seed, v_spread=1.0):
    """A cache whose every slot is written: normal rows of differing magnitudes; what no sequence may see
    (the ends of last pages, spare pages) is NaN rows."""
    B = len(lens)
    per = max(1, max((n + page - 1) // page for n in lens))
    pages = B * per + 2
    rng = np.random.default_rng(seed)
    table = rng.permutation(pages)[:B * per].reshape(B, per).astype(np.int32)
    codes, scales = [], []
    for spread in (1.0, v_spread):
        x = rng.standard_normal((pages, H, page, D)).astype(np.float32)
        x *= np.exp(spread * rng.standard_normal((pages, H, page, 1))).astype(np.float32)
        c, s = so.quant_row(x)
        hidden = np.ones((pages, page), bool)
        for b, n in enumerate(lens):
            for i in range(n):
                hidden[table[b, i // page], i % page] = False
        hidden = np.broadcast_to(hidden[:, None], s.shape)
        s = np.where(hidden, np.float32(np.nan), s)
        codes.append(c)
        scales.append(s)
    f8 = [torch.from_numpy(c).cuda().view(torch.float8_e4m3fn) for c in codes]
    cache = KVCache(f8[0], f8[1], *(torch.from_numpy(s).cuda() for s in scales))
    return cache, table, codes, scales


def _sequence(codes, scales, table, b, h, n, page):
    """Rows 0..n-1 of a sequence's head, [n, D] fp64."""
    i = np.arange(n)
    at = table[b, i // page], h, i % page
    return so.dequant(codes[at], scales[at])


def _check(q, lens, Hkv, page, cache, table, codes, scales, quant, sm_scale=None, heads=None, **kw):
    B, Hq, T, D = q.shape
    sm = D ** -0.5 if sm_scale is None else sm_scale
    o, lse = qat_attention_decode(q, cache, _i32(table), _i32(lens), sm_scale, quant, return_lse=True,
                                  check=True, **kw)
    fq, fo, fl = host_f64(q), host_f64(o), host_f64(lse)
    for b in range(B):
        for h in (range(Hkv) if heads is None else heads):
            k, v = (_sequence(c, s, table, b, h, lens[b], page) for c, s in zip(codes, scales))
            for g in range(Hq // Hkv):
                hq = h * (Hq // Hkv) + g
                w, wl, tol, ltol = so.decode_head(fq[b, hq], k, v, lens[b] - T + np.arange(T), sm, quant)
                err = np.abs(fo[b, hq] - w)
                assert (err <= tol).all(), (b, hq, float((err / np.maximum(tol, 1e-300)).max()))
                seen = np.isfinite(wl)
                assert np.array_equal(np.isneginf(fl[b, hq]), ~seen)
                assert (np.abs(fl[b, hq][seen] - wl[seen]) <= ltol[seen]).all()
    return o, lse


@pytest.mark.parametrize("quant", [0, 1])
@pytest.mark.parametrize("lens,Hq,Hkv,T,D,page", [
    ([1], 1, 1, 1, 128, 16),
    ([0], 4, 2, 1, 64, 16),
    ([64], 4, 4, 1, 64, 64),
    ([65, 63, 0, 1], 8, 2, 1, 128, 16),
    ([300], 8, 1, 1, 128, 32),
    ([17, 129, 1000], 6, 2, 1, 64, 128),
    ([40, 3, 200], 5, 1, 5, 128, 16),        # 25 rows: two row tiles; a sequence shorter than its tokens
    ([77, 1], 32, 2, 16, 64, 32),            # 256 rows; more tokens than keys
    ([513, 255, 256, 257], 16, 16, 2, 128, 256),
    ([1500, 2], 40, 8, 3, 128, 64),
])
def test_decode(lens, Hq, Hkv, T, D, page, quant):
    cache, table, codes, scales = _cache(lens, Hkv, D, page, 17 + Hq)
    q = dev_bf16(normal_bf16(40 + T, (len(lens), Hq, T, D)))
    o, lse = _check(q, lens, Hkv, page, cache, table, codes, scales, quant)
    again = qat_attention_decode(q, cache, _i32(table), _i32(lens), None, quant, return_lse=True)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_many_sequences():
    """More sequences than a block has threads, most of them short or empty: the prefix sums and the
    ranges that cut items anywhere."""
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 150, 700)]
    lens[13], lens[14], lens[699] = 2500, 0, 0
    cache, table, codes, scales = _cache(lens, 1, 64, 16, 3)
    q = dev_bf16(normal_bf16(9, (700, 3, 1, 64)))
    _check(q, lens, 1, 16, cache, table, codes, scales, 1)


def test_largest_batch():
    """4096 sequences, the most a call takes; one more is refused."""
    lens = [int(x) for x in np.random.default_rng(8).integers(0, 40, 4096)]
    cache, table, codes, scales = _cache(lens, 1, 64, 16, 3)
    q = dev_bf16(normal_bf16(9, (4096, 1, 1, 64)))
    o = qat_attention_decode(q, cache, _i32(table), _i32(lens), check=True)
    for b in (0, 1, 2047, 4094, 4095):
        k, v = (_sequence(c, s, table, b, 0, lens[b], 16) for c, s in zip(codes, scales))
        w, _, tol, _ = so.decode_head(host_f64(q[b, 0]), k, v, np.array([lens[b] - 1]), 0.125, 1)
        assert (np.abs(host_f64(o[b, 0]) - w) <= tol).all()
    with pytest.raises(QatError) as e:
        qat_attention_decode(dev_bf16(normal_bf16(9, (4097, 1, 1, 64))), cache,
                             _i32(np.zeros((4097, 1), np.int32)), _i32([0] * 4097))
    assert e.value.status == Status.UNSUPPORTED


def test_long_sequence():
    lens = [20011]
    cache, table, codes, scales = _cache(lens, 2, 128, 64, 4)
    q = dev_bf16(normal_bf16(10, (1, 8, 1, 128)))
    _check(q, lens, 2, 64, cache, table, codes, scales, 1)


@pytest.mark.parametrize("lens,Hq,Hkv,T,D", [
    ([20011], 4, 1, 1, 64),                         # one item: some blocks share its partials
    ([131071], 3, 1, 1, 128),                       # many
    ([70000, 5, 0, 300], 8, 1, 2, 64),              # beside items that are whole
    ([2900 + 17 * i for i in range(40)], 8, 1, 1, 64),   # more rows than fit at once
    ([3000] + [1 + i % 60 for i in range(199)], 2, 1, 1, 64),    # one long chain among short ones
    ([9000 + i for i in range(24)], 4, 4, 1, 64),   # long chains of every warp
    ([1100] * 12, 1, 1, 1, 128),
])
def test_cut_items(lens, Hq, Hkv, T, D):
    """What ranges leave of the items they cut, added up by a warp, a block or several blocks: every row
    right, the same bits again, and a NaN in one sequence's keys in that sequence's rows alone."""
    cache, table, codes, scales = _cache(lens, Hkv, D, 64, 23)
    q = dev_bf16(normal_bf16(12, (len(lens), Hq, T, D)))
    o, lse = _check(q, lens, Hkv, 64, cache, table, codes, scales, 1, heads=[Hkv - 1])
    args = (q, cache, _i32(table), _i32(lens))
    again = qat_attention_decode(*args, return_lse=True)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = qat_attention_decode(*args, return_lse=True)
    for _ in range(2):
        again[0].zero_()
        graph.replay()
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    at = lens[0] // 3
    cache.k_scale[int(table[0, at // 64]), 0, at % 64] = float("nan")
    bad, bad_lse = qat_attention_decode(*args, return_lse=True, check=True)
    rows = Hq // Hkv
    assert torch.isnan(bad[0, :rows]).all() and torch.isnan(bad_lse[0, :rows]).all()
    assert torch.equal(bad[1:], o[1:]) and torch.equal(bad_lse[1:], lse[1:])
    assert torch.equal(bad[0, rows:], o[0, rows:]) and torch.equal(bad_lse[0, rows:], lse[0, rows:])


@pytest.mark.parametrize("D,Hq,Hkv,T", [(64, 16, 8, 1), (128, 8, 8, 1), (64, 24, 8, 3), (128, 16, 4, 4)])
def test_batch_of_long_sequences(D, Hq, Hkv, T):
    """Many tiles for every warp, items cut anywhere, one item cut many times: every row right, the same
    bits in every run and in every replay of a captured call, with a workspace that holds anything."""
    B, page = 24, 64
    rng = np.random.default_rng(6)
    lens = [int(x) for x in rng.integers(4000, 9000, B)]
    lens[3], lens[7] = 65000, 1
    if Hkv == 4:
        lens = [2 * n for n in lens]
    per = [(n + page - 1) // page for n in lens]
    pages = sum(per)
    order = rng.permutation(pages).astype(np.int32)
    table = np.zeros((B, max(per)), np.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    g = torch.Generator(device="cuda").manual_seed(3)
    codes = [(torch.randn(pages, Hkv, page, D, generator=g, device="cuda") * 100).clamp(-448, 448).to(
        torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.rand(pages, Hkv, page, generator=g, device="cuda") * 0.02 + 0.002 for _ in range(2)]
    cache = KVCache(codes[0], codes[1], scales[0], scales[1])
    q = dev_bf16(normal_bf16(77, (B, Hq, T, D)))
    args = (q, cache, _i32(table), _i32(lens))
    o, lse = qat_attention_decode(*args, return_lse=True, check=True)
    for b, h in ((0, 0), (3, Hkv - 1), (7, 1), (B - 1, Hkv - 1), (11, 2)):
        n = lens[b]
        t = torch.from_numpy(table[b, :per[b]]).cuda().long()
        k, v = (so.dequant(c[t][:, h].reshape(-1, D)[:n].view(torch.uint8).cpu().numpy(),
                           s[t][:, h].reshape(-1)[:n].cpu().numpy()) for c, s in zip(codes, scales))
        for hq in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
            w, wl, tol, ltol = so.decode_head(host_f64(q[b, hq]), k, v, n - T + np.arange(T), D ** -0.5, 1)
            assert (np.abs(host_f64(o[b, hq]) - w) <= tol).all()
            seen = np.isfinite(wl)
            assert (np.abs(host_f64(lse[b, hq])[seen] - wl[seen]) <= ltol[seen]).all()
    ws = torch.randint(0, 256, (capi.qat_attn_decode_workspace_bytes(Hq, Hkv, T, D),), dtype=torch.uint8,
                       device="cuda")
    for _ in range(3):
        again = qat_attention_decode(*args, return_lse=True, workspace=ws)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = qat_attention_decode(*args, workspace=ws)
    for _ in range(4):
        out.zero_()
        graph.replay()
        assert torch.equal(out, o)


@pytest.mark.parametrize("quant", [0, 1])
def test_peaked_scores_and_scales(quant):
    """Scores hundreds apart (tiles that underflow, the maximum rising tile by tile) and rows of V whose
    magnitudes differ by 2^20."""
    lens, D, page = [700], 64, 16
    cache, table, codes, scales = _cache(lens, 1, D, page, 6, v_spread=3.0)
    q = dev_bf16(normal_bf16(11, (1, 2, 1, D)))
    _check(q, lens, 1, page, cache, table, codes, scales, quant, sm_scale=2.0)


def test_queries_of_extreme_magnitude():
    lens, D, page = [200], 128, 16
    cache, table, codes, scales = _cache(lens, 2, D, page, 7)
    q = dev_bf16(normal_bf16(12, (1, 8, 1, D))).clone()
    for h, s in enumerate((1.0, 2.0 ** -60, 2.0 ** -126, 0.0, 2.0 ** 60, 2.0 ** 100, 1e-20, 3e4)):
        q[0, h] *= s
    sm = 2.0 ** -104  # the largest row's scores stay finite; the others' weights are all equal
    _check(q, lens, 2, page, cache, table, codes, scales, 0, sm_scale=sm)


def test_nonfinite_rows_stay_with_who_sees_them():
    """A NaN row of the cache reaches the tokens that see it and no other; a NaN query its own row."""
    lens, D, page = [90], 64, 16
    cache, table, codes, scales = _cache(lens, 1, D, page, 8)
    q = dev_bf16(normal_bf16(13, (1, 2, 3, D)))
    clean = qat_attention_decode(q, cache, _i32(table), _i32(lens))
    at = table[0, 89 // page], 0, 89 % page  # the newest token's row
    for s in (cache.k_scale, cache.v_scale):
        keep = s[at].clone()
        s[at] = float("nan")
        o, lse = qat_attention_decode(q, cache, _i32(table), _i32(lens), return_lse=True)
        assert torch.isnan(o[:, :, 2]).all() and torch.equal(o[:, :, :2], clean[:, :, :2])
        assert torch.isfinite(lse[:, :, :2]).all()
        s[at] = keep
    q[0, 1, 1, 5] = float("nan")
    o = qat_attention_decode(q, cache, _i32(table), _i32(lens))
    assert torch.isnan(o[0, 1, 1]).all()
    o[0, 1, 1] = clean[0, 1, 1]
    assert torch.equal(o, clean)


@pytest.mark.parametrize("bad", [-7, 99])
def test_bad_pages_give_nan_and_are_reported(bad):
    lens, D, page = [40, 30], 64, 16
    cache, table, codes, scales = _cache(lens, 1, D, page, 9)
    q = dev_bf16(normal_bf16(13, (2, 2, 1, D)))
    good = qat_attention_decode(q, cache, _i32(table), _i32(lens))
    table[0, 1] = bad
    with pytest.raises(QatError) as e:
        qat_attention_decode(q, cache, _i32(table), _i32(lens), check=True)
    assert e.value.status == Status.BAD_PAGE
    o = qat_attention_decode(q, cache, _i32(table), _i32(lens))
    assert torch.isnan(o[0]).all() and torch.equal(o[1], good[1])
    capi.qat_attn_device_status()
    # behind the sequence's end the entry is never looked at
    assert torch.isfinite(qat_attention_decode(q, cache, _i32(table), _i32([16, 30]), check=True)).all()


def test_lengths_beyond_the_table():
    cache, table, codes, scales = _cache([32], 1, 64, 16, 9)
    q = dev_bf16(normal_bf16(13, (1, 1, 1, 64)))
    with pytest.raises(QatError):
        qat_attention_decode(q, cache, _i32(table), _i32([10 ** 9]), check=True)
    # as many keys as the table holds, and a negative length none
    o = qat_attention_decode(q, cache, _i32(table), _i32([33]))
    assert torch.isfinite(o).all()
    assert capi.qat_attn_device_status() == Status.BAD_PAGE
    o, lse = qat_attention_decode(q, cache, _i32(table), _i32([-5]), return_lse=True, check=True)
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_shared_pages():
    """Sequences whose tables name the same pages read the same prefix."""
    cache, table, codes, scales = _cache([100], 2, 64, 16, 10)
    q = dev_bf16(normal_bf16(14, (1, 4, 1, 64)))
    one = qat_attention_decode(q, cache, _i32(table), _i32([100]))
    three = qat_attention_decode(q.expand(3, 4, 1, 64).contiguous(), cache,
                                 _i32(np.repeat(table, 3, 0)), _i32([100, 100, 37]))
    assert torch.allclose(three[0].float(), one[0].float(), rtol=2.0 ** -7, atol=1e-5)
    assert torch.allclose(three[1].float(), one[0].float(), rtol=2.0 ** -7, atol=1e-5)
    _check(q, [37], 2, 16, cache, table, codes, scales, 1)


@pytest.mark.parametrize("change", [
    lambda a: a.update(q=a["q"].float()),
    lambda a: a.update(q=a["q"][:, :3]),
    lambda a: a.update(q=a["q"][:1]),
    lambda a: a.update(q=a["q"].transpose(1, 2)),
    lambda a: a.update(q=a["q"].repeat(1, 1, 9, 1)),
    lambda a: a.update(q=a["q"][..., :32].contiguous()),
    lambda a: a.update(block_table=a["block_table"][0]),
    lambda a: a.update(seq_lens=a["seq_lens"].long()),
    lambda a: a.update(sm_scale=-1.0),
    lambda a: a.update(quant_mode=2),
    lambda a: a.update(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
    lambda a: a.update(workspace=torch.empty(64, dtype=torch.uint8)),
])
def test_refusals(change):
    cache = KVCache.empty(4, 2, 16, 64)
    args = dict(q=dev_bf16(normal_bf16(5, (2, 4, 2, 64))), cache=cache,
                block_table=_i32([[0, 1], [2, 3]]), seq_lens=_i32([0, 0]))
    assert (qat_attention_decode(**args) == 0).all()
    change(args)
    with pytest.raises((ValueError, TypeError, QatError)):
        qat_attention_decode(**args)
    check_device_status()
