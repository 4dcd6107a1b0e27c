"""Decoding over caches whose values differ much in magnitude: what a row does not see, or weighs with nearly
nothing, takes no bits from the weights that make its output.  The oracle's tolerances hold each weight to f16's
half step, relative to the row's own largest weight where it is far below that."""

import numpy as np
import pytest
import torch

from oracle import serving_oracle as so
from quantization_aware_attention_gb300 import KVCache, qat_attention_decode
from quantization_aware_attention_gb300 import build as qbuild
from quantization_aware_attention_gb300.inputs import normal_bf16

from gpu_util import dev_bf16, host_f64

pytestmark = pytest.mark.gpu

PAGE, HKV = 16, 2


@pytest.fixture(scope="module", autouse=True)
def built():
    qbuild.build()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _case(scores, sizes, D, Hq, T, copies, seed):
    """A sequence whose key j has about the natural-log score scores[j] for every query row and a normal value
    of magnitude sizes[j], and `copies` sequences that share its pages."""
    n = len(scores)
    per = -(-n // PAGE)
    rng = np.random.default_rng(seed)
    k = 0.02 * rng.standard_normal((HKV, per * PAGE, D))
    k[:, :n, 0] = np.asarray(scores) / 8 + 0.05 * rng.standard_normal((HKV, n))
    v = rng.standard_normal((HKV, per * PAGE, D))
    v[:, :n] *= np.asarray(sizes, np.float64)[:, None]
    table = np.arange(per)[::-1].copy()
    quants, tensors = [], []
    for x in (k, v):
        paged = np.ascontiguousarray(x.reshape(HKV, per, PAGE, D).transpose(1, 0, 2, 3)[table])
        c, s = so.quant_row(paged)
        quants.append([so.dequant(c, s)[table].transpose(1, 0, 2, 3).reshape(HKV, per * PAGE, D)[h, :n]
                       for h in range(HKV)])
        tensors.append((torch.from_numpy(c).cuda().view(torch.float8_e4m3fn), torch.from_numpy(s).cuda()))
    q = dev_bf16(normal_bf16(seed, (1, Hq, T, D))).clone()
    q[..., 0] = 8.0
    cache = KVCache(tensors[0][0], tensors[1][0], tensors[0][1], tensors[1][1])
    return (q.expand(copies, Hq, T, D).contiguous(), cache, _i32(np.tile(table, (copies, 1))), _i32([n] * copies),
            *quants)


def _check(case, quant):
    q, cache, table, lens, k, v = case
    B, Hq, T, D = q.shape
    n = int(lens[0])
    o, lse = qat_attention_decode(q, cache, table, lens, 1.0, quant, return_lse=True, check=True)
    fq, fo, fl = host_f64(q[0]), host_f64(o), host_f64(lse)
    for hq in range(Hq):
        h = hq // (Hq // HKV)
        w, wl, tol, ltol = so.decode_head(fq[hq], k[h], v[h], n - T + np.arange(T), 1.0, quant)
        err = np.abs(fo[:, hq] - w)
        assert (err <= tol).all(), (hq, float((err / np.maximum(tol, 1e-300)).max()))
        assert (np.abs(fl[:, hq] - wl) <= ltol).all()


SHAPES = [(64, 4, 3), (128, 4, 3), (64, 8, 3), (128, 8, 3)]  # D, query heads, tokens: 6 or 12 rows a KV head


@pytest.mark.parametrize("D,Hq,T", SHAPES)
@pytest.mark.parametrize("n", [50, 65, 66, 300])  # the newest tokens in the only tile, and in one of their own
@pytest.mark.parametrize("quant", [0, 1])
def test_values_that_a_row_does_not_see(D, Hq, T, n, quant):
    """The newest token's value, 1e12 or 1e30 times as large as the others, reaches the newest token alone: the
    tokens before it give the same bits."""
    rng = np.random.default_rng(1)
    scores, sizes = rng.standard_normal(n), np.ones(n)
    clean = _case(scores, sizes, D, Hq, T, 1, 5)
    want = qat_attention_decode(*clean[:4], 1.0, quant)
    _check(clean, quant)
    for big in (1e12, 1e30):
        sizes[-1] = big
        case = _case(scores, sizes, D, Hq, T, 1, 5)
        _check(case, quant)
        assert torch.equal(qat_attention_decode(*case[:4], 1.0, quant)[:, :, :-1], want[:, :, :-1])


def _spread(name, n, rng):
    scores, sizes = rng.standard_normal(n), np.ones(n)
    if name == "behind":      # one key of weight 2^-130 beside the others, one of weight 0
        scores[40], sizes[40] = -90.0, 2.0 ** 60
        scores[n - 20], sizes[n - 20] = -250.0, 2.0 ** 90
    elif name == "first":     # large values first, then scores 87 octaves above theirs
        sizes[:70] = 2.0 ** 60
        scores[70:] += 60.0
    elif name == "last":
        sizes[-70:] = 2.0 ** 60
        scores[-70:] -= 120.0
    elif name == "falling":   # the maximum rises with every tile, the values fall as fast
        scores += 15.0 * (np.arange(n) // 64)
        sizes *= 2.0 ** (40.0 - 21.0 * (np.arange(n) // 64))
    elif name == "zero":      # the key that takes nearly all the weight has no value
        scores[10], sizes[10] = 60.0, 0.0
    elif name == "wide":      # 2^-100 .. 2^100 at random
        sizes *= 2.0 ** rng.uniform(-100, 100, n)
    elif name == "small":     # near the least and the largest that the cache stores
        sizes *= 2.0 ** -104
    elif name == "large":
        sizes *= 2.0 ** 110
    return scores, sizes


@pytest.mark.parametrize("name", ["behind", "first", "last", "falling", "zero", "wide", "small", "large"])
@pytest.mark.parametrize("D,Hq,T", SHAPES)
@pytest.mark.parametrize("copies", [1, 500])  # ranges of one tile, and of several
@pytest.mark.parametrize("quant", [0, 1])
def test_values_of_little_weight(name, D, Hq, T, copies, quant):
    _check(_case(*_spread(name, 300, np.random.default_rng(2)), D, Hq, T, copies, 6), quant)


@pytest.mark.parametrize("D,Hq,T", SHAPES)
@pytest.mark.parametrize("keys,queries,sm_scale", [
    (2.0 ** 122, 2.0 ** -90, 2.0 ** -32), (2.0 ** 122, 1.0, 2.0 ** -122), (2.0 ** 60, 2.0 ** -60, 1.0),
    (2.0 ** -100, 2.0 ** 100, 1.0), (2.0 ** -100, 1.0, 2.0 ** 100), (2.0 ** 20, 2.0 ** 80, 2.0 ** -100),
    (2.0 ** 100, 2.0 ** -80, 2.0 ** -20),
])
@pytest.mark.parametrize("quant", [0, 1])
def test_keys_of_extreme_magnitude(D, Hq, T, keys, queries, sm_scale, quant):
    """Scores of ordinary size from keys, queries and a scale that are not: the same bits as from ordinary ones,
    as all are powers of two times those."""
    rng = np.random.default_rng(3)
    q, cache, table, lens, _, _ = _case(rng.standard_normal(300), np.ones(300), D, Hq, T, 1, 7)
    want = qat_attention_decode(q, cache, table, lens, 1.0, quant, return_lse=True)
    cache.k_scale.mul_(keys)
    got = qat_attention_decode(q * queries, cache, table, lens, sm_scale, quant, return_lse=True, check=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
