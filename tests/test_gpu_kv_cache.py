"""GPU parity of the FP8 key/value cache: codes and scales bit for bit with the rule's fp32 steps, every
other slot untouched, reads exact, bad pages refused on the device without touching memory."""

import numpy as np
import pytest
import torch

from oracle import qat_oracle as orc
from oracle import serving_oracle as so
from quantization_aware_attention_gb300 import KVCache, QatError, check_device_status
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


def _table(B, per, pages, seed):
    return np.random.default_rng(seed).permutation(pages)[:B * per].reshape(B, per).astype(np.int32)


def _filled(pages, H, page, D, seed=0):
    """A cache whose every byte is a known finite code."""
    c = KVCache.empty(pages, H, page, D)
    rng = np.random.default_rng(seed)
    for t, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        bits = rng.integers(0, 0x7F, (pages, H, page, D)).astype(np.uint8)
        t.view(torch.uint8).copy_(torch.from_numpy(bits))
        s.copy_(torch.from_numpy(rng.random((pages, H, page)).astype(np.float32)))
    return c


def _state(c):
    return [t.view(torch.uint8).cpu().numpy().copy() for t in (c.k, c.v)] + [
        t.cpu().numpy().copy() for t in (c.k_scale, c.v_scale)]


def _rows(B, H, N, D, seed, inner):
    """Rows with outliers, zeros, tiny and non-finite ones, heads inner or not; bits [B, H, N, D]."""
    bits = normal_bf16(seed, (B, N, H, D))
    f = orc.bf16_bits_to_f64(bits).astype(np.float32)
    f[..., 3] *= 30
    flat = f.reshape(-1, D)
    for i, s in ((1, 0.0), (2, 2.0 ** -115), (3, 2.0 ** -100), (5, 1e36)):
        flat[i % len(flat)] *= np.float32(s)
    if len(flat) > 8:
        flat[6, 5], flat[7, D - 1] = np.inf, np.nan
    bits = (f.view(np.uint32) >> 16).astype(np.uint16)
    bits[np.isnan(f)] = 0x7FC0
    d = dev_bf16(bits).transpose(1, 2)
    return (d if inner else d.contiguous()), orc.bf16_bits_to_f64(bits).transpose(0, 2, 1, 3)


@pytest.mark.parametrize("B,H,N,D,page,lens,new", [
    (1, 1, 1, 128, 16, [1], None),
    (3, 2, 1, 64, 16, [17, 16, 1], None),
    (2, 3, 37, 128, 32, [37, 70], None),
    (4, 1, 20, 64, 16, [20, 5, 40, 0], [20, 5, 3, 0]),
    (3, 8, 100, 128, 64, [100, 64, 300], [100, 1, 77]),
    (2, 2, 40, 128, 256, [40, 513], [50, 40]),        # a count above N counts as N
    (2, 2, 9, 64, 128, [4, 20], [9, 9]),              # rows before position 0 are dropped
])
@pytest.mark.parametrize("inner", [False, True])
def test_append_and_read(B, H, N, D, page, lens, new, inner):
    per = (max(lens) + page - 1) // page + 1
    pages = B * per + 3
    table = _table(B, per, pages, 3)
    c = _filled(pages, H, page, D)
    want = _state(c)
    k, fk = _rows(B, H, N, D, 10, inner)
    v, fv = _rows(B, H, N, D, 11, not inner)
    c.append(k, v, _i32(table), _i32(lens), None if new is None else _i32(new), check=True)
    for which, f in ((0, fk), (1, fv)):
        codes, scales = so.quant_row(f)
        for b in range(B):
            count = N if new is None else min(new[b], N)
            for n in range(count):
                pos = lens[b] - count + n
                if pos < 0:
                    continue
                at = table[b, pos // page], slice(None), pos % page
                want[which][at], want[2 + which][at] = codes[b, :, n], scales[b, :, n]
    got = _state(c)
    for g, w in zip(got[:2], want[:2]):  # -0 and 0 are one value
        assert np.array_equal(np.where(g == 0x80, 0, g), np.where(w == 0x80, 0, w))
    for g, w in zip(got[2:], want[2:]):
        assert np.array_equal(g, w, equal_nan=True)
    # read all back, beyond the ends too
    length = per * page
    rk, rv = c.read(_i32(table), _i32(lens))
    for r, code, scale in ((rk, got[0], got[2]), (rv, got[1], got[3])):
        exact = so.dequant(code, scale)  # [pages, H, page, D]
        for b in range(B):
            rows = exact[table[b]].transpose(1, 0, 2, 3).reshape(H, length, D)
            w = orc.f32_to_bf16_rn((rows[:, :lens[b]]).astype(np.float32)).astype(np.float64)
            g = host_f64(r[b])
            assert np.array_equal(g[:, :lens[b]], w, equal_nan=True)
            assert (g[:, lens[b]:] == 0).all()
    part = c.read(_i32(table), _i32(lens), begin=5, length=7)
    assert torch.equal(part[0].view(torch.int16), rk[:, :, 5:12].view(torch.int16))
    assert torch.equal(part[1].view(torch.int16), rv[:, :, 5:12].view(torch.int16))
    past = c.read(_i32(table), _i32(lens), begin=length - 2, length=9)[0]
    assert past.shape == (B, H, 9, D) and (host_f64(past[:, :, 2:]) == 0).all()
    check_device_status()


def test_broadcast_rows():
    c = KVCache.empty(3, 2, 16, 64)
    k = dev_bf16(normal_bf16(1, (1, 1, 4, 64)))
    c.append(k.expand(2, 2, 4, 64), k.expand(2, 2, 4, 64), _i32([[2], [0]]), _i32([4, 9]))
    r = c.read(_i32([[2], [0]]), _i32([4, 9]), length=9)[0]
    assert torch.equal(r[0, 0, :4], r[1, 1, 5:9])


def test_empty_calls():
    c = KVCache.empty(1, 1, 16, 64)
    z = torch.empty(0, 1, 3, 64, dtype=torch.bfloat16, device="cuda")
    none, no_seq = _i32([]), torch.empty(0, 1, dtype=torch.int32, device="cuda")
    c.append(z, z, no_seq, none, check=True)
    assert c.read(no_seq, none)[0].shape == (0, 1, 16, 64)
    z = torch.empty(1, 1, 0, 64, dtype=torch.bfloat16, device="cuda")
    c.append(z, z, _i32([[0]]), _i32([0]), check=True)
    assert c.read(_i32([[0]]), _i32([0]), begin=16)[0].shape == (1, 1, 0, 64)


def test_far_pages():
    """A cache of more than 2^32 bytes: rows beyond the 32-bit offsets land where they belong."""
    H, page, D = 8, 256, 128
    pages = (1 << 32) // (H * page * D) + 8
    c = KVCache.empty(pages, H, page, D)
    far = pages - 1
    k = dev_bf16(normal_bf16(5, (1, H, 4, D)))
    c.append(k, -k, _i32([[far]]), _i32([4]), check=True)
    codes, scales = so.quant_row(host_f64(k))
    assert np.array_equal(c.k[far, :, :4].view(torch.uint8).cpu().numpy()[0] & 0x7F, codes[0, 0] & 0x7F)
    assert np.array_equal(c.k_scale[far, :, :4].cpu().numpy(), scales[0])
    rk, rv = c.read(_i32([[far]]), _i32([4]), length=4)
    assert torch.equal(rk, -rv)
    assert np.array_equal(host_f64(rk), orc.f32_to_bf16_rn(so.dequant(codes, scales).astype(np.float32)))


@pytest.mark.parametrize("bad", [-1, 5, 2 ** 31 - 1, -2 ** 31])
def test_bad_pages_are_reported_and_not_followed(bad):
    """The kernels check every page index against the cache before they use it."""
    c = _filled(5, 2, 16, 64)
    before = _state(c)
    k = dev_bf16(normal_bf16(5, (1, 2, 20, 64)))
    table = _i32([[3, bad]])
    with pytest.raises(QatError) as e:
        c.append(k, k, table, _i32([20]), check=True)
    assert e.value.status == Status.BAD_PAGE
    check_device_status()  # read and cleared
    after = _state(c)
    codes, scales = so.quant_row(host_f64(k))
    before[2][3], before[3][3] = scales[0, :, :16], scales[0, :, :16]
    assert np.array_equal(after[2], before[2]) and np.array_equal(after[3], before[3])
    with pytest.raises(QatError):
        c.read(table, _i32([20]), check=True)
    r = c.read(table, _i32([20]))[0]
    assert torch.isnan(r[:, :, 16:20]).all() and torch.isfinite(r[:, :, :16]).all()
    assert (r[:, :, 20:] == 0).all()
    capi.qat_attn_device_status()


def test_lengths_beyond_the_table():
    c = _filled(5, 1, 16, 64)
    before = _state(c)
    k = dev_bf16(normal_bf16(5, (1, 1, 2, 64)))
    with pytest.raises(QatError):
        c.append(k, k, _i32([[0, 1]]), _i32([2 ** 31 - 1]), check=True)
    assert all(np.array_equal(a, b) for a, b in zip(before, _state(c)))
    r = c.read(_i32([[0, 1]]), _i32([33]))[0]  # the table's 32 positions can be read
    assert torch.isfinite(r).all()
    assert capi.qat_attn_device_status() == Status.BAD_PAGE


@pytest.mark.parametrize("change", [
    lambda a: a.update(k=a["k"].float()),
    lambda a: a.update(k=a["k"][:, :1]),
    lambda a: a.update(v=a["v"][..., :32]),
    lambda a: a.update(v=a["v"][:, :, :2]),
    lambda a: a.update(block_table=a["block_table"].long()),
    lambda a: a.update(block_table=a["block_table"][:1]),
    lambda a: a.update(block_table=a["block_table"][:, :0]),
    lambda a: a.update(seq_lens=a["seq_lens"].cpu()),
    lambda a: a.update(seq_lens=a["seq_lens"][None]),
    lambda a: a.update(new_lens=_i32([1, 1, 1])),
    lambda a: a.update(new_lens=_i32([1, 1]).long()),
])
def test_refusals(change):
    c = KVCache.empty(4, 2, 16, 64)
    k = dev_bf16(normal_bf16(5, (2, 2, 3, 64)))
    args = dict(k=k, v=k, block_table=_i32([[0, 1], [2, 3]]), seq_lens=_i32([3, 3]))
    c.append(**args)
    change(args)
    with pytest.raises((ValueError, TypeError)):
        c.append(**args)
    with pytest.raises(ValueError):
        KVCache(c.k, c.v, c.k_scale, c.v_scale[:2])
    with pytest.raises(ValueError):
        KVCache(c.k.view(torch.uint8), c.v, c.k_scale, c.v_scale)
    with pytest.raises(ValueError):
        KVCache.empty(4, 2, 48, 64)
    with pytest.raises(ValueError):
        c.read(args["block_table"], args["seq_lens"], begin=-1)
