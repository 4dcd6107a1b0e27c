"""The norm + rotation, the cache and decoding as they are used together: a prompt and then single steps of
a serving loop (eager, and captured into a graph), other streams, the training path through attention,
and a cached prefix read back for the training forward."""

import numpy as np
import pytest
import torch

from oracle import qat_oracle as orc
from oracle import serving_oracle as so
from quantization_aware_attention_gb300 import (QUANT_NONE, KVCache, RopePlan, attention,
                                                check_device_status, qat_attention_decode,
                                                qat_attention_forward, qat_qk_norm_rope,
                                                qat_qk_norm_rope_backward)
from quantization_aware_attention_gb300 import build as qbuild
from quantization_aware_attention_gb300 import capi
from quantization_aware_attention_gb300.inputs import normal_bf16

from gpu_util import TOL_HP, dev_bf16, host_f64, rel_l2

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, PAGE = 3, 8, 2, 64, 16


@pytest.fixture(scope="module", autouse=True)
def built():
    qbuild.build()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """One layer's attention as a serving program runs it."""

    def __init__(self):
        self.cache = KVCache.empty(30, HKV, PAGE, D)
        self.table = _i32(np.random.default_rng(1).permutation(30)[:B * 8].reshape(B, 8))
        self.rope = RopePlan(32, base=500000.0, layout="interleaved", scaling="yarn", factor=4.0,
                             original_len=64)
        w = np.random.default_rng(2)
        self.wq, self.wk = (torch.from_numpy((1 + 0.2 * w.standard_normal(D)).astype(np.float32)).cuda()
                            for _ in range(2))

    def qkv(self, x, positions):
        """x [B, N, HQ + 2 HKV, D], a fused projection's output."""
        x = x.transpose(1, 2)
        q, k = qat_qk_norm_rope(x[:, :HQ], x[:, HQ:HQ + HKV], positions, self.rope, self.wq, self.wk)
        return q, k, x[:, HQ + HKV:]

    def step(self, x, positions, lens):
        q, k, v = self.qkv(x, positions)
        self.cache.append(k, v, self.table, lens)
        return qat_attention_decode(q, self.cache, self.table, lens)


def _x(n, seed):
    return dev_bf16(normal_bf16(seed, (B, n, HQ + 2 * HKV, D)))


def test_prompt_then_steps():
    """Each step's output against the oracle on every key and value so far: those of the prompt, padded to
    its longest, and those of the steps; a sequence that is idle for a step keeps its cache."""
    s = Server()
    lens = [21, 5, 40]
    x = _x(40, 100)
    n = torch.arange(40, dtype=torch.int32, device="cuda")
    q, k, v = s.qkv(x, n)
    s.cache.append(k, v, s.table, _i32(lens), _i32(lens), check=True)
    keys = [[host_f64(k)[b, :, i] for i in range(lens[b])] for b in range(B)]
    values = [[host_f64(v)[b, :, i] for i in range(lens[b])] for b in range(B)]
    # the rotation itself, from the raw projection
    pos = np.broadcast_to(np.arange(40), (B, 40))
    want = so.norm_rope(host_f64(x).transpose(0, 2, 1, 3)[:, HQ:HQ + HKV], host_f64(s.wk), pos,
                        s.rope.frequencies, "interleaved", s.rope.amplitude)
    assert rel_l2(host_f64(k), want) <= 2.0 ** -8
    for t in range(4):
        idle = 1 if t == 2 else None
        x = _x(1, 200 + t)
        pos = [[n] for n in lens]
        q, k, v = s.qkv(x, _i32(pos))
        new = [0 if b == idle else 1 for b in range(B)]
        lens = [n + m for n, m in zip(lens, new)]
        s.cache.append(k, v, s.table, _i32(lens), _i32(new), check=True)
        o, lse = qat_attention_decode(q, s.cache, s.table, _i32(lens), return_lse=True, check=True)
        for b in range(B):
            if b != idle:
                keys[b].append(host_f64(k)[b, :, 0])
                values[b].append(host_f64(v)[b, :, 0])
            for h in range(HKV):
                kk = so.dequant(*so.quant_row(np.stack([r[h] for r in keys[b]])))
                vv = so.dequant(*so.quant_row(np.stack([r[h] for r in values[b]])))
                for hq in range(h * HQ // HKV, (h + 1) * HQ // HKV):
                    w, wl, tol, ltol = so.decode_head(host_f64(q)[b, hq], kk, vv, np.array([lens[b] - 1]),
                                                      D ** -0.5, 1)
                    assert (np.abs(host_f64(o)[b, hq] - w) <= tol).all(), (t, b, hq)
                    assert (np.abs(host_f64(lse)[b, hq] - wl) <= ltol).all()


def test_a_captured_step_follows_the_lengths():
    """The whole step captured once; each replay reads the positions and lengths of its time."""
    eager, graphed = Server(), Server()
    graphed.table.copy_(eager.table)
    x, lens = _x(1, 300), _i32([0, 3, 30])
    pos = lens.view(B, 1).clone()
    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        graphed.step(x, pos, lens + 1)
    warm.synchronize()
    for c in (eager.cache, graphed.cache):
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            t.view(torch.uint8).zero_()
    gx, gpos, glens = x.clone(), pos.clone(), lens.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        glens.add_(1)
        out = graphed.step(gx, gpos, glens)
        gpos.add_(1)
    for t in range(5):
        new = _x(1, 400 + t)
        gx.copy_(new)
        graph.replay()
        lens = lens + 1
        want = eager.step(new, pos, lens)
        pos = pos + 1
        assert torch.equal(out, want), t
        for a, b in zip((eager.cache.k, eager.cache.v), (graphed.cache.k, graphed.cache.v)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    check_device_status()


def test_two_streams_at_once():
    """Calls on two streams, each with its own tensors, give what they give alone."""
    servers = [Server(), Server()]
    lens = [_i32([100, 17, 64]), _i32([3, 128, 90])]
    for i, s in enumerate(servers):
        x = _x(128, 500 + i)
        _, k, v = s.qkv(x, torch.arange(128, dtype=torch.int32, device="cuda"))
        s.cache.append(k, v, s.table, lens[i], lens[i])
    xs = [_x(1, 600 + i) for i in range(2)]
    pos = [(n - 1).view(B, 1) for n in lens]
    alone = [s.step(x, p, n) for s, x, p, n in zip(servers, xs, pos, lens)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        outs = []
        for st, s, x, p, n in zip(streams, servers, xs, pos, lens):
            with torch.cuda.stream(st):
                outs.append(s.step(x, p, n))
        torch.cuda.synchronize()
        for a, b in zip(alone, outs):
            assert torch.equal(a, b)


def test_cached_prefix_read_back():
    """The training forward on a prefix read back from the cache against decoding over the cache: the rows
    read back are rounded to bf16 (2^-8 relative at most, 2^-9 in the mean), the two kernels are within
    their own tolerances of 5e-3 and a bf16 rounding."""
    s = Server()
    n = 100
    x = _x(n, 700)
    q, k, v = s.qkv(x, torch.arange(n, dtype=torch.int32, device="cuda"))
    lens = _i32([n] * B)
    s.cache.append(k, v, s.table, lens)
    kr, vr = s.cache.read(s.table, lens, length=n)
    g = HQ // HKV
    kr, vr = (t.repeat_interleave(g, 1).contiguous() for t in (kr, vr))
    last = q[:, :, -1:].contiguous()
    o = qat_attention_decode(last, s.cache, s.table, lens, quant_mode=QUANT_NONE)
    want = qat_attention_forward(last, kr, vr, quant_mode=QUANT_NONE)[0]
    assert rel_l2(host_f64(o), host_f64(want)) <= TOL_HP + 2 * 2.0 ** -8


@pytest.mark.parametrize("D,R,layout", [(64, 64, "half"), (128, 64, "interleaved")])
def test_training_through_attention(D, R, layout):
    """Norm + rotation, then quantization-aware attention, causal, and back to the projection and both
    weights, against fp64 autograd of the plain formulas.  Tolerance: the attention's gradients are held to
    1e-2 (relative L2); q and k rounded to bf16 move the scores by 2^-9 of themselves, and every gradient
    is rounded once more: 2 x 2^-9 on top."""
    Bt, H, N = 2, 3, 130
    bits = normal_bf16(900 + D, (Bt, N, 3 * H, D))
    x = dev_bf16(bits).requires_grad_(True)
    w = np.random.default_rng(3).standard_normal((2, D)).astype(np.float32) * 0.2 + 1
    ws = [torch.from_numpy(a).cuda().requires_grad_(True) for a in w]
    rope = RopePlan(R, layout=layout)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    y = x.transpose(1, 2)
    q, k = qat_qk_norm_rope(y[:, :H], y[:, H:2 * H], pos, rope, *ws)
    o = attention(q, k, y[:, 2 * H:].contiguous(), causal=True)
    do = normal_bf16(901, (Bt, H, N, D))
    o.backward(dev_bf16(do))
    # fp64
    x64 = torch.from_numpy(orc.bf16_bits_to_f64(bits)).requires_grad_(True)
    w64 = [torch.from_numpy(a.astype(np.float64)).requires_grad_(True) for a in w]
    z = x64.transpose(1, 2)
    ang = torch.arange(N, dtype=torch.float64)[:, None] * torch.tensor(rope.frequencies, dtype=torch.float64)

    def turned(u, weight):
        u = u / (u.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight
        a, b = (u[..., :R // 2], u[..., R // 2:R]) if layout == "half" else (u[..., 0:R:2], u[..., 1:R:2])
        c, s = a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()
        part = torch.cat((c, s), -1) if layout == "half" else torch.stack((c, s), -1).flatten(-2)
        return torch.cat((part, u[..., R:]), -1)

    sc = turned(z[:, :H], w64[0]) @ turned(z[:, H:2 * H], w64[1]).transpose(-1, -2) * D ** -0.5
    sc = sc.masked_fill(torch.ones(N, N).triu(1).bool(), -torch.inf)
    (torch.softmax(sc, -1) @ z[:, 2 * H:]).backward(torch.from_numpy(orc.bf16_bits_to_f64(do)))
    tol = 1e-2 + 2 * 2.0 ** -9
    for i in range(3):  # the q, k and v parts of the projection
        part = slice(i * H, (i + 1) * H)
        assert rel_l2(host_f64(x.grad[:, :, part]), x64.grad[:, :, part].numpy()) <= tol, i
    for a, b in zip(ws, w64):
        assert rel_l2(host_f64(a.grad), b.grad.numpy()) <= tol


def test_calls_without_a_backward_say_so():
    s = Server()
    x = _x(1, 800).requires_grad_(True)
    q, k, v = s.qkv(x, _i32([[0]] * B))
    with pytest.raises(ValueError, match="no backward"):
        s.cache.append(k, v, s.table, _i32([1] * B))
    with pytest.raises(ValueError, match="no backward"):
        qat_attention_decode(q, s.cache, s.table, _i32([1] * B))
    with torch.no_grad():
        assert s.step(x, _i32([[0]] * B), _i32([1] * B)).shape == (B, HQ, 1, D)
    assert capi.qat_attn_device_status() == capi.Status.OK


@pytest.mark.parametrize("captured", [False, True])
def test_a_chain_of_calls_in_flight(captured):
    """Forty steps of one stream, each call's inputs the ones before it have just written -- lengths and
    positions included -- and the scratch memory used again by the next: queued without a pause, they give
    the bits that they give one at a time."""
    def steps(s, x, lens, wait):
        pos = torch.empty(B, 1, dtype=torch.int32, device="cuda")
        outs = []
        for _ in range(40):
            torch.add(lens, 0, out=pos[:, 0])
            lens.add_(1)
            o = s.step(x, pos, lens)
            kr, vr = s.cache.read(s.table, lens, length=64)
            x = torch.cat([o.transpose(1, 2), kr[:, :, 5:6].transpose(1, 2), vr[:, :, 5:6].transpose(1, 2)], 2)
            g = qat_qk_norm_rope_backward(x[:, :, :HQ].transpose(1, 2), None, pos, s.rope, s.wq, None, o, None)
            x = torch.cat([g[0].transpose(1, 2), x[:, :, HQ:]], 2)
            s.wq.copy_(1 + g[2].tanh() / 4)
            outs += [o, kr, vr, *[t for t in g if t is not None]]
            if wait:
                torch.cuda.synchronize()
        return outs

    runs = []
    for wait in (True, False):
        s = Server()
        for t in (s.cache.k, s.cache.v):
            t.view(torch.uint8).zero_()
        for t in (s.cache.k_scale, s.cache.v_scale):
            t.zero_()
        x, lens = _x(1, 500), _i32([0, 11, 3])
        if captured and not wait:
            first = (s.wq.clone(), lens.clone())
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                steps(s, x, lens.clone(), False)
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs = steps(s, x, lens, False)
            for t in (s.cache.k, s.cache.v):
                t.view(torch.uint8).zero_()
            for t in (s.cache.k_scale, s.cache.v_scale):
                t.zero_()
            s.wq.copy_(first[0])
            lens.copy_(first[1])
            graph.replay()
        else:
            outs = steps(s, x, lens, wait)
        torch.cuda.synchronize()
        runs.append([t.clone() for t in outs])
    for i, (a, b) in enumerate(zip(*runs)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
    check_device_status()


@pytest.mark.parametrize("captured", [False, True])
def test_calls_that_alternate_between_streams(captured):
    """Every call on the other stream than the one before, ordered by events alone, the workspace shared:
    the bits of one stream."""
    def steps(s, x, lens, streams, ws):
        pos = torch.empty(B, 1, dtype=torch.int32, device="cuda")
        keep, turn = [], 0

        def on(f):
            nonlocal turn
            turn += 1
            a, b = streams[turn % 2], streams[(turn + 1) % 2]
            a.wait_stream(b)
            with torch.cuda.stream(a):
                out = f()
            keep.append(out)  # alive until the end: no memory is handed on
            return out

        for _ in range(25):
            on(lambda: torch.add(lens, 0, out=pos[:, 0]))
            on(lambda: lens.add_(1))
            q, k, v = on(lambda: s.qkv(x, pos))
            on(lambda: s.cache.append(k, v, s.table, lens))
            o = on(lambda: qat_attention_decode(q, s.cache, s.table, lens, workspace=ws))
            kr, vr = on(lambda: s.cache.read(s.table, lens, length=48))
            x = on(lambda: torch.cat([o, kr[:, :, 3:4], vr[:, :, 3:4]], 1).transpose(1, 2).contiguous())
        streams[0].wait_stream(streams[1])
        return [t for out in keep for t in (out if isinstance(out, tuple) else (out,)) if t is not None]

    ws = torch.empty(capi.qat_attn_decode_workspace_bytes(HQ, HKV, 1, D), dtype=torch.uint8, device="cuda")
    runs = []
    for two in (False, True):
        s = Server()
        for t in (s.cache.k, s.cache.v):
            t.view(torch.uint8).zero_()
        for t in (s.cache.k_scale, s.cache.v_scale):
            t.zero_()
        x, lens = _x(1, 501), _i32([2, 30, 0])
        main = torch.cuda.current_stream()
        if captured and two:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                main = torch.cuda.current_stream()
                outs = steps(s, x, lens, (main, torch.cuda.Stream()), ws)
            graph.replay()
        else:
            outs = steps(s, x, lens, (main, torch.cuda.Stream() if two else main), ws)
        torch.cuda.synchronize()
        runs.append([t.clone() for t in outs])
    for i, (a, b) in enumerate(zip(*runs)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
    check_device_status()
