"""GPU parity of the query/key norm with rotary positions, forward and backward, against the fp64 oracle.

Tolerances, per element.  A bf16 output is off by at most half a step, 2^-8 relative.  Before that
rounding: the angle's fraction of a turn has 32 bits and becomes an fp32 angle below pi (2^-22 absolute),
the hardware sine and cosine are within 2^-20.5 there, and the sums of 128 squares and the few fp32
products are within 2^-20 relative; each rotated channel is a sum of two products of a channel with one
of these, so it is off by at most 2^-18 (under 4e-6) of the row's largest |z| times the amplitude.
A term dz n of a weight's gradient carries dz's error, which like a rotated channel's is relative to the
row's largest |dy| and not to |dz| (dz is a difference of two products, and may cancel): 4e-6 of
max|dy| |n| times the amplitude, and 4e-6 of |dz n| for n, the product and the fp32 sum."""

import numpy as np
import pytest
import torch

from oracle import qat_oracle as orc
from oracle import serving_oracle as so
from quantization_aware_attention_gb300 import (RopePlan, check_device_status, qat_qk_norm_rope,
                                                qat_qk_norm_rope_backward)
from quantization_aware_attention_gb300 import build as qbuild
from quantization_aware_attention_gb300.inputs import normal_bf16

from gpu_util import dev_bf16, host_f64

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def built():
    qbuild.build()


def _make(B, Hq, Hk, N, D, seed, inner=True):
    """Seeded q, k (slices of a fused projection, heads inner, or contiguous) and their fp64 values."""
    H = Hq + 2 * Hk
    bits = normal_bf16(seed, (B, N, H, D))
    x = dev_bf16(bits)
    f = orc.bf16_bits_to_f64(bits).transpose(0, 2, 1, 3)
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2)
    if not inner:
        q, k = q.contiguous(), k.contiguous()
    return q, k, f[:, :Hq], f[:, Hq:Hq + Hk]


def _weights(D, seed, dtype):
    rng = np.random.default_rng(seed)
    w = [torch.from_numpy((1 + 0.3 * rng.standard_normal(D)).astype(np.float32)).cuda().to(dtype)
         for _ in range(2)]
    return w, [host_f64(t) for t in w]


def _positions(B, N, seed, top):
    return np.random.default_rng(seed).integers(-5 if top > 1 << 20 else 0, top, (B, N)).astype(np.int32)


def _near(got, want, slack):
    err = np.abs(host_f64(got) - want)
    lim = HALF * np.abs(want) * 1.001 + slack
    assert (err <= lim).all(), float((err / np.maximum(lim, 1e-300)).max())


def _forward_slack(x, w, amplitude, eps=1e-6):
    z = so.norm_rope(x, w, None, [], "half", eps=eps)
    return 4e-6 * max(1.0, abs(amplitude)) * np.abs(z).max(-1, keepdims=True)


PLANS = [
    ("half", dict(scaling="none")),
    ("interleaved", dict(scaling="none", base=500000.0)),
    ("half", dict(scaling="linear", factor=3.0)),
    ("interleaved", dict(scaling="ntk", factor=4.0)),
    ("half", dict(scaling="yarn", factor=8.0, original_len=2048)),
]


@pytest.mark.parametrize("layout,kw", PLANS)
@pytest.mark.parametrize("B,Hq,Hk,N,D,R", [
    (1, 1, 1, 1, 128, 128), (2, 5, 3, 9, 128, 64), (3, 7, 1, 17, 64, 64), (1, 9, 2, 33, 64, 16),
    (2, 40, 8, 3, 128, 16),
])
@pytest.mark.parametrize("wtype", [torch.float32, torch.bfloat16])
def test_forward(layout, kw, B, Hq, Hk, N, D, R, wtype):
    q, k, fq, fk = _make(B, Hq, Hk, N, D, 100 + N)
    (wq, wk), (fwq, fwk) = _weights(D, 7, wtype)
    rope = RopePlan(R, layout=layout, **kw)
    pos = _positions(B, N, 5, 1 << 17)
    got_q, got_k = qat_qk_norm_rope(q, k, torch.from_numpy(pos).cuda(), rope, wq, wk, eps=1e-5)
    assert got_q.is_contiguous() and got_k.shape == (B, Hk, N, D)
    for got, x, w in ((got_q, fq, fwq), (got_k, fk, fwk)):
        want = so.norm_rope(x, w, pos, rope.frequencies, layout, rope.amplitude, 1e-5)
        _near(got, want, _forward_slack(x, w, rope.amplitude, 1e-5))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_forward_far_and_negative_positions(layout):
    q, k, fq, fk = _make(2, 3, 2, 40, 128, 11)
    rope = RopePlan(128, layout=layout)
    pos = _positions(2, 40, 6, 2 ** 31 - 1)
    pos[0, :4] = (0, -1, 2 ** 31 - 1, -2 ** 31)
    got_q, got_k = qat_qk_norm_rope(q, k, torch.from_numpy(pos).cuda(), rope)
    # a frequency in fp64 is off by 2^-53 of itself: at position 2^31 and one radian, 2.4e-7 rad
    for got, x in ((got_q, fq), (got_k, fk)):
        want = so.norm_rope(x, None, pos, rope.frequencies, layout)
        _near(got, want, 5e-6 * np.abs(x).max(-1, keepdims=True))


def test_one_step_alone_and_single_tensors():
    q, k, fq, fk = _make(2, 4, 2, 7, 64, 21, inner=False)
    (wq, wk), (fwq, fwk) = _weights(64, 8, torch.float32)
    rope = RopePlan(32)
    pos = np.arange(7, dtype=np.int32)  # one row for every sequence
    dpos = torch.from_numpy(pos).cuda()
    both = np.broadcast_to(pos, (2, 7))
    norm_q, norm_k = qat_qk_norm_rope(q, k, q_weight=wq, k_weight=wk)
    _near(norm_q, so.norm_rope(fq, fwq, both, [], "half"), _forward_slack(fq, fwq, 1.0))
    _near(norm_k, so.norm_rope(fk, fwk, both, [], "half"), _forward_slack(fk, fwk, 1.0))
    only = qat_qk_norm_rope(q, None, dpos, rope, wq)
    pair = qat_qk_norm_rope(q, k, dpos, rope, wq, wk)
    assert torch.equal(only, pair[0])
    same = qat_qk_norm_rope(q, k)  # neither step: a copy, bit for bit
    assert torch.equal(same[0], q) and torch.equal(same[1], k)
    _near(only, so.norm_rope(fq, fwq, both, rope.frequencies, "half"), _forward_slack(fq, fwq, 1.0))


def test_channels_behind_the_rotation_keep_infinities_apart():
    """Without a norm, a channel that is not rotated is its input, whatever its neighbour holds."""
    for layout in ("half", "interleaved"):
        q, _, _, _ = _make(1, 2, 1, 3, 64, 31, inner=False)
        q[..., 40] = float("inf")
        q[..., 50] = float("nan")
        out = qat_qk_norm_rope(q, None, torch.arange(3, dtype=torch.int32, device="cuda"),
                               RopePlan(32, layout=layout))
        a, b = out[..., 32:], q[..., 32:]
        assert torch.equal(torch.isnan(a), torch.isnan(b))
        assert torch.equal(a.nan_to_num(0.0), b.nan_to_num(0.0))
        assert torch.isfinite(out[..., :32]).all()


def test_empty_sizes():
    rope = RopePlan(64)
    for B, H, N in ((0, 2, 3), (2, 0, 3), (2, 2, 0)):
        q = torch.empty(B, H, N, 64, dtype=torch.bfloat16, device="cuda").requires_grad_(True)
        w = torch.ones(64, device="cuda", requires_grad=True)
        pos = torch.zeros(N, dtype=torch.int32, device="cuda")
        out = qat_qk_norm_rope(q, None, pos, rope, w)
        assert out.shape == (B, H, N, 64)
        dq, dw = torch.autograd.grad(out, (q, w), torch.empty_like(out))
        assert dq.shape == q.shape and (dw == 0).all()


def test_no_second_derivative():
    q, _, _, _ = _make(1, 2, 1, 3, 64, 41)
    q = q.detach().requires_grad_(True)
    out = qat_qk_norm_rope(q, None, q_weight=torch.ones(64, device="cuda"))
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(out.float().square().sum(), q, create_graph=True)


def test_a_tensor_of_no_key_heads():
    q, _, fq, _ = _make(2, 3, 1, 5, 64, 42)
    k = torch.empty(2, 0, 5, 64, dtype=torch.bfloat16, device="cuda")
    a, b = qat_qk_norm_rope(q, k)
    assert torch.equal(a, q) and b.shape == k.shape


def _backward_case(B, Hq, Hk, N, D, R, layout, wtype, amplitude=1.0, inner=True):
    q, k, fq, fk = _make(B, Hq, Hk, N, D, 300 + N, inner)
    ws, fws = _weights(D, 9, wtype)
    rope = RopePlan(R, layout=layout, amplitude=amplitude)
    pos = _positions(B, N, 5, 1 << 17)
    gb = [normal_bf16(400 + i, (B, h, N, D)) for i, h in enumerate((Hq, Hk))]
    return q, k, fq, fk, ws, fws, rope, pos, [dev_bf16(b) for b in gb], [orc.bf16_bits_to_f64(b) for b in gb]


def _check_grads(x, w, dy, pos, rope, got_dx, got_dw, eps=1e-6):
    dx, dw = so.norm_rope_backward(x, w, dy, pos, rope.frequencies, rope.layout, rope.amplitude, eps)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    dz = so._rotate(dy, pos, rope.frequencies, rope.layout, rope.amplitude, -1.0)
    dn = np.abs(dz * w)
    scale = r * (dn.max(-1, keepdims=True) + np.abs(n).max(-1, keepdims=True) * (dn * np.abs(n)).mean(-1, keepdims=True))
    _near(got_dx, dx, 1e-5 * scale * max(1.0, rope.amplitude))
    lim = 4e-6 * (np.abs(dz * n) + max(1.0, rope.amplitude) * np.abs(dy).max(-1, keepdims=True) * np.abs(n)
                  ).sum((0, 1, 2)) + (HALF * np.abs(dw) * 1.001 if got_dw.dtype == torch.bfloat16 else 0)
    assert (np.abs(host_f64(got_dw) - dw) <= lim).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,Hq,Hk,N,D,R,wtype", [
    (1, 1, 1, 1, 128, 128, torch.float32), (2, 5, 3, 19, 128, 64, torch.bfloat16),
    (3, 7, 1, 70, 64, 64, torch.float32), (1, 24, 8, 333, 64, 16, torch.bfloat16),
    (2, 12, 4, 600, 128, 128, torch.float32),
])
def test_backward(layout, B, Hq, Hk, N, D, R, wtype):
    q, k, fq, fk, ws, fws, rope, pos, g, fg = _backward_case(B, Hq, Hk, N, D, R, layout, wtype, 1.25)
    leaves = [t.detach().requires_grad_(True) for t in (q, k, *ws)]
    out = qat_qk_norm_rope(leaves[0], leaves[1], torch.from_numpy(pos).cuda(), rope, leaves[2], leaves[3])
    dq, dk, dwq, dwk = torch.autograd.grad(out, leaves, g)
    assert dwq.dtype == wtype
    _check_grads(fq, fws[0], fg[0], pos, rope, dq, dwq)
    _check_grads(fk, fws[1], fg[1], pos, rope, dk, dwk)
    again = torch.autograd.grad(qat_qk_norm_rope(leaves[0], leaves[1], torch.from_numpy(pos).cuda(), rope,
                                                 leaves[2], leaves[3]), leaves, g)
    for a, b in zip((dq, dk, dwq, dwk), again):
        assert torch.equal(a, b)


# Few heads: a warp's rows are then of 2, 4 or 8 tokens (D = 64: 8 rows, D = 128: 4), a different number
# for the queries than for the keys, and the last warp's tokens end among its rows.
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,Hq,Hk,N,D,R", [
    (1, 1, 1, 5, 64, 64), (3, 3, 1, 43, 64, 16), (2, 4, 2, 65, 64, 32), (1, 5, 4, 130, 64, 64),
    (1, 1, 1, 3, 128, 128), (5, 3, 1, 21, 128, 64), (2, 2, 2, 4001, 128, 128), (1, 3, 0, 63, 128, 128),
])
def test_few_heads(layout, B, Hq, Hk, N, D, R):
    q, k, fq, fk, ws, fws, rope, pos, g, fg = _backward_case(B, Hq, Hk, N, D, R, layout, torch.float32)
    dpos = torch.from_numpy(pos).cuda()
    out = qat_qk_norm_rope(q, k if Hk else None, dpos, rope, ws[0], ws[1] if Hk else None)
    if Hk == 0:  # the queries alone, not a pair
        out = (out, None)
    dq, dk, dwq, dwk = qat_qk_norm_rope_backward(q, k if Hk else None, dpos, rope, ws[0], ws[1] if Hk else None,
                                                 g[0], g[1] if Hk else None)
    for got, x, w, dy, fdy, dx, dw in ((out[0], fq, fws[0], g[0], fg[0], dq, dwq),
                                       (out[1], fk, fws[1], g[1], fg[1], dk, dwk))[:2 if Hk else 1]:
        want = so.norm_rope(x, w, pos, rope.frequencies, layout, rope.amplitude)
        _near(got, want, _forward_slack(x, w, rope.amplitude))
        _check_grads(x, w, fdy, pos, rope, dx, dw)


def test_backward_against_differences():
    """<dy, y> moves with an input as its gradient says, by the kernel's own forward: the step is large
    enough that bf16 roundings of y (2^-9 of each, random) average out over the 2^18 elements."""
    q, k, fq, fk, ws, fws, rope, pos, g, fg = _backward_case(1, 8, 1, 256, 128, 128, "half", torch.float32)
    dpos = torch.from_numpy(pos).cuda()
    dq, _, dwq, _ = qat_qk_norm_rope_backward(q, k, dpos, rope, *ws, *g)
    d = torch.from_numpy(np.random.default_rng(3).standard_normal(128).astype(np.float32)).cuda()
    h = 0.125
    up = qat_qk_norm_rope(q, k, dpos, rope, ws[0] + h * d, ws[1])[0]
    down = qat_qk_norm_rope(q, k, dpos, rope, ws[0] - h * d, ws[1])[0]
    num = ((up.double() - down.double()) * g[0].double()).sum().item() / (2 * h)
    want = (dwq.double() * d.double()).sum().item()  # y is linear in the weight
    noise = (2.0 ** -8 * up.double().abs() * g[0].double().abs()).square().sum().sqrt().item() / h
    assert abs(num - want) <= 4 * noise


def test_without_norm_and_shared_gradients():
    """No weights: the backward is the inverse rotation alone.  Gradients of broadcast inputs, and an
    upstream gradient that is itself broadcast (the sum's)."""
    B, H, N, D = 2, 3, 11, 64
    q, k, fq, fk = _make(1, H, H, N, D, 51, inner=False)
    pos = _positions(B, N, 4, 5000)
    dpos = torch.from_numpy(pos).cuda()
    rope = RopePlan(64)
    leaf = q.detach().requires_grad_(True)
    wide = leaf.expand(B, H, N, D)  # one sequence's rows at two sets of positions
    qat_qk_norm_rope(wide, None, dpos, rope).sum().backward()
    dx = so.norm_rope_backward(np.broadcast_to(fq, (B, H, N, D)), None, np.ones((B, H, N, D)), pos,
                               rope.frequencies, "half")[0]
    # two bf16 rows, added by torch in bf16: two roundings each within half a step of at most sqrt(2)
    assert (np.abs(host_f64(leaf.grad) - dx.sum(0, keepdims=True)) <= 2.0 ** -8 * 2 * 3 * np.sqrt(2)).all()


def test_only_some_inputs_need_gradients():
    q, k, _, _ = _make(1, 2, 1, 5, 64, 61)
    ws, _ = _weights(64, 3, torch.float32)
    w = ws[1].requires_grad_(True)
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    a, b = qat_qk_norm_rope(q, k, pos, RopePlan(64), ws[0], w)
    b.float().square().sum().backward()  # only k's output is used
    assert w.grad is not None and torch.isfinite(w.grad).all() and not a.grad_fn is None


@pytest.mark.parametrize("change", [
    lambda a: a.update(q=a["q"].float()),
    lambda a: a.update(q=a["q"][..., :60]),
    lambda a: a.update(q=a["q"][..., ::2]),
    lambda a: a.update(q=a["q"][0]),
    lambda a: a.update(k=a["k"][:, :, :3]),
    lambda a: a.update(q_weight=a["q_weight"].half()),
    lambda a: a.update(k_weight=None),
    lambda a: a.update(k_weight=a["k_weight"].bfloat16()),
    lambda a: a.update(q_weight=a["q_weight"][:32]),
    lambda a: a.update(positions=a["positions"].long()),
    lambda a: a.update(positions=a["positions"][:3]),
    lambda a: a.update(positions=a["positions"].cpu()),
    lambda a: a.update(positions=None),
    lambda a: a.update(rope=None),
    lambda a: a.update(rope=RopePlan(128)),
])
def test_refusals(change):
    q, k, _, _ = _make(2, 2, 1, 5, 64, 71, inner=False)
    ws, _ = _weights(64, 3, torch.float32)
    args = dict(q=q, k=k, positions=torch.arange(5, dtype=torch.int32, device="cuda"), rope=RopePlan(64),
                q_weight=ws[0], k_weight=ws[1])
    qat_qk_norm_rope(**args)
    change(args)
    with pytest.raises((ValueError, TypeError)):
        qat_qk_norm_rope(**args)
    check_device_status()


def test_captured_forward_and_backward():
    """Forward and backward in one graph, through the functions and through autograd; replays follow new
    inputs, and give the eager call's bits."""
    q, k, fq, fk, ws, fws, rope, pos, g, fg = _backward_case(2, 6, 2, 37, 64, 64, "half", torch.float32)
    dpos = torch.from_numpy(pos).cuda()
    q, k = q.contiguous(), k.contiguous()

    def run():
        leaves = [t.detach().requires_grad_(True) for t in (q, k, *ws)]
        out = qat_qk_norm_rope(leaves[0], leaves[1], dpos, rope, leaves[2], leaves[3])
        grads = torch.autograd.grad(out, leaves, g)
        return [t.detach() for t in out] + list(grads) + list(
            qat_qk_norm_rope_backward(q, k, dpos, rope, *ws, *g))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()  # loads the kernels
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for seed in (1, 2):
        new = dev_bf16(normal_bf16(seed, tuple(q.shape)))
        q.copy_(new)
        dpos.add_(seed)
        graph.replay()
        for a, b in zip(captured, run()):
            assert torch.equal(a, b)
    for a, b in zip(captured[2:6], captured[6:]):
        assert torch.equal(a, b)


def test_a_capture_beside_a_living_eager_graph_of_the_leaves_is_refused():
    """The leaves' accumulation nodes belong to the default stream while the eager graph lives; with it
    gone, or made on another stream, the same capture goes through.  Only the forward is called here where
    the call has to be refused."""
    q, k, fq, fk, ws, fws, rope, pos, g, fg = _backward_case(1, 2, 1, 9, 64, 64, "half", torch.float32)
    dpos = torch.from_numpy(pos).cuda()
    leaves = [t.contiguous().detach().requires_grad_(True) for t in (q, k, *ws)]

    def forward():
        return qat_qk_norm_rope(leaves[0], leaves[1], dpos, rope, leaves[2], leaves[3])

    eager = forward()
    want = torch.autograd.grad(eager, leaves, g, retain_graph=True)
    torch.cuda.synchronize()
    with pytest.raises(ValueError, match="default stream"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            forward()
    torch.cuda.synchronize()
    del eager
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(forward(), leaves, g)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(forward(), leaves, g)
    graph.replay()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_sizes_beyond_32_bits_are_refused():
    x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="too large"):
        qat_qk_norm_rope(x.expand(1, 1, 2 ** 32 + 1, 64))
