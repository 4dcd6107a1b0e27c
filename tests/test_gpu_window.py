"""GPU parity of attention with a sliding window and sinks, forward and backward, against the fp64 oracle
(oracle/drafted_oracle.py).  Tolerances are the training kernels' (gpu_util): relative L2 over a tensor."""

import numpy as np
import pytest
import torch

from oracle import drafted_oracle as do_
from oracle import qat_oracle as orc
from quantization_aware_attention_gb300 import (QUANT_P_FP8E4M3_ROW_TILE64_PAGE_BWD, QatError, attention,
                                                check_device_status, qat_attention_backward, qat_attention_forward,
                                                qat_prepare_qkv)
from quantization_aware_attention_gb300 import build as qbuild
from quantization_aware_attention_gb300 import capi
from quantization_aware_attention_gb300.inputs import custom_inputs

from gpu_util import TOL_HP, TOL_Q, dev_bf16, host_f64, oracle_f64, rel_l2

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    qbuild.build()


def _inputs(seed, B, H, N, D):
    inp = custom_inputs(seed, B, H, N, N, D)
    return oracle_f64(inp), [dev_bf16(inp[n]) for n in ("q", "k", "v", "do")]


def _want(f, sm, seen, heads, **kw):
    r = [do_.head_train(f["q"][b, h], f["k"][b, h], f["v"][b, h], f["do"][b, h], sm, seen, **kw) for b, h in heads]
    return {n: np.stack([x[n] for x in r]) for n in r[0]}


def _check(got, want, heads, names=("o_q", "o_hp", "lse", "dq", "dk", "dv"), what=""):
    for n in names:
        g = np.stack([host_f64(got[n][b, h]) for b, h in heads])
        err = rel_l2(g, want[n])
        assert err <= (TOL_HP if n in ("o_hp", "lse") else TOL_Q), (what, n, err)


def _run(t, window, sinks, sm=None, quant=1, **kw):
    q, k, v, do = t
    o_q, o_hp, lse = qat_attention_forward(q, k, v, True, sm, quant, window, sinks)
    o = o_q if quant == QUANT_P_FP8E4M3_ROW_TILE64_PAGE_BWD else o_hp
    dq, dk, dv = qat_attention_backward(q, k, v, o, lse, do, True, sm, quant, window=window, sinks=sinks, **kw)
    check_device_status()
    return dict(o_q=o_q, o_hp=o_hp, lse=lse, dq=dq, dk=dk, dv=dv)


@pytest.mark.parametrize("B,H,N,D,window,sinks", [
    (1, 1, 2, 64, 2, 0),
    (1, 2, 64, 128, 3, 0),
    (2, 1, 127, 64, 63, 1),
    (1, 2, 128, 128, 64, 64),
    (1, 3, 129, 64, 65, 4),          # one row behind the first block
    (1, 2, 257, 128, 128, 0),
    (1, 1, 257, 64, 129, 127),
    (2, 2, 300, 128, 100, 5),
    (1, 1, 520, 64, 1, 3),           # the row itself and the sinks
    (1, 1, 777, 128, 127, 130),      # sinks in two blocks
    (1, 2, 777, 64, 2, 700),
    (1, 1, 1025, 128, 300, 64),
    (1, 1, 1400, 64, 1000, 17),      # more than eight blocks a row
    (1, 1, 1400, 128, 900, 300),
    (1, 1, 333, 64, 1 << 40, 0),     # no limit
    (1, 1, 333, 128, 5, 1 << 40),
])
@pytest.mark.parametrize("quant", [0, 1])
def test_window(B, H, N, D, window, sinks, quant):
    f, t = _inputs(50 + N, B, H, N, D)
    heads = [(b, h) for b in range(B) for h in range(H)]
    got = _run(t, window, sinks, quant=quant)
    want = _want(f, D ** -0.5, do_.window_seen(range(N), N, window, sinks), heads, quant=bool(quant))
    _check(got, want, heads, what=(N, window, sinks))
    again = _run(t, window, sinks, quant=quant)
    assert all(torch.equal(got[n], again[n]) for n in got)


def test_a_window_of_one_is_the_value():
    """Each row sees itself alone: its value comes back, and with P constant no gradient reaches q or k.  dS =
    P (dP - Delta) is the difference of two fp32 sums of the same D products (o is v exactly): 2^-16 of their sum."""
    f, t = _inputs(3, 1, 2, 200, 64)
    got = _run(t, 1, 0)
    assert torch.equal(got["o_q"], t[2]) and torch.equal(got["o_hp"], t[2].float())
    assert rel_l2(host_f64(got["dv"]), f["do"]) <= TOL_Q
    ds = 2.0 ** -16 * np.abs(f["do"] * f["v"]).sum(-1, keepdims=True)
    assert (np.abs(host_f64(got["dq"])) <= 0.125 * ds * np.abs(f["k"]) * 1.01 + 1e-30).all()
    assert (np.abs(host_f64(got["dk"])) <= 0.125 * ds * np.abs(f["q"]) * 1.01 + 1e-30).all()


@pytest.mark.parametrize("H,N,D,window,sinks", [(1, 4000, 64, 128, 4), (2, 2500, 128, 50, 200), (1, 3900, 128, 700, 129)])
def test_sinks_cut_into_pieces(H, N, D, window, sinks):
    """The sinks' dK and dV are sums over all queries, in pieces that one more kernel adds; what the workspace holds
    before is of no account, and the bits are the same in every run and replay."""
    assert capi.qat_attn_bwd_window_workspace_bytes(1, H, N, D, window, sinks) > \
        capi.qat_attn_bwd_window_workspace_bytes(1, H, N, D, window, 0)
    f, t = _inputs(7, 1, H, N, D)
    got = _run(t, window, sinks)
    heads = [(0, H - 1)]
    _check(got, _want(f, D ** -0.5, do_.window_seen(range(N), N, window, sinks), heads), heads)
    ws = torch.full((capi.qat_attn_bwd_window_workspace_bytes(1, H, N, D, window, sinks),), 0xff, dtype=torch.uint8,
                    device="cuda")
    q, k, v, do = t
    args = (q, k, v, got["o_hp"], got["lse"], do, True)
    for _ in range(2):
        again = qat_attention_backward(*args, workspace=ws, window=window, sinks=sinks)
        assert all(torch.equal(got[n], x) for n, x in zip(("dq", "dk", "dv"), again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = qat_attention_backward(*args, workspace=ws, window=window, sinks=sinks)
    for _ in range(2):
        for x in out:
            x.zero_()
        graph.replay()
        assert all(torch.equal(got[n], x) for n, x in zip(("dq", "dk", "dv"), out))
    with pytest.raises(QatError):
        qat_attention_backward(*args, workspace=ws[:-1], window=window, sinks=sinks)


@pytest.mark.parametrize("window,sinks", [(100, 4), (700, 0)])
def test_page_backward(window, sinks):
    B, H, N, D = 1, 2, 900, 128
    f, t = _inputs(9, B, H, N, D)
    got = _run(t, window, sinks, quant=QUANT_P_FP8E4M3_ROW_TILE64_PAGE_BWD)
    heads = [(0, 0), (0, 1)]
    want = _want(f, D ** -0.5, do_.window_seen(range(N), N, window, sinks), heads, page=True)
    _check(got, want, heads)


def test_quantized_inputs_and_smooth_k():
    """The options of the full path: fake-quantized q, k and v, with the mean of K taken out and its term in dQ."""
    B, H, N, D, window, sinks = 1, 2, 500, 64, 90, 3
    f, (q, k, v, do) = _inputs(10, B, H, N, D)
    leaves = [x.clone().requires_grad_(True) for x in (q, k + 2, v)]
    o = attention(*leaves, causal=True, quant_mode=2, qkv_quant=True, smooth_k=True, window=window, sinks=sinks, check=True)
    grads = torch.autograd.grad(o, leaves, do)
    qf, kf, vf, k_mean = qat_prepare_qkv(*(x.detach() for x in leaves), True)
    f = dict(q=host_f64(qf), k=host_f64(kf), v=host_f64(vf), do=f["do"])
    heads = [(0, 0), (0, 1)]
    want = _want(f, D ** -0.5, do_.window_seen(range(N), N, window, sinks), heads, page=True, k_mean=host_f64(k_mean))
    _check(dict(o_q=o, dq=grads[0], dk=grads[1], dv=grads[2]), want, heads, ("o_q", "dq", "dk", "dv"))


def test_sampled_heads_of_a_large_call():
    """Enough items that every SM takes several: sampled heads against the oracle, the rest against themselves."""
    B, H, N, D, window, sinks = 2, 24, 2000, 128, 500, 4
    f, t = _inputs(11, B, H, N, D)
    got = _run(t, window, sinks)
    heads = [(0, 0), (1, 23), (1, 7)]
    _check(got, _want(f, D ** -0.5, do_.window_seen(range(N), N, window, sinks), heads), heads)
    one = _run([x[1:, 7:8].contiguous() for x in t], window, sinks)
    assert torch.equal(one["o_q"][0, 0], got["o_q"][1, 7]) and torch.equal(one["dq"][0, 0], got["dq"][1, 7])


def test_whole_windows_are_causal_attention():
    """A window that holds every key is plain causal attention, up to the order of sums: both within the tolerance of
    the same values, and 2^-7 of each other where a bf16 step is all that lies between."""
    _, t = _inputs(12, 1, 2, 700, 128)
    a = _run(t, 700, 0)
    o_q, o_hp, lse = qat_attention_forward(t[0], t[1], t[2], True)
    grads = qat_attention_backward(t[0], t[1], t[2], o_hp, lse, t[3], True)
    for n, x in zip(("o_q", "o_hp", "lse", "dq", "dk", "dv"), (o_q, o_hp, lse) + grads):
        assert rel_l2(host_f64(a[n]), host_f64(x)) <= 2 * TOL_Q, n


def test_autograd_streams_and_graphs():
    """Through autograd; on a stream of its own; captured forward and backward, replayed on new inputs."""
    B, H, N, D, window, sinks = 1, 3, 400, 64, 70, 4
    f, (q, k, v, do) = _inputs(13, B, H, N, D)
    heads = [(0, h) for h in range(H)]
    want = _want(f, D ** -0.5, do_.window_seen(range(N), N, window, sinks), heads)
    leaves = [x.clone().requires_grad_(True) for x in (q, k, v)]
    o = attention(*leaves, causal=True, window=window, sinks=sinks)
    o.backward(do)
    got = dict(o_q=o, dq=leaves[0].grad, dk=leaves[1].grad, dv=leaves[2].grad)
    _check(got, want, heads, ("o_q", "dq", "dk", "dv"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on = _run([q, k, v, do], window, sinks)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(on["o_q"], o) and torch.equal(on["dk"], leaves[1].grad)
    bufs = [torch.zeros_like(x) for x in (q, k, v, do)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o_q, o_hp, lse = qat_attention_forward(*bufs[:3], True, window=window, sinks=sinks)
        grads = qat_attention_backward(*bufs[:3], o_hp, lse, bufs[3], True, window=window, sinks=sinks)
    for b, x in zip(bufs, (q, k, v, do)):
        b.copy_(x)
    graph.replay()
    assert torch.equal(o_q, o) and all(torch.equal(g, x.grad) for g, x in zip(grads, leaves))


def test_refusals():
    _, (q, k, v, do) = _inputs(14, 1, 1, 64, 64)
    for how in (dict(causal=False, window=4), dict(causal=True, window=0), dict(causal=True, window=4, sinks=-1),
                dict(causal=True, sinks=2)):
        with pytest.raises(ValueError):
            attention(q, k, v, **how)
    with pytest.raises(ValueError):
        attention(q, k[:, :, :32].contiguous(), v[:, :, :32].contiguous(), causal=True, window=4)
    with pytest.raises(ValueError):
        attention(q.float(), k, v, causal=True, window=4)
    with pytest.raises(ValueError):
        attention(q[..., :32], k, v, causal=True, window=4)
    check_device_status()


def test_without_gradients_the_output_is_the_same():
    """A call without gradients leaves O_hp out (null through the C ABI); its output is the training forward's."""
    for N, D, window, sinks in ((700, 128, 200, 4), (1500, 64, 1400, 0), (130, 128, 20, 1)):
        _, (q, k, v, _) = _inputs(15, 1, 2, N, D)
        o_q, _, lse = qat_attention_forward(q, k, v, True, window=window, sinks=sinks)
        with torch.no_grad():
            assert torch.equal(attention(q, k, v, causal=True, window=window, sinks=sinks, check=True), o_q)
        o = torch.full_like(q, float("nan"))
        stats = torch.empty_like(lse)
        assert capi.qat_attn_fwd_window(q, k, v, o, None, stats, 1, 2, N, D, D ** -0.5, window, sinks, 1) == 0
        assert torch.equal(o, o_q) and torch.equal(stats, lse)


def test_derivatives_that_are_not_there():
    """A second derivative, forward-mode derivatives, and a captured backward of leaves in which a graph of the default
    stream ends (torch would wait for the capture on that stream) are refused."""
    import torch.autograd.forward_ad as fwad
    _, (q, k, v, do) = _inputs(16, 1, 1, 128, 64)
    how = dict(causal=True, window=30, sinks=2)
    leaves = [x.clone().requires_grad_(True) for x in (q, k, v)]
    o = attention(*leaves, **how)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(o, leaves, do, create_graph=True)
    with fwad.dual_level():
        with pytest.raises(ValueError, match="forward-mode"):
            attention(fwad.make_dual(q, q), k, v, **how)
    want = torch.autograd.grad(o, leaves, do, retain_graph=True)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(ValueError, match="default stream"):
        with torch.cuda.graph(graph, stream=side):
            attention(*leaves, **how)
    del o, graph
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # warm, on the capturing stream
        torch.autograd.grad(attention(*leaves, **how), leaves, do)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = torch.autograd.grad(attention(*leaves, **how), leaves, do)
    for _ in range(2):
        for g in got:
            g.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_gradient_layouts():
    """An upstream gradient that is broadcast, strided or off the 16-byte boundary."""
    _, (q, k, v, do) = _inputs(17, 1, 2, 130, 64)
    how = dict(causal=True, window=30, sinks=2)
    leaves = [x.clone().requires_grad_(True) for x in (q, k, v)]
    want = torch.autograd.grad(attention(*leaves, **how), leaves, do)
    flat = torch.empty(do.numel() + 1, dtype=do.dtype, device="cuda")
    off = flat[1:].view(do.shape)
    off.copy_(do)
    for g in (do.transpose(1, 2).contiguous().transpose(1, 2), off):
        got = torch.autograd.grad(attention(*leaves, **how), leaves, g)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    ones = torch.autograd.grad(attention(*leaves, **how).sum(), leaves)
    full = torch.autograd.grad(attention(*leaves, **how), leaves, torch.ones_like(do))
    assert all(torch.equal(x, y) for x, y in zip(ones, full))
    only_v = [q, k, v.clone().requires_grad_(True)]
    assert torch.equal(torch.autograd.grad(attention(*only_v, **how), only_v[2:], do)[0], want[2])


def test_offsets_beyond_32_bits():
    """Tensors of more than 2^31 elements: the last head's results are those of a call with that head alone."""
    H, N, D, window, sinks = 136, 131072, 128, 200, 4
    x = torch.empty((1, H, N, D), dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator("cuda").manual_seed(3))
    how = dict(window=window, sinks=sinks)
    o_q, o_hp, lse = qat_attention_forward(x, x, x, True, **how)
    last = x[:, -1:].contiguous()
    want = qat_attention_forward(last, last, last, True, **how)
    for got, w in zip((o_q, o_hp, lse), want):
        assert torch.equal(got[:, -1:], w)
    del o_q
    grads = qat_attention_backward(x, x, x, o_hp, lse, x, True, **how)
    alone = qat_attention_backward(last, last, last, want[1], want[2], last, True, **how)
    assert torch.equal(grads[0][:, -1:], alone[0])
    keys = slice((sinks + 127) // 128 * 128, None)  # the sinks' own sums are cut into other pieces
    for got, w in zip(grads[1:], alone[1:]):
        assert torch.equal(got[:, -1:, keys], w[:, :, keys])
        assert rel_l2(host_f64(got[:, -1:, :sinks]), host_f64(w[:, :, :sinks])) <= TOL_Q
    check_device_status()


def test_scale():
    f, t = _inputs(18, 1, 1, 300, 64)
    heads = [(0, 0)]
    _check(_run(t, 50, 3, sm=0.3), _want(f, 0.3, do_.window_seen(range(300), 300, 50, 3), heads), heads)


def test_expired_waits():
    """With the waits' limit at nothing forward and backward give up, report it, and the next calls are whole."""
    _, t = _inputs(19, 1, 8, 2048, 128)
    want = _run(t, 700, 4)
    q, k, v, do = t
    assert capi.qat_debug_set_wait_limit_us(0) == 0
    try:
        with pytest.raises(QatError):
            for _ in range(5):
                attention(q, k, v, causal=True, window=700, sinks=4, check=True)
        seen = False
        for _ in range(5):
            qat_attention_backward(q, k, v, want["o_hp"], want["lse"], do, True, window=700, sinks=4)
            seen |= capi.qat_attn_device_status() == capi.Status.TIMEOUT
        assert seen
    finally:
        assert capi.qat_debug_set_wait_limit_us(4000000) == 0
        capi.qat_attn_device_status()
    got = _run(t, 700, 4)
    assert all(torch.equal(got[n], want[n]) for n in want)


def test_one_tensor_three_times_and_none():
    """q, k and v as one leaf: its gradient is the sum of the three; an empty batch; a single token."""
    f, (q, k, v, do) = _inputs(20, 1, 2, 200, 64)
    how = dict(causal=True, window=30, sinks=2)
    x = q.clone().requires_grad_(True)
    got = torch.autograd.grad(attention(x, x, x, **how), x, do)[0]
    each = [q.clone().requires_grad_(True) for _ in range(3)]
    parts = torch.autograd.grad(attention(*each, **how), each, do)
    assert rel_l2(host_f64(got), sum(host_f64(p) for p in parts)) <= 2.0 ** -7  # two sums rounded to bf16
    none = [x[:0].clone().requires_grad_(True) for x in (q, k, v)]
    assert all(g.shape == (0, 2, 200, 64) for g in torch.autograd.grad(attention(*none, **how).sum(), none))
    one = [x[:, :, :1].contiguous().requires_grad_(True) for x in (q, k, v)]
    o = attention(*one, **how, check=True)
    assert torch.equal(o, one[2]) and torch.equal(torch.autograd.grad(o, one[2:], do[:, :, :1])[0], do[:, :, :1])


def test_threads_on_streams_of_their_own():
    """Training passes of four host threads at once, each on its stream, give the same bits."""
    import threading
    _, t = _inputs(21, 2, 4, 700, 128)
    out, errors = {}, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                leaves = [x.clone().requires_grad_(True) for x in t[:3]]
                for _ in range(5):
                    o = attention(*leaves, causal=True, window=100, sinks=3)
                    grads = torch.autograd.grad(o, leaves, t[3])
                torch.cuda.current_stream().synchronize()
                out[i] = (o,) + grads
        except Exception as e:  # shown by the test, not by the thread
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not errors
    assert all(torch.equal(a, b) for i in range(1, 4) for a, b in zip(out[0], out[i]))


@pytest.mark.parametrize("N,D,window,sinks", [(700, 64, 1, 1), (700, 128, 2, 0), (700, 64, 3, 0), (900, 64, 10, 1),
                                              (1500, 128, 100, 5)])
def test_gradients_of_rows_that_see_few_keys(N, D, window, sinks):
    """P near 1 makes dS = P (dP - Delta) a small difference.  Roundings to bf16 are off by 1.7e-3 of a value (rms of
    half a step over mantissas); in quadrature the output once, dS once, which keys with an offset of half their spread
    make sqrt(1.25) of dQ, and P in O_hp and with it in Delta, at most as much: 1.7e-3 sqrt(1 + 1.25 + 1) = 3.1e-3."""
    g = torch.Generator("cuda").manual_seed(N + window)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    q, v, do = normal(1, 2, N, D) * 1.5, normal(1, 2, N, D), normal(1, 2, N, D)
    k = normal(1, 2, N, D) + 0.5 * normal(D)
    t = [q, k, v, do]
    f = {n: host_f64(x) for n, x in zip(("q", "k", "v", "do"), t)}
    heads = [(0, 0), (0, 1)]
    want = _want(f, D ** -0.5, do_.window_seen(range(N), N, window, sinks), heads)
    got = _run(t, window, sinks)
    for n in ("dq", "dk"):
        assert rel_l2(np.stack([host_f64(got[n][0, h]) for h in range(2)]), want[n]) <= 3.1e-3, n
