"""Calls at the edges of what the norm + rotation, the cache and decoding take: several host threads, tensors
without heads, derivatives that are not there, wrappers, a captured backward, wide tables."""

import gc
import sys
import threading

import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as fwad

from oracle import serving_oracle as so
from quantization_aware_attention_gb300 import (KVCache, RopePlan, qat_attention_decode, qat_qk_norm_rope,
                                                qat_qk_norm_rope_backward)
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


def test_decode_from_threads_with_different_batches():
    """Host threads that decode batches of 1 and of 4096 sequences at the same time, through the C ABI: the
    kernel's shared memory, which grows with the batch, is enough for every one of them."""
    D, page = 128, 16
    cache = KVCache.empty(1, 1, page, D)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).zero_()
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(1.0)
    calls, bad = [], []
    for B in (1, 4096) * 3:
        q = torch.ones(B, 1, 1, D, dtype=torch.bfloat16, device="cuda")
        o = torch.empty_like(q)
        ws = torch.empty(capi.qat_attn_decode_workspace_bytes(1, 1, 1, D), dtype=torch.uint8, device="cuda")
        calls.append((q, cache.k, cache.v, cache.k_scale, cache.v_scale, _i32(np.zeros((B, 1))), _i32([5] * B), o,
                      None, B, 1, 1, 1, D, 1, page, 1, 0.1, 1, ws, ws.numel(), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(args):
        for _ in range(10000):
            st = capi.qat_attn_decode(*args)
            if st != Status.OK:
                bad.append((args[9], st))

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    switch = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(switch)
    torch.cuda.synchronize()
    assert not bad, (len(bad), bad[:3])
    assert all((c[7] == 0).all() for c in calls)


@pytest.mark.parametrize("Hq,Hk", [(3, 0), (0, 2), (0, 0)])
@pytest.mark.parametrize("wtype", [torch.float32, torch.bfloat16])
def test_gradients_where_a_tensor_has_no_heads(Hq, Hk, wtype):
    """Both weights given, one tensor (or each) without heads: its weight's gradient is zero, the other's what
    it is alone."""
    D, rope = 64, RopePlan(32)
    q, k = (dev_bf16(normal_bf16(80 + h, (2, 3, 5, D)))[:, :h] for h in (Hq, Hk))
    g = [dev_bf16(normal_bf16(90 + h, (2, 3, 5, D)))[:, :h] for h in (Hq, Hk)]
    w = [torch.linspace(0.5, 1.5, D, device="cuda").to(wtype).requires_grad_(True) for _ in range(2)]
    pos = _i32(range(5))
    leaves = [q.detach().requires_grad_(True), k.detach().requires_grad_(True), *w]
    out = qat_qk_norm_rope(leaves[0], leaves[1], pos, rope, *w)
    grads = torch.autograd.grad(out, leaves, g)
    direct = qat_qk_norm_rope_backward(q, k, pos, rope, *(t.detach() for t in w), *g)
    for x, y, leaf in zip(grads, direct, leaves):
        assert x.shape == leaf.shape and x.dtype == leaf.dtype and torch.equal(x, y)
    for i, (t, h) in enumerate(((q, Hq), (k, Hk))):
        if h == 0:
            assert (grads[2 + i] == 0).all()
        else:
            alone = qat_qk_norm_rope_backward(t, None, pos, rope, w[i].detach(), None, g[i], None)
            assert torch.equal(alone[0], grads[i]) and torch.equal(alone[2], grads[2 + i])


def test_forward_mode_derivatives_are_refused():
    """A tangent that a call would drop is an error, on tensors that need gradients and on others."""
    q, k = (dev_bf16(normal_bf16(70 + h, (2, h, 5, 64))) for h in (4, 2))
    w = [torch.ones(64, device="cuda") for _ in range(2)]
    pos, table, lens = _i32(range(5)), _i32([[0], [1]]), _i32([5, 5])
    cache = KVCache.empty(2, 2, 16, 64)
    cache.append(k, k, table, lens)
    args = [q, k, *w]
    for needs in (False, True):
        for i in range(4):
            with fwad.dual_level():
                a = [t.detach().requires_grad_(needs) for t in args]
                a[i] = fwad.make_dual(a[i], torch.ones_like(a[i]))
                with pytest.raises((ValueError, RuntimeError), match="forward-mode|jvp"):
                    qat_qk_norm_rope(a[0], a[1], pos, RopePlan(64), a[2], a[3])
    with fwad.dual_level():
        dual = fwad.make_dual(k, torch.ones_like(k))
        for call in (lambda: cache.append(dual, k, table, lens), lambda: cache.append(k, dual, table, lens),
                     lambda: qat_attention_decode(fwad.make_dual(q, torch.ones_like(q)), cache, table, lens),
                     lambda: qat_qk_norm_rope_backward(q, k, pos, RopePlan(64), *w, q, dual)):
            with pytest.raises(ValueError, match="forward-mode"):
                call()
        leaf = q.detach().requires_grad_(True)
        out = qat_qk_norm_rope(leaf, q_weight=w[0])
        with pytest.raises(ValueError, match="forward-mode"):  # forward over reverse
            torch.autograd.grad(out, leaf, fwad.make_dual(q, torch.ones_like(q)))
        scaled = KVCache(cache.k, cache.v, fwad.make_dual(cache.k_scale, torch.ones_like(cache.k_scale)),
                         cache.v_scale)
        with pytest.raises(ValueError, match="forward-mode"):
            scaled.read(table, lens)
    # and the same calls without a tangent go through
    assert len(qat_qk_norm_rope(q, k, pos, RopePlan(64), *w)) == 2
    assert qat_attention_decode(q, cache, table, lens, check=True).shape == q.shape


def test_function_transforms_are_refused():
    """torch.func's wrapped tensors have no memory of their own: an error, not a result without the transform."""
    q = dev_bf16(normal_bf16(75, (3, 2, 4, 5, 64)))
    w = torch.ones(64, device="cuda")
    for call in (lambda: torch.func.vmap(lambda x: qat_qk_norm_rope(x, q_weight=w))(q),
                 lambda: torch.func.grad(lambda x: qat_qk_norm_rope(x, q_weight=w).float().sum())(q[0]),
                 lambda: torch.func.jvp(lambda x: qat_qk_norm_rope(x, q_weight=w), (q[0],), (q[0],))):
        with pytest.raises((ValueError, RuntimeError)):
            call()


class _Wrapper(torch.Tensor):
    """Sizes and a device, no memory."""

    @staticmethod
    def __new__(cls, like):
        return torch.Tensor._make_wrapper_subclass(cls, like.shape, dtype=like.dtype, device=like.device)

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError(str(func))


def test_tensors_without_memory_are_refused():
    """Optional arguments among them: they are not taken for absent."""
    q, k = (dev_bf16(normal_bf16(76 + h, (2, h, 5, 64))) for h in (4, 2))
    w, pos, table, lens = torch.ones(64, device="cuda"), _i32(range(5)), _i32([[0], [1]]), _i32([5, 5])
    cache = KVCache.empty(2, 2, 16, 64)
    rope = RopePlan(64)
    for call in (lambda: qat_qk_norm_rope(q, k, pos, rope, _Wrapper(w), _Wrapper(w)),
                 lambda: qat_qk_norm_rope(q, k, _Wrapper(pos), rope, w, w),
                 lambda: qat_qk_norm_rope(q, _Wrapper(k), pos, rope, w, w),
                 lambda: qat_qk_norm_rope_backward(q, k, pos, rope, w, w, q, _Wrapper(k)),
                 lambda: cache.append(k, k, table, lens, _Wrapper(lens)),
                 lambda: cache.append(k, k, _Wrapper(table), lens),
                 lambda: qat_attention_decode(q, cache, table, lens,
                                              workspace=_Wrapper(torch.empty(1 << 20, dtype=torch.uint8,
                                                                             device="cuda")))):
        with pytest.raises(ValueError, match="memory"):
            call()


@pytest.mark.parametrize("alive", ["projection", "input"])
def test_a_captured_backward_beside_a_living_eager_graph_of_a_projection(alive):
    """q and k are slices of a projection, whose weight's accumulation node (or the projection itself) belongs to
    the default stream: the captured backward is refused before gradients leave the operator.  With the eager graph
    gone, or where the backward ends before it, the same capture goes through with the eager call's bits."""
    H, D, N = 2, 64, 9
    gen = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(1, N, 128, generator=gen, device="cuda").bfloat16()
    big = (torch.randn(128, 2 * H * D, generator=gen, device="cuda") / 12).bfloat16().requires_grad_(True)
    w = torch.ones(D, device="cuda", requires_grad=True)
    pos, rope = _i32(range(N)), RopePlan(D)
    g = [torch.randn(1, H, N, D, generator=gen, device="cuda").bfloat16() for _ in range(2)]

    def project():
        return (h @ big).view(1, N, 2 * H, D).transpose(1, 2)

    def forward(x):
        return qat_qk_norm_rope(x[:, :H], x[:, H:], pos, rope, w, w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = torch.autograd.grad(forward(project()), (big, w), g)  # and loads the kernels
    torch.cuda.current_stream().wait_stream(side)
    eager = project()
    torch.cuda.synchronize()
    with pytest.raises(ValueError, match="default stream"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            out = forward(project() if alive == "projection" else eager)
            torch.autograd.grad(out, (big, w), g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # the weight of the norm alone: nothing goes further
        got = torch.autograd.grad(forward(project()), w, g)
    graph.replay()
    assert torch.equal(got[0], want[1])
    del eager, out
    gc.collect()  # the refused call's frames
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(forward(project()), (big, w), g)
    graph.replay()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("n,Hkv,T", [(500, 8, 1), (1100, 2, 2), (3000, 1, 3)])
def test_the_same_lengths_in_tables_of_different_widths(n, Hkv, T):
    """A block table that could hold far longer sequences changes the order in which partials are added, and no
    more: every width gives rows within the oracle's tolerance, and its own bits again; entries behind the
    sequence's end are never followed."""
    D, G, page = 64, 4, 16
    per = -(-n // page)
    k, v = (dev_bf16(normal_bf16(60 + i, (1, Hkv, n, D))) for i in range(2))
    q = dev_bf16(normal_bf16(62, (1, Hkv * G, T, D)))
    cache = KVCache.empty(per, Hkv, page, D)
    narrow = torch.randperm(per, device="cuda", dtype=torch.int32)[None]
    cache.append(k, v, narrow, _i32([n]), check=True)
    kk, vv = (so.dequant(*so.quant_row(host_f64(x)[0])) for x in (k, v))
    for width in (per, 4 * per, 8192):
        table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
        table[:, :per] = narrow
        o, lse = qat_attention_decode(q, cache, table, _i32([n]), return_lse=True, check=True)
        for h in range(Hkv * G):
            w, wl, tol, ltol = so.decode_head(host_f64(q)[0, h], kk[h // G], vv[h // G], n - T + np.arange(T),
                                              D ** -0.5, 1)
            assert (np.abs(host_f64(o)[0, h] - w) <= tol).all()
            assert (np.abs(host_f64(lse)[0, h] - wl) <= ltol).all()
        again = qat_attention_decode(q, cache, table, _i32([n]), return_lse=True)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
