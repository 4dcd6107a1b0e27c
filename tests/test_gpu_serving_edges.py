"""Calls at the edges of what the norm + rotation, the cache and decoding take."""

import sys
import threading

import numpy as np
import pytest
import torch

from quantization_aware_attention_gb300 import (KVCache, RopePlan, qat_qk_norm_rope,
                                                qat_qk_norm_rope_backward)
from quantization_aware_attention_gb300 import build as qbuild
from quantization_aware_attention_gb300 import capi
from quantization_aware_attention_gb300.capi import Status
from quantization_aware_attention_gb300.inputs import normal_bf16

from gpu_util import dev_bf16

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
