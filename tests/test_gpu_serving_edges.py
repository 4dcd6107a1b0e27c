"""Calls at the edges of what the norm + rotation, the cache and decoding take."""

import sys
import threading

import numpy as np
import pytest
import torch

from quantization_aware_attention_gb300 import KVCache
from quantization_aware_attention_gb300 import build as qbuild
from quantization_aware_attention_gb300 import capi
from quantization_aware_attention_gb300.capi import Status

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
