"""GPU tests of a drafted tree's attention at its edges, the narrow and the wide kernel alike: codes that are not a number,
and pages that no token's window reaches."""

import numpy as np
import pytest
import torch

from oracle import drafted_oracle as do_
from quantization_aware_attention_gb300 import check_device_status, qat_attention_tree
from quantization_aware_attention_gb300 import build as qbuild
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
    that sees the key and of no other, in a value its channel."""
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
            others = [c for c in range(D) if c != d]
            assert torch.equal(o[..., others], clean[..., others]) and torch.equal(lse, clean_lse)
    assert torch.equal(qat_attention_tree(*args)[0], clean)
    check_device_status()
