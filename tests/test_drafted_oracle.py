"""Pins of the oracle of windows, trees and kept paths (oracle/drafted_oracle.py): the plain causal oracle, counting
by hand and finite differences, on the CPU."""

import numpy as np
import pytest

from oracle import drafted_oracle as do_
from oracle import qat_oracle as orc
from oracle import serving_oracle as so


def _rng(seed):
    return np.random.default_rng(seed)


def test_windows_by_counting():
    seen = do_.window_seen(range(6), 6, 2, 1)
    want = ["100000", "110000", "111000", "101100", "100110", "100011"]
    assert ["".join("01"[int(x)] for x in row) for row in seen] == want
    assert (do_.window_seen(range(50), 50, 50, 0) == np.tril(np.ones((50, 50), bool))).all()
    assert (do_.window_seen(range(50), 50, 1, 50) == np.tril(np.ones((50, 50), bool))).all()
    assert not do_.window_seen([-1], 4, 3, 2).any()


@pytest.mark.parametrize("quant", [False, True])
def test_wide_windows_are_causal_attention(quant):
    rng = _rng(1)
    q, k, v, do = (rng.standard_normal((90, 64)) for _ in range(4))
    r = do_.head_train(q, k, v, do, 0.2, do_.window_seen(range(90), 90, 1000, 0), quant)
    f = orc.head_forward(q, k, v, 0.2, True, quant)
    assert np.allclose(r["o_q"], f["o_q" if quant else "o_hp"], atol=1e-12) and np.allclose(r["lse"], f["lse"])
    for n, want in zip(("dq", "dk", "dv"), orc.head_backward(q, k, v, do, 0.2, True)):
        assert np.allclose(r[n], want, atol=1e-12)
    page = do_.head_train(q, k, v, do, 0.2, do_.window_seen(range(90), 90, 1000, 0), True, page=True)
    for n, want in zip(("dq", "dk", "dv"), orc.head_backward_page(q, k, v, do, 0.2, True)):
        assert np.allclose(page[n], want, atol=1e-12)


@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 0), (7, 3), (1, 5)])
def test_gradients_against_differences(window, sinks):
    rng = _rng(2)
    n, D = 40, 8
    q, k, v, do = (rng.standard_normal((n, D)) for _ in range(4))
    seen = do_.window_seen(range(n), n, window, sinks)
    r = do_.head_train(q, k, v, do, 0.3, seen, False)

    def value(q, k, v):
        return float((do * do_.head_train(q, k, v, do, 0.3, seen, False)["o_hp"]).sum())

    h = 1e-5
    for _ in range(5):
        for i, name in enumerate(("dq", "dk", "dv")):
            d = [np.zeros((n, D))] * 3
            d[i] = rng.standard_normal((n, D))
            num = (value(q + h * d[0], k + h * d[1], v + h * d[2]) - value(q - h * d[0], k - h * d[1], v - h * d[2]))
            assert abs(num / (2 * h) - (r[name] * d[i]).sum()) <= 1e-7 * max(1.0, abs(num / (2 * h)))


def test_a_chain_is_decoding():
    """A tree whose tokens each continue the one before is the plain decoding of its tokens, windows included."""
    T, length = 5, 90
    masks, pos = do_.draft([-1, 0, 1, 2, 3], length)
    assert masks == [1, 3, 7, 15, 31] and list(pos) == [85, 86, 87, 88, 89]
    assert (do_.tree_seen(length, masks) == do_.window_seen(range(85, 90), 90, 1000, 0)).all()
    assert (do_.tree_seen(length, masks, 9, 3) == do_.window_seen(range(85, 90), 90, 9, 3)).all()
    rng = _rng(3)
    q, k, v = rng.standard_normal((T, 64)), rng.standard_normal((length, 64)), rng.standard_normal((length, 64))
    one = do_.attend_rows(q, k, v, do_.tree_seen(length, masks), 0.125, True, do_.F16)
    two = so.decode_head(q, k, v, np.arange(85, 90), 0.125, True)
    for x, y in zip(one, two):
        assert np.allclose(x, y, atol=1e-12)


def test_trees_by_hand():
    #        0   1  2  3   4  5   6: padding, as is what continues it
    masks, pos = do_.draft([-1, 0, 0, 2, -1, 4, 9, 6], 100)
    assert masks == [1, 0b11, 0b101, 0b1101, 0b10000, 0b110000, 0, 0]
    assert list(pos) == [92, 93, 93, 94, 92, 93, 91, 91]
    seen = do_.tree_seen(4, [0b1, 0b11, 0b101, 0b1000, 0, 0b100000])  # slots -2 .. 3
    assert seen.astype(int).tolist() == [[0] * 4, [0] * 4, [1, 0, 0, 0], [0, 1, 0, 0], [0] * 4, [0, 0, 0, 1]]


def test_kept_paths():
    moves, new = do_.keep([10, 3, 4], 4, [[0, 2, 3], [1, 3, 0], [7, 1, -1]], [3, 9, 3])
    assert moves == [(0, 6, 6), (0, 8, 7), (0, 9, 8), (1, 2, 0), (2, 1, 1)]
    assert new == [9, 2, 3]
