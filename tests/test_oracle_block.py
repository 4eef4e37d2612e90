"""Pins of oracle/block.py: closed forms, hand-worked rows, invariants."""
import math

import numpy as np
import pytest

from oracle import block as B
from oracle import moe as M


def test_rmsnorm_closed_form():
    y, n = B.add_rmsnorm([[3.0, 4.0]], None, 0.0)
    assert np.allclose(n, [[3 / math.sqrt(12.5), 4 / math.sqrt(12.5)]], rtol=1e-15)
    y, n = B.add_rmsnorm([[1.0, -1.0]], [2.0, 3.0], 3.0, res=[[0.0, 2.0]])
    assert y.tolist() == [[1.0, 1.0]] and np.allclose(n, [[1.0, 1.5]], rtol=1e-15)
    assert B.add_rmsnorm([[0.0, 0.0]], None, 1e-6)[1].tolist() == [[0.0, 0.0]]


def test_route_matches_plain_routing():
    """Softmax scores, no bias, one group, renormalised: the softmax top-k."""
    rng = np.random.default_rng(0)
    l = rng.standard_normal((20, 37)).astype(np.float32)
    ids, w, nan = B.route_scored(l, 5)
    rid, rw, rnan = M.route(l, 5)
    assert np.array_equal(ids, rid) and np.allclose(w, rw, atol=1e-7) and nan == rnan == False  # noqa: E712


def test_route_hand_worked():
    l = np.array([[0.0, 0.0, 1.0, -np.inf, 2.0, 0.0]], dtype=np.float32)
    s = [0.5, 0.5, 1 / (1 + math.exp(-1)), 0.0, 1 / (1 + math.exp(-2)), 0.5]
    # the bias selects, the score weighs; a masked expert is not saved by its bias
    ids, w, _ = B.route_scored(l, 2, bias=[0.0, 0.9, 0.0, 9.0, 0.0, 0.0], score="sigmoid", renorm=False, scale=2.0)
    assert ids.tolist() == [[1, 4]] and np.allclose(w, [[2 * s[1], 2 * s[4]]], rtol=1e-15)
    # groups {0,1,2} and {3,4,5}: best two sum .5+.73 against .88+.5; best one .73 against .88
    assert B.route_scored(l, 2, score="sigmoid", n_group=2, group_top=2)[0].tolist() == [[4, 5]]
    assert B.route_scored(l, 3, score="sigmoid", n_group=2, group_top=1)[0].tolist() == [[4, 5, 3]]
    # ties to the lowest group and expert
    z = np.zeros((1, 6), dtype=np.float32)
    assert B.route_scored(z, 2, n_group=3, topk_group=1)[0].tolist() == [[0, 1]]


def test_route_rows_without_an_expert():
    l = np.full((1, 4), -np.inf, dtype=np.float32)
    for score in ("softmax", "sigmoid"):
        ids, w, nan = B.route_scored(l, 2, score=score)
        assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]] and not nan
    ids, w, nan = B.route_scored(np.array([[np.nan, -np.inf, 0.0]], dtype=np.float32), 3)
    assert ids.tolist() == [[2, 1, 0]] and w.tolist() == [[1.0, 0.0, 0.0]] and nan


@pytest.mark.parametrize("act,f", [("none", lambda v: v), ("silu", lambda v: v / (1 + math.exp(-v))),
                                   ("gelu", lambda v: 0.5 * v * math.erfc(-v / math.sqrt(2)))])
def test_linear_activations(act, f):
    x, w = [[1.0, 2.0]], [[0.5, -1.0], [1.0, 1.0]]
    got = B.linear(x, w, bias=[0.25, 0.0], act=act, res=[[1.0, -1.0]])
    assert np.allclose(got, [[f(-1.25) + 1, f(3.0) - 1]], rtol=1e-14)


def test_linear_swiglu_order():
    got = B.linear([[1.0]], [[2.0], [3.0]], act="swiglu")
    assert np.allclose(got, [[2 / (1 + math.exp(-2)) * 3]], rtol=1e-14)


def test_mxfp8_rows_pins():
    bits = np.zeros((1, 32), dtype=np.uint16)
    bits[0, 0] = 0x3F80  # 1.0: X = -8, code of 256
    q, s = B.mxfp8_rows(bits)
    assert s.tolist() == [[119]] and q[0, 0] == 0x78 and not q[0, 1:].any()
