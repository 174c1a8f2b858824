"""Pins of the oracle's norms around a block: hand cases and closed forms."""
import numpy as np


def test_hand_case(orc):
    # y = (3, 4): mean square 12.5; eps 3.5 -> divided by 4
    y = np.array([[3.0, 4.0]], np.float32)
    res = np.array([[1.0, -1.0]], np.float32)
    r, h = orc.norm_residual(res, y, w_post=np.array([1.0, 2.0], np.float32), scale=2.0, eps=3.5)
    np.testing.assert_array_equal(r, [[1 + 2 * 0.75, -1 + 2 * 2.0]])
    assert h is None
    # no norm of y, a gate, then a norm of r' = (7, 1): mean square 25, eps 0
    g = np.array([[2.0, 0.5]], np.float32)
    r, h = orc.norm_residual(res, y, w_pre=np.array([1.0, 3.0], np.float32), gate=g, eps=0.0)
    np.testing.assert_array_equal(r, [[7.0, 1.0]])
    np.testing.assert_allclose(h, [[7 / 5, 3 / 5]], rtol=1e-15)
    # weights about zero
    _, h = orc.norm_residual(res, y, w_pre=np.zeros(2, np.float32), gate=g, eps=0.0, w_offset=1.0)
    np.testing.assert_allclose(h, [[7 / 5, 1 / 5]], rtol=1e-15)


def test_gate_rows_and_sigmoid(orc):
    res, y = np.zeros((4, 1), np.float32), np.ones((4, 1), np.float32)
    g = np.array([[0.0], [np.log(3.0)]], np.float32)
    r, _ = orc.norm_residual(res, y, gate=g, gate_rep=2, sigmoid=True)
    np.testing.assert_allclose(r, [[0.5], [0.5], [0.75], [0.75]], rtol=1e-7)
    r, _ = orc.norm_residual(res, y, gate=g[1:], gate_rep=4)
    np.testing.assert_allclose(r, np.full((4, 1), np.log(3.0)), rtol=1e-7)
