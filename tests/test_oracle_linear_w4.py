"""Pins of the oracle's product with 4-bit weights and group scales: hand
cases, exact in fp64, that fix the order of the codes in a byte, the zero
point, the group of a column and the conv's tap order."""
import numpy as np
import pytest

import synth
from w4_inputs import activations, weights


def test_hand_case(orc):
    # K = 4, groups of 2: byte 0 holds k = 0 (low), 1 (high)
    q = np.array([[0x8F, 0x09], [0x10, 0xFF]], np.uint8)
    scale = np.array([[1.0, 2.0], [0.5, 4.0]], np.float32)
    x = np.array([[1, 10, 100, 1000]], np.float32)
    # row 0: codes 15 8 | 9 0, zero 8: 7 0 | 2 * (1, -8) -> 7 + 200 - 16000
    # row 1: codes 0 1 | 15 15: 0.5 * (-8, -7) | 4 * (7, 7) -> -4 - 35 + 2800 + 28000
    y, mag = orc.linear_w4(x, q, scale)
    np.testing.assert_array_equal(y, [[7 + 200 - 16000, -39 + 30800]])
    np.testing.assert_array_equal(mag, [[7 + 200 + 16000, 39 + 30800]])
    # zero points 15, 0 | 1, 15
    zero = np.array([[15, 0], [1, 15]], np.uint8)
    # row 0: (0, -7) | 2 * (9, 0) -> -70 + 1800; row 1: 0.5 * (-1, 0) | 0
    y, _ = orc.linear_w4(x, q, scale, zero)
    np.testing.assert_array_equal(y, [[-70 + 1800, -0.5]])


@pytest.mark.parametrize("group", [32, 64])
def test_against_a_dense_product(orc, group):
    rng = np.random.default_rng(5)
    N, K = 7, 128
    q, s, z = weights(rng, N, K, group, zeros=True, f32_scale=True)
    x = activations(rng, (3, K), "f32")
    codes = np.empty((N, K))
    codes[:, 0::2], codes[:, 1::2] = q & 15, q >> 4
    w = (codes - np.repeat(z, group, 1).astype(float)) * np.repeat(s, group, 1).astype(float)
    y, mag = orc.linear_w4(x, q, s, z)
    np.testing.assert_allclose(y, x.astype(float) @ w.T, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(mag, np.abs(x).astype(float) @ np.abs(w).T, rtol=1e-12)


def test_conv_is_the_dense_conv_on_the_same_taps(orc):
    """bf16 scales times integers are exact in fp32, so the conv's own oracle takes the same weights."""
    rng = np.random.default_rng(6)
    B, T, H = 2, 3, 64
    q, s, z = weights(rng, 2 * H, H, 32, zeros=True)
    codes = np.empty((2 * H, H), np.float32)
    codes[:, 0::2], codes[:, 1::2] = q & 15, q >> 4
    w = (codes - np.repeat(z, 32, 1)) * np.repeat(synth.bf16_bits_to_f32(s), 32, 1)
    x, xp = activations(rng, (B, T, H), "f32"), activations(rng, (B, H), "f32")
    out, _ = orc.dynconv2_w4(x, xp, q, s, z)
    np.testing.assert_allclose(out, orc.dynconv2(x, xp, w.astype(np.float32)), rtol=1e-12, atol=1e-12)
