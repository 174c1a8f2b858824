"""Seeded inputs and error bounds of the 4-bit-weight tests."""
import numpy as np

import synth


def weights(rng, N, K, group, zeros=False, f32_scale=False):
    """Codes [N, K/2] (even k low), scales [N, K/group] (float32 or bf16 bits), zero points."""
    q = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    s = (rng.uniform(0.5, 1.5, (N, K // group)) * 0.4 / np.sqrt(K)).astype(np.float32)
    z = rng.integers(0, 16, (N, K // group)).astype(np.uint8) if zeros else None
    return q, s if f32_scale else synth.to_bf16_bits(s), z


def activations(rng, shape, dt):
    x = rng.standard_normal(shape).astype(np.float32)
    return synth.to_bf16_bits(x) if dt == "bf16" else x


def sum_bound(K, planes):
    """Bound on |fp32 result - exact| / sum of |products|.

    A product of a code (integer, at most 8 bits) and a bf16 value is exact.
    Inside a 64-wide chunk an element passes through 4 matrix instructions per
    plane; each may cut its aligned fp32 sum off by one unit of 2^-22 of the
    magnitude (twice the step of fp32, for instructions that keep two guard
    bits and truncate), the planes' magnitudes adding up to at most
    (1 + 2^-7) of |x|.  Then come one fp32 fma per chunk (half a step, 2^-24,
    each), at most 16 runs' sums in a cluster's CTA and 8 CTAs, and the scale's
    fma.  The products of the planes below the first are cut at 2^-24 |x|
    (all 24 bits are kept, so nothing is lost there)."""
    chunks = -(-K // 64)
    return (4 * planes * 4 * (1 + 2.0 ** -7) + chunks + 16 + 8 + 2) * 2.0 ** -24
