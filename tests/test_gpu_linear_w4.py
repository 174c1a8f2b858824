"""GPU parity of the products with 4-bit weights (linear_w4) and of the
two-tap conv on 4-bit taps (dynconv2 with a PackedW4) against the fp64 oracle.

Error bound: the fp32 sum's (w4_inputs.sum_bound, relative to the sum of the
products' magnitudes) plus, for bf16 outputs, half a step: 2^-8 of the value."""
import numpy as np
import pytest
import torch

import block_draft_verification_b200 as dfl
import synth
from parity import bf16_to_f64, gpu, need_cuda, to_dev, to_host
from w4_inputs import activations, sum_bound, weights

pytestmark = gpu


def f64(t):
    a = to_host(t)
    return bf16_to_f64(a) if a.dtype == np.uint16 else a.astype(np.float64)


def assert_within(got, ref, mag, K, planes, out_bf16, what="", factor=1.0):
    err = np.abs(got - ref)
    bound = factor * sum_bound(K, planes) * mag
    if out_bf16:
        bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
    bad = err > bound
    assert not bad.any(), "%s: %d of %d outside, worst %g of the bound" % (
        what, bad.sum(), bad.size, (err[bad] / bound[bad]).max())


def packed(q, s, z, taps=False):
    return dfl.PackedW4(to_dev(q), to_dev(s), None if z is None else to_dev(z), taps=taps)


def check(orc, seed, tokens, N, K, group, zeros=False, f32_scale=False, dt="bf16", out="bf16", rows=None):
    need_cuda()
    rng = np.random.default_rng(seed)
    q, s, z = weights(rng, N, K, group, zeros, f32_scale)
    x = activations(rng, (tokens, K), dt)
    w = packed(q, s, z)
    odt = torch.bfloat16 if out == "bf16" else torch.float32
    y = dfl.linear_w4(to_dev(x), w, out_dtype=odt)
    torch.cuda.synchronize()
    assert y.dtype == odt and y.shape == (tokens, N)
    sel = np.arange(N) if rows is None else np.asarray(rows)
    ref, mag = orc.linear_w4(x, q[sel], s[sel], None if z is None else z[sel])
    assert_within(f64(y)[:, sel], ref, mag, K, 3 if dt == "f32" else 1, out == "bf16", "linear")
    assert dfl.device_errors() == 0


@pytest.mark.parametrize("tokens", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 64, 65, 100, 127, 129, 256, 257])
def test_token_counts(orc, tokens):
    check(orc, tokens, tokens, 160, 256, 64, out="f32")


@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (1, 64, 64), (31, 96, 32), (33, 160, 32),
                                       (45, 128, 128), (17, 1088, 64), (300, 416, 32), (64, 384, 192),
                                       (129, 1024, 1024), (1000, 64, 32), (4999, 128, 64)])
@pytest.mark.parametrize("zeros,f32_scale", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_shapes_and_formats(orc, N, K, group, zeros, f32_scale, dt):
    for tokens in (1, 5, 12, 24, 70):
        check(orc, N + K + tokens, tokens, N, K, group, zeros, f32_scale, dt, "f32")
    check(orc, N + K, 3, N, K, group, zeros, f32_scale, dt, "bf16")


@pytest.mark.parametrize("tokens,N,K,group,dt", [(1, 5120, 5120, 128, "bf16"), (8, 10240, 5120, 128, "bf16"),
                                                 (64, 2048, 5120, 64, "bf16"), (256, 1024, 5120, 128, "bf16"),
                                                 (8, 600, 20480, 128, "bf16"), (40, 600, 20480, 128, "bf16"),
                                                 (6, 200, 49152, 128, "bf16"), (9, 300, 20480, 32, "f32"),
                                                 (30, 70, 17408, 64, "f32")])
def test_large(orc, tokens, N, K, group, dt):
    check(orc, 3, tokens, N, K, group, True, False, dt, "f32",
          rows=np.unique(np.concatenate([[0, 1, N // 2, N - 1], np.arange(0, N, max(1, N // 24))])))


def test_head_of_a_block(orc):
    """The vocabulary head for a block of 8: rows at either end and in between."""
    check(orc, 4, 8, 151936, 5120, 128, rows=[0, 31, 32, 63, 75967, 75968, 151000, 151935])


def test_offsets_past_32_bits(orc):
    """Codes of more than 2^31 bytes, and outputs of more than 2^31 elements."""
    need_cuda()
    N, K, group = 300000, 16384, 128
    gen = torch.Generator(device="cuda")
    gen.manual_seed(21)
    q = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    s = (torch.rand((N, K // group), device="cuda", generator=gen) * 0.01).bfloat16()
    w = dfl.PackedW4(q, s)
    rows = np.array([0, 131071, 262144, 262145, N - 33, N - 1])
    qh, sh = to_host(q[rows]), to_host(s[rows])
    del q, s
    rng = np.random.default_rng(22)
    x = activations(rng, (20, K), "bf16")
    ref, mag = orc.linear_w4(x, qh, sh)
    for tokens in (3, 20):
        y = dfl.linear_w4(to_dev(x[:tokens]), w, out_dtype=torch.float32)
        assert_within(f64(y[:, rows.tolist()]), ref[:tokens], mag[:tokens], K, 1, False, "packed")
    del w, y
    tokens, N, K = 2 ** 18, 8300, 32
    q, s, _ = weights(rng, N, K, 32)
    x = torch.randn((tokens, K), device="cuda", generator=gen).bfloat16()
    y = dfl.linear_w4(x, packed(q, s, None))
    at = [0, 2 ** 17, tokens - 2, tokens - 1]
    ref, mag = orc.linear_w4(to_host(x[at]), q, s)
    assert_within(f64(y[at]), ref, mag, K, 1, True, "output")
    assert dfl.device_errors() == 0


def test_exact_small_integers(orc):
    """Integer activations and power-of-two scales: every sum is exact, so every bit is."""
    need_cuda()
    rng = np.random.default_rng(9)
    N, K = 96, 320
    q, _, z = weights(rng, N, K, 32, True)
    s = synth.to_bf16_bits((2.0 ** rng.integers(-3, 4, (N, K // 32))).astype(np.float32))
    for tokens in (1, 8, 20, 150):
        x = synth.to_bf16_bits(rng.integers(-4, 5, (tokens, K)).astype(np.float32))
        y = dfl.linear_w4(to_dev(x), packed(q, s, z), out_dtype=torch.float32)
        np.testing.assert_array_equal(f64(y), orc.linear_w4(x, q, s, z)[0])


def test_fp32_activations_keep_24_bits(orc):
    """x = 1 + 2^-23 and codes that cancel all but the last bit."""
    need_cuda()
    K = 64
    q = np.full((32, K // 2), 0x79, np.uint8)        # codes 9 (even k), 7 (odd k): +1, -1
    s = np.ones((32, 1), np.float32)
    x = np.ones((2, K), np.float32)
    x[0, 0] = 1 + 2.0 ** -23
    y = dfl.linear_w4(to_dev(x), packed(q, s, None))
    np.testing.assert_array_equal(to_host(y)[0], np.full(32, 2.0 ** -23, np.float32))
    np.testing.assert_array_equal(to_host(y)[1], np.zeros(32, np.float32))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("offset,extra", [(0, 8), (0, 3), (1, 0), (5, 11)])
def test_strided_and_unaligned_rows(orc, dt, offset, extra):
    """A column slice of a wider tensor: rows that start anywhere."""
    need_cuda()
    rng = np.random.default_rng(11)
    N, K = 70, 192
    q, s, z = weights(rng, N, K, 64, True)
    for tokens in (1, 6, 40, 140):
        wide = activations(rng, (tokens, K + offset + extra), dt)
        x = wide[:, offset:offset + K]
        w = packed(q, s, z)
        y = dfl.linear_w4(to_dev(wide)[:, offset:offset + K], w, out_dtype=torch.float32)
        same = dfl.linear_w4(to_dev(x), w, out_dtype=torch.float32)
        ref, mag = orc.linear_w4(x, q, s, z)
        assert_within(f64(y), ref, mag, K, 3 if dt == "f32" else 1, False, "strided")
        np.testing.assert_array_equal(to_host(y), to_host(same))


def test_leading_shapes_out_and_nothing_else_written(orc):
    need_cuda()
    rng = np.random.default_rng(12)
    N, K = 50, 64
    q, s, _ = weights(rng, N, K, 64)
    w = packed(q, s, None)
    x = activations(rng, (2, 3, K), "bf16")
    ref, mag = orc.linear_w4(x.reshape(6, K), q, s)
    guard = torch.full((6 * N + 64,), -7.0, dtype=torch.bfloat16, device="cuda")
    out = guard[32:32 + 6 * N].view(2, 3, N)
    y = dfl.linear_w4(to_dev(x), w, out=out)
    assert y is out
    assert_within(f64(y).reshape(6, N), ref, mag, K, 1, True, "lead")
    assert bool((guard[:32] == -7).all()) and bool((guard[32 + 6 * N:] == -7).all())
    assert dfl.linear_w4(torch.empty((0, K), dtype=torch.bfloat16, device="cuda"), w).shape == (0, N)
    t = to_dev(x).transpose(0, 1)                       # rows that no 2-D view covers
    np.testing.assert_array_equal(to_host(dfl.linear_w4(t, w)), to_host(y).transpose(1, 0, 2))


def test_one_bad_token_leaves_the_others(orc):
    """NaN and infinity in one token's activations reach that token's outputs only."""
    need_cuda()
    rng = np.random.default_rng(13)
    N, K = 64, 128
    q, s, z = weights(rng, N, K, 32, True)
    w = packed(q, s, z)
    for tokens in (5, 20, 70, 130):
        x = to_dev(activations(rng, (tokens, K), "bf16"))
        good = dfl.linear_w4(x, w)
        x[3, 5] = float("nan")
        x[4, 7] = float("inf")
        bad = dfl.linear_w4(x, w)
        keep = [t for t in range(tokens) if t not in (3, 4)]
        np.testing.assert_array_equal(to_host(good[keep]), to_host(bad[keep]))
        assert bool(torch.isnan(bad[3]).all()) and not bool(torch.isfinite(bad[4]).any())


CONV = [(1, 1, 64, 32), (3, 5, 64, 64), (2, 7, 192, 64), (5, 3, 320, 32), (1, 40, 128, 128), (40, 8, 128, 32),
        (3, 200, 64, 64), (300, 1, 64, 32)]


@pytest.mark.parametrize("B,T,H,group", CONV)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("zeros,f32_scale", [(False, False), (True, False), (True, True)])
def test_conv(orc, B, T, H, group, dt, zeros, f32_scale):
    need_cuda()
    rng = np.random.default_rng(B * 100 + T * 10 + H)
    q, s, z = weights(rng, 2 * H, H, group, zeros, f32_scale)
    x, xp = activations(rng, (B, T, H), dt), activations(rng, (B, H), dt)
    out = dfl.dynconv2(to_dev(x), to_dev(xp), packed(q, s, z, taps=True))
    ref, mag = orc.dynconv2_w4(x, xp, q, s, z)
    # two more fp32 fmas, each half a step of the running magnitude
    assert_within(f64(out), ref, mag, H, 3 if dt == "f32" else 1, dt == "bf16", "conv", factor=1.0 + 2 / 34)
    assert dfl.device_errors() == 0


@pytest.mark.parametrize("name,B", [("b1", 1), ("b8", 8), ("b32", 32)])
def test_conv_workloads(orc, name, B):
    """The decode workloads' conv (H = 5,120, blocks of 8); the oracle takes 32 channels."""
    need_cuda()
    rng = np.random.default_rng(B)
    H, T = 5120, 8
    q, s, z = weights(rng, 2 * H, H, 128, True)
    x, xp = activations(rng, (B, T, H), "bf16"), activations(rng, (B, H), "bf16")
    out = f64(dfl.dynconv2(to_dev(x), to_dev(xp), packed(q, s, z, taps=True)))
    ch = np.unique(np.concatenate([np.arange(0, H, 317), [15, 16, H - 1]]))
    rows = np.concatenate([ch, H + ch])
    y, mag = orc.linear_w4(x.reshape(B * T, H), q[rows], s[rows], z[rows])
    cur = bf16_to_f64(x)
    prev = np.concatenate([bf16_to_f64(xp)[:, None], cur[:, :-1]], 1)[..., ch].reshape(B * T, -1)
    cur = cur[..., ch].reshape(B * T, -1)
    n = len(ch)
    ref = cur + y[:, :n] * cur + y[:, n:] * prev
    m = np.abs(cur) + mag[:, :n] * np.abs(cur) + mag[:, n:] * np.abs(prev)
    assert_within(out.reshape(B * T, H)[:, ch], ref, m, H, 1, True, name, factor=1.0 + 2 / 34)


def test_zero_point_out_of_range_is_flagged(orc):
    need_cuda()
    dfl.device_errors(clear=True)
    rng = np.random.default_rng(14)
    q, s, z = weights(rng, 64, 64, 32, True)
    z[5, 1] = 77
    w = packed(q, s, z)
    torch.cuda.synchronize()
    assert dfl.device_errors() & 32
    x = activations(rng, (4, 64), "bf16")
    z[5, 1] = 15                                        # counts as 15
    ref, mag = orc.linear_w4(x, q, s, z)
    assert_within(f64(dfl.linear_w4(to_dev(x), w)), ref, mag, 64, 1, True, "clamped")
    assert dfl.device_errors() == 0


def test_binding_refusals():
    need_cuda()
    rng = np.random.default_rng(15)
    q, s, z = (to_dev(a) for a in weights(rng, 128, 64, 32, True))
    w, taps = dfl.PackedW4(q, s, z), dfl.PackedW4(q, s, z, taps=True)
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: dfl.linear_w4(x, taps), lambda: dfl.linear_w4(x[:, :32], w),
                lambda: dfl.linear_w4(x.cpu(), w), lambda: dfl.linear_w4(x, w, out=torch.empty_like(x)),
                lambda: dfl.linear_w4(x, w, out=torch.empty((128, 4), device="cuda").T),
                lambda: dfl.dynconv2(x.view(2, 2, 64), x[:2], w),
                lambda: dfl.dynconv2(x.view(2, 2, 64), x[:2].float(), taps),
                lambda: dfl.dynconv2(x.view(2, 2, 64), x, taps),
                lambda: dfl.PackedW4(q, s[:64], z), lambda: dfl.PackedW4(q, s, z[:, :1]),
                lambda: dfl.PackedW4(q, s[:, :0])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: dfl.PackedW4(q.int(), s), lambda: dfl.PackedW4(q, s.half()),
                lambda: dfl.PackedW4(q, s, z.int()), lambda: dfl.linear_w4(x.half(), w),
                lambda: dfl.linear_w4(x, w, out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(dfl.DFlash2Error):
        dfl.PackedW4(q, s[:, :1].expand(128, 4).contiguous())     # groups of 16


def test_streams_graphs_and_calls_at_once(orc):
    """Two streams at once on the same weights, and a captured call replayed on new
    inputs while eager calls run: no state is shared between calls."""
    need_cuda()
    rng = np.random.default_rng(16)
    N, K = 600, 1024
    q, s, z = weights(rng, N, K, 128, True)
    w = packed(q, s, z)
    for tokens in (3, 100):
        xs = [to_dev(activations(rng, (tokens, K), "bf16")) for _ in range(4)]
        want = [dfl.linear_w4(x, w) for x in xs]
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        got = [None] * 4
        for i, x in enumerate(xs):
            with torch.cuda.stream((s1, s2)[i & 1]):
                for _ in range(5):
                    got[i] = dfl.linear_w4(x, w)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        static = xs[0].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = dfl.linear_w4(static, w)
        for x, b in zip(xs, want):
            static.copy_(x)
            g.replay()
            eager = dfl.linear_w4(xs[1], w)
            torch.cuda.synchronize()
            assert torch.equal(y, b) and torch.equal(eager, want[1])


def test_a_pass_of_head_and_step(orc):
    """The run these belong to: conv on 4-bit taps -> 4-bit head -> top-16 -> greedy
    verify, against the oracle's chain on the same inputs (tokens compared where the
    oracle's margin between its two best logits exceeds the logits' error)."""
    need_cuda()
    rng = np.random.default_rng(17)
    B, T, H, V = 2, 8, 128, 997
    q, s, z = weights(rng, 2 * H, H, 64, True)
    hq, hs, _ = weights(rng, V, H, 64)
    x, xp = activations(rng, (B, T, H), "bf16"), activations(rng, (B, H), "bf16")
    h = dfl.dynconv2(to_dev(x), to_dev(xp), packed(q, s, z, taps=True))
    logits = dfl.linear_w4(h, packed(hq, hs, None), out_dtype=torch.float32)
    idx, prob, logp, logz = dfl.topk_softmax(logits)
    oi, *_ = orc.topk_softmax(to_host(logits).reshape(-1, V))
    np.testing.assert_array_equal(to_host(idx).reshape(-1, 16), oi)
    ref, mag = orc.linear_w4(to_host(h).reshape(-1, H), hq, hs)
    assert_within(f64(logits).reshape(-1, V), ref, mag, H, 1, False, "head")
    n, tok = dfl.verify_greedy(logits, idx[:, :-1, 0].contiguous())
    assert to_host(n).tolist() == [T - 1] * B           # drafted from the same rows: all accepted
    top = np.sort(ref, 1)[:, -2:]
    clear = (top[:, 1] - top[:, 0]) > 2 * sum_bound(H, 1) * mag.max(1)
    np.testing.assert_array_equal(to_host(tok).reshape(-1)[clear], ref.argmax(1)[clear])


def silence(q, z, group, ks):
    """Sets every row's code at the columns ks to its zero point: their products are zero."""
    q = q.copy()
    for k in ks:
        c = np.full(len(q), 8, np.uint8) if z is None else z[:, k // group]
        q[:, k // 2] = (q[:, k // 2] & 0x0F) | (c << 4) if k & 1 else (q[:, k // 2] & 0xF0) | c
    return q


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros,f32_scale", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("large", [1e3, 1e6, 1e9])
def test_large_activations_on_zero_points_leave_no_trace(orc, group, zeros, f32_scale, large):
    """Channels far above the rest whose codes are the zero point: their products are exactly
    zero, so the others keep the bound of a sum without them, whatever the output's type."""
    need_cuda()
    rng = np.random.default_rng(group + int(np.log10(large)))
    N, K = 70, 1024
    q, s, z = weights(rng, N, K, group, zeros, f32_scale)
    ks = [0, 5, 130, 131, 600, 1023]
    q = silence(q, z, group, ks)
    w = packed(q, s, z)
    for tokens in (1, 3, 8, 11, 16, 20, 70):
        x = activations(rng, (tokens, K), "f32") + np.float32(0.5)
        x[:, ks] *= np.float32(large)
        x = synth.to_bf16_bits(x)
        ref, mag = orc.linear_w4(x, q, s, z)
        for out in (torch.bfloat16, torch.float32):
            y = dfl.linear_w4(to_dev(x), w, out_dtype=out)
            assert_within(f64(y), ref, mag, K, 1, out == torch.bfloat16, "%d tokens" % tokens)
    B, T = 2, 4
    q, s, z = weights(rng, 2 * K, K, group, zeros, f32_scale)
    q = silence(q, z, group, ks)
    x, xp = activations(rng, (B, T, K), "f32"), activations(rng, (B, K), "f32")
    x[:, :, ks] *= np.float32(large)
    x, xp = synth.to_bf16_bits(x), synth.to_bf16_bits(xp)
    out = dfl.dynconv2(to_dev(x), to_dev(xp), packed(q, s, z, taps=True))
    ref, mag = orc.dynconv2_w4(x, xp, q, s, z)
    assert_within(f64(out), ref, mag, K, 1, True, "conv", factor=1.0 + 2 / 34)
    assert dfl.device_errors() == 0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_dense_rows_off_16_bytes(orc, dt):
    """A dense x whose storage starts anywhere goes the way of an aligned copy, strided or not."""
    need_cuda()
    rng = np.random.default_rng(23)
    N, K = 200, 1024
    q, s, z = weights(rng, N, K, 64, True)
    w = packed(q, s, z)
    for tokens in (3, 16, 17, 20, 140):
        x = activations(rng, (tokens, K), dt)
        flat = torch.zeros(tokens * K + 9, dtype=torch.bfloat16 if dt == "bf16" else torch.float32, device="cuda")
        for off in (0, 1, 3, 8):
            v = flat[off:off + tokens * K].view(tokens, K)
            v.copy_(to_dev(x))
            assert v.is_contiguous()
            y = dfl.linear_w4(v, w, out_dtype=torch.float32)
            assert torch.equal(y, dfl.linear_w4(to_dev(x), w, out_dtype=torch.float32)), (tokens, off)
        ref, mag = orc.linear_w4(x, q, s, z)
        assert_within(f64(y), ref, mag, K, 3 if dt == "f32" else 1, False, "dense")
