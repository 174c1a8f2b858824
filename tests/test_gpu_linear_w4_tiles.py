"""Every tile width, cluster size, group kind and format of the tensor-core products
with 4-bit weights, with one tile a cluster and with several, against the formula in
fp64 over the whole output; and the few-token kernel where it is given more tokens.

Shapes are searched for at run time, smallest first, by what dflash2_linear_w4_plan
says of them: a change of the plan's costs moves the shapes, not what is covered.
Error bound: w4_inputs.sum_bound, and half a step of a bf16 output."""
import ctypes as C
import functools
import itertools

import pytest
import torch

import block_draft_verification_b200 as dfl
from parity import gpu, need_cuda
from w4_inputs import sum_bound

pytestmark = gpu

CLUSTERS = {1: 148, 2: 74, 4: 33, 8: 15}     # of a B200: only to tell one tile a cluster from several


@functools.lru_cache(maxsize=None)
def plan(tokens, N, K, group, fmt, dtype=dfl.BF16):
    tile, cluster = C.c_int(-1), C.c_int(-1)
    assert dfl.lib().dflash2_linear_w4_plan(tokens, N, K, group, fmt, dtype, C.byref(tile), C.byref(cluster)) == 0
    return tile.value, cluster.value


def turns(tokens, N, tile, S):
    return -(-(-(-N // 128) * -(-tokens // tile)) // CLUSTERS[S])


@functools.lru_cache(maxsize=None)
def shapes(taps):
    """(tokens, N, K), smallest first."""
    if taps:
        s = [(t, 2 * h, h) for t in (33, 64, 65, 100, 128, 200, 225, 256, 300, 512)
             for h in (64, 128, 256, 512, 1024, 1536, 2048, 2560, 3584, 4096, 5120)]
    else:
        s = list(itertools.product((33, 64, 65, 100, 128, 200, 225, 300),
                                   (125, 637, 1000, 2557, 5000, 10237, 20480, 40000),
                                   (128, 256, 512, 1024, 2048, 5120, 8192, 20480)))
    return sorted(s, key=lambda v: v[0] * (v[1] + v[2]) + v[1] * v[2])


def find(group, fmt, tile, S, several, taps=False):
    for t, n, k in shapes(taps):
        if k % group == 0 and plan(t, n, k, group, fmt) == (tile, S) and (turns(t, n, tile, S) > 2) == several:
            return t, n, k
    return None


def inputs(seed, N, K, group, fmt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    s = (torch.rand((N, K // group), device="cuda", generator=g) + 0.5) * (0.4 / K ** 0.5)
    z = torch.randint(0, 16, (N, K // group), dtype=torch.uint8, device="cuda", generator=g) if fmt & 1 else None
    return q, s if fmt & 2 else s.bfloat16(), z, g


def product(x, q, s, z):
    """x W^T and |x| |W|^T in fp64."""
    y, mag = (torch.empty((x.shape[0], len(q)), dtype=torch.float64, device="cuda") for _ in range(2))
    step = max(1, (1 << 27) // x.shape[1])
    for i in range(0, len(q), step):
        c = torch.stack((q[i:i + step] & 15, q[i:i + step] >> 4), -1).double().reshape(*s[i:i + step].shape, -1)
        w = (c - (8.0 if z is None else z[i:i + step, :, None].double())) * s[i:i + step, :, None].double()
        w = w.reshape(len(w), -1)
        y[:, i:i + step], mag[:, i:i + step] = x.double() @ w.T, x.double().abs() @ w.abs().T
    return y, mag


def assert_within(got, ref, mag, K, what, planes=1):
    bound = sum_bound(K, planes) * mag
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (ref.abs() + bound)
    err = (got.double() - ref).abs()
    assert bool((err <= bound).all()), (what, float((err / bound).max()))


KINDS = [(g, f) for g in (32, 64, 128) for f in (0, 1, 2, 3)]


@pytest.mark.parametrize("S", [1, 2, 4, 8])
@pytest.mark.parametrize("tile,several", [(32, False), (64, False), (64, True), (128, False), (128, True)])
def test_tiles(tile, several, S):
    need_cuda()
    dfl.device_errors(clear=True)
    reached = set()
    for i, (group, fmt) in enumerate(KINDS):
        at = find(group, fmt, tile, S, several)
        if at is None:
            continue
        reached.add((group, fmt))
        tokens, N, K = at
        q, s, z, gen = inputs(i, N, K, group, fmt)
        w = dfl.PackedW4(q, s, z)
        assert w.format == fmt
        # this many tokens, and others of the same tiles that end elsewhere in the last one
        more = [t for t in (33, 47, 64, 65, 97, 128, 129, 193, 256, 257) if t != tokens and
                plan(t, N, K, group, fmt) == (tile, S)]
        for t in [tokens] + more[i % 3::3][:2]:
            x = torch.randn((t, K), device="cuda", generator=gen).bfloat16()
            ref, mag = product(x, q, s, z)
            for out in (torch.float32, torch.bfloat16):
                assert_within(dfl.linear_w4(x, w, out_dtype=out), ref, mag, K, (group, fmt, t, N, K))
            del ref, mag
        assert dfl.device_errors() == 0, (group, fmt, at)
    # every combination is to be had but these (32-token tiles are for few tiles: one a cluster)
    none = {(tile, several, S, *k) for k in KINDS} - {(tile, several, S, *k) for k in reached}
    assert none <= {(128, True, 8, 128, 2), (128, True, 8, 128, 3), (32, False, 2, 128, 0), (32, False, 2, 128, 1),
                    (32, False, 4, 128, 0), (32, False, 4, 128, 1)}


@pytest.mark.parametrize("S", [1, 2, 4])
@pytest.mark.parametrize("tile", [32, 64, 128])
def test_conv_tiles(tile, S):
    need_cuda()
    dfl.device_errors(clear=True)
    reached = set()
    for i, ((group, fmt), several) in enumerate(itertools.product(KINDS, (False, True))):
        at = find(group, fmt | 4, tile, S, several, taps=True)
        if at is None:
            continue
        reached.add(group)
        tokens, _, H = at
        T = next(t for t in (8, 13, 11, 5, 15, 1) if tokens % t == 0)
        q, s, z, gen = inputs(50 + i, 2 * H, H, group, fmt)
        x = torch.randn((tokens // T, T, H), device="cuda", generator=gen).bfloat16()
        xp = torch.randn((tokens // T, H), device="cuda", generator=gen).bfloat16()
        out = dfl.dynconv2(x, xp, dfl.PackedW4(q, s, z, taps=True))
        y, mag = (v.view(tokens // T, T, 2, H) for v in product(x.view(-1, H), q, s, z))
        cur = x.double()
        prev = torch.cat((xp.double()[:, None], cur[:, :-1]), 1)
        ref = cur + y[:, :, 0] * cur + y[:, :, 1] * prev
        m = cur.abs() + mag[:, :, 0] * cur.abs() + mag[:, :, 1] * prev.abs()
        # two more fp32 fmas, each half a step of the running magnitude
        assert_within(out, ref, m * (1 + 2 / 34), H, (group, fmt, tokens, H))
        assert dfl.device_errors() == 0, (group, fmt, at)
    assert reached == ({32, 128} if (tile, S) == (128, 4) else {32, 64, 128})


@pytest.mark.parametrize("group,fmt", KINDS)
def test_rows_off_16_bytes_through_the_library(group, fmt):
    """Rows that start off 16 bytes, more of them than a few: the library's call takes them
    element by element (the binding copies them first)."""
    need_cuda()
    N, K = 133, 768
    q, s, z, gen = inputs(7, N, K, group, fmt)
    w = dfl.PackedW4(q, s, z)
    for tokens, stride, off in ((20, K + 1, 0), (33, K, 1), (140, K + 4, 3)):
        for dt, planes in ((torch.bfloat16, 1), (torch.float32, 3)):
            flat = torch.randn(tokens * stride + 8, device="cuda", generator=gen).to(dt)
            x = flat[off:].as_strided((tokens, K), (stride, 1))
            for out in (torch.float32, torch.bfloat16):
                y = torch.empty((tokens, N), dtype=out, device="cuda")
                dfl._call("dflash2_linear_w4", w.index, x.data_ptr(), dfl._dtype(x), stride, tokens, w.ptr, N, K,
                          group, w.format, y.data_ptr(), dfl._dtype(y))
                ref, mag = product(x, q, s, z)
                assert_within(y, ref, mag, K, (tokens, dt, out), planes)
    assert dfl.device_errors() == 0


def test_plan_of_known_shapes():
    need_cuda()
    assert plan(1, 5120, 5120, 128, 0)[0] == 0                  # a few tokens
    assert plan(64, 5120, 5120, 128, 0, dfl.F32)[0] == 0        # fp32 activations
    assert plan(64, 20480, 5120, 64, 1)[0] == 64
