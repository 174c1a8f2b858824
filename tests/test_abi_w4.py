"""Refusals of the 4-bit-weight entry points: bad arguments come back as the
documented status before any CUDA call (no device needed)."""
import ctypes as C

import pytest
import torch

OK, EINVAL, EDTYPE, ESHAPE, EWORKSPACE, ECUDA, EALIGN = range(7)
P, P2, ODD = C.c_void_p(0x10000), C.c_void_p(0x20000), C.c_void_p(0x10001)
S0 = C.c_void_p(0)


@pytest.fixture(scope="module")
def L():
    from block_draft_verification_b200 import build
    build.build()
    import block_draft_verification_b200 as d
    return d.lib()


def test_packed_bytes(L):
    f = L.dflash2_w4_packed_bytes
    n = f(5120, 5120, 128, 0)
    assert n == 5120 * 5120 // 2 + 5120 * 40 * 2
    assert f(5120, 5120, 128, 1) == 5120 * 5120 // 2 + 5120 * 40 * 4      # zero points beside the scales
    assert f(5120, 5120, 128, 2) == 5120 * 5120 // 2 + 5120 * 40 * 8      # float scales
    assert f(5119, 5120, 128, 0) == n                                      # rows in tiles of 128
    assert f(1, 32, 32, 0) == 4 * (1024 + 2 * 64)                          # K in chunks of 64
    assert f(2 ** 31 - 1, 2 ** 20, 128, 0) > 2 ** 50                       # 64-bit sizes
    for bad in [(0, 64, 32, 0), (8, 0, 32, 0), (8, 100, 32, 0), (8, 64, 48, 0), (8, 96, 64, 0),
                (8, 64, 0, 0), (8, 64, -32, 0), (2 ** 31, 64, 32, 0), (8, 2 ** 20 + 64, 64, 0),
                (8, 64, 32, 8), (8, 64, 32, -1)]:
        assert f(*bad) == 0, bad


def test_pack_validation(L):
    def pack(q=P, s=P, z=None, N=128, K=64, g=32, fmt=0, out=P2):
        return L.dflash2_w4_pack(q, s, z, N, K, g, fmt, out, S0)
    assert pack(fmt=8) == EINVAL
    assert pack(fmt=-1) == EINVAL
    assert pack(K=100) == ESHAPE
    assert pack(g=48) == ESHAPE
    assert pack(N=0) == ESHAPE
    assert pack(fmt=4, N=130) == ESHAPE          # taps: N = 2 K
    assert pack(fmt=4, N=64, K=32) == ESHAPE     # taps: K a multiple of 64
    assert pack(q=None) == EINVAL
    assert pack(s=None) == EINVAL
    assert pack(out=None) == EINVAL
    assert pack(fmt=1) == EINVAL                 # zero points announced, not given
    assert pack(z=P) == EINVAL                   # given, not announced
    assert pack(q=C.c_void_p(0x10004)) == EALIGN
    assert pack(s=ODD) == EALIGN
    assert pack(fmt=2, s=C.c_void_p(0x10002)) == EALIGN
    assert pack(out=C.c_void_p(0x20010)) == EALIGN


def test_linear_validation(L):
    def lin(x=P, dt=1, xs=64, tok=3, w=P2, N=128, K=64, g=32, fmt=0, y=P, odt=1):
        return L.dflash2_linear_w4(x, dt, xs, tok, w, N, K, g, fmt, y, odt, S0)
    assert lin(dt=2) == EDTYPE
    assert lin(odt=-1) == EDTYPE
    assert lin(fmt=4) == EINVAL                  # taps are for the conv
    assert lin(fmt=16) == EINVAL
    assert lin(K=80) == ESHAPE
    assert lin(g=96) == ESHAPE
    assert lin(xs=63) == ESHAPE
    assert lin(tok=-1) == ESHAPE
    assert lin(tok=2 ** 18 + 1) == ESHAPE
    assert lin(tok=0, x=None) == OK              # nothing to do, nothing launched
    assert lin(x=None) == EINVAL
    assert lin(w=None) == EINVAL
    assert lin(y=None) == EINVAL
    assert lin(x=ODD) == EALIGN
    assert lin(dt=0, x=C.c_void_p(0x10002)) == EALIGN
    assert lin(w=C.c_void_p(0x20080)) == EALIGN
    assert lin(y=ODD) == EALIGN
    assert lin(odt=0, y=C.c_void_p(0x10002)) == EALIGN


def test_conv_validation(L):
    def conv(x=P, xp=P, w=P2, g=32, fmt=4, dt=1, B=2, T=8, H=128, out=P):
        return L.dflash2_dynconv2_w4(x, xp, w, g, fmt, dt, B, T, H, out, S0)
    assert conv(dt=3) == EDTYPE
    assert conv(fmt=0) == EINVAL                 # weights not packed as taps
    assert conv(fmt=12) == EINVAL
    assert conv(H=100) == ESHAPE
    assert conv(H=0) == ESHAPE
    assert conv(B=-1) == ESHAPE
    assert conv(T=-1) == ESHAPE
    assert conv(g=256) == ESHAPE
    assert conv(B=2 ** 10, T=2 ** 9) == ESHAPE
    assert conv(T=0) == OK
    assert conv(B=0, x=None) == OK
    assert conv(x=None) == EINVAL
    assert conv(xp=None) == EINVAL
    assert conv(out=None) == EINVAL
    assert conv(x=C.c_void_p(0x10008)) == EALIGN
    assert conv(w=C.c_void_p(0x20010)) == EALIGN


def test_binding_refuses_host_tensors(L):
    import block_draft_verification_b200 as d
    with pytest.raises(ValueError):
        d.PackedW4(torch.zeros((32, 32), dtype=torch.uint8), torch.ones((32, 2)))


def test_plan_validation(L):
    t, c = C.c_int(), C.c_int()
    def plan(tok=8, N=128, K=128, g=128, fmt=0, dt=1, tile=C.byref(t), cl=C.byref(c)):
        return L.dflash2_linear_w4_plan(tok, N, K, g, fmt, dt, tile, cl)
    assert plan(tok=0) == ESHAPE
    assert plan(tok=2 ** 18 + 1) == ESHAPE
    assert plan(K=100) == ESHAPE
    assert plan(g=48) == ESHAPE
    assert plan(fmt=8) == EINVAL
    assert plan(dt=7) == EDTYPE
    assert plan(tile=None) == EINVAL
    assert plan(cl=None) == EINVAL
