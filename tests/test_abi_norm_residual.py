"""Refusals of the norms around a block: bad arguments come back as the
documented status before any CUDA call (no device needed)."""
import ctypes as C

import pytest
import torch

OK, EINVAL, EDTYPE, ESHAPE, EWORKSPACE, ECUDA, EALIGN = range(7)
P, P2, ODD = C.c_void_p(0x10000), C.c_void_p(0x20000), C.c_void_p(0x10001)


@pytest.fixture(scope="module")
def L():
    from block_draft_verification_b200 import build
    build.build()
    import block_draft_verification_b200 as d
    return d.lib()


def test_validation(L):
    def norm(res=P, rdt=1, rs=64, y=P, dt=1, ys=64, g=P, gs=64, rep=1, act=0, wo=P, wi=P, off=0.0, al=1.0,
             eps=1e-6, rows=3, H=64, ro=P2, h=P2):
        return L.dflash2_norm_residual(res, rdt, rs, y, dt, ys, g, gs, rep, act, wo, wi, off, al, eps, rows, H,
                                       ro, h, C.c_void_p(0))
    assert norm(dt=2) == EDTYPE
    assert norm(rdt=-1) == EDTYPE
    assert norm(dt=0, rdt=1) == EDTYPE           # a residual narrower than y
    assert norm(rows=-1) == ESHAPE
    assert norm(rows=2 ** 30 + 1) == ESHAPE
    assert norm(H=0) == ESHAPE
    assert norm(H=2 ** 24 + 1, rs=2 ** 25, ys=2 ** 25, gs=2 ** 25) == ESHAPE
    assert norm(rs=63) == ESHAPE
    assert norm(ys=63) == ESHAPE
    assert norm(gs=63) == ESHAPE
    assert norm(rep=0) == ESHAPE
    nan, inf = float("nan"), float("inf")
    for bad in (dict(al=nan), dict(al=inf), dict(off=nan), dict(eps=nan), dict(eps=-1e-6), dict(eps=inf),
                dict(act=2), dict(act=-1), dict(res=None), dict(y=None), dict(ro=None), dict(h=None),
                dict(wi=None)):
        assert norm(**bad) == EINVAL, bad
    assert norm(res=P, ro=P, rs=72) == EINVAL    # written over a strided residual
    assert norm(rows=0, res=None) == OK
    for k in ("res", "y", "g", "wo", "wi", "ro", "h"):
        assert norm(**{k: ODD}) == EALIGN, k
    assert norm(rdt=0, res=C.c_void_p(0x10002)) == EALIGN
    assert norm(rdt=0, ro=C.c_void_p(0x10002)) == EALIGN


def test_binding_refuses_host_tensors(L):
    import block_draft_verification_b200 as d
    with pytest.raises(ValueError):
        d.norm_residual(torch.zeros(2, 8), torch.zeros(2, 8))
