"""GPU parity of the norms around a block (norm_residual) against the fp64
oracle.

Error bound, in steps of fp32 (2^-24 relative, half a step per rounding): a sum
of H squares in fp32, added in runs of at most 32 per thread and then over a
tree, is off by at most (32 + 10 + 2) of them relative (the long rows' loop: H /
512 + 10 + 2), half of that in its root; the reciprocal root and the division
are within 2 more each, the products within 4, and the gate's sigmoid within 8
(expf's two steps, relative to a value below 1, and a division): at most
E = (H / 512 + 70) 2^-24 of alpha * act(g) * rms(y), plus 2^-24 of r'.  In h the
error of r' comes in again, relative to the row's largest terms.  Outputs of
bf16 add half a step, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import block_draft_verification_b200 as dfl
import synth
from parity import bf16_to_f64, gpu, need_cuda, to_dev, to_host

pytestmark = gpu


def f64(a):
    a = to_host(a) if isinstance(a, torch.Tensor) else a
    return bf16_to_f64(a) if a.dtype == np.uint16 else a.astype(np.float64)


def make(rng, shape, dt, std=1.0, mean=0.0):
    a = (rng.standard_normal(shape) * std + mean).astype(np.float32)
    return synth.to_bf16_bits(a) if dt == "bf16" else a


def inputs(rng, B, T, H, dt, rdt, gate, post, pre):
    gshape = {"none": None, "channel": (H,), "sequence": (B, H), "token": (B, T, H)}[gate]
    return dict(res=make(rng, (B, T, H), rdt, 2.0), y=make(rng, (B, T, H), dt, 0.7),
                gate=None if gshape is None else make(rng, gshape, dt, 0.5, 0.8),
                w_post=make(rng, (H,), dt, 0.1, 1.0) if post else None,
                w_pre=make(rng, (H,), dt, 0.1, 1.0) if pre else None)


def oracle(orc, d, B, T, H, **kw):
    rep = {None: 1, 1: B * T, 2: T, 3: 1}[None if d["gate"] is None else d["gate"].ndim]
    r, h = orc.norm_residual(d["res"].reshape(-1, H), d["y"].reshape(-1, H), d["w_post"], d["w_pre"],
                             None if d["gate"] is None else d["gate"].reshape(-1, H), rep, **kw)
    return r.reshape(B, T, H), None if h is None else h.reshape(B, T, H)


def compare(got, want, d, H, eps, w_offset=0.0):
    r, h = got if isinstance(got, tuple) else (got, None)
    rr, hh = want
    E = (H / 512 + 70) * 2.0 ** -24
    branch = np.abs(rr - f64(d["res"]))
    er = E * branch + 2.0 ** -24 * (np.abs(rr) + branch)
    tol = er + (2.0 ** -8 * (np.abs(rr) + er) if r.dtype == torch.bfloat16 else 0.0)
    err = np.abs(f64(r) - rr)
    assert (err <= tol).all(), ("r'", (err / np.maximum(tol, 1e-300)).max())
    if hh is None:
        assert h is None
        return
    scale = 1 / np.sqrt((rr ** 2).mean(-1, keepdims=True) + eps)
    w = np.abs(f64(d["w_pre"]) + w_offset)
    # rms error of r' moves the root: at most max |er| / rms; then E of the value itself
    eh = w * scale * er + np.abs(hh) * (E + (er * np.abs(rr)).mean(-1, keepdims=True) * scale ** 2)
    tol = eh + (2.0 ** -8 * (np.abs(hh) + eh) if h.dtype == torch.bfloat16 else 0.0)
    err = np.abs(f64(h) - hh)
    assert (err <= tol).all(), ("h", (err / np.maximum(tol, 1e-300)).max())


def dev(d):
    return {k: None if v is None else to_dev(v) for k, v in d.items()}


TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


@pytest.mark.parametrize("dt,rdt", TYPES)
@pytest.mark.parametrize("B,T,H", [(1, 1, 1), (1, 1, 8), (2, 3, 7), (1, 8, 64), (3, 5, 100), (2, 2, 264), (1, 3, 1023),
                                   (2, 4, 4096), (1, 8, 5120), (2, 3, 8200), (1, 2, 16384), (1, 2, 20000), (301, 2, 40)])
def test_shapes(orc, dt, rdt, B, T, H):
    need_cuda()
    for n, (gate, sig, post, pre) in enumerate([("none", False, True, True), ("channel", False, True, True),
                                                ("sequence", True, True, True), ("token", True, False, True),
                                                ("token", False, True, False), ("none", False, False, False)]):
        rng = np.random.default_rng(B * 10000 + H + n)
        d = inputs(rng, B, T, H, dt, rdt, gate, post, pre)
        got = dfl.norm_residual(**dev(d), gate_act=dfl.GATE_SIGMOID if sig else dfl.GATE_LINEAR, scale=0.7071, eps=1e-5)
        scale = float(np.float32(0.7071))
        compare(got, oracle(orc, d, B, T, H, sigmoid=sig, scale=scale, eps=float(np.float32(1e-5))), d, H, 1e-5)


def test_many_rows_of_a_prompt(orc):
    need_cuda()
    B, T, H = 2, 1500, 512
    rng = np.random.default_rng(5)
    d = inputs(rng, B, T, H, "bf16", "f32", "sequence", True, True)
    got = dfl.norm_residual(**dev(d), gate_act=dfl.GATE_SIGMOID)
    compare(got, oracle(orc, d, B, T, H, sigmoid=True, eps=float(np.float32(1e-6))), d, H, 1e-6)


@pytest.mark.parametrize("H", [256, 100, 17000])
def test_written_over_the_residual(orc, H):
    need_cuda()
    rng = np.random.default_rng(6)
    d = inputs(rng, 2, 9, H, "bf16", "f32", "channel", True, True)
    g = dev(d)
    apart = dfl.norm_residual(**g)
    h = torch.empty_like(g["y"])
    res = g["res"]
    r, h2 = dfl.norm_residual(**g, out=(res, h))
    assert r is res and h2 is h
    assert torch.equal(r, apart[0]) and torch.equal(h, apart[1])


@pytest.mark.parametrize("offset,extra", [(0, 8), (8, 0), (1, 0), (3, 2)])
@pytest.mark.parametrize("dt,rdt", TYPES)
def test_strided_rows(orc, dt, rdt, offset, extra):
    """Column slices of wider tensors: the same bits as dense copies within the formula's bound."""
    need_cuda()
    rng = np.random.default_rng(7)
    rows, H = 11, 192
    wy, wr = make(rng, (rows, H + offset + extra), dt), make(rng, (rows, H + offset + extra), rdt)
    wg = make(rng, (rows, H + offset + extra), dt, 0.5, 1.0)
    cut = slice(offset, offset + H)
    d = dict(res=wr[:, cut], y=wy[:, cut], gate=wg[:, cut], w_post=make(rng, (H,), dt), w_pre=make(rng, (H,), dt))
    got = dfl.norm_residual(to_dev(wr)[:, cut], to_dev(wy)[:, cut], to_dev(d["w_post"]), to_dev(d["w_pre"]),
                            gate=to_dev(wg)[:, cut])
    r, h = orc.norm_residual(d["res"], d["y"], d["w_post"], d["w_pre"], d["gate"], 1, eps=float(np.float32(1e-6)))
    compare(got, (r, h), d, H, 1e-6)


def test_offset_weights_zero_rows_and_large_values(orc):
    need_cuda()
    rng = np.random.default_rng(8)
    H = 128
    d = inputs(rng, 1, 6, H, "f32", "f32", "none", True, True)
    d["y"][0, 1] = 0                       # a block that gives nothing: eps alone under the root
    d["res"][0, 2] = 0
    d["y"][0, 2] = 0                       # and a residual of zeros: h = 0
    d["y"][0, 3] *= 1e15                   # squares near 1e30
    d["y"][0, 4] *= 1e-18
    got = dfl.norm_residual(**dev(d), w_offset=1.0, eps=1e-6)
    want = oracle(orc, d, 1, 6, H, w_offset=1.0, eps=float(np.float32(1e-6)))
    compare(got, want, d, H, 1e-6, w_offset=1.0)
    assert not bool(got[1][0, 2].any())


def test_a_bad_row_leaves_the_others():
    need_cuda()
    rng = np.random.default_rng(9)
    d = dev(inputs(rng, 1, 40, 320, "bf16", "bf16", "token", True, True))
    good = dfl.norm_residual(**d)
    d["y"][0, 7, 3] = float("nan")
    d["res"][0, 9, 5] = float("inf")
    bad = dfl.norm_residual(**d)
    keep = [t for t in range(40) if t not in (7, 9)]
    for a, b in zip(good, bad):
        assert torch.equal(a[:, keep], b[:, keep])
    assert bool(torch.isnan(bad[0][0, 7]).all())


def test_rows_do_not_depend_on_the_batch_and_nothing_else_is_written():
    need_cuda()
    rng = np.random.default_rng(10)
    for H in (640, 77):
        d = dev(inputs(rng, 1, 33, H, "bf16", "f32", "token", True, True))
        r, h = dfl.norm_residual(**d)
        one = {k: v[:, 5:6] if v is not None and v.dim() == 3 else v for k, v in d.items()}
        guard = torch.full((H + 32,), 7.0, device="cuda")
        ro = guard[16:16 + H].view(1, 1, H)
        r1, h1 = dfl.norm_residual(**one, out=(ro, torch.empty_like(one["y"])))
        assert torch.equal(r1, r[:, 5:6]) and torch.equal(h1, h[:, 5:6])
        assert bool((guard[:16] == 7).all()) and bool((guard[16 + H:] == 7).all())
    e = torch.empty((0, 64), device="cuda")
    assert dfl.norm_residual(e, e, w_pre=torch.ones(64, device="cuda"))[1].shape == (0, 64)


def test_offsets_past_32_bits(orc):
    """More than 2^31 elements, vectors and single elements."""
    need_cuda()
    for H in (4096, 4097):
        rows = 530000
        y = torch.empty((rows, H), dtype=torch.bfloat16, device="cuda").normal_()
        res = y.clone()
        w = torch.full((H,), 1.25, dtype=torch.bfloat16, device="cuda")
        r, h = dfl.norm_residual(res, y, w, w, out=(res, torch.empty_like(y)))
        at = [0, 524287, 524288, rows - 1]
        d = dict(res=to_host(y[at]), y=to_host(y[at]), gate=None, w_post=to_host(w), w_pre=to_host(w))
        want = orc.norm_residual(d["res"], d["y"], d["w_post"], d["w_pre"], eps=float(np.float32(1e-6)))
        compare((r[at], h[at]), want, d, H, 1e-6)
        del y, res, r, h


def test_binding_refusals():
    need_cuda()
    y = torch.zeros((2, 3, 16), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(16, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: dfl.norm_residual(y[:, :2], y), lambda: dfl.norm_residual(y, y, w[:8]),
                lambda: dfl.norm_residual(y, y, w_pre=w[:8]), lambda: dfl.norm_residual(y, y, gate=w[:8]),
                lambda: dfl.norm_residual(y, y, gate=y[:, 0, :8]), lambda: dfl.norm_residual(y.cpu(), y),
                lambda: dfl.norm_residual(y, y, out=y.float()), lambda: dfl.norm_residual(y, y, w_pre=w, out=(y, y.transpose(0, 1)))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: dfl.norm_residual(y, y, w.float()), lambda: dfl.norm_residual(y.half(), y),
                lambda: dfl.norm_residual(y.half(), y.half())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(dfl.DFlash2Error):
        dfl.norm_residual(y, y.float())             # a bf16 residual beside float
    with pytest.raises(dfl.DFlash2Error):
        dfl.norm_residual(y, y, eps=-1.0)


def test_capture_and_streams():
    need_cuda()
    rng = np.random.default_rng(11)
    d = dev(inputs(rng, 4, 8, 5120, "bf16", "bf16", "sequence", True, True))
    want = dfl.norm_residual(**d)
    other = dev(inputs(rng, 4, 8, 5120, "bf16", "bf16", "sequence", True, True))
    want2 = dfl.norm_residual(**other)
    static = {k: v.clone() for k, v in d.items()}
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = dfl.norm_residual(**static)
    s = torch.cuda.Stream()
    for src, ref in ((d, want), (other, want2), (d, want)):
        for k in src:
            static[k].copy_(src[k])
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(s):
            eager = dfl.norm_residual(**other)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
        assert all(torch.equal(a, b) for a, b in zip(eager, want2))


def compare_denormal(got, want, d, H, eps):
    """compare()'s bound where values below 2^-126 are steps of 2^-149 (bf16: 2^-133): an
    fp32 result that small is off by at most 2^-150 (r' by one such rounding, h by that of
    v / rms, times w, and of the product), an output of bf16 by 2^-134 more.  A row's
    reciprocal below 2^-126 (rms above 2^126) is off by 2^-150 of at least 2^-128.2, so 2.3
    steps of 2^-24; it and its products with w and the gate, 7 steps, fit in E, whose
    terms add up to H / 1024 + 38 of its H / 512 + 70 steps."""
    r, h = got if isinstance(got, tuple) else (got, None)
    rr, hh = want
    E = (H / 512 + 70) * 2.0 ** -24
    branch = np.abs(rr - f64(d["res"]))
    er = E * branch + 2.0 ** -24 * (np.abs(rr) + branch) + 2.0 ** -150
    tol = er + (2.0 ** -8 * (np.abs(rr) + er) + 2.0 ** -134 if r.dtype == torch.bfloat16 else 0.0)
    err = np.abs(f64(r) - rr)
    assert (err <= tol).all(), ("r'", (err / tol).max(-1))
    if hh is None:
        return
    scale = 1 / np.sqrt((rr ** 2).mean(-1, keepdims=True) + eps)
    w = np.abs(f64(d["w_pre"]))
    eh = w * scale * er + np.abs(hh) * (E + (er * np.abs(rr)).mean(-1, keepdims=True) * scale ** 2) + \
        (w + 1) * 2.0 ** -150
    tol = eh + (2.0 ** -8 * (np.abs(hh) + eh) + 2.0 ** -134 if h.dtype == torch.bfloat16 else 0.0)
    err = np.abs(f64(h) - hh)
    assert (err <= tol).all(), ("h", (err / tol).max(-1))


@pytest.mark.parametrize("dt,rdt", TYPES)
@pytest.mark.parametrize("H", [8, 31, 264, 1023, 5120, 6001, 8200, 16384, 20000])
def test_squares_beyond_fp32(orc, dt, rdt, H):
    """Finite rows whose squares (or their sum alone) leave fp32: the same bound as any
    other row's.  Rows far below one are taken with eps = 0, where eps does not cover them."""
    need_cuda()
    rng = np.random.default_rng(H)
    rows = 8
    d = inputs(rng, 1, rows, H, "f32", "f32", "none", True, True)
    flat = lambda size: rng.choice([-1.0, 1.0], H) * rng.uniform(0.5, 1.0, H) * size
    d["y"][0, 0] = flat(3e38)
    d["y"][0, 1] = flat(1.8e19)              # each square fits, a few of them do not
    d["y"][0, 2] = flat(4e37) * (np.arange(H) == H - 1)   # one element alone
    d["res"][0, 3] = flat(3e38)
    d["res"][0, 4] = flat(1e20)
    d["y"][0, 5] = flat(2e25)
    d["res"][0, 5] = flat(2e25)
    low = {k: None if v is None else v.copy() for k, v in d.items()}
    for i, size in enumerate([1e-19, 1e-21, 1e-25, 1e-30, 1e-36]):
        low["y"][0, i] = flat(size)
        low["res"][0, i] = flat(1e-30)
    for case, eps in ((d, 1e-6), (low, 0.0), (low, 1e-44)):
        for post, pre in ((True, True), (False, True), (True, False)):
            c = dict(case, w_post=case["w_post"] if post else None, w_pre=case["w_pre"] if pre else None)
            if dt == "bf16":
                c = {k: v if v is None or (k == "res" and rdt == "f32") else synth.to_bf16_bits(v) for k, v in c.items()}
            got = dfl.norm_residual(**dev(c), eps=eps)
            want = oracle(orc, c, 1, rows, H, eps=float(np.float32(eps)))
            compare_denormal(got, want, c, H, float(np.float32(eps)))
