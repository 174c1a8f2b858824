"""The operators of a drafter's sub-block at decode time, as measured cases.

  linear  y = x W^T with W held in 4 bits: W[n, k] = scale[n, k / group] * (q[n, k] - zero[n, k / group]),
          zero = 8 where none is given
  conv    the two-tap dynamic conv whose tap projection W [2H, H] is held the same way:
          [a; b] = W x_t,  out_t = x_t + a * x_t + b * x_{t-1}
  norm    the norms around a block with its gate and residual scale:
          r' = r + alpha * act(gate) * rms(y; w_post),  h = rms(r'; w_pre),
          rms(v; w) = v / sqrt(mean(v^2) + eps) * w

Where `own` is false, run() computes them in elementary torch operations (fp32, rounded once at the
end); where it is true, it makes the calls a user makes of block_draft_verification_b200.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _named(name):
    return {} if name is None else {"name": name}


def _linear(name, tokens, n, k, group, zeros, x, out):
    return _named(name) | {"op": "linear", "tokens": tokens, "n": n, "k": k, "group": group, "zeros": zeros, "x": x, "out": out}


def _conv(name, seqs, tokens, h, group, zeros, x="bf16"):
    return _named(name) | {"op": "conv", "seqs": seqs, "tokens": tokens, "h": h, "group": group, "zeros": zeros, "x": x}


def _norm(name, seqs, tokens, h, gate, act, x, res, pre=True, post=True):
    return _named(name) | {"op": "norm", "seqs": seqs, "tokens": tokens, "h": h, "gate": gate, "act": act, "x": x,
            "res": res, "pre": pre, "post": post}


def listed():
    return [
        # one token through a square projection at the drafter's hidden size: the smallest step of a decode
        _linear("linear_1x5120x5120", 1, 5120, 5120, 128, False, "bf16", "bf16"),
        # a block of 8 through the vocabulary head, whose logits the top-16 softmax reads
        _linear("linear_8x151936x5120", 8, 151936, 5120, 128, False, "bf16", "bf16"),
        # 8 sequences' blocks into an MLP of four times the hidden size, weights with zero points
        _linear("linear_64x20480x5120", 64, 20480, 5120, 64, True, "bf16", "bf16"),
        # 32 sequences' blocks out of that MLP, kept in fp32 for the residual sum
        _linear("linear_256x5120x20480", 256, 5120, 20480, 128, False, "bf16", "f32"),
        # fp32 activations and odd sizes: a small model whose layers fit no tile
        _linear("linear_13x4099x1600_f32", 13, 4099, 1600, 32, True, "f32", "f32"),
        # the conv of one sequence's block, of 32 sequences' blocks, and of a small ragged batch
        _conv("conv_1x8x5120", 1, 8, 5120, 128, False),
        _conv("conv_32x8x5120", 32, 8, 5120, 128, True),
        _conv("conv_5x3x320", 5, 3, 320, 32, True),
        # one sequence's block, gated by channel; 32 sequences, gated per sequence
        _norm("norm_1x8x5120", 1, 8, 5120, "channel", "linear", "bf16", "bf16"),
        _norm("norm_32x8x5120", 32, 8, 5120, "sequence", "sigmoid", "bf16", "bf16"),
        # prompts of 2 x 2,048 tokens with the residual stream kept in fp32 and a gate per token
        _norm("norm_2x2048x5120_f32", 2, 2048, 5120, "token", "sigmoid", "bf16", "f32"),
        # an odd width, everything in fp32, no gate
        _norm("norm_7x143x1023_f32", 7, 143, 1023, "none", "linear", "f32", "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "conv", "norm"])
    if op == "linear":
        tokens = _log(rng, 1, 256)
        group = rng.choice([32, 64, 128])
        k = group * max(1, _log(rng, 64, 20480) // group)
        most = min(151936 * 5120 // 4, 256 * 5120 * 20480 // tokens) // k
        n = min(_log(rng, 48, 60000), most)
        x = rng.choice(["bf16", "bf16", "bf16", "f32"])
        if x == "f32":
            tokens = min(tokens, 32)
        return _linear(None, tokens, n, k, group, rng.random() < 0.5, x, rng.choice(["bf16", "f32"]) if x == "bf16" else "f32")
    if op == "conv":
        x = rng.choice(["bf16", "bf16", "bf16", "f32"])
        h = 64 * _log(rng, 1, 80)
        group = rng.choice([32, 64, 128] if h % 128 == 0 else [32, 64])
        return _conv(None, _log(rng, 1, 32 if x == "bf16" else 4), rng.randint(1, 8), h, group, rng.random() < 0.5, x)
    h = _log(rng, 64, 8192)
    rows = min(_log(rng, 1, 16384), 4096 * 5120 // h)
    seqs = _log(rng, 1, min(32, rows))
    x, res = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
    return _norm(None, seqs, max(1, rows // seqs), h, rng.choice(["none", "channel", "sequence", "token"]),
                 rng.choice(["linear", "sigmoid"]), x, res, rng.random() < 0.8, rng.random() < 0.8)


def _weights(gen, n, k, group, zeros):
    """Random 4-bit weights as a quantiser leaves them: bell-shaped codes about the zero point, two to a
    byte (the even k in the low half), bf16 group scales, zero points near the middle."""
    q = torch.empty((n, k // 2), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // k)
    for i in range(0, n, step):
        c = torch.randn((min(step, n - i), k), generator=gen, device="cuda", dtype=torch.float32)
        c = c.mul_(2.6).add_(8).round_().clamp_(0, 15).to(torch.uint8)
        q[i:i + step] = c[:, 0::2] | (c[:, 1::2] << 4)
    scale = torch.rand((n, k // group), generator=gen, device="cuda").add_(0.5).mul_(0.38 / math.sqrt(k))
    zero = torch.randint(5, 12, (n, k // group), generator=gen, device="cuda", dtype=torch.uint8) if zeros else None
    return q, scale.to(torch.bfloat16), zero


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device="cuda").mul_(std).add_(mean).to(dtype)

    dt = DTYPES[case["x"]]
    if case["op"] == "norm":
        B, T, H = case["seqs"], case["tokens"], case["h"]
        gate = {"none": None, "channel": (H,), "sequence": (B, H), "token": (B, T, H)}[case["gate"]]
        return {"case": case, "res": normal(B, T, H, std=3.0, dtype=DTYPES[case["res"]]), "y": normal(B, T, H, std=0.7, dtype=dt),
                "gate": None if gate is None else normal(*gate, std=0.5, mean=0.8, dtype=dt),
                "post": normal(H, std=0.1, mean=1.0, dtype=dt) if case["post"] else None,
                "pre": normal(H, std=0.1, mean=1.0, dtype=dt) if case["pre"] else None, "alpha": 0.70710678}
    taps = case["op"] == "conv"
    n, k = (2 * case["h"], case["h"]) if taps else (case["n"], case["k"])
    q, scale, zero = _weights(gen, n, k, case["group"], case["zeros"])
    state = {"case": case, "q": q, "scale": scale, "zero": zero}
    if taps:
        state["x"] = normal(case["seqs"], case["tokens"], k, dtype=dt)
        state["x_prev"] = normal(case["seqs"], k, dtype=dt)
    else:
        state["x"] = normal(case["tokens"], k, dtype=dt)
    if own:
        import block_draft_verification_b200 as dfl
        state["w4"] = dfl.PackedW4(q, scale, zero, taps=taps)  # laid out once, as a program keeps its weights
    return state


def _dequantise(q, scale, zero):
    n, groups = scale.shape
    codes = torch.stack((q & 15, q >> 4), dim=-1).reshape(n, groups, -1)
    w = codes.float() - (8.0 if zero is None else zero.float().unsqueeze(-1))
    return (w * scale.float().unsqueeze(-1)).reshape(n, -1)


def _rms(v, w):
    v = v * torch.rsqrt((v * v).mean(dim=-1, keepdim=True) + EPS)
    return v if w is None else v * w.float()


def run(state):
    c = state["case"]
    if own:
        import block_draft_verification_b200 as dfl
        if c["op"] == "linear":
            return dfl.linear_w4(state["x"], state["w4"], out_dtype=DTYPES[c["out"]])
        if c["op"] == "conv":
            return dfl.dynconv2(state["x"], state["x_prev"], state["w4"])
        return dfl.norm_residual(state["res"], state["y"], state["post"], state["pre"], gate=state["gate"],
                                 gate_act=dfl.GATE_SIGMOID if c["act"] == "sigmoid" else dfl.GATE_LINEAR, scale=state["alpha"], eps=EPS)
    if c["op"] == "linear":
        w = _dequantise(state["q"], state["scale"], state["zero"])
        return (state["x"].float() @ w.T).to(DTYPES[c["out"]])
    if c["op"] == "conv":
        x = state["x"].float()
        a, b = (x @ _dequantise(state["q"], state["scale"], state["zero"]).T).chunk(2, dim=-1)
        before = torch.cat((state["x_prev"].float().unsqueeze(1), x[:, :-1]), dim=1)
        return (x + a * x + b * before).to(DTYPES[c["x"]])
    y = state["y"].float()
    if state["post"] is not None:
        y = _rms(y, state["post"])
    if state["gate"] is not None:
        g = state["gate"].float()
        g = 1 / (1 + torch.exp(-g)) if c["act"] == "sigmoid" else g
        y = y * (g.unsqueeze(1) if c["gate"] == "sequence" else g)
    r = state["res"].float() + state["alpha"] * y
    res_out = r.to(DTYPES[c["res"]])
    return (res_out, _rms(r, state["pre"]).to(DTYPES[c["x"]])) if state["pre"] is not None else res_out


def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "norm":
        e = case["seqs"] * case["tokens"] * case["h"]
        gate = {"none": 0, "channel": case["h"], "sequence": case["seqs"] * case["h"], "token": e}[case["gate"]]
        x = size[case["x"]]
        per = 2 * size[case["res"]] + x + (x if case["pre"] else 0)
        return {"bytes": e * per + gate * x + case["h"] * x * (case["pre"] + case["post"]), "flops": 10 * e}
    taps = case["op"] == "conv"
    n, k = (2 * case["h"], case["h"]) if taps else (case["n"], case["k"])
    tokens = case["seqs"] * case["tokens"] if taps else case["tokens"]
    weights = n * k // 2 + n * (k // case["group"]) * (3 if case["zeros"] else 2)
    x = size[case["x"]]
    ends = (2 * tokens + case["seqs"]) * k * x if taps else tokens * (k * x + n * size[case["out"]])
    return {"bytes": weights + ends, "flops": 2 * tokens * n * k}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        r, y = s["res"].double(), s["y"].double()
        H = case["h"]
        if s["post"] is not None:
            y = y / (y.square().sum(-1, keepdim=True) / H + EPS).sqrt() * s["post"].double()
        if s["gate"] is not None:
            g = s["gate"].double()
            g = g.sigmoid() if case["act"] == "sigmoid" else g
            y = y * (g[:, None, :] if case["gate"] == "sequence" else g)
        r = r + s["alpha"] * y
        return (r, r / (r.square().sum(-1, keepdim=True) / H + EPS).sqrt() * s["pre"].double()) if s["pre"] is not None else r
    taps = case["op"] == "conv"
    x = s["x"].double().reshape(-1, s["x"].shape[-1])
    n, groups = s["scale"].shape
    group = x.shape[1] // groups
    xg = x.reshape(-1, groups, group).transpose(0, 1)  # the groups apart: their products, then the scales
    y = torch.empty((x.shape[0], n), dtype=torch.float64, device="cuda")
    rows = max(1, (1 << 25) // max(x.shape[1], x.shape[0] * groups))
    for i in range(0, n, rows):
        q = s["q"][i:i + rows].long()
        c = torch.zeros((q.shape[0], x.shape[1]), dtype=torch.float64, device="cuda")
        c[:, 0::2], c[:, 1::2] = (q % 16).double(), (q // 16).double()
        c = c.reshape(-1, groups, group) - (8 if s["zero"] is None else s["zero"][i:i + rows].double()[..., None])
        part = torch.bmm(xg, c.permute(1, 2, 0))  # [groups, tokens, rows]
        y[:, i:i + rows] = (part * s["scale"][i:i + rows].double().T[:, None, :]).sum(0)
    if not taps:
        return y
    B, T, H = s["x"].shape
    x3, y = s["x"].double(), y.reshape(B, T, 2 * H)
    out = x3 * (1 + y[..., :H])
    out[:, 0] += y[:, 0, H:] * s["x_prev"].double()
    out[:, 1:] += y[:, 1:, H:] * x3[:, :-1]
    return out
