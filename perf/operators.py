"""The sequence-layer operators, as they are measured: the gated linear
recurrence (forward, backward, single-token step), the gated norm after a
block and the residual norm before one.

Where `own` is false, run() computes them in elementary torch operations in 32
bits, rounded once at the end; where it is true, it makes the calls a user
makes of this package.  Sizes follow the package's own workloads (8x12x2048x64,
2x16x32768x128, decode of 64 sequences with 16 heads of 128) or are odd.
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
#: elements of the largest listed case
MOST = 65536 * 2048


def listed():
    return [
        # one training step of a recurrent layer at the benchmark's layer width (12 heads of 64), x and f the two
        # halves of one projection
        dict(name="scan_train_8x2048x768_bf16", op="scan", way="train", type="bf16", n=8, l=2048, d=768, halves=True, reset=False, initial=False),
        # prefill of two long prompts that continue a state
        dict(name="scan_prefill_2x32768x2048_bf16", op="scan", way="fwd", type="bf16", n=2, l=32768, d=2048, halves=True, reset=False, initial=True),
        # training on packed documents, in fp32, odd in every size
        dict(name="scan_packed_5x1537x515_f32", op="scan", way="train", type="f32", n=5, l=1537, d=515, halves=False, reset=True, initial=True),
        # one token of 64 sequences being decoded
        dict(name="scan_step_64x2048_bf16", op="scan", way="step", type="bf16", n=64, l=1, d=2048, halves=True, reset=False, initial=True),
        # the gated norm behind a long prefill
        dict(name="gate_fwd_2x16x32768x128_bf16", op="gate", way="fwd", type="bf16", b=2, h=16, l=32768, d=128, per_head=False),
        # the gated norm of one decoded token of 64 sequences
        dict(name="gate_fwd_64x16x1x128_bf16", op="gate", way="fwd", type="bf16", b=64, h=16, l=1, d=128, per_head=True),
        # the gated norm's backward in the benchmark's training shape
        dict(name="gate_bwd_8x12x2048x64_bf16", op="gate", way="bwd", type="bf16", b=8, h=12, l=2048, d=64, per_head=False),
        # its backward in fp32 at odd sizes, a weight for each head
        dict(name="gate_bwd_3x7x1021x48_f32", op="gate", way="bwd", type="f32", b=3, h=7, l=1021, d=48, per_head=True),
        # the residual norm over the benchmark's 8 x 2048 tokens
        dict(name="residual_fwd_16384x768_bf16", op="residual", way="fwd", type="bf16", r=16384, d=768),
        # the residual norm of one decoded token of 64 sequences
        dict(name="residual_fwd_64x2048_bf16", op="residual", way="fwd", type="bf16", r=64, d=2048),
        # its backward over two long sequences
        dict(name="residual_bwd_65536x2048_bf16", op="residual", way="bwd", type="bf16", r=65536, d=2048),
        # its backward in fp32 at odd sizes
        dict(name="residual_bwd_1003x1111_f32", op="residual", way="bwd", type="f32", r=1003, d=1111),
    ]


def _spread(rng, low, high):
    """A whole number, evenly spread over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "gate", "residual"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    most = MOST // (2 if kind == "f32" else 1)  # fp32 costs twice the bytes
    if op == "scan":
        way = rng.choice(["train", "fwd", "step"])
        most //= 2 if way == "train" else 1
        d = _spread(rng, 64, 4096) // rng.choice([1, 1, 8, 64])
        d = max(1, d) * rng.choice([1, 8])
        n = _spread(rng, 1, 256 if way == "step" else 32)
        l = 1 if way == "step" else max(1, min(_spread(rng, 1, 32768), most // (n * d)))
        return dict(op=op, way=way, type=kind, n=n, l=l, d=d, halves=rng.random() < 0.5, reset=way != "step" and rng.random() < 0.4,
                    initial=way == "step" or rng.random() < 0.5)
    if op == "gate":
        way = rng.choice(["fwd", "bwd"])
        most //= 2 if way == "bwd" else 1
        d = rng.choice([16, 32, 64, 128, 256, rng.randint(1, 300), _spread(rng, 257, 4096)])
        h = _spread(rng, 1, 32)
        b = _spread(rng, 1, 64)
        l = max(1, min(_spread(rng, 1, 32768), most // (b * h * d)))
        return dict(op=op, way=way, type=kind, b=b, h=h, l=l, d=d, per_head=rng.random() < 0.5)
    way = rng.choice(["fwd", "bwd"])
    d = rng.choice([768, 1024, 2048, 4096, 8192, _spread(rng, 16, 8192)])
    return dict(op=op, way=way, type=kind, r=max(1, min(_spread(rng, 1, 65536), most // d)), d=d)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 13)
    t = TYPES[case["type"]]

    def normal(*shape, scale=1.0, shift=0.0, dtype=t):
        return torch.randn(shape, generator=gen, device=dev).mul_(scale).add_(shift).to(dtype)

    s = dict(case=dict(case))
    if case["op"] == "scan":
        n, l, d = case["n"], case["l"], case["d"]
        shape = (n, d) if case["way"] == "step" else (n, l, d)
        # forget gates with a bias for each channel: memories of two to some hundred tokens
        bias = torch.rand(d, generator=gen, device=dev) * 6.0
        if case["halves"]:  # the two halves of one projection
            both = normal(*shape[:-1], 2 * d, dtype=torch.float32)
            both[..., d:] += bias
            both = both.to(t)
            s["x"], s["f"] = both[..., :d], both[..., d:]
        else:
            s["x"] = normal(*shape)
            s["f"] = normal(*shape, dtype=torch.float32).add_(bias).to(t)
        s["reset"] = None
        if case["reset"]:  # documents of 300 tokens on average, packed one behind the other
            s["reset"] = torch.rand((n, l), generator=gen, device=dev) < 1.0 / 300
        s["initial"] = normal(n, d, scale=0.5, dtype=torch.float32) if case["initial"] else None
        if case["way"] == "train":
            s["dout"] = normal(n, l, d)
            s["dstate"] = normal(n, d, dtype=torch.float32)
        if case["way"] == "step":
            s["next"] = torch.empty_like(s["initial"])
    elif case["op"] == "gate":
        b, h, l, d = case["b"], case["h"], case["l"], case["d"]
        s["o"] = normal(b, h, l, d, scale=0.3)
        s["gate"] = normal(b, l, h * d)
        s["weight"] = normal(*((h, d) if case["per_head"] else (d,)), scale=0.1, shift=1.0, dtype=torch.float32)
        if case["way"] == "bwd":
            s["dout"] = normal(b, l, h * d)
    else:
        r, d = case["r"], case["d"]
        # in the backward, r is the residual stream as the forward left it
        s["r"] = normal(r, d, scale=2.0)
        s["y"] = normal(r, d)
        s["scale"] = normal(d, scale=0.1, shift=0.5, dtype=torch.float32)
        s["weight"] = normal(d, scale=0.1, shift=1.0, dtype=torch.float32)
        if case["way"] == "bwd":
            s["dh"] = normal(r, d)
            s["dr"] = normal(r, d)
    return s


# ---------------------------------------------------------------- the package's calls

def _own(s):
    import linear_attention_sequence_falcon_b200 as F
    c = s["case"]
    if c["op"] == "scan":
        if c["way"] == "step":
            out, state = F.scan_step(s["x"], s["f"], s["initial"], state_out=s["next"])
            return {"out": out, "state": state}
        if c["way"] == "fwd":
            out, state = F.scan(s["x"], s["f"], reset=s["reset"], initial_state=s["initial"])
            return {"out": out, "state": state}
        out, state, marks = F.scan(s["x"], s["f"], reset=s["reset"], initial_state=s["initial"], want_marks=True)
        g = F.scan_bwd(s["x"], s["f"], s["dout"], dstate=s["dstate"], reset=s["reset"], initial_state=s["initial"], marks=marks)
        return {"out": out, "state": state, "dx": g["dx"], "df": g["df"], "dinitial": g["dinitial"]}
    if c["op"] == "gate":
        if c["way"] == "fwd":
            return {"out": F.norm_gate(s["o"], s["gate"], s["weight"], EPS)}
        g = F.norm_gate_bwd(s["o"], s["gate"], s["weight"], EPS, s["dout"])
        return {"do": g["do"], "dgate": g["dgate"], "dweight": g["dweight"]}
    if c["way"] == "fwd":
        r, h = F.residual_norm(s["r"], s["weight"], EPS, y=s["y"], scale=s["scale"])
        return {"r": r, "h": h}
    g = F.residual_norm_bwd(s["r"], s["weight"], EPS, s["dh"], dr_out=s["dr"], y=s["y"], scale=s["scale"])
    return {"dr": g["dr"], "dy": g["dy"], "dscale": g["dscale"], "dweight": g["dweight"]}


# ---------------------------------------------------------------- the plain form

def _linear(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1, with h before the first step zero:
    neighbours joined over doubling distances, log2(L) times (a loop over the
    doublings; one over tokens would launch thousands of kernels)."""
    s = 1
    while s < a.shape[1]:
        b = torch.cat([b[:, :s], b[:, s:] + a[:, s:] * b[:, :-s]], 1)
        a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return b


def _plain_scan(s):
    c, t = s["case"], s["x"].dtype
    x, f = s["x"].float(), s["f"].float()
    keep = 1.0 / (1.0 + torch.exp(-f))
    take = 1.0 / (1.0 + torch.exp(f))
    if c["way"] == "step":
        h = keep * s["initial"] + take * x
        return {"out": h.to(t), "state": h}
    held = keep if s["reset"] is None else torch.where(s["reset"][..., None], 0.0, keep)  # what the state is multiplied by
    b = take * x
    if s["initial"] is not None:
        b[:, 0] += held[:, 0] * s["initial"]
    h = _linear(held, b)
    if c["way"] == "fwd":
        return {"out": h.to(t), "state": h[:, -1].clone()}
    first = torch.zeros_like(h[:, :1]) if s["initial"] is None else s["initial"][:, None]
    before = torch.cat([first, h[:, :-1]], 1)
    if s["reset"] is not None:
        before = torch.where(s["reset"][..., None], 0.0, before)
    dout = s["dout"].to(torch.float32, copy=True)  # the state's own dout stays as it is
    dout[:, -1] += s["dstate"]
    # the reverse recurrence g_t = dout_t + held_{t+1} g_{t+1}, as a forward one over the flipped tokens
    after = torch.cat([held[:, 1:], torch.zeros_like(held[:, :1])], 1)
    g = _linear(after.flip(1), dout.flip(1)).flip(1)
    dx = g * take
    df = g * (before - x) * (keep * take)
    return {"out": h.to(t), "state": h[:, -1].clone(), "dx": dx.to(t), "df": df.to(t), "dinitial": held[:, 0] * g[:, 0]}


def _plain_gate(s):
    c, t = s["case"], s["o"].dtype
    b, h, l, d = (c[k] for k in "bhld")
    o = s["o"].float().transpose(1, 2)  # [b,l,h,d]
    gate = s["gate"].float().reshape(b, l, h, d)
    rstd = 1.0 / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS)
    n = o * rstd
    sig = 1.0 / (1.0 + torch.exp(-gate))
    act = gate * sig
    if c["way"] == "fwd":
        return {"out": (n * s["weight"] * act).to(t).reshape(b, l, h * d)}
    dout = s["dout"].float().reshape(b, l, h, d)
    e = dout * act
    dn = e * s["weight"]
    do = rstd * (dn - n * (dn * n).mean(-1, keepdim=True))
    dgate = dout * n * s["weight"] * (sig * (1.0 + gate * (1.0 - sig)))
    dweight = (e * n).sum((0, 1) if c["per_head"] else (0, 1, 2))
    return {"do": do.transpose(1, 2).to(t).contiguous(), "dgate": dgate.to(t).reshape(b, l, h * d), "dweight": dweight}


def _plain_residual(s):
    c, t = s["case"], s["r"].dtype
    r, y = s["r"].float(), s["y"].float()
    if c["way"] == "fwd":
        r = r + s["scale"] * y
        h = r * (1.0 / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS)) * s["weight"]
        return {"r": r.to(t), "h": h.to(t)}
    rstd = 1.0 / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS)
    n = r * rstd
    dh = s["dh"].float()
    dn = dh * s["weight"]
    dr = s["dr"].float() + rstd * (dn - n * (dn * n).mean(-1, keepdim=True))
    return {"dr": dr.to(t), "dy": (dr * s["scale"]).to(t), "dscale": (dr * y).sum(0), "dweight": (dh * n).sum(0)}


def run(state):
    if own:
        return _own(state)
    return {"scan": _plain_scan, "gate": _plain_gate, "residual": _plain_residual}[state["case"]["op"]](state)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "scan":
        return _exact_scan(case, s)
    grad = case["way"] == "bwd"
    if case["op"] == "gate":
        b, h, l, d = (case[k] for k in "bhld")
        o, gate, weight = (s[k].double().requires_grad_(grad) for k in ("o", "gate", "weight"))
        unit = o / (torch.linalg.vector_norm(o, dim=-1, keepdim=True).square() / d + EPS).sqrt()
        w = weight[None, :, None, :] if case["per_head"] else weight
        out = (unit * w).permute(0, 2, 1, 3).reshape(b, l, h * d) * torch.nn.functional.silu(gate)
        if not grad:
            return {"out": out}
        out.backward(s["dout"].double())
        return {"do": o.grad, "dgate": gate.grad, "dweight": weight.grad}
    r, y, scale, weight = (s[k].double().requires_grad_(grad) for k in ("r", "y", "scale", "weight"))
    if not grad:
        stream = torch.addcmul(r, scale, y)
        return {"r": stream, "h": stream * torch.rsqrt(stream.square().mean(-1, keepdim=True) + EPS) * weight}
    # the stream as the forward left it, plus nothing: its gradient reaches r and, through the scale, y
    stream = r + scale * (y - s["y"].double())
    h = stream * torch.rsqrt(stream.square().mean(-1, keepdim=True) + EPS) * weight
    stream.retain_grad()
    torch.autograd.backward([h, stream], [s["dh"].double(), s["dr"].double()])
    # (y - y is zero, so the scale takes its gradient from the formula: the sum of the gradient of the stream times y)
    dscale = torch.einsum("rd,rd->d", r.grad, s["y"].double())
    return {"dr": r.grad, "dy": y.grad, "dscale": dscale, "dweight": weight.grad}


def _exact_scan(case, s):
    x, f = s["x"].double(), s["f"].double()
    a = torch.sigmoid(f)
    if case["way"] == "step":
        h = torch.lerp(x, s["initial"].double(), a)
        return {"out": h, "state": h}
    n, l, d = x.shape
    if s["reset"] is not None:
        a_held = a.masked_fill(s["reset"][..., None], 0.0)
    else:
        a_held = a
    h = torch.empty_like(x)
    state = torch.zeros_like(x[:, 0]) if s["initial"] is None else s["initial"].double()
    b = torch.sigmoid(-f) * x
    for t in range(l):
        state = torch.addcmul(b[:, t], a_held[:, t], state)
        h[:, t] = state
    if case["way"] == "fwd":
        return {"out": h, "state": state}
    dx, df = torch.empty_like(x), torch.empty_like(x)
    slope = a * torch.sigmoid(-f)
    g = s["dstate"].double()
    none = torch.zeros_like(g) if s["initial"] is None else s["initial"].double()
    dout = s["dout"].double()
    for t in range(l - 1, -1, -1):
        g = g + dout[:, t]
        prev = h[:, t - 1] if t else none
        if s["reset"] is not None:
            prev = prev.masked_fill(s["reset"][:, t, None], 0.0)
        dx[:, t] = g
        df[:, t] = g * (prev - x[:, t])
        g = g * a_held[:, t]
    return {"out": h, "state": state, "dx": dx * torch.sigmoid(-f), "df": df * slope, "dinitial": g}


def work(case):
    z = BYTES[case["type"]]
    if case["op"] == "scan":
        n, e = case["n"] * case["d"], case["n"] * case["l"] * case["d"]
        mask = case["n"] * case["l"] if case["reset"] else 0
        if case["way"] == "train":
            # x, f, dout read and out, dx, df written; the states at the ends
            return {"bytes": 6 * e * z + 4 * n * (3 + (1 if case["initial"] else 0)) + mask, "flops": 22 * e}
        return {"bytes": 3 * e * z + 4 * n * (1 + (1 if case["initial"] else 0)) + mask, "flops": 8 * e}
    if case["op"] == "gate":
        e = case["b"] * case["h"] * case["l"] * case["d"]
        w = 4 * case["d"] * (case["h"] if case["per_head"] else 1)
        if case["way"] == "bwd":
            return {"bytes": 5 * e * z + 2 * w, "flops": 26 * e}
        return {"bytes": 3 * e * z + w, "flops": 10 * e}
    e = case["r"] * case["d"]
    if case["way"] == "bwd":
        return {"bytes": 6 * e * z + 16 * case["d"], "flops": 16 * e}
    return {"bytes": 4 * e * z + 8 * case["d"], "flops": 7 * e}
