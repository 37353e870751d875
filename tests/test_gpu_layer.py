"""The layer operators on the GPU against the plain fp64 forms of
layer_ref.py, element by element within the bounds derived there."""
import numpy as np
import pytest
import torch

from tests import layer_ref as ref
from tests.layer_ref import np64

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for the gpu tests")
    from linear_attention_sequence_falcon_b200 import build
    build.build()
    import linear_attention_sequence_falcon_b200 as F
    F.load()
    return F


def normal(gen, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=gen) * scale + shift).to(dtype).cuda()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def reset_mask(kind, g, N, L):
    if kind == "none":
        return None
    if kind == "all":
        return torch.ones((N, L), dtype=torch.bool, device="cuda")
    if kind == "first":
        m = torch.zeros((N, L), dtype=torch.bool, device="cuda")
        m[:, 0] = True
        return m
    return (torch.rand((N, L), generator=g) < 0.05).cuda()


# ---------------------------------------------------------------- the recurrence

SCAN = [
    # N, L, D, reset, initial state
    (1, 1, 1, "none", False), (3, 1, 64, "first", True), (2, 2, 7, "all", True), (2, 15, 33, "random", False),
    (1, 16, 64, "none", True), (2, 17, 128, "random", True), (1, 127, 40, "none", False), (3, 128, 64, "random", True),
    (2, 129, 66, "none", True), (1, 255, 2, "random", True), (2, 300, 130, "random", True), (1, 513, 96, "none", True),
    (1, 1025, 72, "random", True), (5, 257, 515, "random", True), (1, 2200, 8, "random", True), (40, 140, 16, "none", True),
    (1, 5000, 24, "random", False), (300, 3, 64, "random", True),
]


def scan_case(N, L, D, reset, initial, dtype, seed, halves=False):
    g = gen(seed)
    both = torch.randn((N, L, 2 * D), generator=g)
    both[..., D:] += 6 * torch.rand(D, generator=g)
    both = both.to(dtype).cuda()
    x, f = both[..., :D], both[..., D:]
    if not halves:
        x, f = x.contiguous(), f.contiguous()
    h0 = normal(g, N, D) if initial else None
    return x, f, reset_mask(reset, g, N, L), h0, normal(g, N, L, D, dtype=dtype), normal(g, N, D)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,L,D,reset,initial", SCAN)
def test_scan_forward_backward(F, N, L, D, reset, initial, dtype):
    t = TYPES[dtype]
    x, f, m, h0, dout, dstate = scan_case(N, L, D, reset, initial, t, 100 * N + L + D, halves=(L + D) % 2 == 1)
    out, state, marks = F.scan(x, f, reset=m, initial_state=h0, want_marks=True)
    args = np64(x), np64(f), None if m is None else m.cpu().numpy(), np64(h0)
    h, b, before, eb = ref.scan(*args)
    ref.check(out, h, b, t, "out")
    ref.check(state, h[:, -1], b[:, -1], torch.float32, "state")
    # the state before a block is what entered it: a reset on its first token acts after the mark
    blocks = range(0, L, F.SCAN_BLOCK)
    want = np.stack([(h[:, i - 1] if i else (args[3] if initial else np.zeros((N, D)))) for i in blocks], 1)
    wantb = np.stack([(b[:, i - 1] if i else np.zeros((N, D))) for i in blocks], 1)
    ref.check(marks, want, wantb, torch.float32, "marks")
    g = F.scan_bwd(x, f, dout, dstate=dstate, reset=m, initial_state=h0, marks=marks)
    r = ref.scan_bwd(args[0], args[1], np64(dout), np64(dstate), args[2], args[3])
    ref.check(g["dx"], *r["dx"], t, "dx")
    ref.check(g["df"], *r["df"], t, "df")
    ref.check(g["dinitial"], *r["dinitial"], torch.float32, "dinitial")
    # marks formed again are the same marks, and the same call gives the same bits
    again = F.scan_bwd(x, f, dout, dstate=dstate, reset=m, initial_state=h0)
    for k in g:
        assert torch.equal(g[k], again[k]), k
    assert torch.equal(out, F.scan(x, f, reset=m, initial_state=h0, want_state=False)[0])


# Long sequences of few channels: five turns of the cluster's walk at least, so
# that every place of the tiles' ring and both halves of the cluster's exchange
# are used again, and a ragged end.  (A tile is 64 tokens beyond 32 channels,
# and 4096 tokens over the channels rounded up to 8, 16 or 32 below that.)
STEPS = [
    (1, 6001, 64), (1, 6001, 66), (1, 6001, 67),                  # bf16: the three ways tiles come; fp32: two
    (1, 10001, 24), (1, 17001, 16), (1, 33001, 5), (2, 5185, 96),
    (197, 330, 130),                                              # blocks that need no neighbours: six turns of their own
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("reset", ["none", "random"])
@pytest.mark.parametrize("N,L,D", STEPS)
def test_scan_many_steps(F, N, L, D, reset, dtype):
    t = TYPES[dtype]
    tile = 64 if D > 32 else 4096 // max(8, 1 << (D - 1).bit_length())
    assert N > 2 or -(-(-(-L // tile)) // 16) >= 5 and L % tile
    x, f, m, h0, dout, dstate = scan_case(N, L, D, reset, True, t, N + L + D)
    out, state, marks = F.scan(x, f, reset=m, initial_state=h0, want_marks=True)
    args = np64(x), np64(f), None if m is None else m.cpu().numpy(), np64(h0)
    h, b, _, _ = ref.scan(*args)
    ref.check(out, h, b, t, "out")
    ref.check(state, h[:, -1], b[:, -1], torch.float32, "state")
    blocks = range(F.SCAN_BLOCK, L, F.SCAN_BLOCK)
    ref.check(marks[:, 1:], h[:, [i - 1 for i in blocks]], b[:, [i - 1 for i in blocks]], torch.float32, "marks")
    r = ref.scan_bwd(args[0], args[1], np64(dout), np64(dstate), args[2], args[3])
    first = F.scan_bwd(x, f, dout, dstate=dstate, reset=m, initial_state=h0, marks=marks)
    for g in (first, F.scan_bwd(x, f, dout, dstate=dstate, reset=m, initial_state=h0)):
        ref.check(g["dx"], *r["dx"], t, "dx")
        ref.check(g["df"], *r["df"], t, "df")
        ref.check(g["dinitial"], *r["dinitial"], torch.float32, "dinitial")
        assert all(torch.equal(first[k], g[k]) for k in g)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_gradients_against_differences(F, dtype):
    """The kernel's gradient along a direction against a central difference of
    the fp64 formula: a step of 1e-5 leaves 1e-10 of the terms (truncation and
    rounding); the stored gradients are off by half a step of their type each,
    and by less than 2^-14 of it in fp32 arithmetic."""
    t = TYPES[dtype]
    x, f, m, h0, dout, dstate = scan_case(2, 150, 20, "random", True, t, 5)
    g = F.scan_bwd(x, f, dout, dstate=dstate, reset=m, initial_state=h0)
    a = dict(x=np64(x), f=np64(f), initial=np64(h0))
    rng = np.random.default_rng(0)
    for k, got in (("x", g["dx"]), ("f", g["df"]), ("initial", g["dinitial"])):
        v = rng.standard_normal(a[k].shape)

        def loss(s):
            b = {**a, k: a[k] + s * v}
            h = ref.scan(b["x"], b["f"], m.cpu().numpy(), b["initial"])[0]
            return (h * np64(dout)).sum() + (h[:, -1] * np64(dstate)).sum()
        terms = np.abs(np64(got) * v).sum()
        tol = (ref.half(got.dtype) + 2.0 ** -14 + 1e-8) * terms
        assert abs((loss(1e-5) - loss(-1e-5)) / 2e-5 - (np64(got) * v).sum()) <= tol, k


def test_scan_extreme_gates(F):
    """f = +inf keeps the state to the bit, f = -inf replaces it; a reset drops
    infinities and NaN, and what is not reset keeps them; gates far out."""
    N, L, D = 2, 300, 64
    x, f, _, h0, _, _ = scan_case(N, L, D, "none", True, torch.float32, 9)
    keep = torch.full_like(f, float("inf"))
    out, state = F.scan(x, keep, initial_state=h0)
    assert torch.equal(state, h0) and torch.equal(out[:, 17], h0)
    out, state = F.scan(x, -keep, initial_state=h0)
    assert torch.equal(out, x) and torch.equal(state, x[:, -1])
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[0, 40, 3] = bad
        m = torch.zeros((N, L), dtype=torch.bool, device="cuda")
        m[:, 200] = True
        clean, _ = F.scan(x, f, reset=m, initial_state=h0)
        got, _ = F.scan(y, f, reset=m, initial_state=h0)
        assert not torch.isfinite(got[0, 40:200, 3]).any()
        assert torch.equal(got[0, 200:], clean[0, 200:]) and torch.equal(got[0, :40], clean[0, :40])
        assert torch.equal(got[1], clean[1]) and torch.equal(got[0, :, :3], clean[0, :, :3])
        s = h0.clone()
        s[1, 5] = bad
        m[1, 0] = True
        assert torch.isfinite(F.scan(x, f, reset=m, initial_state=s)[0]).all()
    big = f.clone().fill_(80.0)
    big[:, ::2] = -80.0
    args = np64(x), np64(big), None, np64(h0)
    h, b, _, _ = ref.scan(*args)
    ref.check(F.scan(x, big, initial_state=h0)[0], h, b, torch.float32, "far gates")


def test_scan_backward_nonfinite_documents(F):
    """A document that overflowed leaves the gradients of its neighbours alone."""
    N, L, D = 1, 400, 64
    x, f, _, h0, dout, dstate = scan_case(N, L, D, "none", True, torch.float32, 11)
    m = torch.zeros((N, L), dtype=torch.bool, device="cuda")
    m[:, 130] = m[:, 260] = True
    clean = F.scan_bwd(x, f, dout, dstate, m, h0)
    y, do = x.clone(), dout.clone()
    y[0, 150, 7] = float("inf")
    do[0, 170, 9] = float("nan")
    got = F.scan_bwd(y, f, do, dstate, m, h0)
    for k in ("dx", "df"):
        assert torch.equal(got[k][:, :130], clean[k][:, :130]) and torch.equal(got[k][:, 260:], clean[k][:, 260:])
        assert torch.isnan(got[k][0, 130:171, 9]).all()
    assert torch.equal(got["dinitial"], clean["dinitial"])


# Gates far below zero.  Beside layer_ref's (|f| + 12) U, log2(e) as an fp32 is
# 0.22 U off, so the exponent's argument is off by 1.22 |f| U at most.
FAR = 1.25


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,L,D,low", [(1, 1, 64, 20), (2, 300, 64, 79), (3, 130, 7, 79), (1, 200, 70, 20), (2, 90, 67, 14), (1, 500, 96, 79)])
def test_scan_closed_gates(F, N, L, D, low, dtype):
    """A closed gate lets little through, but that little to the accuracy of
    its type: df and dinitial are proportional to it, and the state where x is 0."""
    t = TYPES[dtype]
    x, f, m, h0, dout, dstate = scan_case(N, L, D, "random", True, t, 19)
    g = gen(N + L + D)
    shut = torch.rand((N, L, D), generator=g).cuda() < 0.5
    shut[:, 0] |= shut[:, -1]
    f = torch.where(shut, (-low * torch.rand((N, L, D), generator=g)).to(t).cuda(), f)
    x = torch.where(shut & (torch.rand((N, L, D), generator=g) < 0.5).cuda(), 0, x)
    m[:, 0] = m[:, -1] = False
    args = np64(x), np64(f), m.cpu().numpy(), np64(h0)
    out, state, marks = F.scan(x, f, m, h0, want_marks=True)
    h, b, _, _ = ref.scan(*args, far=FAR)
    ref.check(out, h, b, t, "out")
    ref.check(state, h[:, -1], b[:, -1], torch.float32, "state")
    blocks = range(F.SCAN_BLOCK, L, F.SCAN_BLOCK)
    if len(blocks):
        ref.check(marks[:, 1:], h[:, [i - 1 for i in blocks]], b[:, [i - 1 for i in blocks]], torch.float32, "marks")
    got = F.scan_bwd(x, f, dout, dstate, m, h0, marks)
    want = ref.scan_bwd(args[0], args[1], np64(dout), np64(dstate), args[2], args[3], far=FAR)
    ref.check(got["dx"], *want["dx"], t, "dx")
    ref.check(got["df"], *want["df"], t, "df")
    ref.check(got["dinitial"], *want["dinitial"], torch.float32, "dinitial")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_closed_gates_against_differences(F, dtype):
    """df of single tokens against central differences of the fp64 formula, each
    element by itself.  A step of 1e-4 leaves s^2/6 = 2e-9 of it; with x = 0 the
    state is a h0, so the difference's rounding is 2^-52 / 1e-4 of it; the
    kernel's own is layer_ref's bound, at most 2^-15, and half a step of its type."""
    t = TYPES[dtype]
    n = 64
    f = torch.linspace(-79, -1, n).to(t).cuda()[None, None]
    h0, dout = normal(gen(3), 1, n, shift=2.0), normal(gen(4), 1, 1, n, dtype=t)
    got = np64(F.scan_bwd(torch.zeros_like(f), f, dout, initial_state=h0)["df"])[0, 0]
    loss = lambda s: ref.scan(np.zeros((1, 1, n)), np64(f) + s, None, np64(h0))[0][0, 0] * np64(dout)[0, 0]  # noqa: E731
    d = (loss(1e-4) - loss(-1e-4)) / 2e-4
    assert (np.abs(got - d) <= (ref.half(t) + 2.0 ** -15 + 1e-8) * np.abs(d)).all(), np.abs(got / d - 1).max()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 67])
def test_scan_step_closed_gates(F, D, dtype):
    t = TYPES[dtype]
    g = gen(D)
    N = 40
    f = (-79 * torch.rand((N, D), generator=g)).to(t).cuda()
    x, s = normal(g, N, D, dtype=t), normal(g, N, D)
    x[:, ::2] = 0
    out, nxt = F.scan_step(x, f, s, state_out=torch.empty_like(s))
    h, b, _, _ = ref.scan(np64(x)[:, None], np64(f)[:, None], None, np64(s), far=FAR)
    ref.check(out, h[:, 0], b[:, 0], t, "out")
    ref.check(nxt, h[:, 0], b[:, 0], torch.float32, "state")


@pytest.mark.parametrize("D", [24, 64, 66, 67])
def test_scan_infinite_gates_bf16(F, D):
    """In bf16 too f = +inf keeps the state to the bit and f = -inf replaces it,
    backward and in a single step as well."""
    x, f, _, h0, dout, dstate = scan_case(2, 300, D, "none", True, torch.bfloat16, 21)
    keep = torch.full_like(f, float("inf"))
    out, state = F.scan(x, keep, initial_state=h0)
    assert torch.equal(state, h0) and torch.equal(out[:, 17], h0.bfloat16())
    assert torch.equal(F.scan_step(x[:, 0], keep[:, 0], h0.clone())[1], h0)
    out, state = F.scan(x, -keep, initial_state=h0)
    assert torch.equal(out, x) and torch.equal(state, x[:, -1].float())
    assert torch.equal(F.scan_step(x[:, 0], -keep[:, 0], h0.clone())[1], x[:, 0].float())
    got = F.scan_bwd(x, -keep, dout, dstate, initial_state=h0)
    last = (dout[:, -1].float() + dstate).bfloat16()
    assert torch.equal(got["dx"][:, :-1], dout[:, :-1]) and torch.equal(got["dx"][:, -1], last)
    assert (got["df"] == 0).all() and (got["dinitial"] == 0).all()
    got = F.scan_bwd(x, keep, torch.zeros_like(dout), dstate, initial_state=h0)
    assert torch.equal(got["dinitial"], dstate) and (got["dx"] == 0).all() and (got["df"] == 0).all()


def test_scan_in_segments_and_steps(F):
    """Two segments with the state handed on, and single-token steps, give the
    forward of the whole within twice its bound."""
    N, L, D = 3, 330, 70
    x, f, _, h0, _, _ = scan_case(N, L, D, "none", True, torch.float32, 13, halves=True)
    h, b, _, _ = ref.scan(np64(x), np64(f), None, np64(h0))
    o1, s1 = F.scan(x[:1, :200], f[:1, :200], initial_state=h0[:1])
    o2, s2 = F.scan(x[:1, 200:], f[:1, 200:], initial_state=s1, final_state=s1)  # the state in place
    assert s2 is s1
    ref.check(torch.cat([o1, o2], 1), h[:1], b[:1], torch.float32, "segments")
    ref.check(s1, h[:1, -1], b[:1, -1], torch.float32, "state")
    state = h0.clone()
    outs = []
    for t in range(40):
        o, same = F.scan_step(x[:, t], f[:, t], state)
        assert same is state
        outs.append(o)
    ref.check(torch.stack(outs, 1), h[:, :40], b[:, :40], torch.float32, "steps")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D", [(1, 1), (1, 3), (5, 64), (64, 2048), (7, 515), (2, 8190)])
def test_scan_step(F, N, D, dtype):
    t = TYPES[dtype]
    g = gen(N + D)
    both = normal(g, N, 2 * D, dtype=t)
    x, f, s = both[:, :D], both[:, D:], normal(g, N, D)
    nxt = torch.empty_like(s)
    out, got = F.scan_step(x, f, s, state_out=nxt)
    assert got is nxt
    h, b, _, _ = ref.scan(np64(x)[:, None], np64(f)[:, None], None, np64(s))
    ref.check(out, h[:, 0], b[:, 0], t, "out")
    ref.check(nxt, h[:, 0], b[:, 0], torch.float32, "state")


def guarded(shape, dtype, offset=0):
    """A view of a larger buffer filled with a mark, `offset` elements in, and the buffer."""
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * 64 + offset,), 77.0, dtype=dtype, device="cuda")
    return buf[64 + offset:64 + offset + n].view(shape), buf, 64 + offset, n


def untouched(buf, start, n):
    assert (buf[:start] == 77.0).all() and (buf[start + n:] == 77.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("N,L,D", [(2, 130, 64), (1, 300, 67), (3, 20, 128), (1, 700, 70), (2, 333, 18)])
def test_scan_alignment_and_borders(F, N, L, D, offset, dtype):
    """Arrays that begin off any vector's boundary, and nothing written beside the outputs."""
    t = TYPES[dtype]
    x, f, m, h0, dout, dstate = scan_case(N, L, D, "random", True, t, 17)
    shift = lambda a: guarded(a.shape, a.dtype, offset)[0].copy_(a)  # noqa: E731
    marks = F.scan(x, f, m, h0, want_marks=True)[2]
    h, b, _, _ = ref.scan(np64(x), np64(f), m.cpu().numpy(), np64(h0))
    wantg = ref.scan_bwd(np64(x), np64(f), np64(dout), np64(dstate), m.cpu().numpy(), np64(h0))
    out, ob, os_, on = guarded((N, L, D), t, offset)
    st, sb, ss, sn = guarded((N, D), torch.float32, offset)
    mk, mb, ms, mn = guarded(marks.shape, torch.float32, offset)
    F.scan(shift(x), shift(f), m, shift(h0), out=out, final_state=st, marks=mk)
    for buf, s, n in ((ob, os_, on), (sb, ss, sn), (mb, ms, mn)):
        untouched(buf, s, n)
    ref.check(out, h, b, t, "out")
    ref.check(st, h[:, -1], b[:, -1], torch.float32, "state")
    blocks = list(range(F.SCAN_BLOCK, L, F.SCAN_BLOCK))
    ref.check(mk[:, 1:], h[:, [i - 1 for i in blocks]], b[:, [i - 1 for i in blocks]], torch.float32, "marks")
    assert torch.equal(mk[:, 0], h0)
    both = torch.full((N, L, 2 * D + 3), 77.0, dtype=t, device="cuda")
    g = F.scan_bwd(shift(x), shift(f), shift(dout), shift(dstate), m, shift(h0), marks=shift(marks),
                   dx=both[..., 1:D + 1], df=both[..., D + 2:2 * D + 2])
    ref.check(g["dx"], *wantg["dx"], t, "dx")
    ref.check(g["df"], *wantg["df"], t, "df")
    ref.check(g["dinitial"], *wantg["dinitial"], torch.float32, "dinitial")
    assert (both[..., 0] == 77).all() and (both[..., D + 1] == 77).all() and (both[..., 2 * D + 2:] == 77).all()


# ---------------------------------------------------------------- the gated norm

GATE = [
    # B, H, L, d, weight, gate
    (1, 1, 1, 1, "shared", True), (2, 3, 5, 16, "head", True), (1, 2, 33, 48, "shared", True), (64, 16, 1, 128, "head", True),
    (2, 12, 100, 64, "shared", True), (1, 1, 70, 2048, "shared", True), (1, 2, 9, 300, "head", True), (2, 1, 4, 16384, "none", True),
    (1, 5, 40, 33, "head", False), (2, 2, 17, 256, "none", False), (1, 1, 3, 5001, "shared", True), (3, 7, 121, 48, "head", True),
    (1, 40, 300, 32, "shared", True), (1, 3, 1, 511, "shared", True), (1, 1, 200, 260, "head", True), (2, 130, 2, 8, "head", True),
    (1, 2, 3, 2056, "head", True), (1, 1, 9, 8190, "shared", True), (2, 1, 5, 6000, "none", False), (1, 4, 1200, 2, "head", True),
]


def gate_case(B, H, L, d, weight, gated, dtype, seed):
    g = gen(seed)
    o = normal(g, B, H, L, d, dtype=dtype, scale=0.3)
    gate = normal(g, B, L, H * d, dtype=dtype, scale=2.0) if gated else None
    w = {"none": None, "shared": normal(g, d, scale=0.2, shift=1.0), "head": normal(g, H, d, scale=0.2, shift=1.0)}[weight]
    return o, gate, w, normal(g, B, L, H * d, dtype=dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,L,d,weight,gated", GATE)
def test_norm_gate(F, B, H, L, d, weight, gated, dtype):
    t = TYPES[dtype]
    o, gate, w, dout = gate_case(B, H, L, d, weight, gated, t, B + H + L + d)
    eps = 1e-5
    want, b = ref.norm_gate(np64(o), np64(gate), np64(w), eps)
    ref.check(F.norm_gate(o, gate, w, eps), want, b, t, "out")
    g = F.norm_gate_bwd(o, gate, w, eps, dout)
    r = ref.norm_gate_bwd(np64(o), np64(gate), np64(w), eps, np64(dout))
    for k in ("do", "dgate", "dweight"):
        assert (g[k] is None) == (k not in r)
        if k in r:
            ref.check(g[k], *r[k], torch.float32 if k == "dweight" else t, k)
    again = F.norm_gate_bwd(o, gate, w, eps, dout)
    assert all(g[k] is None or torch.equal(g[k], again[k]) for k in g)
    part = F.norm_gate_bwd(o, gate, w, eps, dout, want_dweight=False)
    assert part["dweight"] is None and torch.equal(part["do"], g["do"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,offset", [(64, 0), (64, 1), (50, 2), (300, 0), (300, 1)])
def test_norm_gate_layouts(F, d, offset, dtype):
    """Heads-last input, the gate as half of a projection, arrays off a vector's
    boundary, gradients written into given places, nothing beside them."""
    t = TYPES[dtype]
    B, H, L = 2, 3, 21
    o, gate, w, dout = gate_case(B, H, L, d, "head", True, t, 23)
    want, b = ref.norm_gate(np64(o), np64(gate), np64(w), 1e-6)
    wantg = ref.norm_gate_bwd(np64(o), np64(gate), np64(w), 1e-6, np64(dout))
    last = guarded((B, L, H, d), t, offset)[0]
    last.copy_(o.transpose(1, 2))
    proj = torch.full((B, L, 2 * H * d + 5), 77.0, dtype=t, device="cuda")
    proj[..., 5:5 + H * d] = gate
    shift = lambda a: guarded(a.shape, a.dtype, offset)[0].copy_(a)  # noqa: E731
    out, ob, s, n = guarded((B, L, H * d), t, offset)
    F.norm_gate(last.transpose(1, 2), proj[..., 5:5 + H * d], shift(w), 1e-6, out=out)
    untouched(ob, s, n)
    ref.check(out, want, b, t, "out")
    do, db, s, n = guarded((B, L, H, d), t, offset)
    dproj = torch.full_like(proj, 77.0)
    g = F.norm_gate_bwd(last.transpose(1, 2), proj[..., 5:5 + H * d], shift(w), 1e-6, shift(dout), do=do.transpose(1, 2),
                        dgate=dproj[..., 5:5 + H * d])
    untouched(db, s, n)
    assert (dproj[..., :5] == 77).all() and (dproj[..., 5 + H * d:] == 77).all()
    ref.check(g["do"], *wantg["do"], t, "do")
    ref.check(g["dgate"], *wantg["dgate"], t, "dgate")
    ref.check(g["dweight"], *wantg["dweight"], torch.float32, "dweight")


def test_norm_gate_zero_and_nonfinite_rows(F):
    """Rows of zeros give zeros (eps = 0 too) and finite gradients; a row with a
    NaN spoils itself and no other; far gates."""
    o, gate, w, dout = gate_case(2, 3, 20, 64, "shared", True, torch.float32, 29)
    o[0, 1] = 0
    for eps in (0.0, 1e-6):
        out = F.norm_gate(o, gate, w, eps).view(2, 20, 3, 64)
        assert (out[0, :, 1] == 0).all() and torch.isfinite(out).all()
        g = F.norm_gate_bwd(o, gate, w, eps, dout)
        assert all(torch.isfinite(v).all() for v in g.values())
    clean = F.norm_gate(o, gate, w, 1e-6).view(2, 20, 3, 64).clone()
    o[1, 2, 7, 5] = float("nan")
    got = F.norm_gate(o, gate, w, 1e-6).view(2, 20, 3, 64)
    assert torch.isnan(got[1, 7, 2]).all()
    got[1, 7, 2] = clean[1, 7, 2]
    assert torch.equal(got, clean)
    gate = torch.where(gate > 0, 200.0, -200.0)
    o[1, 2, 7, 5] = 1
    want, b = ref.norm_gate(np64(o), np64(gate), np64(w), 1e-6)
    ref.check(F.norm_gate(o, gate, w, 1e-6), want, b, torch.float32, "far gates")
    assert all(torch.isfinite(v).all() for v in F.norm_gate_bwd(o, gate, w, 1e-6, dout).values())


# ---------------------------------------------------------------- the residual norm

RESIDUAL = [
    # rows, D, y, scale, weight, dr_out
    (1, 1, True, True, True, True), (3, 16, True, True, True, True), (64, 2048, True, True, True, True), (5, 33, True, False, True, True),
    (130, 768, True, True, True, True), (7, 1111, True, True, True, False), (2, 16384, True, True, True, True), (9, 4096, False, False, True, True),
    (1, 5003, True, True, False, True), (300, 64, True, True, True, True), (4, 8192, True, False, False, True), (1000, 24, True, True, True, True),
    (33, 260, False, False, True, False), (2, 9001, True, True, True, True),
    (3, 2056, True, True, True, True), (5, 7096, True, True, True, True), (4, 6002, True, True, True, True),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,D,has_y,scaled,weighted,stream", RESIDUAL)
def test_residual_norm(F, R, D, has_y, scaled, weighted, stream, dtype):
    t = TYPES[dtype]
    g = gen(R + D)
    r, dh = normal(g, R, D, dtype=t, scale=2.0), normal(g, R, D, dtype=t)
    y = normal(g, R, D, dtype=t) if has_y else None
    s = normal(g, D, scale=0.3, shift=0.5) if scaled else None
    w = normal(g, D, scale=0.2, shift=1.0) if weighted else None
    dr = normal(g, R, D, dtype=t) if stream else None
    eps = 1e-5
    r_out, h = F.residual_norm(r, w, eps, y=y, scale=s)
    (ws, bs), (wh, bh) = ref.residual_norm(np64(r), np64(y), np64(s), np64(w), eps)
    ref.check(r_out, ws, bs, t, "r_out")
    ref.check(h, wh, bh, t, "h")
    assert has_y or r_out is r
    got = F.residual_norm_bwd(r_out, w, eps, dh, dr_out=dr, y=y, scale=s)
    want = ref.residual_norm_bwd(np64(r_out), np64(y), np64(s), np64(w), eps, np64(dh), np64(dr))
    for k in ("dr", "dy", "dscale", "dweight"):
        assert (got[k] is None) == (k not in want), k
        if k in want:
            ref.check(got[k], *want[k], t if k in ("dr", "dy") else torch.float32, k)
    assert scaled or not has_y or got["dy"] is got["dr"]
    again = F.residual_norm_bwd(r_out, w, eps, dh, dr_out=dr, y=y, scale=s)
    assert all(got[k] is None or torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,D,offset", [(40, 64, 0), (40, 64, 1), (9, 1111, 1), (6, 2048, 0), (6, 2048, 3)])
def test_residual_norm_in_place_and_borders(F, R, D, offset, dtype):
    t = TYPES[dtype]
    g = gen(R * D + offset)
    r, y, dh, dr = (normal(g, R, D, dtype=t) for _ in range(4))
    s, w = normal(g, D), normal(g, D)
    (ws, bs), (wh, bh) = ref.residual_norm(np64(r), np64(y), np64(s), np64(w), 1e-6)
    rr, rb, st, n = guarded((R, D), t, offset)
    yy, yb, _, _ = guarded((R, D), t, offset)
    rr.copy_(r)
    yy.copy_(y)
    got_r, got_h = F.residual_norm(rr, w, 1e-6, y=yy, scale=s, r_out=rr, h=yy)  # the stream in place, h over y
    assert got_r is rr and got_h is yy
    for buf in (rb, yb):
        untouched(buf, st, n)
    ref.check(rr, ws, bs, t, "r_out")
    ref.check(yy, wh, bh, t, "h")
    want = ref.residual_norm_bwd(np64(rr), np64(y), np64(s), np64(w), 1e-6, np64(dh), np64(dr))
    dd, db, _, _ = guarded((R, D), t, offset)

    def same(got):
        untouched(db, st, n)
        untouched(yb, st, n)
        for k in want:
            ref.check(got[k], *want[k], t if k in ("dr", "dy") else torch.float32, k)
    yy.copy_(y)
    dd.copy_(dr)
    same(F.residual_norm_bwd(rr, w, 1e-6, dh, dr_out=dd, y=yy, scale=s, dr=dd, dy=yy))
    yy.copy_(y)
    dd.copy_(dh)
    same(F.residual_norm_bwd(rr, w, 1e-6, dd, dr_out=dr, y=yy, scale=s, dr=dd))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,D", [(5003, 281), (2999, 1111), (700, 2047), (301, 4097), (40, 8185), (40, 8187), (2501, 33), (4001, 12), (9000, 1), (1501, 1110), (3, 7)])
def test_residual_norm_rows_off_the_pieces(F, R, D, dtype):
    """Rows that do not start on 16 bytes, in arrays that do: many rows to a
    thread, neighbours of NaN and infinities, the ends of each row, in place."""
    t = TYPES[dtype]
    g = gen(R * 3 + D)
    r, y, dh, dr = (normal(g, R, D, dtype=t) for _ in range(4))
    s, w = normal(g, D), normal(g, D)
    (ws, bs), (wh, bh) = ref.residual_norm(np64(r), np64(y), np64(s), np64(w), 1e-6)
    rr, rb, st, n = guarded((R, D), t, 0)
    yy, yb, _, _ = guarded((R, D), t, 0)
    assert rr.data_ptr() % 16 == 0 and yy.data_ptr() % 16 == 0
    rr.copy_(r)
    yy.copy_(y)
    F.residual_norm(rr, w, 1e-6, y=yy, scale=s, r_out=rr, h=yy)
    untouched(rb, st, n)
    untouched(yb, st, n)
    ref.check(rr, ws, bs, t, "r_out")
    ref.check(yy, wh, bh, t, "h")
    got = F.residual_norm_bwd(rr, w, 1e-6, dh, dr_out=dr, y=y, scale=s)
    want = ref.residual_norm_bwd(np64(rr), np64(y), np64(s), np64(w), 1e-6, np64(dh), np64(dr))
    for k in want:
        ref.check(got[k], *want[k], t if k in ("dr", "dy") else torch.float32, k)
    dd, db, _, _ = guarded((R, D), t, 0)
    dd.copy_(dr)
    again = F.residual_norm_bwd(rr, w, 1e-6, dh, dr_out=dd, y=y, scale=s, dr=dd)
    untouched(db, st, n)
    assert all(torch.equal(got[k], again[k]) for k in got)
    # a row's outputs are its own: bad numbers in every third row stay there
    bad = dh.clone()
    bad[::3] = float("nan")
    bad[1::6] = float("inf")
    kept = [i for i in range(R) if i % 3 and i % 6 != 1]
    if kept:
        ill = F.residual_norm_bwd(rr, w, 1e-6, bad, dr_out=dr, y=y, scale=s)
        assert torch.equal(ill["dr"][kept], got["dr"][kept]) and torch.equal(ill["dy"][kept], got["dy"][kept])
        worse = r.clone()
        worse[::3] = float("nan")
        worse[1::6] = float("inf")
        assert torch.equal(F.residual_norm(worse, w, 1e-6, y=y, scale=s)[1][kept], yy[kept])


def test_norms_gradients_against_differences(F):
    """The kernels' gradients along a direction against central differences of
    the fp64 formulas (a step of 1e-5: 1e-10 of the terms; the fp32 gradients
    are off by less than 2^-14 of themselves)."""
    rng = np.random.default_rng(4)
    o, gate, w, dout = gate_case(2, 2, 9, 40, "head", True, torch.float32, 31)
    g = F.norm_gate_bwd(o, gate, w, 1e-5, dout)
    a = [np64(o), np64(gate), np64(w)]
    for i, k in enumerate(("do", "dgate", "dweight")):
        v = rng.standard_normal(a[i].shape)
        f = lambda s: (ref.norm_gate(*[b + s * v if j == i else b for j, b in enumerate(a)], 1e-5)[0] * np64(dout)).sum()  # noqa: E731,B023
        tol = (2.0 ** -14 + 1e-8) * np.abs(np64(g[k]) * v).sum()
        assert abs((f(1e-5) - f(-1e-5)) / 2e-5 - (np64(g[k]) * v).sum()) <= tol, k
    q = gen(33)
    r, y, dh, dr = (normal(q, 11, 70) for _ in range(4))
    s, w = normal(q, 70), normal(q, 70)
    a = [np64(r), np64(y), np64(s), np64(w)]
    # the stream in fp64 is the sum itself; the kernel continues from it rounded to fp32, 2^-24 of it
    r_out, _ = F.residual_norm(r, w, 1e-5, y=y, scale=s)
    g = F.residual_norm_bwd(r_out, w, 1e-5, dh, dr_out=dr, y=y, scale=s)
    for i, k in enumerate(("dr", "dy", "dscale", "dweight")):
        v = rng.standard_normal(a[i].shape)

        def f(z):
            (u, _), (h, _) = ref.residual_norm(*[b + z * v if j == i else b for j, b in enumerate(a)], 1e-5)
            return (u * np64(dr)).sum() + (h * np64(dh)).sum()
        tol = (2.0 ** -14 + 1e-8) * np.abs(np64(g[k]) * v).sum()
        assert abs((f(1e-5) - f(-1e-5)) / 2e-5 - (np64(g[k]) * v).sum()) <= tol, k


# ---------------------------------------------------------------- empty sizes, streams, graphs

def test_empty_sizes(F):
    f32 = dict(dtype=torch.float32, device="cuda")
    h0 = torch.randn(2, 8, **f32)
    e = torch.empty(2, 0, 8, **f32)
    out, state, marks = F.scan(e, e, initial_state=h0, want_marks=True)
    assert out.shape == (2, 0, 8) and marks.shape == (2, 0, 8) and torch.equal(state, h0)
    assert (F.scan(e, e)[1] == 0).all()
    assert torch.equal(F.scan_bwd(e, e, e, dstate=h0)["dinitial"], h0)
    assert (F.scan_bwd(e, e, e)["dinitial"] == 0).all()
    for shape in ((0, 4, 8), (2, 4, 0)):
        z = torch.empty(shape, **f32)
        assert F.scan(z, z)[0].shape == shape and F.scan_bwd(z, z, z)["dx"].shape == shape
    assert F.scan_step(h0[:0], h0[:0], h0[:0])[0].shape == (0, 8)
    w = torch.ones(8, **f32)
    o, g = torch.empty(2, 3, 0, 8, **f32), torch.empty(2, 0, 24, **f32)
    assert F.norm_gate(o, g, w, 1e-6).shape == (2, 0, 24)
    assert (F.norm_gate_bwd(o, g, w, 1e-6, g)["dweight"] == 0).all()
    r = torch.empty(0, 8, **f32)
    assert F.residual_norm(r, w, 1e-6, y=r, scale=w)[1].shape == (0, 8)
    got = F.residual_norm_bwd(r, w, 1e-6, r, y=r, scale=w)
    assert (got["dscale"] == 0).all() and (got["dweight"] == 0).all()


def layer_calls(F, a, stream=None):
    """One pass through every operator; the results in a list."""
    k = dict(stream=stream)
    out, state, marks = F.scan(a["x"], a["f"], a["m"], a["h0"], want_marks=True, **k)
    g = F.scan_bwd(a["x"], a["f"], a["dout"], a["dstate"], a["m"], a["h0"], marks=marks, **k)
    g2 = F.scan_bwd(a["x"], a["f"], a["dout"], a["dstate"], a["m"], a["h0"], **k)
    o = out.view(a["N"], a["L"], 2, -1).transpose(1, 2)
    y = F.norm_gate(o, a["gate"], a["w"], 1e-6, **k)
    gg = F.norm_gate_bwd(o, a["gate"], a["w"], 1e-6, a["dout"], **k)
    r, h = F.residual_norm(a["x2"], a["w2"], 1e-6, y=y, scale=a["s"], **k)
    rg = F.residual_norm_bwd(r, a["w2"], 1e-6, a["dout"], dr_out=a["x2"], y=y, scale=a["s"], **k)
    so, ss = F.scan_step(a["x"][:, 0], a["f"][:, 0], a["h0"], state_out=torch.empty_like(a["h0"]), **k)
    return [out, state, marks, *g.values(), *g2.values(), y, *gg.values(), r, h, *rg.values(), so, ss]


def layer_args(N, L, D, dtype, seed):
    x, f, m, h0, dout, dstate = scan_case(N, L, D, "random", True, dtype, seed)
    g = gen(seed + 1)
    return dict(N=N, L=L, x=x, f=f, m=m, h0=h0, dout=dout, dstate=dstate, gate=normal(g, N, L, D, dtype=dtype),
                w=normal(g, D // 2), w2=normal(g, D), s=normal(g, D), x2=normal(g, N, L, D, dtype=dtype))


def test_streams_side_by_side(F):
    """Two streams at once, each with its own calls, give what one alone gives."""
    a, b = layer_args(2, 700, 128, torch.bfloat16, 41), layer_args(3, 333, 64, torch.float32, 43)
    wa, wb = layer_calls(F, a), layer_calls(F, b)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        ga, gb = layer_calls(F, a, sa), layer_calls(F, b, sb)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(wa, ga)) and all(torch.equal(p, q) for p, q in zip(wb, gb))


def test_two_threads_at_once(F):
    """Two threads that call at once, each on a stream of its own, give what one gives."""
    import threading
    args = [layer_args(2, 700, 128, torch.bfloat16, 73), layer_args(3, 333, 66, torch.float32, 79)]
    want = [layer_calls(F, a) for a in args]
    torch.cuda.synchronize()
    wrong, begin = [], threading.Barrier(2)

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            begin.wait()
            for _ in range(30):
                got = layer_calls(F, args[i])
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(p, q) for p, q in zip(want[i], got)):
                    wrong.append(i)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join(300)
    assert not wrong and not any(th.is_alive() for th in threads)


def test_two_graphs_share_nothing(F):
    """Two captured graphs, replayed side by side and with new inputs."""
    args = [layer_args(2, 260, 64, torch.bfloat16, 47), layer_args(1, 515, 130, torch.float32, 53)]
    for a in args:
        layer_calls(F, a)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer_calls(F, a))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(3):
        for a in args:
            a["x"].copy_(a["x"].flip(1))
            a["gate"].mul_(-1)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, got in zip(args, outs):
            assert all(torch.equal(p, q) for p, q in zip(layer_calls(F, a), got)), turn


def test_short_and_long_way_agree(F, monkeypatch):
    """layer.py's short way and the way through ctypes: the same kernels, the
    same bits, the same refusals."""
    from linear_attention_sequence_falcon_b200 import layer
    assert layer._quick is not None
    for a in (layer_args(2, 260, 64, torch.bfloat16, 67), layer_args(1, 130, 34, torch.float32, 71)):
        short = layer_calls(F, a)
        monkeypatch.setattr(layer, "_quick", None)
        long = layer_calls(F, a)
        monkeypatch.undo()
        assert len(short) == len(long) and all(torch.equal(p, q) for p, q in zip(short, long))
        assert all(p.shape == q.shape and p.dtype == q.dtype and p.is_contiguous() == q.is_contiguous() for p, q in zip(short, long))
    x, f = a["x"], a["f"]
    assert F.scan(x, f, want_state=0)[1] is None and len(F.scan(x, f, want_marks=1)) == 3
    with pytest.raises(F.FalconError):
        F.scan(x, f.bfloat16())
    with pytest.raises(F.FalconError):
        F.scan(x, f, initial_state=a["h0"].cpu())
    with pytest.raises(F.FalconError):
        F.norm_gate(x[None], None, None, -1.0)
    with pytest.raises(F.FalconError):
        F.residual_norm(x.transpose(0, 1), None, 1e-6) if x.shape[0] > 1 else F.residual_norm(x[..., ::2], None, 1e-6)


def test_short_way_lets_other_threads_run(F):
    """A launch releases Python's lock: another thread gets on during calls of
    the short way, without the interpreter taking the lock from the caller."""
    import sys
    import threading
    from linear_attention_sequence_falcon_b200 import layer
    assert layer._quick is not None
    w = torch.ones(64, device="cuda")
    x, o, r = torch.ones(1, 1, 64, device="cuda"), torch.ones(1, 1, 1, 64, device="cuda"), torch.ones(1, 64, device="cuda")
    out, state = torch.empty_like(x), torch.empty_like(r)
    calls = [lambda: F.scan(x, x, None, None, out, state), lambda: F.scan_bwd(x, x, x), lambda: F.scan_step(r, r, state, None, r),
             lambda: F.norm_gate(o, x, w, 1e-6), lambda: F.norm_gate_bwd(o, x, w, 1e-6, x),
             lambda: F.residual_norm(r, w, 1e-6), lambda: F.residual_norm_bwd(r, w, 1e-6, r)]
    for i, call in enumerate(calls):
        call()
        torch.cuda.synchronize()
        gate, ran = threading.Lock(), []
        gate.acquire()
        other = threading.Thread(target=lambda: (gate.acquire(), ran.append(1)))
        other.start()
        before = sys.getswitchinterval()
        sys.setswitchinterval(1000.0)
        try:
            gate.release()
            turns = 0
            while not ran and turns < 50000:
                call()
                turns += 1
            got = bool(ran)
        finally:
            sys.setswitchinterval(before)
        other.join(60)
        assert got, "call %d held the lock throughout" % i


FIRST_CALL = """
import torch
import linear_attention_sequence_falcon_b200 as F
g = torch.Generator(device="cuda").manual_seed(3)
x, f, d = (torch.randn(2, 200, 96, device="cuda", generator=g).bfloat16() for _ in range(3))
w = torch.ones(48, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
def calls():
    out, state, marks = F.scan(x, f, want_marks=True)
    b = F.scan_bwd(x, f, d, marks=marks)
    o = out.view(2, 200, 2, 48).transpose(1, 2)
    n = F.norm_gate_bwd(o, f, w, 1e-6, d)
    r = F.residual_norm(x, None, 1e-6, y=F.norm_gate(o, f, w, 1e-6))
    return [out, state, b["df"], n["dweight"], n["do"], r[1]]
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, calls()))
"""


def test_first_call_is_captured(F):
    """A process whose first calls are captured into a graph (nothing warmed up)."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_short_way_refuses_what_the_long_way_refuses(F):
    """The checks stand in layer.py and in the short way: what the first refuses the
    second does not take.  (Wrong arrays are larger than right ones here, or views
    of larger ones.)"""
    from linear_attention_sequence_falcon_b200 import layer
    q = layer._quick
    big = torch.zeros(1 << 16, device="cuda")
    f32 = lambda *s: big[:int(np.prod(s))].view(s)  # noqa: E731
    t = lambda *s: f32(*s).bfloat16()  # noqa: E731
    x, st, marks, wide = t(2, 70, 8), f32(2, 8), f32(2, 2, 8), t(2, 70, 16)
    strided, uneven, lying = t(2, 8, 70).transpose(1, 2), t(70, 2, 8).transpose(0, 1), t(2, 1, 8).expand(2, 70, 8)
    rows = [t(2, 71, 8), x.float(), x.cpu(), x.half(), strided, uneven, lying, x[0]]
    whole = rows[:4] + [wide[..., :8], strided]          # where an array has to be contiguous
    states = [f32(3, 8), st.double(), st.cpu(), f32(2, 16)[:, :8], st.bfloat16()]
    resets = [torch.zeros(2, 70, device="cuda"), torch.zeros(2, 71, dtype=torch.bool, device="cuda"),
              torch.zeros(2, 70, dtype=torch.bool), torch.zeros(70, 2, dtype=torch.bool, device="cuda").t()]

    def each(name, good, bad, names):
        for place, choices in bad.items():
            for b in choices:
                args = list(good)
                args[place] = b
                assert getattr(q, name)(*args) is None, (name, names(args))
                with pytest.raises(F.FalconError):
                    getattr(F, name)(**names(args))

    scan = lambda a: dict(zip(("x", "f", "reset", "initial_state", "out", "final_state", "marks", "want_state", "want_marks"), a))  # noqa: E731
    each("scan", [x, x, None, None, None, None, None, True, False],
         {0: rows[1:], 1: rows, 2: resets, 3: states, 4: whole, 5: states, 6: [f32(2, 3, 8), marks.cpu(), marks.bfloat16()]}, scan)
    bwd = lambda a: dict(zip(("x", "f", "dout", "dstate", "reset", "initial_state", "marks", "dx", "df", "workspace"), a))  # noqa: E731
    each("scan_bwd", [x, x, x] + [None] * 7,
         {0: rows[1:], 1: rows, 2: whole, 3: states, 4: resets, 5: states, 6: [f32(2, 3, 8), marks.cpu()], 7: rows, 8: rows}, bwd)
    step = lambda a: dict(zip(("x", "f", "state", "state_out", "out"), a))  # noqa: E731
    one = t(2, 8)
    tokens = [t(3, 8), one.float(), one.cpu(), one.half(), t(8, 2).t(), t(1, 8).expand(2, 8), t(2, 1, 8)]
    each("scan_step", [one, one, st, None, None], {0: tokens, 1: tokens, 2: states, 3: states, 4: tokens[:4] + [t(2, 16)[:, :8]]}, step)
    o, g, w = t(2, 3, 5, 8), t(2, 5, 24), f32(8)
    gates = [t(2, 6, 24), g.float(), g.cpu(), t(2, 24, 5).transpose(1, 2), t(5, 2, 24).transpose(0, 1), t(2, 1, 24).expand(2, 5, 24)]
    weights = [f32(9), f32(2, 8), w.bfloat16(), w.cpu(), f32(16)[::2], f32(3, 16)[:, :8]]
    eps = [-1.0, float("nan")]
    heads = [o.half(), o.cpu(), t(2, 3, 8, 5).transpose(2, 3), o[0], t(2, 3, 5, 0), t(1, 1, 1, 16385)]
    gate = lambda a: dict(zip(("o", "gate", "weight", "eps", "out"), a))  # noqa: E731
    each("norm_gate", [o, g, w, 1e-6, None], {0: heads, 1: gates, 2: weights, 3: eps, 4: gates[:3] + [t(2, 5, 48)[..., :24]]}, gate)
    gbwd = lambda a: dict(zip(("o", "gate", "weight", "eps", "dout", "want_dweight"), a))  # noqa: E731
    each("norm_gate_bwd", [o, g, w, 1e-6, g, True], {0: heads, 1: gates, 2: weights, 3: eps, 4: gates[:3] + [t(2, 5, 48)[..., :24]]}, gbwd)
    r = t(4, 8)
    streams = [t(5, 8), r.float(), r.cpu(), t(4, 16)[:, :8], t(8, 4).t()]
    norm = lambda a: dict(zip(("r", "weight", "eps", "y", "scale"), a))  # noqa: E731
    each("residual_norm", [r, w, 1e-6, r, w], {0: streams, 1: weights, 2: eps, 3: streams + [None], 4: weights}, norm)
    nbwd = lambda a: dict(zip(("r_out", "weight", "eps", "dh", "dr_out", "y", "scale"), a))  # noqa: E731
    each("residual_norm_bwd", [r, w, 1e-6, r, r, r, w], {0: streams, 1: weights, 2: eps, 3: streams, 4: streams, 5: streams + [None], 6: weights}, nbwd)
    assert (big == 0).all()


# ---------------------------------------------------------------- offsets past 31 bits

FAR_ROWS = 2 ** 31 + 64  # elements


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 50, 33])
@pytest.mark.parametrize("far", ["batch", "head", "token", "gate", "dgate"])
def test_norm_gate_far_rows(F, far, d, dtype):
    """Rows that lie past 31 bits from the first, in each of the arrays that have
    strides: the places in 64-bit arithmetic, forward and backward."""
    t = TYPES[dtype]
    B, H, L = 2, 2, 3
    o, gate, w, dout = gate_case(B, H, L, d, "head", True, t, 37)
    want, b = ref.norm_gate(np64(o), np64(gate), np64(w), 1e-6)
    wantg = ref.norm_gate_bwd(np64(o), np64(gate), np64(w), 1e-6, np64(dout))
    D = H * d
    room = torch.empty(FAR_ROWS + 4096, dtype=t, device="cuda")
    strides = {"batch": (FAR_ROWS, L * d, d), "head": (L * d, FAR_ROWS, d), "token": (H * d, d, FAR_ROWS // 2)}
    do = dgate = None
    if far in strides:
        place = room.as_strided((B, H, L, d), strides[far] + (1,))
        place.copy_(o)
        o, do = place, torch.empty_like(room).as_strided((B, H, L, d), strides[far] + (1,))
    else:
        ld = FAR_ROWS // (B * L - 1) // 2 * 2 + 2  # the last token's row
        place = room.as_strided((B, L, D), (L * ld, ld, 1))
        assert (B * L - 1) * ld >= 2 ** 31
        if far == "gate":
            place.copy_(gate)
            gate = place
        else:
            dgate = place
    if far != "dgate":
        ref.check(F.norm_gate(o, gate, w, 1e-6), want, b, t, "out")
    g = F.norm_gate_bwd(o, gate, w, 1e-6, dout, do=do, dgate=dgate)
    ref.check(g["do"], *wantg["do"], t, "do")
    ref.check(g["dgate"], *wantg["dgate"], t, "dgate")
    ref.check(g["dweight"], *wantg["dweight"], torch.float32, "dweight")


def filled(*shape, dtype=torch.bfloat16, seed=0):
    """Standard normal numbers, made in place on the GPU."""
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(seed))


def test_norms_of_more_than_2_31_elements(F):
    """Arrays of more than 2^31 elements, whole: their first rows, the rows around
    that border and the last against the fp64 forms."""
    eps = 1e-5
    B, H, L, d = 1, 16, 1048600, 128
    w = filled(d, dtype=torch.float32, seed=1)
    o, gate, dout = filled(B, L, H, d, seed=2).transpose(1, 2), filled(B, L, H * d, seed=3), filled(B, L, H * d, seed=4)
    assert o.numel() > 2 ** 31
    out, g = F.norm_gate(o, gate, w, eps), F.norm_gate_bwd(o, gate, w, eps, dout)
    for part in (slice(0, 5), slice(2 ** 31 // (H * d) - 3, 2 ** 31 // (H * d) + 3), slice(L - 5, L)):
        a = np64(o[:, :, part]), np64(gate[:, part]), np64(w), eps
        ref.check(out[:, part], *ref.norm_gate(*a), torch.bfloat16, "out")
        want = ref.norm_gate_bwd(*a, np64(dout[:, part]))
        ref.check(g["do"][:, :, part], *want["do"], torch.bfloat16, "do")
        ref.check(g["dgate"][:, part], *want["dgate"], torch.bfloat16, "dgate")
    del o, gate, dout, out, g
    for R, D in ((131100, 16384), (268500, 8001)):
        w, s = filled(D, dtype=torch.float32, seed=5), filled(D, dtype=torch.float32, seed=6)
        r, y, dh = filled(R, D, seed=7), filled(R, D, seed=8), filled(R, D, seed=9)
        assert r.numel() > 2 ** 31
        r_out, h = F.residual_norm(r, w, eps, y=y, scale=s)
        g = F.residual_norm_bwd(r_out, w, eps, dh, dr_out=r, y=y, scale=s)
        for part in (slice(0, 5), slice(2 ** 31 // D - 3, 2 ** 31 // D + 3), slice(R - 5, R)):
            (wr, br), (wh, bh) = ref.residual_norm(np64(r[part]), np64(y[part]), np64(s), np64(w), eps)
            ref.check(r_out[part], wr, br, torch.bfloat16, "r_out")
            ref.check(h[part], wh, bh, torch.bfloat16, "h")
            want = ref.residual_norm_bwd(np64(r_out[part]), np64(y[part]), np64(s), np64(w), eps, np64(dh[part]), np64(r[part]))
            ref.check(g["dr"][part], *want["dr"], torch.bfloat16, "dr")
            ref.check(g["dy"][part], *want["dy"], torch.bfloat16, "dy")
        del r, y, dh, r_out, h, g


@pytest.mark.parametrize("L,D", [(2100, 524288), (2100, 524290), (2101, 524289)])
def test_scan_of_more_than_2_31_elements(F, L, D):
    """Two sequences, together past 31 bits of elements, in the three ways tiles
    come: channels from all over them against the fp64 form."""
    N, t = 2, torch.bfloat16
    x, f, dout = (filled(N, L, D, seed=i) for i in (1, 2, 3))
    h0 = filled(N, D, dtype=torch.float32, seed=4)
    assert x.numel() > 2 ** 31
    f.add_(2.0)
    out, state, marks = F.scan(x, f, initial_state=h0, want_marks=True)
    g = F.scan_bwd(x, f, dout, initial_state=h0, marks=marks)
    at = torch.tensor([0, 1, 63, 64, 131071, 262145, D - 66, D - 2, D - 1], device="cuda")
    pick = lambda a: np64(a.index_select(-1, at))  # noqa: E731
    h, b, _, _ = ref.scan(pick(x), pick(f), None, pick(h0))
    ref.check(out.index_select(-1, at), h, b, t, "out")
    ref.check(state.index_select(-1, at), h[:, -1], b[:, -1], torch.float32, "state")
    want = ref.scan_bwd(pick(x), pick(f), pick(dout), None, None, pick(h0))
    ref.check(g["dx"].index_select(-1, at), *want["dx"], t, "dx")
    ref.check(g["df"].index_select(-1, at), *want["df"], t, "df")
    ref.check(g["dinitial"].index_select(-1, at), *want["dinitial"], torch.float32, "dinitial")


# ---------------------------------------------------------------- the operators together

def test_layer_forward_backward(F):
    """A block as a stack runs it, in fp32: the residual norm, Falcon-1 on its
    output (heads split), the gated norm back to tokens, the recurrence on
    that, the residual norm behind; then the backward of all of it, against the
    same chain in fp64 (Falcon by the oracle).  Tolerances of Falcon's own
    parity (1e-4 of the largest value), times the norms' and the recurrence's
    gain, at most 4 here."""
    import oracle
    oracle.build()
    from linear_attention_sequence_falcon_b200 import inputs as inp
    B, H, L, d = 2, 2, 70, 32
    D = H * d
    q = gen(61)
    d0 = inp.draw("F1", B, H, L, d, d, seed=7, dtype="f32")
    k, v, beta, lam = (d0[n].cuda() for n in ("k", "v", "beta", "lam"))
    eps = d0["eps"]
    r, dtop, dstream = (normal(q, B, L, D) for _ in range(3))
    gate, fg = normal(q, B, L, D), normal(q, B, L, D, shift=2.0)
    w1, w2, w3, s = normal(q, D, shift=1.0, scale=0.1), normal(q, d, shift=1.0, scale=0.1), normal(q, D, shift=1.0, scale=0.1), normal(q, D, scale=0.5)
    heads = lambda t: t.view(B, L, H, d).transpose(1, 2).contiguous()  # noqa: E731
    # forward
    _, x1 = F.residual_norm(r, w1, 1e-5)
    qh = heads(x1)
    o, _ = F.fwd("F1", "recurrent", qh, k, v, beta, lam, eps)
    y = F.norm_gate(o, gate, w2, 1e-5)
    z, _, marks = F.scan(y, fg, want_marks=True)
    r2, h = F.residual_norm(r, w3, 1e-5, y=z, scale=s)
    # backward
    g4 = F.residual_norm_bwd(r2, w3, 1e-5, dtop, dr_out=dstream, y=z, scale=s)
    g3 = F.scan_bwd(y, fg, g4["dy"], marks=marks)
    g2 = F.norm_gate_bwd(o, gate, w2, 1e-5, g3["dx"])
    gf = F.bwd("F1", qh, k, v, beta, lam, eps, g2["do"])
    dx1 = gf["dq"].transpose(1, 2).reshape(B, L, D).contiguous()
    g1 = F.residual_norm_bwd(r, w1, 1e-5, dx1, dr_out=g4["dr"])
    # the same in fp64
    e64 = d0["eps_64"]
    f64 = (d0["k_64"], d0["v_64"], d0["beta_64"], d0["lam_64"], e64)
    X1 = ref.residual_norm(np64(r), None, None, np64(w1), 1e-5)[1][0]
    Q = np.ascontiguousarray(X1.reshape(B, L, H, d).transpose(0, 2, 1, 3))
    O, _ = oracle.fwd("F1", "recurrent", Q, *f64)
    Y = ref.norm_gate(O, np64(gate), np64(w2), 1e-5)[0]
    Z = ref.scan(Y, np64(fg))[0]
    R2, Hh = (t[0] for t in ref.residual_norm(np64(r), Z, np64(s), np64(w3), 1e-5))
    G4 = ref.residual_norm_bwd(R2, Z, np64(s), np64(w3), 1e-5, np64(dtop), np64(dstream))
    G3 = ref.scan_bwd(Y, np64(fg), G4["dy"][0])
    G2 = ref.norm_gate_bwd(O, np64(gate), np64(w2), 1e-5, G3["dx"][0])
    GF = oracle.bwd("F1", Q, *f64, np.ascontiguousarray(G2["do"][0]))
    G1 = ref.residual_norm_bwd(np64(r), None, None, np64(w1), 1e-5, GF["dq"].transpose(0, 2, 1, 3).reshape(B, L, D), G4["dr"][0])
    for name, a, b in (("h", h, Hh), ("r2", r2, R2), ("dscale", g4["dscale"], G4["dscale"][0]), ("df", g3["df"], G3["df"][0]),
                       ("dgate", g2["dgate"], G2["dgate"][0]), ("dw2", g2["dweight"], G2["dweight"][0]),
                       ("dbeta", gf["dbeta"], GF["dbeta"]), ("dk", gf["dk"], GF["dk"]), ("dr", g1["dr"], G1["dr"][0]),
                       ("dw1", g1["dweight"], G1["dweight"][0])):
        assert np.abs(np64(a) - b).max() <= 4e-4 * np.abs(b).max(), name
