"""Plain fp64 forms of the layer operators, with the rounding bounds their
tests use.  Independent of the kernels: loops over tokens for the recurrence,
torch autograd in fp64 for the norms.

Bounds.  U = 2^-24 is half a step of fp32 relative to the value.  A gate
formed in fp32 from f (an exponential whose argument is rounded once, a sum
and a quotient) is off by at most (|f| + 12) U of itself: |f| U from the
argument, 4 U from a 2-ulp exponential, the rest from the sum, the
reciprocal and the products.  An output stored in type t adds half a step of
it, eps(t)/2 of the value.
"""
import numpy as np
import torch

U = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def sigmoid(z):
    with np.errstate(over="ignore"):
        e = np.exp(-np.abs(z))
    return np.where(z < 0, e / (1 + e), 1 / (1 + e))


def scan(x, f, reset=None, initial=None, dtype=torch.float32, far=1.0):
    """h [N,L,D] and its fp32 bound before rounding.  The bound follows the
    recurrence: every step scales what is there by a and adds (|f|+12+4) U of
    the step's two terms in absolute value (their products and sum; the 4
    covers the products of a's formed over runs of tokens, one more rounding
    for each factor).  `far`: how many U of itself a gate is off per unit of |f|."""
    N, L, D = x.shape
    a, c = sigmoid(f), sigmoid(-f)
    h = np.zeros((N, L, D))
    bound = np.zeros((N, L, D))
    s = np.zeros((N, D)) if initial is None else initial.copy()
    mag, e = np.abs(s), np.zeros((N, D))
    before = np.zeros((N, L, D))
    ebefore = np.zeros((N, L, D))
    for t in range(L):
        r = np.zeros((N, 1), bool) if reset is None else reset[:, t, None].astype(bool)
        s, mag, e = np.where(r, 0, s), np.where(r, 0, mag), np.where(r, 0, e)
        before[:, t], ebefore[:, t] = s, e
        k = far * np.minimum(np.abs(f[:, t]), 100) + 16
        step = a[:, t] * mag + c[:, t] * np.abs(x[:, t])
        e = a[:, t] * e + k * U * step
        mag = step
        s = a[:, t] * s + c[:, t] * x[:, t]
        h[:, t], bound[:, t] = s, e
    return h, bound, before, ebefore


def scan_bwd(x, f, dout, dstate=None, reset=None, initial=None, far=1.0):
    """dx, df, dinitial, each with its fp32 bound before rounding."""
    N, L, D = x.shape
    _, _, before, ebefore = scan(x, f, reset, initial, far=far)
    a, c = sigmoid(f), sigmoid(-f)
    g = np.zeros((N, D)) if dstate is None else dstate.copy()
    mag, e = np.abs(g), np.zeros((N, D))
    dx, df, bx, bf = (np.zeros((N, L, D)) for _ in range(4))
    for t in range(L - 1, -1, -1):
        k = far * np.minimum(np.abs(f[:, t]), 100) + 16
        g = g + dout[:, t]
        mag = mag + np.abs(dout[:, t])
        e = e + U * mag
        ac = a[:, t] * c[:, t]
        dx[:, t] = g * c[:, t]
        bx[:, t] = c[:, t] * (e + k * U * mag)
        diff = before[:, t] - x[:, t]
        df[:, t] = g * diff * ac
        bf[:, t] = ac * (e * np.abs(diff) + np.abs(g) * ebefore[:, t] +
                         2 * k * U * mag * (np.abs(before[:, t]) + np.abs(x[:, t])))
        r = np.zeros((N, 1), bool) if reset is None else reset[:, t, None].astype(bool)
        e = np.where(r, 0, a[:, t] * (e + k * U * mag))
        mag = np.where(r, 0, a[:, t] * mag)
        g = np.where(r, 0, a[:, t] * g)
    return dict(dx=(dx, bx), df=(df, bf), dinitial=(g, e))


# The norms.  A sum of squares over a row is formed in runs of at most 64 terms
# and joined by a tree (at most 16 levels): 80 U of itself, 40 U in its root,
# with the reciprocal root (2 ulp) and two products 50 U in n.
ROW = 50


def norm_gate(o, gate, weight, eps):
    """out [B,L,H*d] with its fp32 bound."""
    B, H, L, d = o.shape
    v = np.mean(o * o, -1, keepdims=True) + eps
    n = o * np.where(v == 0, 0, 1 / np.sqrt(np.where(v == 0, 1, v)))
    if weight is not None:
        n = n * (weight[None, :, None, :] if weight.ndim == 2 else weight)
    out = n.transpose(0, 2, 1, 3).reshape(B, L, H * d)
    k = np.full_like(out, ROW + 4)
    if gate is not None:
        out = out * gate * sigmoid(gate)
        k = k + np.minimum(np.abs(gate), 100) + 16
    return out, k * U * np.abs(out)


def norm_gate_bwd(o, gate, weight, eps, dout):
    B, H, L, d = o.shape
    heads = lambda t: t.reshape(B, L, H, d).transpose(0, 2, 1, 3)  # noqa: E731
    flat = lambda t: t.transpose(0, 2, 1, 3).reshape(B, L, H * d)  # noqa: E731
    v = np.mean(o * o, -1, keepdims=True) + eps
    r = np.where(v == 0, 0, 1 / np.sqrt(np.where(v == 0, 1, v)))
    n = o * r
    dy = heads(dout)
    z = None if gate is None else heads(gate)
    s = None if gate is None else sigmoid(z)
    act = 1.0 if gate is None else z * s
    w = 1.0 if weight is None else (weight[None, :, None, :] if weight.ndim == 2 else weight)
    k = ROW + 20 + (0 if gate is None else np.minimum(np.abs(z), 100))
    e = dy * act
    dn = e * w
    dot = np.mean(dn * n, -1, keepdims=True)
    adot = np.mean(k * np.abs(dn * n), -1, keepdims=True)
    do = r * (dn - n * dot)
    # the mean's sum: the terms' own errors and 80 U of their magnitudes
    bdo = U * r * (k * np.abs(dn) + np.abs(n) * (adot + 80 * np.mean(np.abs(dn * n), -1, keepdims=True)) +
                   ROW * np.abs(n * dot) + ROW * np.abs(dn))
    got = dict(do=(do, bdo))
    if gate is not None:
        dg = dy * n * w * s * (1 + z * (1 - s))
        bdg = U * 2 * k * np.abs(dy * n * w) * s * (1 + np.abs(z) * (1 - s))
        got["dgate"] = flat(dg), flat(bdg)
    if weight is not None:
        axes = (0, 2) if weight.ndim == 2 else (0, 1, 2)
        terms = np.abs(e * n)
        count = B * L * (1 if weight.ndim == 2 else H)
        got["dweight"] = (e * n).sum(axes), U * ((2 * k + min(count, 4096)) * terms).sum(axes)
    return got


def residual_norm(r, y, scale, weight, eps):
    mag = np.abs(r)
    if y is not None:
        add = y if scale is None else scale * y
        r, mag = r + add, mag + np.abs(add)
    v = np.mean(r * r, -1, keepdims=True) + eps
    rstd = np.where(v == 0, 0, 1 / np.sqrt(np.where(v == 0, 1, v)))
    w = 1.0 if weight is None else weight
    # the sum's own rounding is 2 U of its terms' magnitudes; the root of the
    # mean square is off by no more than that of the whole row
    rowmag = np.sqrt(np.mean(mag * mag, -1, keepdims=True))
    b = U * np.abs(w) * rstd * (2 * mag + (ROW + 4) * np.abs(r) + 2 * np.abs(r) * rstd * rowmag)
    return (r, 2 * U * mag), (r * rstd * w, b)


def residual_norm_bwd(r, y, scale, weight, eps, dh, dr_out):
    v = np.mean(r * r, -1, keepdims=True) + eps
    rstd = np.where(v == 0, 0, 1 / np.sqrt(np.where(v == 0, 1, v)))
    n = r * rstd
    w = 1.0 if weight is None else weight
    e = dh * w
    dot = np.mean(e * n, -1, keepdims=True)
    t = rstd * (e - n * dot)
    b = U * rstd * ((ROW + 4) * np.abs(e) + (2 * ROW + 4) * np.abs(n * dot) +
                    np.abs(n) * (ROW + 84) * np.mean(np.abs(e * n), -1, keepdims=True))
    if dr_out is not None:
        t = t + dr_out
        b = b + U * np.abs(t)
    rows = int(np.prod(r.shape[:-1]))
    axes = tuple(range(r.ndim - 1))
    got = dict(dr=(t, b))
    if y is not None:
        got["dy"] = (t, b) if scale is None else (t * scale, np.abs(scale) * (b + U * np.abs(t)))
    if scale is not None:
        got["dscale"] = (t * y).sum(axes), (b * np.abs(y) + (min(rows, 4096) + 2) * U * np.abs(t * y)).sum(axes)
    if weight is not None:
        got["dweight"] = (dh * n).sum(axes), ((ROW + 2 + min(rows, 4096)) * U * np.abs(dh * n)).sum(axes)
    return got


def check(got, want, bound, dtype, name):
    """|got - want| <= bound + half a step of the stored type, element by element."""
    got = np64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    tol = bound + half(dtype) * (np.abs(want) + bound) + 1e-40
    off = np.abs(got - want)
    bad = ~(off <= tol)
    assert not bad.any(), "%s: %d of %d outside, the worst %.3g times its bound" % (
        name, bad.sum(), bad.size, float(np.nanmax(np.where(bad, off / tol, 0))))
