"""The plain forms of the layer operators (tests/layer_ref.py): their
gradients against central differences of their own forward in fp64."""
import numpy as np
import pytest

from tests import layer_ref as ref

# A central difference with step s of a smooth function has a truncation of
# s^2/6 of the third derivative (of the order of the values here) and a
# rounding of 2^-53/s of the values: with s = 1e-5 about 1e-11 of each; 1e-7 of
# the sum's terms leaves room for third derivatives of some hundred times the
# values.
STEP, TOL = 1e-5, 1e-7


def _differences(loss, args, grads, rng):
    for name, g in grads.items():
        v = rng.standard_normal(args[name].shape)
        up = loss({**args, name: args[name] + STEP * v})
        down = loss({**args, name: args[name] - STEP * v})
        assert abs((up - down) / (2 * STEP) - (g * v).sum()) <= TOL * (1 + np.abs(g * v).sum()), name


@pytest.mark.parametrize("reset", [False, True])
def test_scan_gradients(reset):
    rng = np.random.default_rng(1)
    N, L, D = 2, 9, 3
    args = dict(x=rng.standard_normal((N, L, D)), f=rng.standard_normal((N, L, D)), initial=rng.standard_normal((N, D)))
    marks = rng.random((N, L)) < 0.3 if reset else None
    do, ds = rng.standard_normal((N, L, D)), rng.standard_normal((N, D))

    def loss(a):
        h = ref.scan(a["x"], a["f"], marks, a["initial"])[0]
        return (h * do).sum() + (h[:, -1] * ds).sum()

    g = ref.scan_bwd(args["x"], args["f"], do, ds, marks, args["initial"])
    _differences(loss, args, {"x": g["dx"][0], "f": g["df"][0], "initial": g["dinitial"][0]}, rng)


@pytest.mark.parametrize("per_head", [False, True])
def test_norm_gate_gradients(per_head):
    rng = np.random.default_rng(2)
    B, H, L, d = 2, 3, 4, 5
    args = dict(o=rng.standard_normal((B, H, L, d)), gate=rng.standard_normal((B, L, H * d)),
                weight=rng.standard_normal((H, d) if per_head else (d,)))
    do = rng.standard_normal((B, L, H * d))
    g = ref.norm_gate_bwd(args["o"], args["gate"], args["weight"], 1e-3, do)
    _differences(lambda a: (ref.norm_gate(a["o"], a["gate"], a["weight"], 1e-3)[0] * do).sum(), args,
                 {"o": g["do"][0], "gate": g["dgate"][0], "weight": g["dweight"][0]}, rng)


def test_residual_norm_gradients():
    rng = np.random.default_rng(3)
    R, D = 4, 7
    args = dict(r=rng.standard_normal((R, D)), y=rng.standard_normal((R, D)), scale=rng.standard_normal(D),
                weight=rng.standard_normal(D))
    dh, dr = rng.standard_normal((R, D)), rng.standard_normal((R, D))

    def loss(a):
        (s, _), (h, _) = ref.residual_norm(a["r"], a["y"], a["scale"], a["weight"], 1e-3)
        return (s * dr).sum() + (h * dh).sum()

    s = ref.residual_norm(args["r"], args["y"], args["scale"], args["weight"], 1e-3)[0][0]
    g = ref.residual_norm_bwd(s, args["y"], args["scale"], args["weight"], 1e-3, dh, dr)
    _differences(loss, args, {"r": g["dr"][0], "y": g["dy"][0], "scale": g["dscale"][0], "weight": g["dweight"][0]}, rng)
