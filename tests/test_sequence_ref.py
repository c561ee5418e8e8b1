"""The 64-bit definitions of the sequence operators: their gradients against
central differences, and simple cases by hand."""
import numpy as np
import pytest

import sequence_ref as ref

H = 1e-5  # differences at H and 2H, extrapolated: error about H^4 times the fifth derivative, and 1e-16 / H


def directional(f, args, grads, rng):
    """sum <grad, d> against differences of f along one random direction over all arguments."""
    ds = {k: rng.standard_normal(args[k].shape) for k in grads}

    def slope(step):
        up = f(**{k: v + step * ds[k] if k in ds else v for k, v in args.items()})
        down = f(**{k: v - step * ds[k] if k in ds else v for k, v in args.items()})
        return (up - down) / (2 * step)

    want = (4 * slope(H) - slope(2 * H)) / 3
    got = sum((grads[k] * ds[k]).sum() for k in grads)
    scale = sum((abs(grads[k]) * abs(ds[k])).sum() for k in grads)
    assert abs(got - want) <= 1e-7 * scale + 1e-9


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("rows,width", [(1, 4), (7, 4), (5, 1), (2, 3)])
def test_conv_gradient(rows, width, act):
    rng = np.random.default_rng(rows * 10 + width)
    ch = 3
    a = {"x": rng.standard_normal((rows, ch)), "w": rng.standard_normal((ch, width)),
         "b": rng.standard_normal(ch), "init": rng.standard_normal((width - 1, ch))}
    dy, df = rng.standard_normal((rows, ch)), rng.standard_normal((width - 1, ch))

    def loss(x, w, b, init):
        y, fin, _ = ref.conv(x, w, b, init, act)
        return (y * dy).sum() + (fin * df).sum()

    g, _ = ref.conv_grad(dy, **a, act=act, dfinal=df)
    directional(loss, a, dict(zip(("x", "w", "b", "init"), g)), rng)


@pytest.mark.parametrize("softplus", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,ch,groups,n", [(1, 2, 1, 1), (6, 4, 2, 3)])
def test_scan_gradient(rows, ch, groups, n, gated, softplus):
    rng = np.random.default_rng(rows + ch)
    a = {"u": rng.standard_normal((rows, ch)), "dt": rng.uniform(0.1, 0.9, (rows, ch)),
         "A": -rng.uniform(0.2, 2.0, (ch, n)), "B": rng.standard_normal((rows, groups, n)),
         "C": rng.standard_normal((rows, groups, n)), "D": rng.standard_normal(ch),
         "bias": rng.uniform(0, 0.1, ch), "init": rng.standard_normal((ch, n))}
    if gated:
        a["z"] = rng.standard_normal((rows, ch))
    dout, df = rng.standard_normal((rows, ch)), rng.standard_normal((ch, n))

    def loss(u, dt, A, B, C, D, bias, init, z=None):
        (y, fin), _ = ref.scan(u, dt, A, B, C, D, z, bias, softplus, init)
        return (y * dout).sum() + (fin * df).sum()

    g, _ = ref.scan_grad(dout, a["u"], a["dt"], a["A"], a["B"], a["C"], a["D"], a.get("z"), a["bias"], softplus,
                         a["init"], df)
    names = {"bias": "dt_bias", "init": "initial_state"}
    directional(loss, a, {k: g[names.get(k, k)] for k in a}, rng)


@pytest.mark.parametrize("form", ["plain", "before", "after"])
@pytest.mark.parametrize("groups", [1, 3])
def test_norm_gradient(form, groups):
    rng = np.random.default_rng(groups)
    a = {"v": rng.standard_normal((4, 6)), "w": rng.standard_normal(6)}
    if form != "plain":
        a["gate"] = rng.standard_normal((4, 6))
    dy, dsum = rng.standard_normal((4, 6)), rng.standard_normal((4, 6))

    def loss(v, w, gate=None):
        return (ref.norm(v, w, gate, form == "after", groups, 1e-5) * dy).sum() + (v * dsum).sum()

    g = ref.norm_grad(dy, a["v"], a["w"], a.get("gate"), form == "after", groups, 1e-5, dsum)
    grads = {"v": g["v"], "w": g["weight"]}
    if form != "plain":
        grads["gate"] = g["gate"]
    directional(loss, a, grads, rng)


def test_scan_of_one_state_is_the_linear_recurrence():
    """a = exp(delta A), b = delta u B: the recurrence h = a h + b read out by C = 1."""
    rng = np.random.default_rng(0)
    u, dt = rng.standard_normal((50, 1)), rng.uniform(0.1, 1, (50, 1))
    one = np.ones((50, 1, 1))
    (y, fin), _ = ref.scan(u, dt, -np.ones((1, 1)), one, one, np.zeros(1), None, np.zeros(1), False, np.zeros((1, 1)))
    h = 0.0
    for t in range(50):
        h = np.exp(-dt[t, 0]) * h + dt[t, 0] * u[t, 0]
        assert abs(y[t, 0] - h) < 1e-14
    assert fin[0, 0] == y[-1, 0]
