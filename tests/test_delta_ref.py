"""The 64-bit definitions of the gated delta rule and the layer norm: their
gradients against differences of the functions, and known small cases."""
import numpy as np
import pytest

import delta_ref as ref

STEP = 1e-5


def unit(x):
    return x / np.sqrt((x * x).sum(-1, keepdims=True))


def differences(f, x):
    """Central differences of the scalar f at each entry of x."""
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += STEP
        down[i] -= STEP
        out[i] = (f(up) - f(down)) / (2 * STEP)
    return out


@pytest.mark.parametrize("rows,keys,values", [(1, 3, 2), (6, 4, 3), (9, 2, 5)])
def test_delta_gradient(rows, keys, values):
    r = np.random.default_rng(rows)
    x = {"q": unit(r.standard_normal((rows, keys))), "k": unit(r.standard_normal((rows, keys))),
         "v": r.standard_normal((rows, values)), "g": -r.uniform(0, 1, rows), "beta": r.uniform(0, 1, rows),
         "initial_state": r.standard_normal((keys, values))}
    dout, dlast = r.standard_normal((rows, values)), r.standard_normal((keys, values))

    def loss(y):
        out, last, *_ = ref.delta(y["q"], y["k"], y["v"], y["g"], y["beta"], 0.7, y["initial_state"])
        return (out * dout).sum() + (last * dlast).sum()

    got, sizes = ref.delta_grad(dout, x["q"], x["k"], x["v"], x["g"], x["beta"], 0.7, x["initial_state"], dlast)
    for name in x:
        want = differences(lambda y: loss(dict(x, **{name: y})), x[name])
        assert np.abs(got[name] - want).max() < 1e-8, name
        assert (sizes[name] >= 0).all()


def test_delta_stores_and_replaces():
    """beta 1 and keys of length one: what is written under a key is read back, and replaced by the next."""
    k = np.eye(3)
    v = np.arange(9.0).reshape(3, 3) + 1
    out, S, *_ = ref.delta(k, k, v, np.zeros(3), np.ones(3), 1.0, np.zeros((3, 3)))
    assert (out == v).all() and (S == v).all()
    out, S, *_ = ref.delta(k[[0, 0]], k[[0, 0]], v[:2], np.zeros(2), np.ones(2), 1.0, np.zeros((3, 3)))
    assert (S[0] == v[1]).all() and (S[1:] == 0).all()


@pytest.mark.parametrize("groups", [1, 2])
def test_layer_norm_gradient(groups):
    r = np.random.default_rng(groups)
    v, w, b, dy, ds = (r.standard_normal(s) for s in ((3, 6), 6, 6, (3, 6), (3, 6)))

    def loss(v, w, b):
        return (ref.layer_norm(v, w, b, groups, 1e-3) * dy).sum() + (v * ds).sum()

    got, _ = ref.layer_norm_grad(dy, v, w, groups, 1e-3, ds)
    assert np.abs(got["v"] - differences(lambda x: loss(x, w, b), v)).max() < 1e-8
    assert np.abs(got["weight"] - differences(lambda x: loss(v, x, b), w)).max() < 1e-8
    assert np.abs(got["bias"] - differences(lambda x: loss(v, w, x), b)).max() < 1e-8
