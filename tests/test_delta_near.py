"""The bounds of test_delta_near_gpu would notice: a gradient of zeros, a part of
a cut sequence that begins from a state of zeros, a start that is off by 2^-12,
forward and back, at the decays and sizes that are tested there."""
import numpy as np
import pytest

import delta_near as near
import delta_ref as ref

# rows, keys, values, decay: one head, as the cases there
CASES = [(1600, 128, 128, 0.01), (1027, 128, 128, 0.02), (500, 64, 24, 0.05)]


def inputs(rows, keys, values, decay):
    r = np.random.default_rng(rows)
    unit = lambda *s: (lambda x: 0.995 * x / np.sqrt((x * x).sum(-1, keepdims=True)))(r.standard_normal(s))  # noqa: E731
    return (r.standard_normal((rows, values)), unit(rows, keys), unit(rows, keys), r.standard_normal((rows, values)),
            -decay * np.abs(r.standard_normal(rows)), r.uniform(0, 1, rows), keys ** -0.5,
            0.3 * r.standard_normal((keys, values)), 0.1 * r.standard_normal((keys, values)))


def noticed(name, got, want):
    """Off by more than the bound, and in bf16 too (its own rounding is at most 2^-8)."""
    with pytest.raises(AssertionError):
        near.check(name, got, want, want)
    return any(near.far(got[w], want[w]) > 4 * (2.0 ** -8 + 2 * near.NEAR[name]) for w in near.windows(len(want)))


@pytest.mark.parametrize("rows,keys,values,decay", CASES)
def test_zeros_and_wrong_starts_are_noticed(rows, keys, values, decay):
    dout, q, k, v, g, beta, scale, s0, dlast = inputs(rows, keys, values, decay)
    out, *_ = ref.delta(q, k, v, g, beta, scale, s0)
    G, _ = ref.delta_grad(dout, q, k, v, g, beta, scale, s0, dlast)
    assert noticed("out", 0 * out, out)
    for name in ("q", "k", "v", "g", "beta"):
        assert noticed(name, 0 * G[name], G[name]), name
    cut = rows // near.CHUNK // 3 * near.CHUNK
    # a later part from zeros, and its walk back from zeros
    part = ref.delta(q[cut:], k[cut:], v[cut:], g[cut:], beta[cut:], scale, 0 * s0)[0]
    assert noticed("out", np.concatenate([out[:cut], part]), out)
    back, _ = ref.delta_grad(dout[:cut], q[:cut], k[:cut], v[:cut], g[:cut], beta[:cut], scale, s0, 0 * dlast)
    for name in ("k", "v", "g", "beta"):
        assert noticed(name, np.concatenate([back[name], G[name][cut:]]), G[name]), name


@pytest.mark.parametrize("rows,keys,values,decay", CASES)
def test_a_start_a_little_off_is_noticed(rows, keys, values, decay):
    """A state that is 2^-12 off, in f32."""
    dout, q, k, v, g, beta, scale, s0, dlast = inputs(rows, keys, values, decay)
    out, *_ = ref.delta(q, k, v, g, beta, scale, s0)
    cut = rows // near.CHUNK // 3 * near.CHUNK
    s1 = ref.delta(q[:cut], k[:cut], v[:cut], g[:cut], beta[:cut], scale, s0)[1]
    part = ref.delta(q[cut:], k[cut:], v[cut:], g[cut:], beta[cut:], scale, s1 * (1 + 2.0 ** -12))[0]
    got = np.concatenate([out[:cut], part])
    with pytest.raises(AssertionError):
        near.check("out", got, out, out)


def test_a_rounding_and_twice_the_error_bound_a_rounded_result():
    """|rnd(w + e) - w| <= |rnd(w) - w| + 2 |e|, number by number, for a grid of bf16's spacing."""
    r = np.random.default_rng(1)
    w, e = r.uniform(1, 2, 10000), r.uniform(-1, 1, 10000) * 2.0 ** -10
    rnd = lambda x: np.round(x * 128) / 128  # noqa: E731
    assert (np.abs(rnd(w + e) - w) <= np.abs(rnd(w) - w) + 2 * np.abs(e) + 1e-15).all()
