"""The layer norm on the GPU against its 64-bit definition, with the bar of the
other sequence operators (test_sequence_gpu): a type's rounding, and 2^-24 of
the terms' magnitudes for each f32 rounding on the way (64 for the statistics
and the products, one for each row or channel that a sum runs over).  The
output's terms are those of (v - mean) r weight + bias."""
import numpy as np
import pytest

import delta_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import device_wide_prefix_gb300 as dwp  # noqa: E402
from device_wide_prefix_gb300 import build as dwp_build  # noqa: E402
from test_sequence_gpu import Draw, TYPES, near  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def lib():
    dwp_build.build()
    return dwp.load()


def magnitude(v, w, b, groups, eps):
    by = v.reshape(v.shape[0], groups, v.shape[1] // groups)
    r = 1 / np.sqrt(by.var(-1, keepdims=True) + eps)
    return ((abs(by) + abs(by.mean(-1, keepdims=True))) * r).reshape(v.shape) * abs(w) + abs(b)


@pytest.mark.parametrize("dtype,residual", [("f32", None), ("f32", "f32"), ("bf16", None), ("bf16", "f32"), ("bf16", "bf16"),
                                            ("f16", "f32")])
@pytest.mark.parametrize("rows,channels,groups,pad", [
    (1, 1, 1, 0), (3, 7, 1, 0), (5, 64, 8, 0), (17, 96, 4, 4), (9, 256, 1, 0), (40, 1024, 8, 8), (3, 1032, 1, 0),
    (2, 4096, 1, 0), (2, 4100, 1, 2), (2, 8192, 1, 0), (1, 16384, 1, 0), (2, 16383, 1, 0), (700, 24, 3, 0), (0, 64, 2, 0)])
def test_layer_norm(rows, channels, groups, pad, dtype, residual):
    d = Draw(rows * 31 + channels, TYPES[dtype])
    x, xv = d.act(rows, channels, pad=pad)
    w, wv = d.f32(channels, lo=0.5, hi=1.5)
    b, bv = d.f32(channels)
    dy, dyv = d.act(rows, channels, pad=pad)
    res, v, dres, dresv = None, xv, None, np.zeros((rows, channels))
    if residual:
        R = TYPES[residual]
        res, rv = d.act(rows, channels, pad=pad, dtype=R)
        dres, dresv = d.act(rows, channels, pad=pad, dtype=R)
        v = rv + xv
    out, total = dwp.layer_norm(x, w, b, residual=res, groups=groups, eps=1e-3)
    if residual:
        near(total, v, abs(v), 2, "sum")
    # what is normed is the sum before it is rounded to be written
    near(out, ref.layer_norm(v, wv, bv, groups, 1e-3), magnitude(v, wv, bv, groups, 1e-3), 64 + channels // groups, "out")
    if residual:
        v = total.double().cpu().numpy()  # as the gradient gets it
    g = dwp.layer_norm_backward(dy, x if total is None else total, w, b, grad_residual=dres, groups=groups, eps=1e-3)
    G, M = ref.layer_norm_grad(dyv, v, wv, groups, 1e-3, dresv)
    r = 1 / np.sqrt(v.reshape(rows, groups, channels // groups).var(-1, keepdims=True) + 1e-3)
    mean = np.broadcast_to(abs(v.reshape(rows, groups, channels // groups)).mean(-1, keepdims=True) * r, (rows, groups, channels // groups))
    mean = mean.reshape(rows, channels)
    steps = 64 + channels // groups
    near(g["x"], G["v"], M["v"] * (1 + mean), steps, "dx")
    if residual:
        near(g["residual"], G["v"], M["v"] * (1 + mean), steps, "dresidual")
    near(g["weight"], G["weight"], M["weight"] + (abs(dyv) * mean).sum(0), steps + rows, "dweight")
    near(g["bias"], G["bias"], M["bias"], steps + rows, "dbias")


def test_without_parameters():
    d = Draw(3, torch.float32)
    x, xv = d.act(4, 40)
    dy, dyv = d.act(4, 40)
    one = np.ones(40)
    near(dwp.layer_norm(x)[0], ref.layer_norm(xv, one, 0 * one, 1, 1e-5), 1 + abs(xv) * 2, 128, "out")
    g = dwp.layer_norm_backward(dy, x)
    assert set(g) == {"x"}
    near(g["x"], ref.layer_norm_grad(dyv, xv, one, 1, 1e-5, 0 * xv)[0]["v"], 4 + abs(dyv) * 8, 128, "dx")


def test_mean_far_from_zero():
    """A mean 2^14 times the spread: squares about the mean, not differences of squares."""
    r = np.random.default_rng(5)
    x = torch.from_numpy(16384.0 + r.integers(-8, 9, (5, 520)) / 8).float().cuda()
    got = dwp.layer_norm(x)[0].double().cpu().numpy()
    want = ref.layer_norm(x.double().cpu().numpy(), 1.0, 0.0, 1, 1e-5)
    # the mean is within a few units of 2^-10 of its own, the spread about 0.6
    assert abs(got - want).max() < 2.0 ** -10 * 4
