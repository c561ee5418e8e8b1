"""Kernels and types that a user's call reaches beside the small ones of
test_delta_gpu and test_layer_norm_gpu: calls of more blocks than the GPU has
SMs (where the chunks' inverses take one team a block), strengths in the
activations' type, the token form without decay, and a norm's weight and bias
in the activations' type or alone."""
import numpy as np
import pytest

import delta_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import device_wide_prefix_gb300 as dwp  # noqa: E402
from device_wide_prefix_gb300 import build as dwp_build  # noqa: E402
from test_delta_edges_gpu import backward, forward  # noqa: E402
from test_delta_gpu import Case, check, rows_near  # noqa: E402
from test_layer_norm_gpu import magnitude  # noqa: E402
from test_sequence_gpu import TYPES, Draw, near  # noqa: E402

SMS = 152


@pytest.fixture(scope="module", autouse=True)
def lib():
    dwp_build.build()
    return dwp.load()


@pytest.mark.parametrize("dtype,batch,rows,key_heads,heads,keys,values", [
    ("bf16", 29, 100, 8, 16, 128, 16), ("bf16", 58, 64, 8, 24, 24, 32), ("f16", 29, 70, 8, 16, 64, 16), ("bf16", 160, 1, 3, 3, 128, 128)])
def test_more_blocks_than_sms(dtype, batch, rows, key_heads, heads, keys, values):
    """The first two batch entries against the definition; every entry, forward and back, against calls of a few
    entries each, which have few blocks."""
    assert batch * -(-rows // 64) * key_heads > 3 * SMS and batch * heads > SMS
    c = Case(50, (batch, rows), None, dtype, key_heads, heads, keys, values)
    out, final, points = forward(c)
    grads = backward(c, points)
    names = ("q", "k", "v", "g", "beta", "grad", "state", "grad_state")
    few = Case(50, (1, 1), None, dtype, key_heads, heads, keys, values)
    for lo in (*range(0, batch - 2, 2), batch - 2):
        for n in names:
            setattr(few, n, getattr(c, n)[lo:lo + 2].contiguous())
        want = forward(few)
        assert torch.equal(out[lo:lo + 2], want[0]) and torch.equal(final[lo:lo + 2], want[1])
        back = backward(few, want[2])
        assert all(torch.equal(grads[n][lo:lo + 2], back[n]) for n in back)
        if lo == 0:
            few.lead, few.values = (2, rows), {n: c.values[n][:2] for n in names}
            check(few, want[0], want[1], back)


def test_more_blocks_than_sms_of_packed_rows():
    """60 segments, some empty, some of one row: against the same segments in calls of their own."""
    lengths = [(37 * i) % 90 if i % 7 else i % 2 for i in range(60)]
    cuts = np.cumsum([0, *lengths]).tolist()
    c = Case(51, (cuts[-1],), cuts, "bf16", 8, 16, 64, 32)
    assert (cuts[-1] // 64 + 60) * 8 > 3 * SMS
    out, final, points = forward(c)
    grads = backward(c, points)
    one = Case(51, (1,), [0, 1], "bf16", 8, 16, 64, 32)
    for i, (lo, hi) in enumerate(zip(cuts[:-1], cuts[1:])):
        for n in ("q", "k", "v", "g", "beta", "grad"):
            setattr(one, n, getattr(c, n)[lo:hi].contiguous())
        one.state, one.grad_state, one.offsets = c.state[i:i + 1], c.grad_state[i:i + 1], [0, hi - lo]
        want = forward(one)
        assert torch.equal(out[lo:hi], want[0]) and torch.equal(final[i:i + 1], want[1]), i
        back = backward(one, want[2])
        for n in back:
            part = grads[n][i:i + 1] if n == "initial_state" else grads[n][lo:hi]
            assert torch.equal(part, back[n]), (i, n)


@pytest.mark.parametrize("dtype,pad", [("bf16", 0), ("bf16", 1), ("f16", 0)])
def test_strengths_of_the_activations_type(dtype, pad):
    c = Case(52, (2, 130), None, dtype, 1, 2, 64, 40, pad, beta_dtype=dtype)
    out, final, points = forward(c)
    grads = backward(c, points)
    assert grads["beta"].dtype == c.T
    check(c, out, final, grads)


@pytest.mark.parametrize("decay", [True, False])
@pytest.mark.parametrize("dtype,beta_dtype,keys,values", [("bf16", "bf16", 128, 128), ("f16", "f16", 40, 30), ("f32", "f32", 64, 64),
                                                         ("bf16", "f32", 16, 7)])
def test_token_form_types(dtype, beta_dtype, keys, values, decay):
    """Strengths of either type, with decays and without."""
    batch, heads = 6, 4
    c = Case(53, (batch,), None, dtype, 2, heads, keys, values, beta_dtype=beta_dtype, count=batch)
    if not decay:
        c.values["g"][:] = 0.0
    cache = c.state.clone()
    out = dwp.gated_delta_rule_step(c.q, c.k, c.v, c.g if decay else None, c.beta, cache, scale=c.scale)
    for i in range(batch):
        for h in range(heads):
            o, last, sizes, size, _ = ref.delta(*c.head(slice(i, i + 1), h), c.scale, c.values["state"][i, h])
            rows_near(out[i:i + 1, h], o, sizes, "out")
            rows_near(cache[i, h].flatten(), last.flatten(), size, "state")


@pytest.mark.parametrize("given", ["both", "weight", "bias"])
@pytest.mark.parametrize("dtype,params,residual", [("bf16", "bf16", None), ("bf16", "bf16", "f32"), ("f16", "f16", None), ("f16", "f16", "f16"),
                                                   ("f16", "f32", None), ("bf16", "f32", "bf16"), ("f32", "f32", None)])
@pytest.mark.parametrize("rows,channels,groups,pad", [(3, 7, 1, 0), (17, 96, 4, 4), (40, 1024, 8, 8), (2, 4100, 1, 2), (3, 8192, 1, 0)])
def test_layer_norm_parameters(rows, channels, groups, pad, dtype, params, residual, given):
    """Weight and bias of either type, both or one of them."""
    d = Draw(rows * 37 + channels, TYPES[dtype])
    x, xv = d.act(rows, channels, pad=pad)
    dy, dyv = d.act(rows, channels, pad=pad)
    w, wv = d.act(channels, dtype=TYPES[params]) if given != "bias" else (None, np.ones(channels))
    b, bv = d.act(channels, dtype=TYPES[params]) if given != "weight" else (None, np.zeros(channels))
    res, v = None, xv
    if residual:
        res, rv = d.act(rows, channels, pad=pad, dtype=TYPES[residual])
        v = rv + xv
    out, total = dwp.layer_norm(x, w, b, residual=res, groups=groups, eps=1e-3)
    near(out, ref.layer_norm(v, wv, bv, groups, 1e-3), magnitude(v, wv, bv, groups, 1e-3), 64 + channels // groups, "out")
    if residual:
        v = total.double().cpu().numpy()
    g = dwp.layer_norm_backward(dy, x if total is None else total, w, b, groups=groups, eps=1e-3, residual=residual is not None)
    assert set(g) == {"x"} | ({"weight"} if w is not None else set()) | ({"bias"} if b is not None else set()) | (
        {"residual"} if residual else set())
    G, M = ref.layer_norm_grad(dyv, v, wv, groups, 1e-3, np.zeros((rows, channels)))
    r = 1 / np.sqrt(v.reshape(rows, groups, channels // groups).var(-1, keepdims=True) + 1e-3)
    mean = np.repeat(abs(v.reshape(rows, groups, channels // groups)).mean(-1) * r[..., 0], channels // groups, 1)
    steps = 64 + channels // groups
    near(g["x"], G["v"], M["v"] * (1 + mean), steps, "dx")
    if residual:
        near(g["residual"], G["v"], M["v"] * (1 + mean), steps, "dresidual")
    if w is not None:
        assert g["weight"].dtype == torch.float32
        near(g["weight"], G["weight"], M["weight"] + (abs(dyv) * mean).sum(0), steps + rows, "dweight")
    if b is not None:
        near(g["bias"], G["bias"], M["bias"], steps + rows, "dbias")
