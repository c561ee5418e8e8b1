"""How near the gated delta rule's results are to its 64-bit definition, head by
head in the relative 2-norm: bounds of the size of what is stated for them
(delta_near, whose bounds are themselves tested in test_delta_near), not of the
largest that could be (test_delta_gpu)."""
import numpy as np
import pytest

import delta_near as near
import delta_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import device_wide_prefix_gb300 as dwp  # noqa: E402
from device_wide_prefix_gb300 import build as dwp_build  # noqa: E402
from test_delta_edges_gpu import backward, forward  # noqa: E402
from test_delta_gpu import Case  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def lib():
    dwp_build.build()
    return dwp.load()


def check(name, got, want, by_rows=True):
    rounded = torch.from_numpy(want).to(got.dtype).double().numpy()
    if got.dtype == torch.float32:
        rounded = want
    near.check(name, got.detach().double().cpu().numpy().reshape(want.shape), want, rounded, by_rows)


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("batch,rows,key_heads,heads,keys,values,pad", [
    (1, 300, 1, 2, 128, 128, 0), (2, 200, 2, 2, 64, 64, 0), (1, 200, 1, 1, 16, 24, 0), (1, 130, 1, 2, 128, 72, 1),
    (1, 1600, 1, 1, 128, 128, 0)])
def test_bf16_outputs_are_off_by_their_own_rounding(batch, rows, key_heads, heads, keys, values, pad, keep):
    """Forward alone, and with what the gradient needs kept: the weights q.k are not rounded to bf16 before the sum."""
    c = Case(31, (batch, rows), None, "bf16", key_heads, heads, keys, values, pad, decay=0.1)
    got = dwp.gated_delta_rule(*c.args(), scale=c.scale, initial_state=c.state, return_checkpoints=keep)
    out = got[0] if keep else got
    for b in range(batch):
        for h in range(heads):
            want = ref.delta(*c.head(slice(b * rows, (b + 1) * rows), h), c.scale, c.values["state"][b, h])[0]
            check("out", out[b, :, h], want)


@pytest.mark.parametrize("dtype,batch,rows,key_heads,heads,keys,values,pad,decay", [
    ("bf16", 1, 1027, 1, 1, 128, 128, 0, 0.02), ("f32", 1, 640, 1, 2, 128, 128, 0, 0.02), ("f16", 2, 500, 1, 2, 64, 24, 0, 0.05),
    ("f32", 1, 300, 2, 4, 16, 16, 0, 0.1), ("bf16", 1, 300, 1, 3, 40, 72, 1, 0.1), ("f16", 1, 260, 1, 1, 128, 128, 3, 1.0),
    # cut in parts, forward and back
    ("bf16", 1, 1600, 1, 1, 128, 128, 0, 0.01), ("bf16", 2, 2049, 1, 2, 64, 128, 0, 0.01), ("bf16", 1, 1984, 2, 2, 16, 16, 0, 0.01)])
def test_every_result_of_many_chunks(dtype, batch, rows, key_heads, heads, keys, values, pad, decay):
    """Outputs, states and gradients of each head, as a whole and chunk by chunk."""
    c = Case(32, (batch, rows), None, dtype, key_heads, heads, keys, values, pad, decay=decay)
    out, final, points = forward(c)
    grads = backward(c, points)
    for b in range(batch):
        span = slice(b * rows, (b + 1) * rows)
        shared = {n: np.zeros((rows, key_heads, keys)) for n in ("q", "k")}
        for h in range(heads):
            x, s0 = c.head(span, h), c.values["state"][b, h]
            want, last, *_ = ref.delta(*x, c.scale, s0)
            check("out", out[b, :, h], want)
            check("final", final[b, h], last, False)
            G, _ = ref.delta_grad(c.grad_of(span, h), *x, c.scale, s0, c.values["grad_state"][b, h])
            for n in ("v", "g", "beta"):
                check(n, grads[n][b, :, h], G[n])
            check("initial_state", grads["initial_state"][b, h], G["initial_state"], False)
            for n in ("q", "k"):
                shared[n][:, h // c.per] += G[n]
        for n in ("q", "k"):
            for kh in range(key_heads):
                check(n, grads[n][b, :, kh], shared[n][:, kh])
