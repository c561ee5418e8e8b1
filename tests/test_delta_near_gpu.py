"""How near the gated delta rule's results are to its 64-bit definition, head by
head in the relative 2-norm: bounds of the size of what is stated for them, not
of the largest that could be (test_delta_gpu)."""
import numpy as np
import pytest

import delta_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import device_wide_prefix_gb300 as dwp  # noqa: E402
from device_wide_prefix_gb300 import build as dwp_build  # noqa: E402
from test_delta_gpu import Case  # noqa: E402

# A rounding to a bf16 leaves at most 2^-9 of each value.  Beside it there are
# products of numbers in two bf16 pieces, which keep 16 bits each: 2^-17 of a
# term, in four products one after another and their sums, whose terms cancel by
# some factors of two.  2^-14 counts eight such terms in line.
PIECES = 2.0 ** -14
BF16 = 2.0 ** -9


@pytest.fixture(scope="module", autouse=True)
def lib():
    dwp_build.build()
    return dwp.load()


def far(got, want):
    got = got.detach().double().cpu().numpy().reshape(want.shape)
    return np.sqrt(((got - want) ** 2).sum() / (want ** 2).sum())


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
            assert far(out[b, :, h], want) <= BF16 + PIECES
