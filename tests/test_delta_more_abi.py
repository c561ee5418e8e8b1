"""More refusals of the gated delta rule's C entry points (test_delta_abi has
the rest): what is finite in 64 bits and not in the kernels' 32."""
import pytest

from test_delta_abi import DELTA, DELTA_BACKWARD, DELTA_STEP, FAR, delta_good
from test_sequence_abi import A, INVALID, call, lib, pytestmark  # noqa: F401


@pytest.mark.parametrize("scale", [1e39, -1e39, 3.5e38])
def test_scale_beyond_f32(scale):
    assert call("dwp_gated_delta_rule", DELTA, delta_good(), scale=scale) == INVALID
    assert call("dwp_gated_delta_rule_backward", DELTA_BACKWARD, delta_good(), scale=scale) == INVALID
    step = dict(delta_good(), num_slots=4, state=A + 20 * FAR, slot_stride=512, slots=A + 21 * FAR)
    assert call("dwp_gated_delta_rule_step", DELTA_STEP, step, scale=scale) == INVALID
