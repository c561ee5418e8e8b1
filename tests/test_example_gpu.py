"""The state space layer of examples/ trains, and generates token by token what it gives for a whole prompt."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from device_wide_prefix_gb300 import build as dwp_build  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_layer_trains_and_generates():
    dwp_build.build()
    import state_space_layer as example
    layer, first, last = example.train()
    assert last < 0.7 * first
    # two bf16 roundings of every intermediate differ at most: a few units of 2^-8 of the largest output
    assert example.generate(layer) < 8 * 2.0 ** -8
