"""The sequence operators at the edges of what they accept: segments that
begin at any row.  The bar and the helpers are test_sequence_gpu's."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import device_wide_prefix_gb300 as dwp  # noqa: E402
import test_sequence_gpu as base  # noqa: E402
from device_wide_prefix_gb300 import build as dwp_build  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def lib():
    dwp_build.build()
    return dwp.load()


# ---------------------------------------------------------------------------
# where a packed stream's first segment begins


@pytest.mark.parametrize("dtype,ch,width,pad", [("f32", 5, 4, 0), ("bf16", 264, 4, 0), ("f16", 33, 3, 2), ("f32", 8, 8, 4),
                                                ("bf16", 8, 2, 0), ("f32", 4, 1, 0)])
@pytest.mark.parametrize("rows,offsets", [(70, [4, 30]), (70, [8, 60]), (200, [68, 140]), (200, [64, 140]),
                                          (70, [8, 8, 60]), (70, [12, 14, 16, 70]), (140, [60, 64, 72])])
def test_conv_of_a_segment_that_begins_after_rows_outside(rows, offsets, dtype, ch, width, pad):
    """At every place within the rows that are loaded together, and at a strip's edge."""
    base.test_conv((rows,), offsets, dtype, ch, width, pad)
