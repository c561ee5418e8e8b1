"""The gated delta rule in a build with test hooks (-DDWP_DELTA_TEST=1): what
happens where no tensor map can be made."""
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import device_wide_prefix_gb300 as dwp  # noqa: E402
from device_wide_prefix_gb300 import build as dwp_build  # noqa: E402
from device_wide_prefix_gb300 import sequence as seq  # noqa: E402
from test_delta_edges_gpu import backward, forward  # noqa: E402
from test_delta_gpu import Case, check  # noqa: E402

HOOKS_LIB = os.path.join(os.path.dirname(dwp.__file__), "libdwp_delta_test.so")


@pytest.fixture(scope="module")
def hooked():
    dwp_build.build(extra=["-DDWP_DELTA_TEST=1"], lib=HOOKS_LIB)
    return dwp.load(HOOKS_LIB)


@pytest.fixture
def lib(hooked, monkeypatch):
    """The helpers on the build with hooks."""
    names = [n for n in dwp.EXPORTS if "delta" in n]
    monkeypatch.setattr(seq, "_ENTRY", {**seq._ENTRY, **{n: getattr(hooked, n) for n in names}})
    return hooked


@pytest.mark.parametrize("batch,rows,heads,keys,values", [(1, 1600, 1, 128, 128), (2, 100, 2, 64, 72), (1, 1550, 2, 16, 128)])
def test_without_tensor_maps(lib, batch, rows, heads, keys, values):
    """Rows are loaded without maps and sequences are not cut, however long they are: the call's result does not go by
    its length."""
    c = Case(40, (batch, rows), None, "bf16", 1, heads, keys, values, decay=0.05)
    lib.dwp_delta_test_no_maps(1)
    try:
        out, final, points = forward(c)
        grads = backward(c, points)
    finally:
        lib.dwp_delta_test_no_maps(0)
    check(c, out, final, grads)
