"""The limits that include/dwp.h states for the sequence operators, on the host:
size queries and refusals, with fake, never-dereferenced addresses."""
import ctypes

import pytest

import device_wide_prefix_gb300 as dwp
import test_sequence_abi as abi
from device_wide_prefix_gb300 import build as dwp_build
from device_wide_prefix_gb300 import sequence as seq

pytestmark = abi.pytestmark

INVALID, ALIASING, SMALL = abi.INVALID, abi.ALIASING, abi.SMALL
A, MB = abi.A, abi.MB


@pytest.fixture(scope="module", autouse=True)
def lib():
    dwp_build.build()
    return dwp.load()


def query(name, names, good, **change):
    """(status, size) of a size query."""
    f = dict(good, **change)
    size = ctypes.c_size_t(0)
    status = getattr(dwp.load(), name)(seq._PACK[name](*(f.get(k, 0) for k in names)), None, ctypes.byref(size), None)
    return status, size.value


NO_ROWS = {k + ".data": 0 for k in ("x", "out", "u", "dt", "z", "B", "C", "residual", "gate", "sum", "grad_out", "grad_sum",
                                    "grad_x", "grad_residual", "grad_gate")}


@pytest.mark.parametrize("name,names,good,change", [
    # enough sequences that no rows are cut into chunks, and no offsets
    ("dwp_selective_scan", abi.SCAN, abi.scan_good, {"batch": 15, "rows": 1024, "channels": 4096, "groups": 1}),
    ("dwp_selective_scan", abi.SCAN, abi.scan_good, {"batch": 2, "rows": 16}),
    ("dwp_selective_scan", abi.SCAN, abi.scan_good, {"rows": 0}),
    ("dwp_selective_scan", abi.SCAN, abi.scan_good, {"batch": 0}),
    ("dwp_selective_scan_backward", abi.SCAN_BACKWARD, abi.scan_good, {"rows": 0}),
    ("dwp_causal_conv_backward", abi.CONV_BACKWARD, abi.conv_good, {"rows": 0}),
    ("dwp_causal_conv_backward", abi.CONV_BACKWARD, abi.conv_good, {"batch": 0}),
    ("dwp_block_norm_backward", abi.NORM_BACKWARD, abi.norm_good, {"rows": 0}),
])
def test_a_size_query_never_answers_zero(name, names, good, change):
    """A caller allocates what the query says: of 0 bytes that is NULL, and the second call another query."""
    if 0 in (change.get("rows"), change.get("batch")):
        change = dict(NO_ROWS, **change)
    good = good()
    if "channels" in change:  # dense rows of that many channels, apart from one another
        for i, k in enumerate(("u", "dt", "z", "out")):
            good.update({k + ".data": A + (100 + 200 * i) * MB, k + ".batch_stride": 1024 * 4096, k + ".row_stride": 4096})
        for i, k in enumerate(("B", "C")):
            good.update({k + ".batch_stride": 1024 * 32})
        good.update(final=A + 1000 * MB, initial=A + 1100 * MB, checkpoints=0)
    status, size = query(name, names, good, **change)
    assert status == dwp.DWP_SUCCESS and size >= 16 and size % 16 == 0
    assert abi.call(name, names, good, size=size - 1, **change) == SMALL
