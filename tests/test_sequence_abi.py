"""Host-side refusals of the sequence operators' C entry points: bad arguments
are reported before any CUDA call (fake, never-dereferenced addresses)."""
import ctypes

import pytest

import device_wide_prefix_gb300 as dwp
from device_wide_prefix_gb300 import build as dwp_build
from device_wide_prefix_gb300 import sequence as seq

A = 0x7F0000000000  # a 16-byte aligned fake device address
MB = 1 << 20

# Every case below is refused on the host; a wrong expectation would hand a
# fake address to the CUDA runtime.
pytestmark = pytest.mark.skipif(
    __import__("torch").cuda.is_available(),
    reason="host-validation tests use fake device addresses; run them without a GPU")

INVALID, MISALIGNED, ALIASING, SMALL = (dwp.DWP_ERR_INVALID_VALUE, dwp.DWP_ERR_MISALIGNED, dwp.DWP_ERR_ALIASING,
                                        dwp.DWP_ERR_SCRATCH_TOO_SMALL)
ROWS3 = ("data", "batch_stride", "row_stride")
CONV = ["dtype", "weight_dtype", "silu", "width", "channels", "batch", "rows", "num_segments",
        *("x." + f for f in ROWS3), *("out." + f for f in ROWS3), "weight", "bias", "offsets", "initial", "final"]
SCAN = ["dtype", "softplus", "channels", "states", "groups", "batch", "rows", "num_segments",
        *("%s.%s" % (t, f) for t in ("u", "dt", "z", "B", "C", "out") for f in ROWS3), "b_group", "c_group", "A", "D",
        "dt_bias", "offsets", "initial", "final", "checkpoints"]
NORM = ["dtype", "weight_dtype", "residual_dtype", "gate_after", "channels", "groups", "rows", "eps",
        *("%s.%s" % (t, f) for t in ("x", "residual", "gate", "sum", "out") for f in ROWS3), "weight", "scale"]


@pytest.fixture(scope="module", autouse=True)
def lib():
    dwp_build.build()
    return dwp.load()


def call(name, names, good, scratch=A + 4000 * MB, size=1 << 40, **change):
    f = dict(good, **change)
    packed = seq._PACK[name](*(f.get(k, 0) for k in names))
    entry = getattr(dwp.load(), name)
    if name in seq._WITH_SCRATCH:
        return entry(packed, scratch, ctypes.byref(ctypes.c_size_t(size)), None)
    return entry(packed, None)


def conv_good():
    """2 x 100 rows of 64 f32 channels, width 4; addresses a few MB apart."""
    g = {"dtype": 0, "weight_dtype": 0, "silu": 1, "width": 4, "channels": 64, "batch": 2, "rows": 100}
    for i, k in enumerate(("x", "out", "grad_out", "grad_x")):
        g.update({k + ".data": A + i * MB, k + ".batch_stride": 6400, k + ".row_stride": 64})
    for i, k in enumerate(("weight", "bias", "initial", "final", "grad_final", "grad_weight", "grad_bias", "grad_initial")):
        g[k] = A + (10 + i) * MB
    return g


CONV_BACKWARD = CONV + ["%s.%s" % (t, f) for t in ("grad_out", "grad_x") for f in ROWS3] + [
    "grad_final", "grad_weight", "grad_bias", "grad_initial"]


@pytest.mark.parametrize("change,status", [
    ({"dtype": 3}, INVALID), ({"dtype": -1}, INVALID), ({"dtype": 1, "weight_dtype": 2}, INVALID), ({"width": 0}, INVALID),
    ({"width": 9}, INVALID), ({"silu": 2}, INVALID), ({"channels": 0}, INVALID), ({"channels": 1 << 18}, INVALID),
    ({"batch": -1}, INVALID), ({"rows": -1}, INVALID), ({"batch": 1 << 20, "rows": 1 << 20}, INVALID),
    ({"batch": 1 << 62, "rows": 4}, INVALID), ({"num_segments": 3}, INVALID), ({"x.data": 0}, INVALID),
    ({"weight": 0}, INVALID), ({"x.row_stride": 63}, INVALID), ({"x.batch_stride": 10}, INVALID),
    ({"x.row_stride": 1 << 60}, INVALID), ({"offsets": A + 30 * MB, "num_segments": 2}, INVALID),  # two batch entries
    ({"x.data": A + 2}, MISALIGNED), ({"weight": A + 10 * MB + 1}, MISALIGNED), ({"initial": A + 12 * MB + 2}, MISALIGNED),
    ({"offsets": A + 30 * MB + 2, "num_segments": 2, "batch": 1}, MISALIGNED)])
def test_conv_refusals(change, status):
    assert call("dwp_causal_conv", CONV, conv_good(), **change) == status
    assert call("dwp_causal_conv_backward", CONV_BACKWARD, conv_good(), **change) == status


@pytest.mark.parametrize("change,status", [
    ({"out.data": A}, ALIASING), ({"out.data": A + 4}, ALIASING), ({"final": A + 12 * MB}, ALIASING),
    ({"out.data": A + 10 * MB}, ALIASING), ({"out.batch_stride": 64}, INVALID),  # the entries' rows would fold
    ({"out.data": A + 200, "x.row_stride": 128, "x.batch_stride": 12800, "out.row_stride": 128,
      "out.batch_stride": 12800}, ALIASING)])
def test_conv_forward_outputs(change, status):
    assert call("dwp_causal_conv", CONV, conv_good(), **change) == status


@pytest.mark.parametrize("change,status", [
    ({"grad_out.data": 0}, INVALID), ({"grad_x.data": 0}, INVALID), ({"grad_weight": 0}, INVALID),
    ({"grad_x.data": A + 2 * MB}, ALIASING), ({"grad_bias": A + 15 * MB}, ALIASING), ({"grad_initial": A}, ALIASING),
    ({"scratch": A + 64}, ALIASING), ({"scratch": A + 4000 * MB + 8}, MISALIGNED), ({"size": 100}, SMALL)])
def test_conv_gradient_refusals(change, status):
    assert call("dwp_causal_conv_backward", CONV_BACKWARD, conv_good(), **change) == status


CONV_STEP = ["dtype", "weight_dtype", "silu", "width", "channels", "batch", "num_slots",
             *("%s.%s" % (t, f) for t in ("x", "out") for f in ROWS3), "weight", "bias", "state", "slot_stride", "slots"]


@pytest.mark.parametrize("change,status", [
    ({"dtype": 5}, INVALID), ({"width": 9}, INVALID), ({"batch": -1}, INVALID), ({"num_slots": -1}, INVALID),
    ({"slots": 0, "num_slots": 1}, INVALID), ({"state": 0}, INVALID), ({"slot_stride": 100}, INVALID),
    ({"x.data": 0}, INVALID), ({"out.data": A}, ALIASING), ({"state": A}, ALIASING), ({"slots": A + 20 * MB + 2}, MISALIGNED),
    ({"state": A + 12 * MB + 1}, MISALIGNED), ({"weight": A + 12 * MB}, ALIASING)])
def test_conv_step_refusals(change, status):
    good = conv_good()
    good.update(batch=2, num_slots=4, state=A + 12 * MB, slot_stride=192, slots=A + 20 * MB)
    assert call("dwp_causal_conv_step", CONV_STEP, good, **change) == status


def scan_good():
    """2 x 100 rows of 64 f32 channels, 16 states in 2 groups."""
    g = {"dtype": 0, "softplus": 1, "channels": 64, "states": 16, "groups": 2, "batch": 2, "rows": 100, "b_group": 16,
         "c_group": 16}
    for i, k in enumerate(("u", "dt", "z", "out", "grad_out")):
        g.update({k + ".data": A + i * MB, k + ".batch_stride": 6400, k + ".row_stride": 64})
    for i, k in enumerate(("B", "C")):
        g.update({k + ".data": A + (6 + i) * MB, k + ".batch_stride": 3200, k + ".row_stride": 32})
    for i, k in enumerate(("A", "D", "dt_bias", "initial", "final", "checkpoints", "grad_final", "grad_u", "grad_dt",
                           "grad_z", "grad_B", "grad_C", "grad_A", "grad_D", "grad_dt_bias", "grad_initial")):
        g[k] = A + (10 + i) * MB
    return g


SCAN_BACKWARD = SCAN + ["grad_out." + f for f in ROWS3] + ["grad_final", "grad_u", "grad_dt", "grad_z", "grad_B",
                                                          "grad_C", "grad_A", "grad_D", "grad_dt_bias", "grad_initial"]
SCAN_STEP = ["dtype", "softplus", "channels", "states", "groups", "batch", "num_slots",
             *("%s.%s" % (t, f) for t in ("u", "dt", "z", "B", "C", "out") for f in ROWS3), "b_group", "c_group", "A", "D",
             "dt_bias", "state", "slot_stride", "slots"]


@pytest.mark.parametrize("change,status", [
    ({"dtype": 7}, INVALID), ({"softplus": 2}, INVALID), ({"states": 0}, INVALID), ({"states": 129}, INVALID),
    ({"groups": 0}, INVALID), ({"groups": 3}, INVALID), ({"channels": 1 << 20}, INVALID), ({"A": 0}, INVALID),
    ({"u.data": 0}, INVALID), ({"B.data": 0}, INVALID), ({"b_group": 8}, INVALID), ({"B.row_stride": 20}, INVALID),
    ({"dt.row_stride": 1}, INVALID), ({"num_segments": 1}, INVALID), ({"C.data": A + 7 * MB + 2}, MISALIGNED),
    ({"A": A + 10 * MB + 2}, MISALIGNED), ({"checkpoints": A + 15 * MB + 2}, MISALIGNED), ({"scratch": A + 4000 * MB + 4},
                                                                                       MISALIGNED)])
def test_scan_refusals(change, status):
    assert call("dwp_selective_scan", SCAN, scan_good(), **change) == status
    assert call("dwp_selective_scan_backward", SCAN_BACKWARD, scan_good(), **change) == status


@pytest.mark.parametrize("change,status", [
    ({"out.data": A}, ALIASING), ({"out.data": A + MB}, ALIASING), ({"final": A + 13 * MB}, ALIASING),
    ({"checkpoints": A + 14 * MB}, ALIASING), ({"out.data": 0}, INVALID)])
def test_scan_forward_outputs(change, status):
    assert call("dwp_selective_scan", SCAN, scan_good(), **change) == status


@pytest.mark.parametrize("change,status", [
    ({"checkpoints": 0}, INVALID), ({"grad_out.data": 0}, INVALID), ({"grad_u": 0}, INVALID), ({"grad_z": 0}, INVALID),
    ({"z.data": 0}, INVALID), ({"grad_A": 0}, INVALID), ({"grad_B": A + 21 * MB}, ALIASING),
    ({"grad_u": A + 4 * MB}, ALIASING), ({"grad_initial": A + 16 * MB}, ALIASING), ({"size": 1000}, SMALL)])
def test_scan_gradient_refusals(change, status):
    assert call("dwp_selective_scan_backward", SCAN_BACKWARD, scan_good(), **change) == status


@pytest.mark.parametrize("change,status", [
    ({"states": 129}, INVALID), ({"groups": 5}, INVALID), ({"state": 0}, INVALID), ({"slot_stride": 1000}, INVALID),
    ({"slots": 0, "num_slots": 1}, INVALID), ({"B.data": 0}, INVALID), ({"out.data": A}, ALIASING),
    ({"state": A + 10 * MB}, ALIASING), ({"state": A + 30 * MB + 2}, MISALIGNED), ({"batch": 1 << 40}, INVALID)])
def test_scan_step_refusals(change, status):
    good = scan_good()
    good.update(num_slots=4, state=A + 30 * MB, slot_stride=1024, slots=A + 31 * MB)
    assert call("dwp_selective_scan_step", SCAN_STEP, good, **change) == status


def norm_good():
    g = {"dtype": 0, "weight_dtype": 0, "channels": 64, "groups": 2, "rows": 100, "eps": 1e-5}
    for i, k in enumerate(("x", "residual", "gate", "sum", "out", "grad_out", "grad_sum", "grad_x", "grad_residual",
                           "grad_gate")):
        g.update({k + ".data": A + i * MB, k + ".row_stride": 64})
    for i, k in enumerate(("weight", "scale", "grad_weight", "grad_scale")):
        g[k] = A + (20 + i) * MB
    return g


NORM_BACKWARD = NORM + ["%s.%s" % (t, f) for t in ("grad_out", "grad_sum", "grad_x", "grad_residual", "grad_gate")
                        for f in ROWS3] + ["grad_weight", "grad_scale"]


@pytest.mark.parametrize("change,status", [
    ({"dtype": 3}, INVALID), ({"dtype": 1, "weight_dtype": 2}, INVALID), ({"dtype": 1, "residual_dtype": 2}, INVALID),
    ({"gate_after": 2}, INVALID), ({"groups": 3}, INVALID), ({"groups": 0}, INVALID), ({"channels": 1 << 16, "groups": 2},
                                                                                      INVALID),
    ({"eps": -1.0}, INVALID), ({"eps": float("nan")}, INVALID), ({"rows": 1 << 31}, INVALID), ({"weight": 0}, INVALID),
    ({"weight": A + 20 * MB + 2}, MISALIGNED)])
def test_norm_refusals(change, status):
    assert call("dwp_block_norm", NORM, norm_good(), **change) == status
    assert call("dwp_block_norm_backward", NORM_BACKWARD, norm_good(), **change) == status


@pytest.mark.parametrize("change,status", [
    ({"x.data": 0}, INVALID), ({"sum.data": 0}, INVALID), ({"residual.data": 0, "sum.data": 0}, INVALID),
    ({"x.row_stride": 60}, INVALID), ({"out.data": A + 4}, ALIASING), ({"sum.data": A}, ALIASING),
    ({"out.data": A + 2 * MB}, ALIASING), ({"sum.data": A + 4 * MB}, ALIASING), ({"out.data": A + 20 * MB}, ALIASING),
    ({"sum.data": A + MB, "sum.row_stride": 128}, ALIASING)])
def test_norm_forward_refusals(change, status):
    assert call("dwp_block_norm", NORM, norm_good(), **change) == status


@pytest.mark.parametrize("change,status", [
    ({"grad_scale": 0}, INVALID), ({"sum.data": 0}, INVALID), ({"grad_gate.data": 0}, INVALID),
    ({"gate.data": 0}, INVALID), ({"grad_out.data": 0}, INVALID), ({"grad_x.data": A + 5 * MB}, ALIASING),
    ({"grad_residual.data": A + 7 * MB}, ALIASING), ({"grad_weight": A + 20 * MB}, ALIASING), ({"size": 64}, SMALL)])
def test_norm_gradient_refusals(change, status):
    assert call("dwp_block_norm_backward", NORM_BACKWARD, norm_good(), **change) == status


def test_null_arguments():
    lib = dwp.load()
    for name in seq._PACK:
        if name in seq._WITH_SCRATCH:
            assert getattr(lib, name)(None, None, ctypes.byref(ctypes.c_size_t(0)), None) == INVALID
        else:
            assert getattr(lib, name)(None, None) == INVALID


def test_size_queries_grow_with_the_work():
    def need(name, names, good, **change):
        f = dict(good, **change)
        return seq.scratch_bytes(name, seq._PACK[name](*(f.get(k, 0) for k in names)))

    for name, names, good in (("dwp_causal_conv_backward", CONV_BACKWARD, conv_good()),
                              ("dwp_selective_scan_backward", SCAN_BACKWARD, scan_good()),
                              ("dwp_block_norm_backward", NORM_BACKWARD, norm_good())):
        small, large = need(name, names, good, rows=1), need(name, names, good, rows=100)
        assert 0 < small <= large and small % 16 == 0 and large % 16 == 0
    packed = dict(batch=1, offsets=A + 40 * MB, num_segments=3)
    assert need("dwp_selective_scan", SCAN, scan_good(), **packed) >= 400
