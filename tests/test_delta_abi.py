"""Host-side refusals of the gated delta rule's and the layer norm's C entry
points (fake, never-dereferenced addresses), the sizes that include/dwp.h
states for them, and what their Python helpers refuse."""
import ctypes

import pytest

import device_wide_prefix_gb300 as dwp
from device_wide_prefix_gb300 import sequence as seq
from test_sequence_abi import A, ALIASING, INVALID, MB, MISALIGNED, ROWS3, SMALL, call, lib, pytestmark  # noqa: F401

HEADS4 = ("data", "batch_stride", "row_stride", "head_stride")
DELTA = ["dtype", "beta_dtype", "keys", "values", "key_heads", "heads", "batch", "rows", "num_segments", "scale",
         *("%s.%s" % (t, f) for t in ("q", "k", "v", "out") for f in HEADS4),
         *("%s.%s" % (t, f) for t in ("g", "beta") for f in ROWS3), "offsets", "initial", "final", "checkpoints"]
DELTA_BACKWARD = DELTA + ["grad_out." + f for f in HEADS4] + ["grad_final", "grad_q", "grad_k", "grad_v", "grad_g",
                                                            "grad_beta", "grad_initial"]
DELTA_STEP = ["dtype", "beta_dtype", "keys", "values", "key_heads", "heads", "batch", "num_slots", "scale",
              *("%s.%s" % (t, f) for t in ("q", "k", "v", "out") for f in HEADS4),
              *("%s.%s" % (t, f) for t in ("g", "beta") for f in ROWS3), "state", "slot_stride", "slots"]
LAYER_NORM = ["dtype", "weight_dtype", "residual_dtype", "channels", "groups", "rows", "eps",
              *("%s.%s" % (t, f) for t in ("x", "residual", "sum", "out") for f in ROWS3), "weight", "bias"]
LAYER_NORM_BACKWARD = LAYER_NORM + ["%s.%s" % (t, f) for t in ("grad_out", "grad_sum", "grad_x", "grad_residual")
                                    for f in ROWS3] + ["grad_weight", "grad_bias"]
FAR = 64 * MB


def delta_good():
    """2 x 100 rows, 2 key heads of 16, 4 heads of 8, f32."""
    g = {"dtype": 0, "beta_dtype": 0, "keys": 16, "values": 8, "key_heads": 2, "heads": 4, "batch": 2, "rows": 100,
         "scale": 0.25}
    for i, (k, heads, size) in enumerate((("q", 2, 16), ("k", 2, 16), ("v", 4, 8), ("out", 4, 8), ("grad_out", 4, 8))):
        g.update({k + ".data": A + i * FAR, k + ".batch_stride": 100 * heads * size, k + ".row_stride": heads * size,
                  k + ".head_stride": size})
    for i, k in enumerate(("g", "beta")):
        g.update({k + ".data": A + (6 + i) * FAR, k + ".batch_stride": 400, k + ".row_stride": 4})
    for i, k in enumerate(("initial", "final", "checkpoints", "grad_final", "grad_q", "grad_k", "grad_v", "grad_g",
                           "grad_beta", "grad_initial")):
        g[k] = A + (10 + i) * FAR
    return g


BOTH = [
    ({"dtype": 3}, INVALID), ({"dtype": -1}, INVALID), ({"beta_dtype": 2}, INVALID), ({"keys": 0}, INVALID),
    ({"keys": 129}, INVALID), ({"values": 0}, INVALID), ({"values": 129}, INVALID), ({"key_heads": 0}, INVALID),
    ({"key_heads": 3}, INVALID), ({"key_heads": 8}, INVALID), ({"heads": 2048, "key_heads": 2}, INVALID),
    ({"batch": -1}, INVALID), ({"rows": -1}, INVALID), ({"batch": 1 << 20, "rows": 1 << 20}, INVALID),
    ({"num_segments": 3}, INVALID), ({"scale": float("nan")}, INVALID), ({"scale": float("inf")}, INVALID),
    ({"q.data": 0}, INVALID), ({"k.data": 0}, INVALID), ({"v.data": 0}, INVALID), ({"beta.data": 0}, INVALID),
    ({"q.head_stride": 15}, INVALID), ({"k.row_stride": 31}, INVALID), ({"v.batch_stride": 3}, INVALID),
    ({"g.row_stride": 3}, INVALID), ({"v.head_stride": 1 << 60}, INVALID), ({"k.row_stride": -32}, INVALID),
    ({"offsets": A + 30 * FAR, "num_segments": 2}, INVALID),  # two batch entries
    ({"q.data": A + 2}, MISALIGNED), ({"g.data": A + 6 * FAR + 1}, MISALIGNED), ({"checkpoints": A + 12 * FAR + 4}, MISALIGNED),
    ({"initial": A + 10 * FAR + 2}, MISALIGNED), ({"offsets": A + 30 * FAR + 2, "num_segments": 2, "batch": 1}, MISALIGNED),
    ({"scratch": A + 4000 * MB + 8}, MISALIGNED)]


@pytest.mark.parametrize("change,status", BOTH)
def test_delta_refusals(change, status):
    assert call("dwp_gated_delta_rule", DELTA, delta_good(), **change) == status
    assert call("dwp_gated_delta_rule_backward", DELTA_BACKWARD, delta_good(), **change) == status


@pytest.mark.parametrize("change,status", [
    ({"out.data": 0}, INVALID), ({"out.data": A}, ALIASING), ({"out.data": A + 2 * FAR}, ALIASING),
    ({"final": A + 10 * FAR}, ALIASING), ({"checkpoints": A + 3 * FAR}, ALIASING), ({"out.data": A + 7 * FAR}, ALIASING),
    ({"out.batch_stride": 32}, INVALID),  # the entries' rows would fold
    ({"scratch": A + FAR}, ALIASING), ({"checkpoints": 0, "size": 100}, SMALL)])
def test_delta_forward_outputs(change, status):
    assert call("dwp_gated_delta_rule", DELTA, delta_good(), **change) == status


@pytest.mark.parametrize("change,status", [
    ({"checkpoints": 0}, INVALID), ({"grad_out.data": 0}, INVALID), ({"grad_q": 0}, INVALID), ({"grad_k": 0}, INVALID),
    ({"grad_v": 0}, INVALID), ({"grad_beta": 0}, INVALID), ({"g.data": 0}, INVALID), ({"grad_q": A}, ALIASING),
    ({"grad_v": A + 4 * FAR}, ALIASING), ({"grad_k": A + 14 * FAR + 64}, ALIASING), ({"grad_g": A + 6 * FAR}, ALIASING),
    ({"grad_initial": A + 13 * FAR}, ALIASING), ({"grad_beta": A + 12 * FAR}, ALIASING), ({"size": 1000}, SMALL)])
def test_delta_gradient_refusals(change, status):
    assert call("dwp_gated_delta_rule_backward", DELTA_BACKWARD, delta_good(), **change) == status


@pytest.mark.parametrize("change,status", [
    ({"keys": 129}, INVALID), ({"key_heads": 3}, INVALID), ({"beta_dtype": 1}, INVALID), ({"batch": -1}, INVALID),
    ({"num_slots": -1}, INVALID), ({"slots": 0, "num_slots": 1}, INVALID), ({"state": 0}, INVALID),
    ({"slot_stride": 511}, INVALID), ({"q.data": 0}, INVALID), ({"beta.data": 0}, INVALID), ({"out.data": A}, ALIASING),
    ({"state": A + 2 * FAR}, ALIASING), ({"state": A + 20 * FAR + 2}, MISALIGNED), ({"slots": A + 21 * FAR + 1}, MISALIGNED)])
def test_delta_step_refusals(change, status):
    good = delta_good()
    good.update(num_slots=4, state=A + 20 * FAR, slot_stride=512, slots=A + 21 * FAR)
    assert call("dwp_gated_delta_rule_step", DELTA_STEP, good, **change) == status


def norm_good():
    g = {"dtype": 0, "weight_dtype": 0, "residual_dtype": 0, "channels": 64, "groups": 2, "rows": 100, "eps": 1e-5}
    for i, k in enumerate(("x", "residual", "sum", "out", "grad_out", "grad_sum", "grad_x", "grad_residual")):
        g.update({k + ".data": A + i * MB, k + ".row_stride": 64})
    for i, k in enumerate(("weight", "bias", "grad_weight", "grad_bias")):
        g[k] = A + (20 + i) * MB
    return g


@pytest.mark.parametrize("change,status", [
    ({"dtype": 3}, INVALID), ({"dtype": 1, "weight_dtype": 2}, INVALID), ({"dtype": 1, "residual_dtype": 2}, INVALID),
    ({"groups": 3}, INVALID), ({"groups": 0}, INVALID), ({"channels": 1 << 16, "groups": 2}, INVALID),
    ({"eps": -1.0}, INVALID), ({"eps": float("nan")}, INVALID), ({"rows": 1 << 31}, INVALID),
    ({"weight": A + 20 * MB + 2}, MISALIGNED), ({"bias": A + 21 * MB + 1}, MISALIGNED)])
def test_layer_norm_refusals(change, status):
    assert call("dwp_layer_norm", LAYER_NORM, norm_good(), **change) == status
    assert call("dwp_layer_norm_backward", LAYER_NORM_BACKWARD, norm_good(), **change) == status


@pytest.mark.parametrize("change,status", [
    ({"x.data": 0}, INVALID), ({"sum.data": 0}, INVALID), ({"residual.data": 0}, INVALID), ({"x.row_stride": 60}, INVALID),
    ({"out.data": A + 4}, ALIASING), ({"sum.data": A}, ALIASING), ({"out.data": A + MB}, ALIASING),
    ({"out.data": A + 20 * MB}, ALIASING), ({"sum.data": A + MB, "sum.row_stride": 128}, ALIASING)])
def test_layer_norm_forward_refusals(change, status):
    assert call("dwp_layer_norm", LAYER_NORM, norm_good(), **change) == status


@pytest.mark.parametrize("change,status", [
    ({"grad_out.data": 0}, INVALID), ({"sum.data": 0}, INVALID), ({"sum.data": 0, "grad_sum.data": 0}, INVALID),
    ({"sum.data": 0, "grad_sum.data": 0, "grad_residual.data": 0, "dtype": 1, "weight_dtype": 1}, INVALID),
    ({"grad_x.data": A + 2 * MB}, ALIASING), ({"grad_residual.data": A + 4 * MB}, ALIASING),
    ({"grad_weight": A + 20 * MB}, ALIASING), ({"grad_bias": A + 22 * MB + 64}, ALIASING), ({"size": 64}, SMALL)])
def test_layer_norm_gradient_refusals(change, status):
    assert call("dwp_layer_norm_backward", LAYER_NORM_BACKWARD, norm_good(), **change) == status


def test_null_arguments():
    for name in ("dwp_gated_delta_rule", "dwp_gated_delta_rule_backward", "dwp_layer_norm_backward"):
        assert getattr(dwp.load(), name)(None, None, ctypes.byref(ctypes.c_size_t(0)), None) == INVALID
    for name in ("dwp_gated_delta_rule_step", "dwp_layer_norm"):
        assert getattr(dwp.load(), name)(None, None) == INVALID


def need(name, names, good, **change):
    f = dict(good, **change)
    return seq.scratch_bytes(name, seq._PACK[name](*(f.get(k, 0) for k in names)))


@pytest.mark.parametrize("batch,rows,segments", [(2, 100, 0), (1, 64, 0), (3, 1, 0), (1, 1000, 7), (1, 63, 1)])
@pytest.mark.parametrize("keys,values", [(16, 8), (65, 128), (128, 65)])
def test_sizes_as_stated(batch, rows, segments, keys, values):
    heads, up = 4, lambda n: -(-n // 64) * 64
    chunks = rows // 64 + segments if segments else batch * -(-rows // 64)
    places = chunks * heads
    change = dict(batch=batch, rows=rows, num_segments=segments, offsets=A + 40 * FAR if segments else 0, keys=keys,
                  values=values)
    for k, h, n in (("q", 2, keys), ("k", 2, keys), ("v", 4, values), ("out", 4, values), ("grad_out", 4, values)):
        change.update({k + ".batch_stride": rows * h * n, k + ".row_stride": h * n, k + ".head_stride": n})
    for k in ("g", "beta"):
        change.update({k + ".batch_stride": rows * 4})
    assert need("dwp_gated_delta_rule", DELTA, delta_good(), **change, checkpoints=0) == 8 * 64 * 64 * places
    assert need("dwp_gated_delta_rule", DELTA, delta_good(), **change) == 16
    want = 4 * (up(keys) * values + 64 * up(values)) * places
    assert need("dwp_gated_delta_rule_backward", DELTA_BACKWARD, delta_good(), **change) == want
    points = seq._delta_points(batch, rows, segments, True if segments else None, heads, keys, values)
    assert points == (chunks, heads, 64 * (2 * 64 + up(values)) + up(keys) * values)


def test_layer_norm_scratch():
    assert need("dwp_layer_norm_backward", LAYER_NORM_BACKWARD, norm_good(), grad_weight=0, grad_bias=0) == 16
    small, large = (need("dwp_layer_norm_backward", LAYER_NORM_BACKWARD, norm_good(), rows=n) for n in (1, 1 << 20))
    assert 2 * 64 * 4 <= small <= large <= 2 * 64 * 4 * 304
