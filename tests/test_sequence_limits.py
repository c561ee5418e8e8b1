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


def halves(rows, batch, *, row, step):
    """x and out as the two halves of one tensor of 2 x 64 channels."""
    return {"batch": batch, "rows": rows, "x.data": A, "x.row_stride": row, "x.batch_stride": step,
            "out.data": A + 64 * 4, "out.row_stride": row, "out.batch_stride": step, "initial": 0, "final": 0}


# The calls below are accepted on the host and get as far as the launch, which reports that there is no GPU.
ACCEPTED = dwp.DWP_ERR_CUDA


@pytest.mark.parametrize("rows,batch,row,step", [
    (100, 2, 128, 12800), (1, 8, 128, 128), (1, 8, 77, 128), (8, 1, 128, 99),
    (100, 4, 512, 128),  # rows first: [rows, batch, 2 x 64]
    (100, 4, 640, 128), (1, 1, 128, 128)])
def test_column_ranges_of_one_tensor_do_not_overlap(rows, batch, row, step):
    change = halves(rows, batch, row=row, step=step)
    assert abi.call("dwp_causal_conv", abi.CONV, abi.conv_good(), **change) == ACCEPTED
    if rows * batch > 1:  # one element into the other half
        change["out.data"] -= 4
        assert abi.call("dwp_causal_conv", abi.CONV, abi.conv_good(), **change) == ALIASING
        change["out.data"] += 8
        assert abi.call("dwp_causal_conv", abi.CONV, abi.conv_good(), **change) == ALIASING


def test_overlap_is_never_missed():
    """Random strides of x and out: whenever they share an element the call is refused."""
    import random
    rng = random.Random(1)
    shared = 0
    for _ in range(4000):
        ch, rows, batch = rng.choice([1, 2, 3, 8]), rng.choice([1, 1, 2, 3, 5]), rng.choice([1, 1, 2, 4])
        def strides():
            row = rng.choice([ch, 2 * ch, 2 * ch + 1, 4 * ch, batch * 2 * ch])
            step = rng.choice([ch, 2 * ch, rows * row, rows * row + ch, 2 * rows * row])
            return row, step
        (xr, xs), (orow, ostep) = strides(), strides()
        if rng.random() < 0.7:
            orow, ostep = xr, xs
        at = rng.randrange(0, 4 * ch + 1)
        places = lambda base, row, step: {base + b * step + t * row + c  # noqa: E731
                                          for b in range(batch) for t in range(rows) for c in range(ch)}
        status = abi.call("dwp_causal_conv", abi.CONV, abi.conv_good(), channels=ch, rows=rows, batch=batch, initial=0,
                          final=0, **{"x.data": A, "x.row_stride": xr, "x.batch_stride": xs, "out.data": A + 4 * at,
                                      "out.row_stride": orow, "out.batch_stride": ostep})
        assert status in (INVALID, ALIASING, ACCEPTED)
        if places(0, xr, xs) & places(at, orow, ostep):
            shared += 1
            assert status != ACCEPTED
    assert shared > 500


@pytest.mark.parametrize("change", [
    {"rows": 1 << 30, "batch": 1, "x.row_stride": 1 << 40}, {"rows": 1 << 30, "batch": 1, "out.row_stride": 1 << 40},
    {"rows": 1, "batch": 1 << 30, "x.batch_stride": 1 << 40}, {"rows": 1 << 24, "batch": 64, "out.row_stride": 1 << 40,
                                                              "out.batch_stride": 1 << 40},
    {"rows": (1 << 31) - 1, "batch": 1, "out.row_stride": 1 << 40}])
def test_a_span_past_the_address_space_is_refused(change):
    """rows x stride of these would wrap around 64 bits, and the overlap checks with it."""
    change = dict({"initial": 0, "final": 0, "x.batch_stride": 1 << 40, "out.batch_stride": 1 << 40,
                   "x.row_stride": 64, "out.row_stride": 64}, **change)
    assert abi.call("dwp_causal_conv", abi.CONV, abi.conv_good(), **change) == INVALID


def many_channels(names, good, channels):
    """`good` with dense rows of that many channels, every tensor 16 GB from the next."""
    g, n = good(), 0
    for k in names:
        if k.endswith(".data") or k in g and g[k] >= A:
            g[k] = A + n * (16 << 30) if g.get(k) else 0
            n += 1
        if k.endswith(".row_stride"):
            g[k] = channels
        if k.endswith(".batch_stride"):
            g[k] = 100 * channels
    return dict(g, channels=channels)


@pytest.mark.parametrize("name,names,good,most,change", [
    ("dwp_causal_conv_backward", abi.CONV_BACKWARD, abi.conv_good, {"channels": 1 << 17}, {}),
    ("dwp_causal_conv_backward", abi.CONV_BACKWARD, abi.conv_good, {"width": 8}, {}),
    ("dwp_selective_scan", abi.SCAN, abi.scan_good, {"channels": 1 << 17}, {"groups": 1}),
    ("dwp_selective_scan_backward", abi.SCAN_BACKWARD, abi.scan_good, {"channels": 1 << 17}, {"groups": 1}),
    ("dwp_selective_scan_backward", abi.SCAN_BACKWARD, abi.scan_good, {"groups": 1024},
     {"channels": 1 << 17, "b_group": 16, "c_group": 16}),
    ("dwp_selective_scan_backward", abi.SCAN_BACKWARD, abi.scan_good, {"states": 128},
     {"groups": 1, "B.row_stride": 129, "C.row_stride": 129, "B.batch_stride": 12900, "C.batch_stride": 12900}),
    ("dwp_block_norm_backward", abi.NORM_BACKWARD, abi.norm_good, {"channels": 1 << 17}, {"groups": 8}),
    ("dwp_block_norm_backward", abi.NORM_BACKWARD, abi.norm_good, {"groups": 1024}, {"channels": 1 << 17}),
    ("dwp_block_norm_backward", abi.NORM_BACKWARD, abi.norm_good, {"rows": (1 << 28) - 1}, {"groups": 8}),
])
def test_stated_sizes_are_accepted_up_to_the_last(name, names, good, most, change):
    """The size query takes the largest size that the header names, and refuses the next."""
    channels = most.get("channels", change.get("channels", 64))
    f = dict(many_channels(names, good, channels), **change)
    key, last = next(iter(most.items()))
    assert query(name, names, f, **{key: last})[0] == dwp.DWP_SUCCESS
    # one more; a step that every other size divides
    more = {"channels": last + f["groups"] if "groups" in f else last + 1, "groups": 2 * last}.get(key, last + 1)
    f["channels"] = more if key == "channels" else f["channels"]
    for k in names:
        if key == "channels" and k.endswith(".row_stride"):
            f[k] = more
        if key == "channels" and k.endswith(".batch_stride"):
            f[k] = 100 * more
    assert query(name, names, f, **{key: more})[0] == INVALID


def test_the_header_states_the_channels_that_the_library_takes():
    import os
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dwp.h")) as f:
        text = " ".join(line.strip(" *\n") for line in f)
    assert "at most 2^17 channels, 1024 groups" in text and "2^20 channels" not in text


@pytest.mark.parametrize("states,block", [(16, 32), (20, 16), (32, 16), (64, 8), (100, 4), (128, 4)])
@pytest.mark.parametrize("rows,channels,groups", [(2048, 4096, 1), (8192, 4096, 4), (4096, 1000, 1),
                                                  (7, 64, 2), (1, 4096, 1)])
@pytest.mark.parametrize("batch", [1, 2, 300])
def test_the_gradients_scratch_is_what_the_header_says(states, block, batch, rows, channels, groups):
    f = dict(many_channels(abi.SCAN_BACKWARD, abi.scan_good, channels), states=states, groups=groups, batch=batch, rows=rows,
             b_group=states, c_group=states)
    wide = max(channels, groups * states)
    for k in abi.SCAN_BACKWARD:
        if k.endswith("_stride"):
            f[k] = {"batch_stride": rows * wide, "row_stride": wide}.get(k.split(".")[-1], states)
    status, size = query("dwp_selective_scan_backward", abi.SCAN_BACKWARD, f)
    shares = 8 * states * batch * rows * groups * -(-channels // groups // block)
    assert status == dwp.DWP_SUCCESS
    assert shares <= size <= shares + max(17e6, 4 * batch * channels * (states + 2)) + 64
