"""The gated delta rule in a build with test hooks (-DDWP_DELTA_TEST=1): what
happens where no tensor map can be made, and where a wait inside a block runs
out.  A stalled wait is for a barrier at which nothing arrives, with a short
limit; the block gives up, lets its copies and products end, and the call
returns with NaN in what it could not compute."""
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


SITES = ("none", "local_rows", "local_product", "issue_rows", "issue_state", "issue_sides", "issue_corrections", "load_room",
         "load_landed", "decay_room", "chain_rows", "chain_keys", "chain_other", "chain_inverse", "chain_state",
         "chain_outputs", "chain_room", "chain_side", "grad_first", "grad_states", "grad_second", "grad_rows", "grad_ends")
WALK = [s for s in SITES if s.startswith(("issue", "load", "decay", "chain"))]


class Stalled:
    """The waits at one site run out, but for each thread's first `skip`."""

    def __init__(self, lib, site, skip=0):
        self.lib, self.site, self.skip = lib, SITES.index(site), skip

    def __enter__(self):
        self.lib.dwp_delta_test_stall(self.site, self.skip)

    def __exit__(self, *_):
        torch.cuda.synchronize()
        self.lib.dwp_delta_test_stall(0, 0)


def nan_or(got, want):
    """Every value is NaN or what the finished call gives."""
    return bool((got.isnan() | (got == want)).all())


def stalled_case(dtype, rows=300, heads=2):
    return Case(41, (1, rows), None, dtype, 1, heads, 128, 64, decay=0.05)


@pytest.mark.parametrize("skip", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("site", ["local_rows", "local_product", *WALK])
def test_a_forward_wait_that_runs_out(lib, site, dtype, skip):
    if site == "chain_side" or (dtype == "f32" and site == "local_rows") or (dtype == "bf16" and site == "chain_room"):
        pytest.skip("no such wait")
    if site.startswith("local") and skip:
        pytest.skip("a block waits there once")
    c = stalled_case(dtype)
    want = forward(c)
    with Stalled(lib, site, skip):
        out, final, points = forward(c)
    assert nan_or(out, want[0]) and out[:, 256:].isnan().all() and final.isnan().all()
    # and what was kept says so to the gradient
    grads = backward(c, points)
    for n in ("q", "k", "g", "beta"):
        assert grads[n][:, 257:].isnan().all(), n
    again = forward(c)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


@pytest.mark.parametrize("skip", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("site", WALK)
def test_a_wait_of_the_walk_back_that_runs_out(lib, site, dtype, skip):
    if site == "chain_outputs" or (dtype == "bf16" and site == "chain_room"):
        pytest.skip("no such wait")
    c = stalled_case(dtype)
    points = forward(c)[2]
    want = backward(c, points)
    with Stalled(lib, site, skip):
        got = backward(c, points)
    for n in ("q", "k", "v", "g", "beta"):
        assert nan_or(got[n], want[n]), n
    # from the walk's last chunk, the first rows
    for n in ("k", "v", "g", "beta"):
        assert got[n][:, :64].isnan().all(), n
    assert got["initial_state"].isnan().all()
    again = backward(c, points)
    assert all(torch.equal(again[n], want[n]) for n in want)


@pytest.mark.parametrize("skip", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("site", [s for s in SITES if s.startswith("grad")])
def test_a_wait_of_the_gradient_that_runs_out(lib, site, dtype, skip):
    """skip 1: the second of two heads that share their keys."""
    c = stalled_case(dtype)
    points = forward(c)[2]
    want = backward(c, points)
    with Stalled(lib, site, skip):
        got = backward(c, points)
    for n in want:
        assert nan_or(got[n], want[n]), n
    assert got["q"].isnan().all() and got["k"].isnan().all()
    for n in ("g", "beta"):
        assert got[n][:, :, skip:].isnan().all() and torch.equal(got[n][:, :, :skip], want[n][:, :, :skip]), n
    if site == "grad_rows":
        assert got["v"][:, :, skip:].isnan().all()
    again = backward(c, points)
    assert all(torch.equal(again[n], want[n]) for n in want)


@pytest.mark.parametrize("site,skip", [("issue_sides", 3), ("load_room", 0), ("chain_state", 2), ("chain_outputs", 1)])
def test_a_part_that_runs_out(lib, site, skip):
    """Of a sequence cut in parts: what the parts after it begin from is not a number either."""
    c = Case(42, (1, 1600), None, "bf16", 1, 1, 128, 64, decay=0.05)
    want = forward(c)
    with Stalled(lib, site, skip):
        out, final, _ = forward(c)
    assert nan_or(out, want[0]) and out[:, 1536:].isnan().all() and final.isnan().all()
    assert torch.equal(forward(c)[0], want[0])
