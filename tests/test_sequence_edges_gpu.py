"""The sequence operators at the edges of what they accept: segments that
begin at any row, values that are not finite, growth and decay past the range
of one f32 factor.  The bar and the helpers are test_sequence_gpu's."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import device_wide_prefix_gb300 as dwp  # noqa: E402
import sequence_ref as ref  # noqa: E402
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


# ---------------------------------------------------------------------------
# values that are not finite


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("dtype,ch", [("f32", 12), ("bf16", 16), ("f16", 7)])
@pytest.mark.parametrize("width", [1, 2, 3, 4, 5, 6, 7, 8])
def test_conv_keeps_bad_values_to_the_taps(width, dtype, ch, act, bad):
    """A value in row t reaches the rows t .. t + width - 1 of its channel and segment, and no others."""
    d = base.Draw(width, base.TYPES[dtype])
    x, _ = d.act(150, ch)
    w, _ = d.f32(ch, width, lo=0.5, hi=1.0)
    dy, _ = d.act(150, ch)
    init, _ = d.act(3, width - 1, ch)
    cuts = [2, 90, 93, 148]
    off, halo, c = base.offs(cuts), width - 1, 5

    def run(x, init):
        y, fin = dwp.causal_conv(x, w, None, off, init, act, return_state=True)
        g = dwp.causal_conv_backward(dy, x, w, None, off, init, act)
        return y, fin, g

    y0, f0, g0 = run(x, init)
    for t in (9, 62, 63, 64, 70, 87, 91, 120, 147):
        x1 = x.clone()
        x1[t, c] = bad
        y1, f1, g1 = run(x1, init)
        end = min(e for e in cuts if e > t)
        lo, hi = max(b for b in cuts if b <= t), min(t + width, end)
        hit = torch.zeros(150, ch, dtype=torch.bool, device="cuda")
        hit[t:hi, c] = True
        inside = slice(2, 148)
        assert not torch.isfinite(y1[hit]).any() or (act and bad == -float("inf"))
        assert torch.equal(y1[inside][~hit[inside]], y0[inside][~hit[inside]]), t
        # the activation's slope is taken at the rows hit, and each goes back to its width - 1 rows before
        hit[max(lo, t - halo):hi, c] = act
        if not act:
            hit[:] = False
        assert torch.equal(g1["x"][inside][~hit[inside]], g0["x"][inside][~hit[inside]]), t
        others = [i for i in range(ch) if i != c]
        assert torch.equal(g1["weight"][others], g0["weight"][others])
        for s in range(3):
            for j in range(halo):
                r = cuts[s + 1] - halo + j
                if not (r == t and cuts[s] <= t < cuts[s + 1]):
                    assert torch.equal(f1[s, j], f0[s, j])
                else:
                    assert not torch.isfinite(f1[s, j, c])
    if halo:
        i1 = init.clone()
        i1[1, 0, c] = bad  # the oldest state row reaches the first row only
        y1, _, _ = run(x, i1)
        keep = torch.ones(150, ch, dtype=torch.bool, device="cuda")
        keep[:2] = keep[148:] = False
        keep[90, c] = False
        assert torch.equal(y1[keep], y0[keep])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("key", ["u", "dt", "z", "dout", "B", "C"])
@pytest.mark.parametrize("ch,n,groups", [(12, 8, 1), (70, 16, 2), (6, 128, 1)])
def test_scan_gradient_keeps_bad_values_to_their_sequence(ch, n, groups, key, bad):
    """Rows outside are in no sum; a value inside reaches its sequence, and its channel but for the sums over channels."""
    c = base.Scan(5, "f32", (700,), [2, 200, 203, 203, 500, 698], ch, n, groups)
    pos, kw = c.args()
    off = base.offs(c.offsets)

    def run():
        out, fin, points = dwp.selective_scan(*pos, **kw, offsets=off, initial_state=c.t["init"], return_state=True,
                                              return_checkpoints=True)
        g = dwp.selective_scan_backward(c.t["dout"], *pos, points, **kw, offsets=off, initial_state=c.t["init"],
                                        grad_final_state=c.t["dfinal"])
        return dict(g, out=out, fin=fin)

    by_row = ("out", "u", "dt", "z", "B", "C")
    r0 = run()
    c.t[key][:2] = bad
    c.t[key][698:] = bad
    r1 = run()
    for k, v in r0.items():
        rows = slice(2, 698) if k in by_row else slice(None)
        assert torch.equal(v[rows], r1[k][rows]), k
    at = (350, 0, 0) if key in "BC" else (350, 5)
    c.t[key][at] = bad
    r2 = run()
    others = [t for t in range(2, 698) if not 203 <= t < 500]
    for k in by_row:
        assert torch.equal(r0[k][others], r2[k][others]), k
    for k in ("fin", "initial_state"):
        assert torch.equal(r0[k][[0, 1, 2, 4]], r2[k][[0, 1, 2, 4]]), k
    if key not in "BC":
        apart = [i for i in range(ch) if i != 5]
        for k in ("out", "u", "dt", "z"):
            assert torch.equal(r0[k][2:698][:, apart], r2[k][2:698][:, apart]), k
        for k in ("A", "D", "dt_bias"):
            assert torch.equal(r0[k][apart], r2[k][apart]), k


@pytest.mark.parametrize("width", [1, 2, 3, 4, 5, 6, 7, 8])
def test_conv_step_is_the_prompt_next_to_an_infinity(width):
    """Where the prompt's output is finite so is the token's, and the same within the bar; the states are equal."""
    d = base.Draw(40 + width, torch.float32)
    x, xv = d.act(1, 12, 8)
    x[0, 3, 2] = float("inf")
    w, _ = d.f32(8, width, lo=0.5, hi=1.0)
    y, fin = dwp.causal_conv(x, w, return_state=True)
    cache = torch.zeros(1, width - 1, 8, device="cuda")
    z = torch.stack([dwp.causal_conv_step(x[:, t], cache, w) for t in range(12)], 1)
    assert torch.equal(torch.isfinite(y), torch.isfinite(z)) and int((~torch.isfinite(y)).sum()) == width
    ok = torch.isfinite(y)
    p, _ = ref.conv_pre(abs(np.where(np.isfinite(x[0].cpu().numpy()), xv[0], 0.0)), w.double().cpu().numpy(), np.zeros(8),
                        np.zeros((width - 1, 8)))
    bound = torch.from_numpy(2 * base.U * (64 + width) * (p + 1)).cuda()[None]
    assert ((y - z).abs()[ok] <= bound[ok]).all()
    assert torch.equal(fin, cache)


# ---------------------------------------------------------------------------
# the scan past the range of one f32 factor


@pytest.mark.parametrize("grow", [True, False])
@pytest.mark.parametrize("ch,n", [(4, 16), (3, 5)])
def test_scan_carries_a_state_over_a_chunk_past_one_factors_range(ch, n, grow):
    """The product of a chunk's decays is past f32's range, what it does to the state is not.

    Rows 16 to 31 have delta 1 and A = +-5.6: e^89.6 over them, for a state of 1e-37 (or e^-89.6 for 1e37);
    the other rows have delta 0, so the walks on both sides keep the state as it is.
    """
    rows = 48
    A = torch.full((ch, n), 5.6 if grow else -5.6, device="cuda")
    dt = torch.zeros(1, rows, ch, device="cuda")
    dt[:, 16:32] = 1.0
    size = 1e-37 if grow else 1e37
    init = torch.linspace(1.0, 2.0, ch * n, device="cuda").view(1, ch, n) * size
    zero, B = torch.zeros(1, rows, ch, device="cuda"), torch.zeros(1, rows, n, device="cuda")
    factor = np.exp(16 * A.double().cpu().numpy())[None]
    want = init.double().cpu().numpy() * factor
    # the exponent's rounding (8.08 in base 2) and the exponential's, for each of 16 rows, as in the bar
    _, fin, points = dwp.selective_scan(zero, dt, A, B, B, initial_state=init, dt_softplus=False, return_state=True,
                                        return_checkpoints=True)
    base.near(fin, want, abs(want), 64 + 16 * rows, "final_state")
    g = dwp.selective_scan_backward(zero, zero, dt, A, B, B, points, initial_state=init, dt_softplus=False,
                                    grad_final_state=init)
    base.near(g["initial_state"], want, abs(want), 2 * (64 + 16 * rows), "grad initial_state")


@pytest.mark.parametrize("ch,n", [(40, 16), (33, 5), (6, 128), (9, 24)])
@pytest.mark.parametrize("size", [-3.4028234663852886e38, -2.5e38])
def test_scan_of_the_lowest_decay_rate(size, ch, n):
    """A at its type's lowest value: such a state is its last input, exp(0 A) is 1, and no other is touched."""
    c = base.Scan(77, "f32", (1, 40), None, ch, n, 1)
    c.t["A"][:, 1] = size
    c.t["A"][ch - 1, :] = size
    c.v["A"] = c.t["A"].double().cpu().numpy()
    base.check_scan(c)
    c.t["dt"][:, 7:9] = -200.0  # softplus gives 0 there in 32 bits; the gradient in 32 bits is then 0 times infinity
    c.v["dt"] = c.t["dt"].double().cpu().numpy()
    pos, kw = c.args()
    out, fin = dwp.selective_scan(*pos, **kw, initial_state=c.t["init"], return_state=True)
    (y, last), (ym, lastm) = ref.scan(*c.ref(0))
    base.near(out[0], y, ym, 64 + 16 * 40, "out")
    base.near(fin[0], last, lastm, 64 + 16 * 40, "final_state")
    for row in (3, 8):
        step = [c.t[k][:, row] for k in ("u", "dt")] + [c.t["A"]] + [c.t[k][:, row] for k in "BC"]
        cache = c.t["init"].clone()
        out = dwp.selective_scan_step(*step, cache, D=c.t["D"], z=c.t["z"][:, row], dt_bias=c.t["dt_bias"])
        args = [v[row:row + 1] if i != 2 else v for i, v in enumerate(c.ref(0)[:5])] + [
            c.v["D"], c.v["z"].reshape(-1, ch)[row:row + 1], c.v["dt_bias"], True, c.v["init"][0]]
        (y, last), (ym, lastm) = ref.scan(*args)
        base.near(out, y, ym, 80, "token out")
        base.near(cache[0], last, lastm, 80, "token state")


@pytest.mark.parametrize("lo,hi", [(-4, 0), (-12, -4), (-16, -12), (-40, -16), (-80, -40), (0, 4), (4, 40)])
def test_softplus_of_far_arguments(lo, hi):
    """delta is the state that one row of u = B = 1 leaves.

    |x| log2(e) is rounded (2^-24) after a constant that is (1.4e-8 off, both relative to |x|), the exponential adds
    2^-22 and the polynomial, with its f32 evaluation, 1.8e-7; all relative, and for x > 0 relative to less.
    """
    x = torch.linspace(lo, hi, 4096, device="cuda")
    one, B = torch.ones(1, 4096, device="cuda"), torch.ones(1, 1, device="cuda")
    A = torch.zeros(4096, 1, device="cuda")
    _, fin = dwp.selective_scan(one, x[None], A, B, B, return_state=True)
    v = x.double().cpu().numpy()
    want = np.logaddexp(v, 0.0)
    bound = (abs(np.minimum(v, 0.0)) * (2.0 ** -24 + 1.4e-8) + 2.0 ** -22 + 1.8e-7 + 2.0 ** -24) * want
    got = fin[0, :, 0].double().cpu().numpy()
    assert (abs(got - want) <= bound).all(), (abs(got - want) / want).max()


# ---------------------------------------------------------------------------
# the caller's scratch


def test_scratch_of_another_place_or_layout_is_refused():
    """The kernels would write to where it points: host memory, or past the one byte of an expanded tensor."""
    x = torch.randn(40, 8, device="cuda")
    w = torch.randn(8, 4, device="cuda")
    A, B = -torch.ones(8, 4, device="cuda"), torch.randn(40, 4, device="cuda")
    ones = torch.ones(8, device="cuda")
    off = torch.tensor([0, 40], dtype=torch.int32).cuda()
    points = dwp.selective_scan(x, x, A, B, B, return_checkpoints=True)[1]
    calls = [lambda s: dwp.causal_conv_backward(x, x, w, scratch=s)["x"],
             lambda s: dwp.selective_scan(x, x, A, B, B, offsets=off, scratch=s),
             lambda s: dwp.selective_scan_backward(x, x, x, A, B, B, points, scratch=s)["u"],
             lambda s: dwp.block_norm_backward(x, x, ones, scratch=s)["x"]]
    for call in calls:
        want = call(None)
        assert torch.equal(call(torch.empty(1 << 20, dtype=torch.uint8, device="cuda")), want)
        assert torch.equal(call(torch.empty(1 << 18, device="cuda")), want)  # bytes, whatever the type
        for bad in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 20)):
            with pytest.raises(ValueError):
                call(bad)


# ---------------------------------------------------------------------------
# padding rows of the token forms


@pytest.mark.parametrize("n", [16, 12])
@pytest.mark.parametrize("slots", [[-1] * 5, [7, -1, 0, 2 ** 31 - 1, -2 ** 31], [0, 0x7000, 1, -1, 2]])
@pytest.mark.parametrize("cache", [0, 1, 4])
def test_padding_rows_leave_every_state_as_it_is(cache, slots, n):
    """A slot outside the cache, whatever its number, and a cache of no slots at all."""
    c = base.Scan(9, "bf16", (5, 1), None, 72, n, 1, slots=cache or 1)
    pos, kw = c.args()
    z = kw.pop("z")[:, 0]
    one = [p if p is pos[2] else p[:, 0] for p in pos]
    d = base.Draw(10, torch.bfloat16)
    taps, _ = d.act(cache, 3, 72)
    w, _ = d.f32(72, 4)
    live = [i for i, s in enumerate(slots) if 0 <= s < cache]
    at = torch.tensor(slots, dtype=torch.int32).cuda()
    state = c.t["init"][:cache].clone()
    before, taps0 = state.clone(), taps.clone()
    out = dwp.selective_scan_step(*one, state, z=z, slots=at, **kw)
    y = dwp.causal_conv_step(one[0], taps, w, slots=at)
    dead = [i for i in range(5) if i not in live]
    assert (out[dead] == 0).all() and (y[dead] == 0).all()
    if live:  # alone, in the same slots
        few, ft = before.clone(), taps0.clone()
        rows = [p if p is pos[2] else p[live] for p in one]
        assert torch.equal(out[live], dwp.selective_scan_step(*rows, few, z=z[live], slots=at[live], **kw))
        assert torch.equal(y[live], dwp.causal_conv_step(one[0][live], ft, w, slots=at[live]))
        assert torch.equal(state, few) and torch.equal(taps, ft)
    else:
        assert torch.equal(state, before) and torch.equal(taps, taps0)
