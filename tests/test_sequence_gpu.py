"""The sequence operators on the GPU against their 64-bit definitions.

The bar, element by element, for an output of type T:

    |got - exact| <= r(T) |exact| + 2^-24 * steps * magnitude + tiny(T)

r(T) is T's rounding (2^-8, 2^-11, 2^-23: a whole unit, half of which is the
rounding itself and the rest its neighbourhood), magnitude the sum of the
absolute values of the terms the definition adds, and steps the f32 roundings
on the longest path from an input to the output: 64 for the activations and
exponentials around it (each a few units, the arguments' own rounding
included), 16 for each row a state passes through, and one for each channel
or row that a sum runs over.
"""
import math

import numpy as np
import pytest

import sequence_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import device_wide_prefix_gb300 as dwp  # noqa: E402
from device_wide_prefix_gb300 import build as dwp_build  # noqa: E402

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {torch.float32: 2.0 ** -23, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-35, torch.bfloat16: 1e-35, torch.float16: 2.0 ** -24}
U = 2.0 ** -24
SENTINEL = 77.0


@pytest.fixture(scope="module", autouse=True)
def lib():
    dwp_build.build()
    return dwp.load()


def near(got, exact, mag, steps, what):
    g = got.detach().double().cpu().numpy()
    assert g.shape == exact.shape, what
    bound = ROUND[got.dtype] * abs(exact) + U * steps * mag + TINY[got.dtype]
    worst = (abs(g - exact) / bound).max() if g.size else 0.0
    assert np.isfinite(g).all() and worst <= 1.0, "%s: %.3g times the bound" % (what, worst)


class Draw:
    """Seeded inputs: numpy 64-bit values that the GPU tensors hold exactly."""

    def __init__(self, seed, dtype):
        self.rng, self.dtype = np.random.default_rng(seed), dtype

    def act(self, *shape, scale=1.0, pad=0, dtype=None):
        """(tensor, its values): rows of a wider tensor where `pad` > 0, starting at an odd place."""
        t = torch.from_numpy(self.rng.standard_normal(shape) * scale).to(dtype or self.dtype)
        v = t.double().numpy()
        if pad:
            wide = torch.full((*shape[:-1], shape[-1] + 2 * pad + 1), SENTINEL, dtype=t.dtype)
            wide[..., pad:pad + shape[-1]] = t
            return wide.cuda()[..., pad:pad + shape[-1]], v
        return t.cuda(), v

    def f32(self, *shape, lo=-1.0, hi=1.0):
        t = torch.from_numpy(self.rng.uniform(lo, hi, shape)).float()
        return t.cuda(), t.double().numpy()


def spans(lead, offsets):
    """(rows of each sequence) as index slices of the flattened stream."""
    if offsets is not None:
        return [slice(a, b) for a, b in zip(offsets[:-1], offsets[1:])]
    batch, rows = lead if len(lead) == 2 else (1, lead[0])
    return [slice(b * rows, (b + 1) * rows) for b in range(batch)]


def offs(o):
    return None if o is None else torch.tensor(o, dtype=torch.int32).cuda()


# lead shape, offsets: batches and packed streams, empty sequences at every place, rows outside, one row, none
SHAPES = [
    ((1, 1), None), ((2, 3), None), ((37,), None), ((3, 0), None), ((0, 5), None), ((1, 130), None),
    ((70,), [0, 70]), ((70,), [0, 0, 1, 1, 33, 64, 65, 70, 70]), ((70,), [5, 5, 20, 50]), ((40,), [7, 7, 7]),
    ((100,), [0, 31, 32, 33, 96, 97, 100]), ((9,), list(range(10))), ((5,), [0]),
    ((70,), [5, 20, 50]), ((200,), [66, 67, 140]),
]
IDS = ["%s-%s" % ("x".join(map(str, s)), "batch" if o is None else "o%d_%d" % (len(o), o[0])) for s, o in SHAPES]


def covered(lead, offsets):
    n = math.prod(lead)
    m = np.zeros(n, bool)
    for s in spans(lead, offsets):
        m[s] = True
    return m


# ---------------------------------------------------------------------------
# causal convolution


@pytest.mark.parametrize("dtype,ch,width,pad", [("f32", 5, 4, 0), ("bf16", 264, 4, 0), ("f16", 33, 3, 2), ("f32", 8, 8, 4),
                                                ("bf16", 1, 1, 0), ("bf16", 1032, 2, 8)])
@pytest.mark.parametrize("lead,offsets", SHAPES, ids=IDS)
def test_conv(lead, offsets, dtype, ch, width, pad):
    d = Draw(len(lead) * 100 + ch, TYPES[dtype])
    cuts = spans(lead, offsets)
    x, xv = d.act(*lead, ch, pad=pad)
    w, wv = d.f32(ch, width)
    b, bv = d.f32(ch)
    init, iv = d.act(len(cuts), width - 1, ch)
    dy, dyv = d.act(*lead, ch, pad=pad)
    df, dfv = d.act(len(cuts), width - 1, ch)
    xv, dyv = xv.reshape(-1, ch), dyv.reshape(-1, ch)
    for act in (True, False):
        out = torch.full((*lead, ch), SENTINEL, dtype=x.dtype, device="cuda")
        out, fin = dwp.causal_conv(x, w, b, offs(offsets), init, act, return_state=True, out=out)
        g = dwp.causal_conv_backward(dy, x, w, b, offs(offsets), init, act, df)
        o2, gx = out.reshape(-1, ch), g["x"].reshape(-1, ch)
        dw, db = np.zeros((ch, width)), np.zeros(ch)
        dwm, dbm = dw.copy(), db.copy()
        for i, s in enumerate(cuts):
            y, last, mag = ref.conv(xv[s], wv, bv, iv[i], act)
            near(o2[s], y, mag + abs(y), 64 + width, "out")
            assert (fin[i].double().cpu().numpy() == last).all()
            (dx, dwi, dbi, di), (dxm, dwim, dbim, dim) = ref.conv_grad(dyv[s], xv[s], wv, bv, iv[i], act, dfv[i])
            near(gx[s], dx, dxm, 80 + width, "dx")
            near(g["initial_state"][i], di, dim, 80 + width, "dinit")
            dw, db, dwm, dbm = dw + dwi, db + dbi, dwm + dwim, dbm + dbim
        near(g["weight"], dw, dwm, 80 + width + math.prod(lead), "dw")
        near(g["bias"], db, dbm, 80 + width + math.prod(lead), "db")
        if offsets is not None and not covered(lead, offsets).all():
            assert (o2[torch.from_numpy(~covered(lead, offsets)).cuda()] == SENTINEL).all()


def test_conv_without_state_or_bias_and_parameters_in_the_activations_type():
    d = Draw(3, torch.bfloat16)
    x, xv = d.act(2, 50, 24)
    w, wv = d.act(24, 4, scale=0.5)
    b, bv = d.act(24)
    zero = np.zeros((3, 24))
    for bias, bval in ((b, bv), (None, np.zeros(24))):
        out = dwp.causal_conv(x, w, bias)
        g = dwp.causal_conv_backward(x, x, w, bias)
        assert set(g) == {"x", "weight"} | ({"bias"} if bias is not None else set())
        dw, dwm = 0, 0
        for i in range(2):
            y, _, mag = ref.conv(xv[i], wv, bval, zero, True)
            near(out[i], y, mag + abs(y), 68, "out")
            (dx, dwi, _, _), (dxm, dwim, _, _) = ref.conv_grad(xv[i], xv[i], wv, bval, zero, True, zero)
            near(g["x"][i], dx, dxm, 84, "dx")
            dw, dwm = dw + dwi, dwm + dwim
        near(g["weight"], dw, dwm, 184, "dw")


@pytest.mark.parametrize("dtype,ch,width,pad", [("f32", 5, 4, 0), ("bf16", 264, 4, 8), ("f16", 33, 3, 2), ("bf16", 8, 1, 0),
                                                ("f32", 8, 8, 0)])
def test_conv_step_continues_the_prompt(dtype, ch, width, pad):
    """Tokens one by one give what the whole prompt gives, bit for bit in the state; padding rows touch nothing."""
    d = Draw(7, TYPES[dtype])
    x, xv = d.act(4, 6, ch, pad=pad)
    w, wv = d.f32(ch, width)
    b, bv = d.f32(ch)
    cache, cv = d.act(9, width - 1, ch)
    slots = torch.tensor([4, -1, 0, 9], dtype=torch.int32).cuda()  # 9 is past the cache
    live = {0: 4, 2: 0}
    before = cache.clone()
    outs = [dwp.causal_conv_step(x[:, t], cache, w, b, slots) for t in range(6)]
    for i in range(4):
        if i not in live:
            assert all((o[i] == 0).all() for o in outs)
            continue
        y, last, mag = ref.conv(xv[i], wv, bv, cv[live[i]], True)
        near(torch.stack([o[i] for o in outs]), y, mag + abs(y), 64 + width, "out")
        assert (cache[live[i]].double().cpu().numpy() == last).all()
    rest = [s for s in range(9) if s not in live.values()]
    assert torch.equal(cache[rest], before[rest])


# ---------------------------------------------------------------------------
# selective scan


class Scan:
    """Inputs of one scan, as tensors and as 64-bit values."""

    def __init__(self, seed, dtype, lead, offsets, ch, n, groups, pad=0, gated=True, softplus=True, slots=None):
        d = Draw(seed, TYPES[dtype])
        self.lead, self.offsets, self.ch = lead, offsets, ch
        self.cuts = spans(lead, offsets)
        t, v = {}, {}
        t["u"], v["u"] = d.act(*lead, ch, pad=pad)
        t["dt"], v["dt"] = d.act(*lead, ch, scale=0.5, pad=pad)
        if not softplus:
            t["dt"] = t["dt"].abs()
            v["dt"] = abs(v["dt"])
        t["z"], v["z"] = d.act(*lead, ch, pad=pad) if gated else (None, None)
        low, lv = d.act(*lead, 2 * groups * n, pad=pad)  # B and C side by side, as a projection gives them
        for i, k in enumerate("BC"):
            t[k] = low[..., i * groups * n:(i + 1) * groups * n].unflatten(-1, (groups, n))
            v[k] = lv[..., i * groups * n:(i + 1) * groups * n].reshape(*lead, groups, n)
        t["A"], v["A"] = d.f32(ch, n, lo=-2.0, hi=-0.05)
        t["D"], v["D"] = d.f32(ch)
        t["dt_bias"], v["dt_bias"] = d.f32(ch, lo=-3.0, hi=0.0) if softplus else d.f32(ch, lo=0.0, hi=0.1)
        t["init"], v["init"] = d.f32(slots or len(self.cuts), ch, n)
        t["dout"], v["dout"] = d.act(*lead, ch, pad=pad)
        t["dfinal"], v["dfinal"] = d.f32(len(self.cuts), ch, n)
        self.t, self.v, self.softplus = t, v, softplus

    def rows(self, k, s):
        x = self.v[k]
        return None if x is None else x.reshape(-1, *x.shape[len(self.lead):])[s]

    def args(self):
        t = self.t
        return [t[k] for k in ("u", "dt", "A", "B", "C")], dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"],
                                                               dt_softplus=self.softplus)

    def ref(self, i):
        s, v = self.cuts[i], self.v
        return [self.rows(k, s) for k in ("u", "dt")] + [v["A"]] + [self.rows(k, s) for k in "BC"] + [
            v["D"], self.rows("z", s), v["dt_bias"], self.softplus, v["init"][i]]


def check_scan(c, steps_extra=0):
    pos, kw = c.args()
    off = offs(c.offsets)
    lead, ch = c.lead, c.ch
    out = torch.full((*lead, ch), SENTINEL, dtype=c.t["u"].dtype, device="cuda")
    out, fin, points = dwp.selective_scan(*pos, **kw, offsets=off, initial_state=c.t["init"], return_state=True,
                                          return_checkpoints=True, out=out)
    g = dwp.selective_scan_backward(c.t["dout"], *pos, points, **kw, offsets=off, initial_state=c.t["init"],
                                    grad_final_state=c.t["dfinal"])
    o2 = out.reshape(-1, ch)
    total = math.prod(lead)
    sums = {k: [0.0, 0.0] for k in ("A", "D", "dt_bias")}
    for i, s in enumerate(c.cuts):
        rows = s.stop - s.start
        steps = 64 + 16 * rows + steps_extra
        (y, last), (ym, lastm) = ref.scan(*c.ref(i))
        near(o2[s], y, ym, steps, "out")
        near(fin[i], last, lastm, steps, "final_state")
        e, m = ref.scan_grad(c.rows("dout", s), *c.ref(i), c.v["dfinal"][i])
        for k in ("u", "dt", "z", "B", "C"):
            if k in g:
                near(g[k].reshape(-1, *e[k].shape[1:])[s], e[k], m[k], 2 * steps + ch, "grad " + k)
        near(g["initial_state"][i], e["initial_state"], m["initial_state"], 2 * steps, "grad initial_state")
        for k in sums:
            sums[k][0] += e[k]
            sums[k][1] += m[k]
    for k, (e, m) in sums.items():
        if np.ndim(e):
            near(g[k], e, m, 2 * (64 + 16 * total) + total, "grad " + k)
        else:
            assert (g[k] == 0).all()
    if c.offsets is not None and not covered(lead, c.offsets).all():
        assert (o2[torch.from_numpy(~covered(lead, c.offsets)).cuda()] == SENTINEL).all()
    return out, fin, g


@pytest.mark.parametrize("dtype,ch,n,groups,pad,gated,softplus", [
    ("f32", 3, 1, 1, 0, True, True), ("f32", 40, 16, 1, 0, True, True), ("bf16", 72, 16, 2, 8, True, True),
    ("f16", 33, 5, 3, 1, False, True), ("f32", 34, 17, 1, 4, True, False), ("bf16", 16, 64, 1, 0, True, True),
    ("f32", 6, 128, 2, 0, False, False), ("f32", 9, 33, 1, 3, True, True)])
@pytest.mark.parametrize("lead,offsets", SHAPES, ids=IDS)
def test_scan(lead, offsets, dtype, ch, n, groups, pad, gated, softplus):
    check_scan(Scan(ch + n, dtype, lead, offsets, ch, n, groups, pad, gated, softplus))


@pytest.mark.parametrize("offsets", [None, [0, 1, 700, 700, 1900, 2500], [3, 2499]])
@pytest.mark.parametrize("dtype,ch,n", [("f32", 20, 16), ("bf16", 24, 8)])
def test_scan_over_many_rows(offsets, dtype, ch, n):
    """Long enough that the rows are split over blocks, with sequences that cross the pieces."""
    check_scan(Scan(11, dtype, (2500,) if offsets else (1, 2500), offsets, ch, n, 1))


def test_scan_without_the_optional_parts():
    c = Scan(5, "f32", (2, 40), None, 12, 8, 1)
    t = c.t
    B, C = t["B"].squeeze(-2), t["C"].squeeze(-2)  # one group: its axis may be left out
    out = dwp.selective_scan(t["u"], t["dt"], t["A"], B, C)
    out2, points = dwp.selective_scan(t["u"], t["dt"], t["A"], B, C, return_checkpoints=True)
    assert torch.equal(out, out2)
    g = dwp.selective_scan_backward(t["dout"], t["u"], t["dt"], t["A"], B, C, points)
    assert set(g) == {"u", "dt", "A", "B", "C"} and g["B"].shape == B.shape
    none = np.zeros(12)
    for i in range(2):
        args = [c.rows(k, c.cuts[i]) for k in ("u", "dt")] + [c.v["A"]] + [c.rows(k, c.cuts[i]) for k in "BC"] + [
            none, None, none, True, np.zeros((12, 8))]
        (y, _), (ym, _) = ref.scan(*args)
        near(out[i], y, ym, 64 + 16 * 40, "out")
        e, m = ref.scan_grad(c.rows("dout", c.cuts[i]), *args, np.zeros((12, 8)))
        for k in ("u", "dt"):
            near(g[k][i], e[k], m[k], 2 * (64 + 16 * 40), "grad " + k)


def test_scan_gradient_against_differences():
    """The kernels' own forward, differenced: loss = <out, dout> + <final, dfinal> along a random direction.

    f32 differences at h carry a rounding of about sqrt(terms) * 2^-24 * |terms| / h and an error h^2 / 6 times the
    third derivative; at h = 2^-6, with terms of order one, both stay below 1e-3 of the terms' norm.
    """
    c = Scan(23, "f32", (1, 96), None, 16, 8, 2)
    pos, kw = c.args()
    h = 2.0 ** -6
    out, fin, points = dwp.selective_scan(*pos, **kw, initial_state=c.t["init"], return_state=True,
                                          return_checkpoints=True)
    g = dwp.selective_scan_backward(c.t["dout"], *pos, points, **kw, initial_state=c.t["init"],
                                    grad_final_state=c.t["dfinal"])
    names = {"u": 0, "dt": 1, "A": 2, "B": 3, "C": 4}
    gen = torch.Generator(device="cuda").manual_seed(1)
    for k in ("u", "dt", "A", "B", "C", "D", "z", "dt_bias", "initial_state"):
        base = pos[names[k]] if k in names else c.t["init"] if k == "initial_state" else kw[k]
        d = torch.randn(base.shape, generator=gen, device="cuda") * (0.1 if k == "A" else 1.0)

        def loss(sign):
            p, q, i = list(pos), dict(kw), c.t["init"]
            v = (base + sign * h * d).contiguous()
            if k in names:
                p[names[k]] = v
            elif k == "initial_state":
                i = v
            else:
                q[k] = v
            o, f = dwp.selective_scan(*p, **q, initial_state=i, return_state=True)
            return (o.double() * c.t["dout"].double()).sum() + (f.double() * c.t["dfinal"].double()).sum()

        want = ((loss(1) - loss(-1)) / (2 * h)).item()
        terms = g[k].double() * d.double()
        assert abs(terms.sum().item() - want) <= 1e-3 * terms.abs().sum().item() + 1e-3, k


@pytest.mark.parametrize("dtype,ch,n,groups,pad", [("f32", 40, 16, 1, 0), ("bf16", 72, 16, 2, 8), ("f16", 33, 5, 3, 1),
                                                   ("f32", 6, 128, 1, 0), ("bf16", 16, 64, 1, 0)])
def test_scan_step_continues_the_prompt(dtype, ch, n, groups, pad):
    c = Scan(31, dtype, (4, 5), None, ch, n, groups, pad, slots=9)
    pos, kw = c.args()
    cache = c.t["init"].clone()
    before = cache.clone()
    slots = torch.tensor([4, -1, 0, 9], dtype=torch.int32).cuda()  # 9 is past the cache
    live = {0: 4, 2: 0}
    z = kw.pop("z")
    outs = [dwp.selective_scan_step(*(a if a.dim() == 2 and a is pos[2] else a[:, t] for a in pos), cache, z=z[:, t],
                                    slots=slots, **kw) for t in range(5)]
    for i in range(4):
        if i not in live:
            assert all((o[i] == 0).all() for o in outs)
            continue
        args = c.ref(i)
        args[-1] = c.v["init"][live[i]]
        (y, last), (ym, lastm) = ref.scan(*args)
        near(torch.stack([o[i] for o in outs]), y, ym, 64 + 16 * 5, "out")
        near(cache[live[i]], last, lastm, 64 + 16 * 5, "state")
    rest = [s for s in range(9) if s not in live.values()]
    assert torch.equal(cache[rest], before[rest])


def test_token_forms_without_slots_use_row_i():
    c = Scan(37, "f32", (3, 1), None, 10, 4, 1)
    pos, kw = c.args()
    z = kw.pop("z")
    a, b = c.t["init"].clone(), c.t["init"].clone()
    one = [p if p is pos[2] else p[:, 0] for p in pos]
    x = dwp.selective_scan_step(*one, a, z=z[:, 0], **kw)
    y = dwp.selective_scan_step(*one, b, z=z[:, 0], slots=torch.arange(3, dtype=torch.int32).cuda(), **kw)
    assert torch.equal(x, y) and torch.equal(a, b)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_bad_values_stay_in_their_sequence_and_channel(bad):
    """A NaN or infinity in one sequence and channel reaches no other, and rows outside are never read."""
    c = Scan(41, "f32", (60,), [2, 20, 40, 58], 12, 8, 1)
    pos, kw = c.args()
    off = offs(c.offsets)
    run = lambda: dwp.selective_scan(*pos, **kw, offsets=off, initial_state=c.t["init"], return_state=True)  # noqa: E731
    out0, fin0 = run()
    for k in ("u", "dt", "z"):  # outside every segment
        c.t[k][:2] = bad
        c.t[k][58:] = bad
    out1, fin1 = run()
    assert torch.equal(out0[2:58], out1[2:58]) and torch.equal(fin0, fin1)
    c.t["u"][25, 7] = bad  # inside the second segment, channel 7
    out2, fin2 = run()
    keep = torch.ones(60, 12, dtype=torch.bool, device="cuda")
    keep[:2], keep[58:], keep[25:40, 7] = False, False, False
    assert torch.equal(out0[keep], out2[keep])
    assert not torch.isfinite(out2[25:40, 7]).any()
    assert torch.equal(fin0[[0, 2]], fin2[[0, 2]])


# ---------------------------------------------------------------------------
# block norm


@pytest.mark.parametrize("rows", [0, 1, 5, 1300])
@pytest.mark.parametrize("dtype,ch,groups,pad,rdtype", [
    ("f32", 6, 1, 0, "f32"), ("bf16", 264, 1, 8, "f32"), ("bf16", 512, 4, 0, "bf16"), ("f16", 77, 7, 1, "f32"),
    ("f32", 1, 1, 0, "f32"), ("bf16", 2056, 1, 0, "f32")])
@pytest.mark.parametrize("form", ["plain", "gate", "gate_after", "residual", "scaled", "scaled_gate"])
def test_norm(rows, dtype, ch, groups, pad, rdtype, form):
    if rows == 1300 and ch > 300 and form != "scaled":
        pytest.skip("many rows are tested at the smaller widths")
    check_norm(rows, dtype, ch, groups, pad, rdtype, form)


@pytest.mark.parametrize("dtype,ch", [("f32", 5001), ("bf16", 8192), ("bf16", 16384), ("f16", 9001), ("f32", 16384),
                                      ("f32", 16383)])
def test_norm_of_wide_rows(dtype, ch):
    check_norm(3, dtype, ch, 1, 0, "f32", "scaled")
    check_norm(2, dtype, ch, 1, 0, dtype, "gate")


def check_norm(rows, dtype, ch, groups, pad, rdtype, form):
    d = Draw(rows + ch, TYPES[dtype])
    after, gated, resid = form == "gate_after", "gate" in form, form in ("residual", "scaled", "scaled_gate")
    x, xv = d.act(rows, ch, pad=pad)
    w, wv = d.f32(ch, lo=0.5, hi=1.5)
    sc, sv = d.f32(ch) if form.startswith("scaled") else (None, np.ones(ch))
    z, zv = d.act(rows, ch, pad=pad) if gated else (None, None)
    r, rv = d.act(rows, ch, scale=2.0, pad=pad, dtype=TYPES[rdtype]) if resid else (None, 0.0)
    dy, dyv = d.act(rows, ch, pad=pad)
    ds, dsv = d.act(rows, ch, pad=pad, dtype=TYPES[rdtype]) if resid else (None, 0.0)
    out, total = dwp.block_norm(x, w, residual=r, scale=sc, gate=z, gate_after=after, groups=groups)
    v = rv + sv * xv if resid else xv
    y = ref.norm(v, wv, zv, after, groups, 1e-5)
    steps = 96 + ch // groups  # the sum of squares, and the functions around it
    # relative in v and in the rms: the magnitude of out is |out|, with v's own cancellation beside it
    vm = abs(rv) + abs(sv * xv) if resid else abs(xv)
    gain = np.divide(abs(y), abs(v), out=np.zeros_like(y), where=v != 0) if rows else abs(y)
    near(out, y, gain * vm + abs(y), steps, "out")
    if resid:
        near(total, v, vm, 4, "sum")
        vin = total
        v = total.double().cpu().numpy()  # the gradient is taken at the sum as written
    else:
        assert total is None
        vin = x
    g = dwp.block_norm_backward(dy, vin, w, x=x if sc is not None else None, scale=sc, gate=z, gate_after=after,
                                grad_residual=ds, groups=groups)
    e = ref.norm_grad(dyv, v, wv, zv, after, groups, 1e-5, dsv)
    # magnitudes: the two terms of the norm's gradient, by Cauchy's bound on the mean
    if rows:
        gate = abs(ref.silu(zv)) if gated else 1.0
        t = abs(v) * gate if gated and not after else abs(v)
        rr = 1 / np.sqrt((t.reshape(rows, groups, -1) ** 2).mean(-1, keepdims=True) + 1e-5)
        gw = (abs(dyv) * wv * (gate if after else 1.0)).reshape(rows, groups, -1)
        h = t.reshape(rows, groups, -1) * rr
        dm = (rr * (gw + h * (gw * h).mean(-1, keepdims=True))).reshape(rows, ch)
        hm = h.reshape(rows, ch)
        if gated:
            near(g["gate"], e["gate"], (abs(dyv) * hm * wv if after else dm * abs(v)) * 1.2, 2 * steps, "grad gate")
        wm = (abs(dyv) * (gate if after else 1.0) * hm).sum(0)
        if gated and not after:
            dm = dm * gate
        dm = dm + abs(dsv)
    else:
        dm, wm = np.zeros((0, ch)), np.zeros(ch)
    near(g["x"], e["v"] * sv, dm * abs(sv), 2 * steps, "grad x")
    near(g["weight"], e["weight"], wm, 2 * steps + rows, "grad weight")
    if resid:
        near(g["residual"], e["v"], dm, 2 * steps, "grad residual")
    if sc is not None:
        near(g["scale"], (e["v"] * xv).sum(0), (dm * abs(xv)).sum(0), 2 * steps + rows, "grad scale")


def test_norm_in_place_and_batched_rows():
    d = Draw(9, torch.bfloat16)
    x, _ = d.act(2, 7, 264)
    r, _ = d.act(2, 7, 264, dtype=torch.float32)
    w, _ = d.f32(264)
    out, total = dwp.block_norm(x, w, residual=r)
    flat, _ = dwp.block_norm(x.view(14, 264), w, residual=r.view(14, 264))
    assert torch.equal(out.view(14, 264), flat)
    x2, r2 = x.clone(), r.clone()
    o2, t2 = dwp.block_norm(x2, w, residual=r2, out=x2, sum_out=r2)
    assert o2 is x2 and t2 is r2 and torch.equal(o2, out) and torch.equal(t2, total)


def test_scan_of_zeros_with_growing_states_is_zero():
    # A > 0: a chunk's product of decays overflows, a zero state stays zero
    rows, ch, n = 4096, 4, 16
    z, one = torch.zeros(1, rows, ch, device="cuda"), torch.ones(1, rows, 1, n, device="cuda")
    args = (z, torch.full_like(z, 8.0), torch.ones(ch, n, device="cuda"), one, one)
    out, fin, points = dwp.selective_scan(*args, dt_softplus=False, return_state=True, return_checkpoints=True)
    assert (out == 0).all() and (fin == 0).all()
    g = dwp.selective_scan_backward(z, *args, points, dt_softplus=False)
    for k, v in g.items():
        assert v is None or (v == 0).all(), k


def test_norm_of_a_row_of_zeros_is_zero():
    x = torch.zeros(2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    out, _ = dwp.block_norm(x, w)
    assert (out == 0).all()
    g = dwp.block_norm_backward(torch.ones_like(x), x, w)
    near(g["x"], np.full((2, 64), 1 / math.sqrt(1e-5)), np.full((2, 64), 1 / math.sqrt(1e-5)), 200, "grad x")


# ---------------------------------------------------------------------------
# streams, repeatability, offsets past 32 bits


def test_results_repeat_bit_for_bit_and_on_another_stream():
    c = Scan(51, "bf16", (700,), [0, 300, 300, 650, 700], 72, 16, 2)
    pos, kw = c.args()
    off = offs(c.offsets)
    side = torch.cuda.Stream()

    def run(stream):
        out, fin, pts = dwp.selective_scan(*pos, **kw, offsets=off, initial_state=c.t["init"], return_state=True,
                                           return_checkpoints=True, stream=stream)
        g = dwp.selective_scan_backward(c.t["dout"], *pos, pts, **kw, offsets=off, initial_state=c.t["init"],
                                        grad_final_state=c.t["dfinal"], stream=stream)
        w = torch.ones(72, 4, device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        y = dwp.causal_conv(c.t["u"], w, offsets=off, stream=stream)
        gy = dwp.causal_conv_backward(c.t["dout"], c.t["u"], w, offsets=off, stream=stream)
        return [out, fin, *(g[k] for k in sorted(g)), y, gy["x"], gy["weight"]]

    torch.cuda.synchronize()
    first = run(None)
    torch.cuda.synchronize()
    second = run(side)
    side.synchronize()
    third = run(None)
    torch.cuda.synchronize()
    for a, b, d in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, d)


def test_token_forms_in_a_graph():
    """A generation step captured once and replayed: the calls allocate through torch's graph pool and wait for nothing."""
    c = Scan(61, "bf16", (6, 1), None, 72, 16, 1)
    pos, kw = c.args()
    z = kw.pop("z")[:, 0]
    one = [p if p is pos[2] else p[:, 0] for p in pos]
    d = Draw(62, torch.bfloat16)
    taps, _ = d.act(6, 3, 72)
    w, _ = d.f32(72, 4)
    g, _ = d.f32(72)

    def step(conv_state, state):
        u = dwp.causal_conv_step(one[0], conv_state, w)
        y = dwp.selective_scan_step(u, *one[1:], state, z=z, **kw)
        return dwp.block_norm(y, g)[0]

    eager = [taps.clone(), c.t["init"].clone()]
    want = [step(*eager).clone() for _ in range(3)]
    state = [taps.clone(), c.t["init"].clone()]
    step(*[t.clone() for t in state])  # the library's first calls, outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*state)
    for t, s in zip(state, (taps, c.t["init"])):
        t.copy_(s)
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[k])
    assert all(torch.equal(a, b) for a, b in zip(state, eager))


@pytest.mark.parametrize("states", [16, 40, 128])
def test_one_step_of_many_sequences(states):
    """More sequences than warps: nothing is cut, and every row is a sequence's first and last."""
    c = Scan(71, "f32", (900, 1), None, 6, states, 1)
    check_scan(c)


def test_places_past_32_bits():
    """Rows and slots whose element offsets pass 2^32: the same numbers as in a small tensor."""
    ch = 32768
    big = torch.empty(140000, ch, dtype=torch.bfloat16, device="cuda")  # 9.2 GB, 4.6e9 elements
    lo = 140000 - 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    big[lo:] = torch.randn(64, ch, generator=gen, device="cuda").bfloat16()
    big[:lo].zero_()
    w = torch.randn(ch, 4, generator=gen, device="cuda")
    off = torch.tensor([0, lo, 140000], dtype=torch.int32).cuda()
    small = dwp.causal_conv(big[lo:].clone(), w)
    out = dwp.causal_conv(big, w, offsets=off)
    assert torch.equal(out[lo:], small) and (out[:lo] == 0).all()
    del out
    cache = big.view(-1, 1, ch)
    x = torch.randn(2, ch, generator=gen, device="cuda").bfloat16()
    w2 = w[:, :2].contiguous()
    few = cache[[139999, 5]].clone()
    want = dwp.causal_conv_step(x, few, w2)
    got = dwp.causal_conv_step(x, cache, w2, slots=torch.tensor([139999, 5], dtype=torch.int32).cuda())
    assert torch.equal(got, want) and torch.equal(cache[139999], few[0]) and torch.equal(cache[5], few[1])


def test_refusals_of_the_tensor_helpers():
    x = torch.zeros(4, 8, device="cuda")
    w = torch.zeros(8, 4, device="cuda")
    st = torch.zeros(4, 8, 2, device="cuda")
    A = -torch.ones(8, 2, device="cuda")
    B = torch.zeros(4, 2, device="cuda")
    for bad in (lambda: dwp.causal_conv(x.cpu(), w), lambda: dwp.causal_conv(x.double(), w),
                lambda: dwp.causal_conv(x.t().contiguous().t(), w), lambda: dwp.causal_conv(x, w[:4]),
                lambda: dwp.causal_conv(x, w.t()), lambda: dwp.causal_conv(x, w.half()),
                lambda: dwp.causal_conv(x, w, offsets=torch.zeros(2, device="cuda")),
                lambda: dwp.causal_conv(x[None], w, offsets=torch.zeros(2, dtype=torch.int32, device="cuda")),
                lambda: dwp.causal_conv(x, w, initial_state=torch.zeros(1, 2, 8, device="cuda")),
                lambda: dwp.causal_conv(x, w, out=x[:2]),
                lambda: dwp.causal_conv_step(x, torch.zeros(4, 2, 8, device="cuda"), w),
                lambda: dwp.causal_conv_step(x, torch.zeros(4, 3, 8, device="cuda"), w, slots=torch.zeros(4, device="cuda")),
                lambda: dwp.selective_scan(x, x, A.half(), B, B), lambda: dwp.selective_scan(x, x[:2], A, B, B),
                lambda: dwp.selective_scan(x, x, A, B, B[:, :1]), lambda: dwp.selective_scan(x, x, A, B.half(), B),
                lambda: dwp.selective_scan(x, x, A, B, B, D=torch.zeros(7, device="cuda")),
                lambda: dwp.selective_scan_backward(x, x, x, A, B, B, None),
                lambda: dwp.selective_scan_step(x, x, A, B, B, st.half()),
                lambda: dwp.block_norm(x, w[:, 0]), lambda: dwp.block_norm(x, w[0, :4]),
                lambda: dwp.block_norm(x, torch.ones(8, device="cuda"), residual=x[:2]),
                lambda: dwp.block_norm_backward(x, x, torch.ones(8, device="cuda"), scale=torch.ones(8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    ones = torch.ones(8, device="cuda")
    for status, bad in ((dwp.DWP_ERR_ALIASING, lambda: dwp.causal_conv(x, w, out=x)),
                        (dwp.DWP_ERR_INVALID_VALUE, lambda: dwp.causal_conv(x, torch.zeros(8, 9, device="cuda"))),
                        (dwp.DWP_ERR_INVALID_VALUE, lambda: dwp.block_norm(x, ones, groups=3)),
                        (dwp.DWP_ERR_INVALID_VALUE, lambda: dwp.block_norm(x, ones, scale=ones)),
                        (dwp.DWP_ERR_INVALID_VALUE,
                         lambda: dwp.causal_conv_step(x, torch.zeros(3, 3, 8, device="cuda"), w)),
                        (dwp.DWP_ERR_SCRATCH_TOO_SMALL,
                         lambda: dwp.causal_conv_backward(x, x, w, scratch=dwp.alloc_scratch(16, "cuda")))):
        with pytest.raises(dwp.DwpError) as err:
            bad()
        assert err.value.status == status
