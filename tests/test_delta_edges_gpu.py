"""The gated delta rule and the layer norm at the edge: values that are not
finite next to a sequence, decays from none to all, many chunks, other streams
and captured graphs, scratch with any contents, determinism, the helpers'
refusals, and the operators together in a layer."""
import math

import numpy as np
import pytest

import delta_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import device_wide_prefix_gb300 as dwp  # noqa: E402
from device_wide_prefix_gb300 import build as dwp_build  # noqa: E402
from test_delta_gpu import Case, E_OUT, check, rows_near  # noqa: E402
from test_sequence_gpu import SENTINEL, offs  # noqa: E402

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def lib():
    dwp_build.build()
    return dwp.load()


def forward(c, **more):
    return dwp.gated_delta_rule(*c.args(), scale=c.scale, offsets=offs(c.offsets), initial_state=c.state, return_state=True,
                                return_checkpoints=True, **more)


def backward(c, points, **more):
    return dwp.gated_delta_rule_backward(c.grad, *c.args(), points, scale=c.scale, offsets=offs(c.offsets),
                                         initial_state=c.state, grad_final_state=c.grad_state, **more)


@pytest.mark.parametrize("dtype,keys,values", [("bf16", 128, 128), ("f32", 40, 24), ("f16", 64, 128)])
@pytest.mark.parametrize("fill", [NAN, math.inf, -65504.0])
def test_rows_outside_the_sequences(dtype, keys, values, fill):
    """Rows outside the segments, before, between and behind them, hold anything."""
    offsets = [3, 40, 40, 130]
    c = Case(5, (170,), offsets, dtype, 2, 4, keys, values)
    outside = torch.ones(170, dtype=torch.bool, device="cuda")
    outside[3:130] = False
    for t in (c.q, c.k, c.v, c.g, c.beta, c.grad):
        t[outside] = fill
    out, final, points = forward(c, out=torch.full((170, 4, values), SENTINEL, dtype=c.T, device="cuda"))
    assert (out[outside] == SENTINEL).all()
    check(c, out, final, backward(c, points))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_another_sequence_is_not_reached(dtype):
    """A sequence that is not finite leaves its neighbours, and their gradients, as they are."""
    offsets = [0, 50, 90, 200]
    c, d = (Case(6, (200,), offsets, dtype, 1, 2, 128, 64) for _ in range(2))
    for t in (d.q, d.k, d.v, d.grad):
        t[50:90] = NAN
    want, got = forward(c), forward(d)
    keep = torch.ones(200, dtype=torch.bool, device="cuda")
    keep[50:90] = False
    assert torch.equal(want[0][keep], got[0][keep]) and torch.equal(want[1][[0, 2]], got[1][[0, 2]])
    want, got = backward(c, want[2]), backward(d, got[2])
    for n in ("q", "k", "v", "g", "beta"):
        assert torch.equal(want[n][keep], got[n][keep]), n
    assert torch.equal(want["initial_state"][[0, 2]], got["initial_state"][[0, 2]])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["none", "zero", "resets", "lowest", "strong", "tiny"])
def test_decays(kind, dtype):
    c = Case(8, (2, 200), None, dtype, 1, 2, 64, 64)
    g = c.g
    if kind in ("none", "zero"):
        g.zero_()
    elif kind == "resets":
        g[:, ::13] = -math.inf
    elif kind == "lowest":
        g[:, 5::9] = torch.finfo(torch.float32).min
    elif kind == "strong":
        g.fill_(-90.0)
        g[:, 70:100] = -0.01
    else:
        g.mul_(1e-6)
    # the definition takes the decays as they count
    c.values["g"] = np.maximum(g.double().cpu().numpy(), -110.0)
    args = list(c.args())
    if kind == "none":
        args[3] = None
    out, final, points = dwp.gated_delta_rule(*args, scale=c.scale, initial_state=c.state, return_state=True,
                                              return_checkpoints=True)
    grads = dwp.gated_delta_rule_backward(c.grad, *args, points, scale=c.scale, initial_state=c.state,
                                          grad_final_state=c.grad_state)
    if kind == "none":
        assert "g" not in grads
        grads["g"] = dwp.gated_delta_rule_backward(c.grad, *c.args(), points, scale=c.scale, initial_state=c.state,
                                                   grad_final_state=c.grad_state)["g"]
    check(c, out, final, grads)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f16"])
@pytest.mark.parametrize("strength", [0.0, 1.0])
def test_strengths(strength, dtype):
    """beta 0 reads and never writes; beta 1 replaces."""
    c = Case(9, (1, 140), None, dtype, 1, 1, 128, 128, decay=0.05)
    c.beta.fill_(strength)
    c.values["beta"][:] = strength
    out, final, points = forward(c)
    check(c, out, final, backward(c, points))


@pytest.mark.parametrize("dtype,rows", [("bf16", 1027), ("f32", 640)])
def test_many_chunks(dtype, rows):
    c = Case(10, (1, rows), None, dtype, 1, 1, 128, 128, decay=0.02)
    out, final, points = forward(c)
    check(c, out, final, backward(c, points))


@pytest.mark.parametrize("dtype,batch,rows,heads,keys,values,pad", [
    ("bf16", 1, 1600, 1, 128, 128, 0), ("bf16", 2, 2049, 1, 64, 128, 0), ("f32", 1, 1537, 2, 40, 72, 0),
    ("f16", 1, 1599, 1, 128, 64, 0), ("bf16", 1, 1600, 1, 72, 24, 1), ("f32", 1, 5184, 1, 16, 16, 0),
    ("bf16", 1, 5185, 1, 16, 16, 0)])
def test_sequences_cut_in_parts(dtype, batch, rows, heads, keys, values, pad):
    """Few heads and many chunks: three parts and more, the last one short, one row long or empty."""
    c = Case(24, (batch, rows), None, dtype, 1, heads, keys, values, pad, decay=0.01)
    out, final, points = forward(c)
    check(c, out, final, backward(c, points))


def test_cut_sequences_scratch_capture_and_neighbours():
    """Sequences cut in parts: any scratch gives the same, captured calls too; a value that is not finite reaches
    neither its neighbours nor, forward, the chunks before it."""
    cases = [Case(s, (2, 2000), None, "bf16", 1, 2, 128, 64, decay=0.01) for s in (25, 26)]
    live = Case(25, (2, 2000), None, "bf16", 1, 2, 128, 64, decay=0.01)
    wants = [forward(c) for c in cases]
    backs = [backward(c, w[2]) for c, w in zip(cases, wants)]
    for byte in (0, 0xFF):
        scratch = torch.full((1 << 25,), byte, dtype=torch.uint8, device="cuda")
        got = forward(cases[0], scratch=scratch)
        assert all(torch.equal(a, b) for a, b in zip(wants[0][:2], got[:2]))
        scratch.fill_(byte)
        again = backward(cases[0], got[2], scratch=scratch)
        assert all(torch.equal(backs[0][k], again[k]) for k in again)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        backward(live, forward(live)[2])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = forward(live)
        grads = backward(live, res[2])
    for c, want, back in list(zip(cases, wants, backs))[::-1]:
        for n in ("q", "k", "v", "g", "beta", "grad", "state", "grad_state"):
            getattr(live, n).copy_(getattr(c, n))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(res[0], want[0]) and torch.equal(res[1], want[1])
        assert all(torch.equal(grads[k], back[k]) for k in back)
    for value in (NAN, math.inf):
        live.v.copy_(cases[0].v)
        live.v[0, 1000, 1, 5] = value
        out, final, points = forward(live)
        assert torch.equal(out[1], wants[0][0][1]) and torch.equal(final[1], wants[0][1][1])
        assert torch.equal(out[0, :, 0], wants[0][0][0, :, 0]) and torch.equal(out[0, :960], wants[0][0][0, :960])
        more = backward(live, points)
        for n in ("v", "g", "beta"):
            assert torch.equal(more[n][1], backs[0][n][1]) and torch.equal(more[n][0, :, 0], backs[0][n][0, :, 0]), n
        assert torch.equal(more["initial_state"][1], backs[0]["initial_state"][1])


def test_keys_all_alike():
    """One key over and over, strength 1, no decay: the worst inverse, whose entries stay bounded."""
    c = Case(11, (1, 192), None, "f32", 1, 1, 64, 64, decay=0.0)
    c.k[:] = c.k[:, :1]
    c.values["k"][:] = c.values["k"][:, :1]
    c.beta.fill_(1.0)
    c.values["beta"][:] = 1.0
    out, final, points = forward(c)
    check(c, out, final, backward(c, points))


def test_gradient_against_differences():
    """The loss's change along random directions, in f32 from f32 inputs."""
    c = Case(12, (1, 100), None, "f32", 1, 2, 32, 32)
    names = ("q", "k", "v", "g", "beta")
    points = forward(c)[2]
    grads = backward(c, points)

    def loss(args, state):
        out, final = dwp.gated_delta_rule(*args, scale=c.scale, initial_state=state, return_state=True)
        return ((out.double() * c.grad.double()).sum() + (final.double() * c.grad_state.double()).sum()).item()

    gen = torch.Generator(device="cuda").manual_seed(1)
    for i, name in enumerate((*names, "initial_state")):
        x = c.state if name == "initial_state" else c.args()[i]
        d = torch.randn(x.shape, generator=gen, device="cuda")
        h = 2.0 ** -7 / d.abs().max().item()
        ends = []
        for sign in (1, -1):
            args, state = list(c.args()), c.state
            if name == "initial_state":
                state = state + sign * h * d
            else:
                args[i] = args[i] + sign * h * d
            ends.append(loss(args, state))
        got, want = (ends[0] - ends[1]) / (2 * h), (grads[name].double() * d).sum().item()
        size = (grads[name].double().norm() * d.double().norm()).item()
        # the third order of steps of at most 2^-7, and the losses' own 2^-16 over the step
        assert abs(got - want) <= 2e-3 * size + 1e-3 * abs(want), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bit_for_bit(dtype):
    c = Case(13, (300,), [0, 100, 130, 300], dtype, 2, 4, 128, 64)
    first = forward(c)
    grads = backward(c, first[2])
    for _ in range(3):
        again = forward(c)
        assert all(torch.equal(a, b) for a, b in zip(first[:2], again[:2]))
        more = backward(c, again[2])
        assert all(torch.equal(grads[k], more[k]) for k in grads)


def test_scratch_of_any_contents():
    c = Case(14, (130,), [0, 1, 70, 130], "bf16", 1, 2, 64, 128)
    want = dwp.gated_delta_rule(*c.args(), scale=c.scale, offsets=offs(c.offsets), initial_state=c.state, return_state=True)
    for byte in (0, 0x7F, 0xFF):
        scratch = torch.full((1 << 22,), byte, dtype=torch.uint8, device="cuda")
        got = dwp.gated_delta_rule(*c.args(), scale=c.scale, offsets=offs(c.offsets), initial_state=c.state,
                                   return_state=True, scratch=scratch)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        points = torch.full(forward(c)[2].shape, NAN, device="cuda")
        again = forward(c, checkpoints=points)
        a, b = backward(c, forward(c)[2]), backward(c, again[2], scratch=scratch)
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_without_states():
    """No initial state is a state of zeros, and a gradient without final states one of zeros."""
    c = Case(15, (2, 90), None, "bf16", 1, 2, 128, 128)
    zero = torch.zeros_like(c.state)
    out, points = dwp.gated_delta_rule(*c.args(), return_checkpoints=True)
    assert torch.equal(out, dwp.gated_delta_rule(*c.args(), scale=128 ** -0.5, initial_state=zero))
    g = dwp.gated_delta_rule_backward(c.grad, *c.args(), points)
    assert set(g) == {"q", "k", "v", "g", "beta"}
    h = dwp.gated_delta_rule_backward(c.grad, *c.args(), points, initial_state=zero, grad_final_state=zero)
    assert all(torch.equal(g[k], h[k]) for k in g)


def test_other_stream_and_captured_graph():
    """A training step and a token step, captured, replayed on new inputs, and on another stream."""
    c, d = (Case(s, (2, 100), None, "bf16", 1, 2, 128, 128) for s in (16, 17))
    names = ("q", "k", "v", "g", "beta", "grad", "state", "grad_state")
    live = Case(16, (2, 100), None, "bf16", 1, 2, 128, 128)
    token = [t[:, 0].contiguous() for t in live.args()]
    cache = live.state.clone()

    def step():
        res = forward(live)
        grads = backward(live, res[2])
        y = dwp.gated_delta_rule_step(*token, cache, scale=live.scale)
        return res, grads, y

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res, grads, y = step()
    for other in (d, c):
        for n in names:
            getattr(live, n).copy_(getattr(other, n))
        cache.copy_(other.state)
        for t, a in zip(token, other.args()):
            t.copy_(a[:, 0])
        graph.replay()
        want = forward(other)
        back = backward(other, want[2])
        state = other.state.clone()
        one = dwp.gated_delta_rule_step(*(a[:, 0].contiguous() for a in other.args()), state, scale=other.scale)
        torch.cuda.synchronize()
        assert torch.equal(res[0], want[0]) and torch.equal(res[1], want[1])
        assert all(torch.equal(grads[k], back[k]) for k in back)
        assert torch.equal(y, one) and torch.equal(cache, state)
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
        on_side = dwp.gated_delta_rule(*other.args(), scale=other.scale, initial_state=other.state, stream=side)
        side.synchronize()
        assert torch.equal(on_side, want[0])


def test_two_streams_at_once():
    cases = [Case(s, (1, 500), None, "bf16", 2, 8, 128, 128) for s in (18, 19)]
    want = [forward(c)[0] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(4):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(forward(c)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 2]) for i, g in enumerate(got))


def test_views_of_a_projection():
    """Queries, keys and values as columns of one wide row, decays and strengths of another; any alignment."""
    rows, heads, n = 150, 3, 64
    c = Case(20, (2, rows), None, "bf16", 3, heads, n, n)
    for shift in (0, 8, 1):
        wide = torch.full((2, rows, 3 * heads * n + 16), SENTINEL, dtype=torch.bfloat16, device="cuda")
        views = [wide[..., shift + i * heads * n:shift + (i + 1) * heads * n].unflatten(-1, (heads, n)) for i in range(3)]
        for v, t in zip(views, (c.q, c.k, c.v)):
            v.copy_(t)
        gates = torch.zeros(2, rows, 2 * heads, device="cuda")
        gates[..., :heads], gates[..., heads:] = c.g, c.beta
        out = dwp.gated_delta_rule(*views, gates[..., :heads], gates[..., heads:], scale=c.scale, initial_state=c.state)
        want = dwp.gated_delta_rule(*c.args(), scale=c.scale, initial_state=c.state)
        assert torch.equal(out, want), shift


def test_output_in_place_of_none():
    """An output whose heads are apart, written through; what lies between stays."""
    c = Case(21, (1, 70), None, "f32", 1, 2, 16, 8)
    wide = torch.full((1, 70, 2, 20), SENTINEL, device="cuda")
    got = dwp.gated_delta_rule(*c.args(), scale=c.scale, initial_state=c.state, out=wide[..., 3:11])
    assert torch.equal(got, dwp.gated_delta_rule(*c.args(), scale=c.scale, initial_state=c.state))
    assert (wide[..., :3] == SENTINEL).all() and (wide[..., 11:] == SENTINEL).all()


@pytest.mark.parametrize("dtype,keys,values,stride", [("bf16", 128, 128, 0), ("f32", 7, 5, 3), ("f16", 64, 36, 4)])
def test_step_slots(dtype, keys, values, stride):
    """Slots in any order, some outside the cache, in a cache with room between the slots."""
    batch, heads = 9, 2
    c = Case(22, (batch,), None, dtype, 1, heads, keys, values, count=12)
    room = torch.full((12, heads * keys * values + stride), SENTINEL, device="cuda")
    cache = room[:, :heads * keys * values].unflatten(1, (heads, keys, values)) if stride == 0 else torch.as_strided(
        room, (12, heads, keys, values), (heads * keys * values + stride, keys * values, values, 1))
    cache.copy_(c.state)
    slots = torch.tensor([11, 0, -1, 5, 12, 7, 2**31 - 1, 3, -2**31], dtype=torch.int32, device="cuda")
    out = dwp.gated_delta_rule_step(*c.args(), cache, scale=c.scale, slots=slots)
    for i, slot in enumerate(slots.tolist()):
        if not 0 <= slot < 12:
            assert (out[i] == 0).all()
            continue
        for h in range(heads):
            o, last, sizes, size, _ = ref.delta(*c.head(slice(i, i + 1), h), c.scale, c.values["state"][slot, h])
            rows_near(out[i:i + 1, h], o, sizes, "out")
            rows_near(cache[slot, h].flatten(), last.flatten(), size, "state")
    rest = [s for s in range(12) if s not in slots.tolist()]
    assert torch.equal(cache[rest], c.state[rest])
    assert stride == 0 or (room[:, heads * keys * values:] == SENTINEL).all()


def test_refusals():
    c = Case(23, (2, 10), None, "bf16", 1, 2, 16, 8)
    q, k, v, g, beta = c.args()
    bad = [lambda: dwp.gated_delta_rule(q.float(), k, v, g, beta), lambda: dwp.gated_delta_rule(q, k[:, :9], v, g, beta),
           lambda: dwp.gated_delta_rule(q, k, v, g.bfloat16(), beta), lambda: dwp.gated_delta_rule(q, k, v, g, beta.half()),
           lambda: dwp.gated_delta_rule(q, k, v, g[..., :1], beta), lambda: dwp.gated_delta_rule(q, k[..., :8], v, g, beta),
           lambda: dwp.gated_delta_rule(q, k, v, g, beta, initial_state=c.state[:1]),
           lambda: dwp.gated_delta_rule(q, k, v, g, beta, offsets=offs([0, 10])),
           lambda: dwp.gated_delta_rule(q.cpu(), k, v, g, beta), lambda: dwp.gated_delta_rule(q, k, v.cpu(), g, beta),
           lambda: dwp.gated_delta_rule(q, k, v, g, beta, out=v[..., :4]),
           lambda: dwp.gated_delta_rule(q, k, v.transpose(-1, -2), g, beta),
           lambda: dwp.gated_delta_rule_backward(c.grad, q, k, v, g, beta, None),
           lambda: dwp.gated_delta_rule_backward(c.grad, q, k, v, g, beta, torch.zeros(2, 2, 5, device="cuda")),
           lambda: dwp.gated_delta_rule_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], c.state.bfloat16()),
           lambda: dwp.gated_delta_rule_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], c.state,
                                             slots=torch.zeros(2, dtype=torch.int64, device="cuda")),
           lambda: dwp.layer_norm(v[..., 0], weight=torch.ones(3, device="cuda")),
           lambda: dwp.layer_norm_backward(v[:, :, 0], v[:, :, 0].float(), residual=False)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d was taken" % i)
    with pytest.raises(dwp.DwpError):  # three heads do not share two key heads
        dwp.gated_delta_rule(q.expand(2, 10, 1, 16).repeat(1, 1, 2, 1), k.repeat(1, 1, 2, 1),
                             torch.zeros(2, 10, 3, 8, dtype=torch.bfloat16, device="cuda"),
                             torch.zeros(2, 10, 3, device="cuda"), torch.zeros(2, 10, 3, device="cuda"))
    with pytest.raises(dwp.DwpError):  # the output over its input
        dwp.gated_delta_rule(q, k, v, g, beta, out=v)


def test_nothing_to_do():
    empty = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    state = torch.ones(2, 3, 8, 4, device="cuda")
    out, final = dwp.gated_delta_rule(empty(2, 0, 1, 8), empty(2, 0, 1, 8), empty(2, 0, 3, 4), empty(2, 0, 3), empty(2, 0, 3),
                                      initial_state=state, return_state=True)
    assert out.shape == (2, 0, 3, 4) and torch.equal(final, state)
    y = dwp.gated_delta_rule_step(empty(0, 1, 8), empty(0, 1, 8), empty(0, 3, 4), empty(0, 3), empty(0, 3), state)
    assert y.shape == (0, 3, 4) and (state == 1).all()
    g = dwp.layer_norm_backward(empty(0, 6), empty(0, 6), empty(6) + 1, empty(6) + 1)
    assert (g["weight"] == 0).all() and (g["bias"] == 0).all()


def test_layer_norm_in_place_and_captured():
    x, r = torch.randn(50, 640, device="cuda").bfloat16(), torch.randn(50, 640, device="cuda")
    w, b = torch.rand(640, device="cuda"), torch.randn(640, device="cuda")
    want, total = dwp.layer_norm(x, w, b, residual=r, groups=5)
    a, s = x.clone(), r.clone()
    dwp.layer_norm(a, w, b, residual=s, groups=5, out=a, sum_out=s)
    assert torch.equal(a, want) and torch.equal(s, total)
    live = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dwp.layer_norm_backward(live, total, w, b, groups=5)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dwp.layer_norm_backward(live, total, w, b, groups=5)
    live.copy_(want)
    graph.replay()
    again = dwp.layer_norm_backward(want, total, w, b, groups=5)
    assert all(torch.equal(got[k], again[k]) for k in again)


@pytest.mark.parametrize("value", [math.inf, NAN])
def test_layer_norm_rows_apart(value):
    """A row or group that is not finite touches no other output row."""
    x = torch.randn(9, 96, device="cuda")
    want = dwp.layer_norm(x, groups=3)[0]
    x[4, 40] = value
    got = dwp.layer_norm(x, groups=3)[0]
    keep = torch.ones(9, 96, dtype=torch.bool, device="cuda")
    keep[4, 32:64] = False
    assert torch.equal(got[keep], want[keep]) and not torch.isfinite(got[4, 32:64]).any()


def plain_layer(layer, y, residual):
    """The example's layer in 64 bits, elementary operations and torch's own gradient."""
    P = {k: v.detach().double().requires_grad_() for k, v in layer.named_parameters()}
    Y, R = y.double().requires_grad_(), residual.double().requires_grad_()
    norm = lambda t, w, b: (t - t.mean(-1, keepdim=True)) * torch.rsqrt(t.var(-1, unbiased=False, keepdim=True) + 1e-5) * w + b  # noqa: E731
    r = R + Y
    x = norm(r, P["norm"], P["norm_bias"])
    u = torch.nn.functional.pad(x @ P["w_qkv"], (0, 0, layer.taps - 1, 0))
    rows = y.shape[1]
    u = torch.nn.functional.silu(sum(P["conv"][:, i] * u[:, i:i + rows] for i in range(layer.taps)) + P["conv_bias"])
    n = layer.key_heads * layer.keys
    q, k, v = u.split([n, n, layer.heads * layer.values], -1)
    unit = lambda t: (lambda s: s * torch.rsqrt(s.square().mean(-1, keepdim=True) + 1e-5) * layer.keys ** -0.5)(  # noqa: E731
        t.unflatten(-1, (layer.key_heads, layer.keys))).repeat_interleave(layer.heads // layer.key_heads, 2)
    q, k, v = unit(q), unit(k), v.unflatten(-1, (layer.heads, layer.values))
    a, b = (x @ P["w_gates"]).split(layer.heads, -1)
    g, beta = -P["rate"].exp() * torch.nn.functional.softplus(a + P["step"]), torch.sigmoid(b)
    S, outs = 0.0, []
    for t in range(rows):
        S = g[:, t].exp()[..., None, None] * (S if t else torch.zeros(*v[:, 0].shape[:2], layer.keys, layer.values,
                                                                     dtype=torch.float64, device="cuda"))
        h = v[:, t] - torch.einsum("bhk,bhkv->bhv", k[:, t], S)
        S = S + k[:, t][..., None] * (beta[:, t][..., None] * h)[..., None, :]
        outs.append(layer.keys ** -0.5 * torch.einsum("bhk,bhkv->bhv", q[:, t], S))
    o = torch.stack(outs, 1)
    o = norm(o, 1.0, 0.0).flatten(-2) * P["head_norm"] + P["head_bias"]
    return o @ P["w_out"], r, P, Y, R


def test_layer_forward_and_gradient():
    """The operators together, trained: outputs and every parameter's gradient against 64 bits."""
    from examples.delta_rule_layer import Layer
    torch.manual_seed(3)
    layer = Layer(width=64, key_heads=1, heads=2, keys=32, values=32, dtype=torch.float32)
    y, res = torch.randn(2, 100, 64, device="cuda", requires_grad=True), torch.randn(2, 100, 64, device="cuda", requires_grad=True)
    was = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        out, r = layer(y, res)
        dy, dr = torch.randn_like(out), torch.randn_like(r)
        torch.autograd.backward((out, r), (dy, dr))
    finally:
        torch.backends.cuda.matmul.allow_tf32 = was
    want, wr, P, Y, R = plain_layer(layer, y.detach(), res.detach())
    torch.autograd.backward((want, wr), (dy.double(), dr.double()))
    # a chain of a dozen f32 operators, the recurrence's products in two bf16 pieces (2^-16 each)
    close = lambda a, b, what: (a.double() - b).norm() <= 2.0 ** -12 * b.norm() or pytest.fail(  # noqa: E731
        "%s: %.2g" % (what, (a.double() - b).norm() / b.norm()))
    close(out, want, "out")
    close(y.grad, Y.grad, "dy")
    close(res.grad, R.grad, "dresidual")
    for name, p in layer.named_parameters():
        close(p.grad, P[name].grad, name)


def test_layer_runs():
    """The example's own run: trained steps are finite, and prompts continue token by token."""
    from examples import delta_rule_layer as ex
    layer, first, last = ex.train(steps=3)
    assert math.isfinite(first) and math.isfinite(last)
    # bf16 activations through a dozen operators: a few of bf16's units of the output's largest value
    assert ex.generate(layer) < 12 * 2.0 ** -8
