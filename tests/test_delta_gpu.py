"""The gated delta rule on the GPU against its 64-bit definition.

Rows of an output of type T are held to r(T) of their own 2-norm plus 2^-14 of
the size that the definition gives (delta_ref): products of two f32 numbers are
taken in two bf16 pieces each, which loses at most 2^-16 of their magnitudes,
and from an input to an output there are at most four such products one after
another (the chunk's inverse, the corrections, the state, the read).  r(T) is
half a unit of T and as much again for its neighbourhood.

A bf16 output's weights are rounded to one bf16: half a unit, 2^-9, of each.
The terms are weight_j u_j for each row j of the chunk, and the size bounds
sum_j |q||k_j||u_j|, decayed.  So this rounding costs at most 2^-9 of the size.
"""
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
from test_sequence_gpu import SHAPES, IDS, SENTINEL, TYPES, covered, offs, spans  # noqa: E402

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -9, torch.float16: 2.0 ** -12}
TINY = {torch.float32: 1e-35, torch.bfloat16: 1e-35, torch.float16: 2.0 ** -24}
E = 2.0 ** -14
E_OUT = {torch.float32: E, torch.float16: E, torch.bfloat16: E + 2.0 ** -9}


@pytest.fixture(scope="module", autouse=True)
def lib():
    dwp_build.build()
    return dwp.load()


def rows_near(got, exact, size, what, e=E):
    """Rows (..., n) in the 2-norm."""
    g = got.detach().double().cpu().numpy()
    assert g.shape == exact.shape, what
    bound = 4 * HALF[got.dtype] * ref.norm(exact) + e * size + TINY[got.dtype] * math.sqrt(max(1, exact.shape[-1]))
    worst = (ref.norm(g - exact) / bound).max() if g.size else 0.0
    assert np.isfinite(g).all() and worst <= 1.0, "%s: %.3g times the bound" % (what, worst)


class Case:
    """Seeded inputs of one call, as tensors and as the 64-bit values they hold."""

    def __init__(self, seed, lead, offsets, dtype, key_heads, heads, keys, values, pad=0, decay=1.0, beta_dtype=None, count=None):
        r = np.random.default_rng(seed)
        self.T, self.lead, self.offsets, self.per = TYPES[dtype], lead, offsets, heads // key_heads
        self.scale = keys ** -0.5
        self.values = {}
        n = len(spans(lead, offsets)) if count is None else count

        def put(name, x, dtype, pad=0):
            t = torch.from_numpy(x).to(dtype)
            self.values[name] = t.double().numpy()
            if pad:  # heads of a wider tensor, from an odd place
                wide = torch.full((*t.shape[:-1], t.shape[-1] + 2 * pad + 1), SENTINEL, dtype=dtype)
                wide[..., pad:pad + t.shape[-1]] = t
                t = wide.cuda()[..., pad:pad + t.shape[-1]]
            setattr(self, name, t.cuda())

        def unit(*shape):
            x = r.standard_normal(shape)
            return x / np.maximum(np.sqrt((x * x).sum(-1, keepdims=True)), 1e-9) * 0.995

        put("q", unit(*lead, key_heads, keys), self.T, pad)
        put("k", unit(*lead, key_heads, keys), self.T, pad)
        put("v", r.standard_normal((*lead, heads, values)), self.T, pad)
        put("grad", r.standard_normal((*lead, heads, values)), self.T, pad)
        put("g", -decay * np.abs(r.standard_normal((*lead, heads))), torch.float32, 1 if pad else 0)
        put("beta", r.uniform(0, 1, (*lead, heads)), TYPES[beta_dtype or "f32"], 1 if pad else 0)
        put("state", r.standard_normal((n, heads, keys, values)) * 0.3, torch.float32)
        put("grad_state", r.standard_normal((n, heads, keys, values)) * 0.1, torch.float32)

    def args(self):
        return self.q, self.k, self.v, self.g, self.beta

    def head(self, rows, h):
        """One head's rows of the flattened stream, as the definition takes them."""
        flat = lambda n: self.values[n].reshape(-1, *self.values[n].shape[len(self.lead):])[rows]  # noqa: E731
        kh = h // self.per
        return (flat("q")[:, kh], flat("k")[:, kh], flat("v")[:, h], flat("g")[:, h], flat("beta")[:, h])

    def grad_of(self, rows, h):
        return self.values["grad"].reshape(-1, *self.values["grad"].shape[len(self.lead):])[rows][:, h]


def check(c, out, final, grads=None):
    """Every output of a call against the definition."""
    lead, offsets = c.lead, c.offsets
    heads, key_heads = c.v.shape[-2], c.k.shape[-2]
    flat = lambda t: t.reshape(-1, *t.shape[len(lead):])  # noqa: E731
    out = flat(out)
    if grads:
        rows_grads = {n: flat(grads[n]) for n in ("q", "k", "v", "g", "beta")}
        shared = {n: (np.zeros(rows_grads[n].shape), np.zeros(rows_grads[n].shape[:2])) for n in ("q", "k")}
    for i, rows in enumerate(spans(lead, offsets)):
        for h in range(heads):
            x, s0 = c.head(rows, h), c.values["state"][i, h]
            want, last, sizes, size, _ = ref.delta(*x, c.scale, s0)
            rows_near(out[rows][:, h], want, sizes, "out", E_OUT[c.T])
            rows_near(final[i, h].flatten(), last.flatten(), size, "final state")
            if grads is None:
                continue
            G, Z = ref.delta_grad(c.grad_of(rows, h), *x, c.scale, s0, c.values["grad_state"][i, h])
            rows_near(rows_grads["v"][rows][:, h], G["v"], Z["v"], "dv")
            for n in ("g", "beta"):
                rows_near(rows_grads[n][rows][:, h, None], G[n][:, None], Z[n], "d" + n)
            rows_near(grads["initial_state"][i, h].flatten(), G["initial_state"].flatten(), Z["initial_state"], "dinitial")
            for n in ("q", "k"):
                shared[n][0][rows, h // c.per] += G[n]
                shared[n][1][rows, h // c.per] += Z[n]
    if grads:
        live = covered(lead, offsets)
        at = torch.from_numpy(live).cuda()
        for n in ("q", "k"):
            rows_near(rows_grads[n][at], shared[n][0][live], shared[n][1][live], "d" + n)


SIZES = [("f32", 1, 1, 5, 3, 0), ("bf16", 2, 4, 128, 128, 0), ("f16", 1, 3, 33, 20, 2), ("f32", 2, 2, 64, 72, 4),
         ("bf16", 1, 1, 1, 1, 0), ("bf16", 1, 2, 64, 64, 8), ("f16", 2, 2, 128, 64, 0)]


@pytest.mark.parametrize("dtype,key_heads,heads,keys,values,pad", SIZES)
@pytest.mark.parametrize("lead,offsets", SHAPES, ids=IDS)
def test_delta(lead, offsets, dtype, key_heads, heads, keys, values, pad):
    c = Case(len(lead) * 100 + keys, lead, offsets, dtype, key_heads, heads, keys, values, pad,
             beta_dtype=dtype if keys == 33 else None)
    out = torch.full((*lead, heads, values), SENTINEL, dtype=c.T, device="cuda")
    out, final, points = dwp.gated_delta_rule(*c.args(), scale=c.scale, offsets=offs(offsets), initial_state=c.state,
                                              return_state=True, return_checkpoints=True, out=out)
    grads = dwp.gated_delta_rule_backward(c.grad, *c.args(), points, scale=c.scale, offsets=offs(offsets),
                                          initial_state=c.state, grad_final_state=c.grad_state)
    check(c, out, final, grads)
    if offsets is not None and not covered(lead, offsets).all():
        outside = torch.from_numpy(~covered(lead, offsets)).cuda()
        assert (out[outside] == SENTINEL).all()
    # without what the gradient needs the results are the same numbers
    again, last = dwp.gated_delta_rule(*c.args(), scale=c.scale, offsets=offs(offsets), initial_state=c.state, return_state=True)
    live = torch.from_numpy(covered(lead, offsets)).cuda()
    flat = lambda t: t.reshape(-1, heads, values)[live]  # noqa: E731
    assert torch.equal(flat(again), flat(out)) and torch.equal(last, final)


@pytest.mark.parametrize("dtype,heads,keys,values", [("bf16", 4, 128, 128), ("f32", 3, 40, 24), ("f16", 2, 128, 64)])
def test_step_continues_a_prompt(dtype, heads, keys, values):
    """A prompt run whole is the prompt cut anywhere and continued row by row; padding rows change nothing."""
    rows, cut, slots = 75, 70, 5
    c = Case(7, (2, rows), None, dtype, 1, heads, keys, values)
    out, final = dwp.gated_delta_rule(*c.args(), scale=c.scale, initial_state=c.state, return_state=True)
    part = [t[:, :cut] for t in c.args()]
    _, mid = dwp.gated_delta_rule(*part, scale=c.scale, initial_state=c.state, return_state=True)
    cache = torch.full((slots, heads, keys, values), SENTINEL, device="cuda")
    place = torch.tensor([3, -1, 1], dtype=torch.int32, device="cuda")
    cache[3], cache[1] = mid[0], mid[1]
    got = []
    for t in range(cut, rows):
        x = [torch.stack([a[0, t], a[1, t], a[1, t]]) for a in c.args()]
        y = dwp.gated_delta_rule_step(*x, cache, scale=c.scale, slots=place)
        assert (y[1] == 0).all()
        got.append(y[[0, 2]])
    assert (cache[[0, 2, 4]] == SENTINEL).all()
    want = [ref.delta(*(a for a in c.head(slice(b * rows, (b + 1) * rows), h)), c.scale, c.values["state"][b, h])
            for b in range(2) for h in range(heads)]
    for b in range(2):
        for h in range(heads):
            o, last, sizes, size, _ = want[b * heads + h]
            rows_near(torch.stack(got)[:, b, h], o[cut:], sizes[cut:], "token form")
            rows_near(cache[[3, 1]][b, h].flatten(), last.flatten(), size, "token state")
            rows_near(final[b, h].flatten(), last.flatten(), size, "prompt state")
