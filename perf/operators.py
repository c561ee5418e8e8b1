"""The sequence operators of a state space layer, as cases to measure.

Each case is one operator: the short causal convolution (prompts, gradient,
single tokens), the selective state space scan (prompts, training step,
single tokens) and the norm around the block (with residual scale or gate,
and its gradient).  `run` computes it in elementary torch operations in 32
bits (own = False) or through device_wide_prefix_gb300 (own = True).
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # prompt processing: many packed requests of uneven length (some empty), each continuing its own state
        {"name": "conv_prompt_packed", "op": "conv", "dtype": "bf16", "batch": 1, "rows": 16384, "segments": 37,
         "channels": 5120, "width": 4},
        # training: gradient of the convolution over a batch of equal sequences
        {"name": "conv_gradient", "op": "conv_grad", "dtype": "bf16", "batch": 4, "rows": 2048, "segments": 0,
         "channels": 4096, "width": 4},
        # generation: one token for each running request, states in a slot cache
        {"name": "conv_token", "op": "conv_step", "dtype": "bf16", "batch": 64, "channels": 4096, "width": 4},
        # one short prompt of a small layer: latency counts
        {"name": "scan_short", "op": "scan", "dtype": "bf16", "batch": 1, "rows": 128, "segments": 0, "channels": 1024,
         "states": 16, "groups": 1},
        # an ordinary batch of prompts
        {"name": "scan_prompt", "op": "scan", "dtype": "bf16", "batch": 4, "rows": 2048, "segments": 0, "channels": 4096,
         "states": 16, "groups": 1},
        # one very long prompt: few channels, many rows
        {"name": "scan_long", "op": "scan", "dtype": "bf16", "batch": 1, "rows": 65536, "segments": 0, "channels": 2048,
         "states": 16, "groups": 1},
        # packed requests at sizes that no tile divides, in 32 bits
        {"name": "scan_packed_f32", "op": "scan", "dtype": "f32", "batch": 1, "rows": 4099, "segments": 23,
         "channels": 1002, "states": 12, "groups": 2},
        # a training step of the scan: forward, then every gradient
        {"name": "scan_train", "op": "scan_train", "dtype": "bf16", "batch": 2, "rows": 2048, "segments": 0,
         "channels": 4096, "states": 16, "groups": 1},
        # generation at a full batch: the state cache is read and written
        {"name": "scan_token", "op": "scan_step", "dtype": "bf16", "batch": 256, "channels": 4096, "states": 16,
         "groups": 1},
        # before a block: residual stream in 32 bits, per-channel residual scale
        {"name": "norm_residual", "op": "norm", "dtype": "bf16", "rows": 8192, "channels": 4096, "groups": 1,
         "form": "residual"},
        # the same for one token of a few requests: latency counts
        {"name": "norm_token", "op": "norm", "dtype": "bf16", "rows": 8, "channels": 4096, "groups": 1,
         "form": "residual"},
        # after a block, training: gradient of the gated norm in groups
        {"name": "norm_gated_gradient", "op": "norm_grad", "dtype": "f16", "rows": 4096, "channels": 8192, "groups": 8,
         "form": "gate"},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of its range; odd values as often as not."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "conv_grad", "conv_step", "scan", "scan_train", "scan_step", "norm", "norm_grad"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if op in ("norm", "norm_grad"):
        groups = rng.choice([1, 1, 2, 4, 8])
        c.update(rows=_size(rng, 1, 8192), channels=groups * _size(rng, 64 // groups, 8192 // groups), groups=groups,
                 form=rng.choice(["residual", "gate", "gate_after", "plain"]))
        return c
    states = rng.choice([4, 8, 12, 16, 16, 32, 64])
    groups = rng.choice([1, 1, 1, 2, 4])
    channels = groups * _size(rng, 64 // groups, 4096 // groups)
    if op in ("conv_step", "scan_step"):
        c.update(batch=_size(rng, 1, 256), channels=channels)
    else:
        batch = rng.choice([1, 1, 2, 4])
        heavy = {"conv": 16384 * 5120, "conv_grad": 8192 * 4096, "scan": 65536 * 2048 * 16, "scan_train": 4096 * 4096 * 16}[op]
        per = channels * (states if op.startswith("scan") else 1)
        rows = _size(rng, 1, max(1, min(16384, heavy // (per * batch))))
        c.update(batch=batch, rows=rows, segments=_size(rng, 1, 40) if batch == 1 and rng.random() < 0.6 else 0,
                 channels=channels)
    if op.startswith("conv"):
        c["width"] = rng.choice([2, 3, 4, 4])
    else:
        c.update(states=states, groups=groups)
    return c


# ---------------------------------------------------------------------------
# inputs


def _offsets(count, rows, seed):
    """CSR offsets of `count` uneven segments over `rows` rows; every seventh is empty."""
    r = random.Random(seed * 7919 + count)
    weight = [0.0 if i % 7 == 3 and count > 1 else math.exp(r.gauss(0.0, 1.0)) for i in range(count)]
    total, acc, off = sum(weight), 0.0, [0]
    for w in weight:
        acc += w
        off.append(min(rows, int(round(rows * acc / total))))
    off[-1] = rows
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo

    op, s = case["op"], {"op": case["op"]}
    if op in ("norm", "norm_grad"):
        rows, ch, form = case["rows"], case["channels"], case["form"]
        s.update(groups=case["groups"], form=form, weight=uniform(ch, lo=0.5, hi=1.5))
        s["x"] = normal(rows, ch, dtype=dt)
        s["residual"] = normal(rows, ch, scale=3.0) if form == "residual" else None
        s["scale"] = uniform(ch, lo=0.1, hi=1.0) if form == "residual" else None
        # the gate is the second half of the projection that feeds the block
        s["gate"] = normal(rows, 2 * ch, dtype=dt)[:, ch:] if form.startswith("gate") else None
        if op == "norm_grad":
            s["grad"] = normal(rows, ch, dtype=dt)
            s["grad_residual"] = normal(rows, ch) if form == "residual" else None
            if form == "residual":
                s["sum"] = s["residual"] + s["scale"] * s["x"].float()
        return s

    ch = case["channels"]
    if op in ("conv_step", "scan_step"):
        batch = case["batch"]
        slots = batch + 8
        perm = torch.randperm(slots, generator=g, device="cuda")[:batch].to(torch.int32)
        if batch > 4:
            perm[batch // 2] = -1  # a padding row of the batch
        s.update(slots=perm)
        lead = (batch,)
    else:
        batch, rows = case["batch"], case["rows"]
        s["offsets"] = _offsets(case["segments"], rows, seed) if case["segments"] else None
        lead = (rows,) if case["segments"] else (batch, rows)
        count = case["segments"] or batch
    proj = normal(*lead, 2 * ch, dtype=dt)  # a projection's output: the block's input beside its gate

    if op.startswith("conv"):
        w = case["width"]
        s.update(x=proj[..., :ch], weight=normal(ch, w, scale=0.5), bias=normal(ch, scale=0.1))
        if op == "conv_step":
            s["state"] = normal(slots, w - 1, ch, dtype=dt)
        else:
            s["state"] = normal(count, w - 1, ch, dtype=dt)
        if op == "conv_grad":
            s["grad"] = normal(*lead, ch, dtype=dt)
            s["grad_state"] = normal(count, w - 1, ch, dtype=dt)
        return s

    n, groups = case["states"], case["groups"]
    rank = 32
    low = normal(*lead, rank + 2 * groups * n, dtype=dt)  # the small projection: dt's factors, B and C
    s["B"] = low[..., rank:rank + groups * n].unflatten(-1, (groups, n))
    s["C"] = low[..., rank + groups * n:].unflatten(-1, (groups, n))
    s["u"], s["z"] = normal(*lead, ch, dtype=dt), proj[..., ch:]
    s["dt"] = normal(*lead, ch, scale=0.5, dtype=dt)
    step = torch.exp(uniform(ch, lo=math.log(1e-3), hi=math.log(1e-1)))
    s["dt_bias"] = torch.log(torch.expm1(step))
    s["A"] = -torch.arange(1, n + 1, device="cuda").float() * torch.exp(normal(ch, n, scale=0.1))
    s["D"] = uniform(ch, lo=0.5, hi=1.5)
    s["state"] = normal(slots if op == "scan_step" else count, ch, n, scale=0.5)
    if op == "scan_train":
        s["grad"] = normal(*lead, ch, dtype=dt)
        s["grad_state"] = normal(count, ch, n, scale=0.1)
    return s


# ---------------------------------------------------------------------------
# one pass


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import device_wide_prefix_gb300 as dwp
    op = s["op"]
    if op == "conv":
        out, final = dwp.causal_conv(s["x"], s["weight"], s["bias"], offsets=s["offsets"], initial_state=s["state"],
                                     silu=True, return_state=True)
        return {"out": out, "final_state": final}
    if op == "conv_grad":
        return dwp.causal_conv_backward(s["grad"], s["x"], s["weight"], s["bias"], offsets=s["offsets"],
                                        initial_state=s["state"], grad_final_state=s["grad_state"], silu=True)
    if op == "conv_step":
        out = dwp.causal_conv_step(s["x"], s["state"], s["weight"], s["bias"], slots=s["slots"], silu=True)
        return {"out": out, "state": s["state"]}
    if op == "scan":
        out, final = dwp.selective_scan(s["u"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
                                        dt_bias=s["dt_bias"], dt_softplus=True, offsets=s["offsets"],
                                        initial_state=s["state"], return_state=True)
        return {"out": out, "final_state": final}
    if op == "scan_train":
        out, final, points = dwp.selective_scan(s["u"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
                                                dt_bias=s["dt_bias"], dt_softplus=True, offsets=s["offsets"],
                                                initial_state=s["state"], return_state=True, return_checkpoints=True)
        grads = dwp.selective_scan_backward(s["grad"], s["u"], s["dt"], s["A"], s["B"], s["C"], points, D=s["D"],
                                            z=s["z"], dt_bias=s["dt_bias"], dt_softplus=True, offsets=s["offsets"],
                                            initial_state=s["state"], grad_final_state=s["grad_state"])
        return {"out": out, "final_state": final, "grads": grads}
    if op == "scan_step":
        out = dwp.selective_scan_step(s["u"], s["dt"], s["A"], s["B"], s["C"], s["state"], D=s["D"], z=s["z"],
                                      dt_bias=s["dt_bias"], dt_softplus=True, slots=s["slots"])
        return {"out": out, "state": s["state"]}
    if op == "norm":
        out, total = dwp.block_norm(s["x"], s["weight"], residual=s["residual"], scale=s["scale"], gate=s["gate"],
                                    gate_after=s["form"] == "gate_after", groups=s["groups"], eps=1e-5)
        return {"out": out, "sum": total} if s["residual"] is not None else {"out": out}
    grads = dwp.block_norm_backward(s["grad"], s["sum"] if s["form"] == "residual" else s["x"], s["weight"],
                                    x=s["x"] if s["form"] == "residual" else None, scale=s["scale"], gate=s["gate"],
                                    gate_after=s["form"] == "gate_after", grad_residual=s["grad_residual"],
                                    groups=s["groups"], eps=1e-5)
    return grads


# The plain forms: 32 bits throughout, rounded once at the end.


def _silu(v):
    return v * torch.sigmoid(v)


def _silu_slope(v):
    p = torch.sigmoid(v)
    return p * (1.0 + v * (1.0 - p))


def _rows(s, t):
    """A row-shaped input as one packed stream (rows, ...)."""
    return t.flatten(0, 1) if s["offsets"] is None else t


def _segments(s, like):
    """First row of each segment, its end, and each row's segment, of the packed stream."""
    if s["offsets"] is not None:
        first, end = s["offsets"][:-1].long(), s["offsets"][1:].long()
        rows = like.shape[0]
    else:
        batch, length = like.shape[:2]
        first = torch.arange(batch, device=like.device) * length
        end, rows = first + length, batch * length
    return first, end, torch.searchsorted(end, torch.arange(rows, device=like.device), right=True)


def _taps(s, x, width):
    """(rows, width) places of each row's taps in the stream that has every segment's state rows before its rows,
    that stream's places of the rows and of the state rows, and of each segment's last width - 1 rows."""
    first, end, seg = _segments(s, x)
    halo = width - 1
    place = torch.arange(seg.numel(), device=seg.device) + halo * (seg + 1)
    back = torch.arange(halo, device=seg.device)
    start = first + halo * torch.arange(first.numel(), device=seg.device)
    return (place[:, None] + torch.arange(-halo, 1, device=seg.device), place, start[:, None] + back,
            (start + (end - first))[:, None] + back)


def _scan(a, x):
    """h[t] = a[t] h[t-1] + x[t] from h[-1] = 0 along the first axis: within blocks of rows, then over the blocks."""
    rows = a.shape[0]
    q = max(1, int(math.isqrt(rows)))
    blocks = -(-rows // q)
    pad = blocks * q - rows
    if pad:
        a = torch.cat([a, a.new_zeros(pad, *a.shape[1:])])
        x = torch.cat([x, x.new_zeros(pad, *x.shape[1:])])
    a, h = a.unflatten(0, (blocks, q)), x.unflatten(0, (blocks, q)).clone()
    run_a = a.clone()
    for i in range(1, q):
        h[:, i] += a[:, i] * h[:, i - 1]
        run_a[:, i] *= run_a[:, i - 1]
    for b in range(1, blocks):
        h[b] += run_a[b] * h[b - 1, -1]
    return h.flatten(0, 1)[:rows]


def _run_plain(s):
    op = s["op"]
    if op.startswith("norm"):
        return _plain_norm(s) if op == "norm" else _plain_norm_grad(s)
    if op == "conv_step":
        return _plain_conv_step(s)
    if op == "scan_step":
        return _plain_scan_step(s)
    return _plain_conv(s) if op.startswith("conv") else _plain_scan(s)


def _plain_conv(s):
    x, w = s["x"], s["weight"]
    taps, place, old, last = _taps(s, x, w.shape[1])
    rows, kind = _rows(s, x), x.dtype
    stream = torch.empty(rows.shape[0] + old.numel(), rows.shape[1], device=x.device)
    stream[place], stream[old] = rows.float(), s["state"].float()
    seen = stream[taps]  # (rows, width, channels)
    p = (seen * w.t()).sum(1) + s["bias"]
    if s["op"] == "conv":
        return {"out": _silu(p).to(kind).view(x.shape), "final_state": stream[last].to(kind)}
    g = _rows(s, s["grad"]).float() * _silu_slope(p)
    back = torch.zeros_like(stream)
    back.index_add_(0, taps.flatten(), (g[:, None, :] * w.t()).flatten(0, 1))
    back.index_add_(0, last.flatten(), s["grad_state"].float().flatten(0, 1))
    return {"x": back[place].to(kind).view(x.shape), "weight": (g[:, None, :] * seen).sum(0).t().contiguous(),
            "bias": g.sum(0), "initial_state": back[old].to(kind)}


def _store(state, new, slots):
    """Row i of `new` in place of slot slots[i] of `state`; a negative slot stores nothing."""
    row = torch.zeros(state.shape[0], dtype=torch.long, device=state.device)
    row.index_add_(0, slots.clamp(min=0),
                   torch.where(slots >= 0, torch.arange(1, slots.numel() + 1, device=state.device), 0))
    hit = row > 0
    state.copy_(torch.where(hit[:, None, None], new[(row - 1).clamp(min=0)].to(state.dtype), state))


def _plain_conv_step(s):
    x, w, state, slots = s["x"], s["weight"], s["state"], s["slots"].long()
    seen = torch.cat([state[slots.clamp(min=0)].float(), x.float()[:, None]], 1)  # (batch, width, channels)
    p = _silu((seen * w.t()).sum(1) + s["bias"])
    _store(state, seen[:, 1:], slots)
    return {"out": torch.where(slots[:, None] >= 0, p, p.new_zeros(())).to(x.dtype), "state": state}


def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(v.clamp(max=20.0))))


def _spread(v, channels):
    """(rows, groups, n) -> (rows, channels, n): each group's values for its channels."""
    return v.repeat_interleave(channels // v.shape[1], 1) if v.shape[1] > 1 else v.expand(-1, channels, -1)


def _plain_scan(s):
    kind, shape = s["u"].dtype, s["u"].shape
    u, raw, z = (_rows(s, s[k]).float() for k in ("u", "dt", "z"))
    ch, groups, n = u.shape[1], s["B"].shape[-2], s["B"].shape[-1]
    B, C = (_spread(_rows(s, s[k]).float(), ch) for k in ("B", "C"))
    first, end, _ = _segments(s, s["u"])
    full = end > first
    head, tail, start = first[full], end[full] - 1, s["state"][full]
    raw = raw + s["dt_bias"]
    delta = _softplus(raw)
    a = torch.exp(delta[..., None] * s["A"])
    x = (delta * u)[..., None] * B
    x[head] += a[head] * start
    cut = a.clone()
    cut[head] = 0.0
    h = _scan(cut, x)
    y = (h * C).sum(-1) + s["D"] * u
    final = s["state"].clone()
    final[full] = h[tail]
    out = (y * _silu(z)).to(kind).view(shape)
    if s["op"] == "scan":
        return {"out": out, "final_state": final}
    g = _rows(s, s["grad"]).float()
    dy = g * _silu(z)
    dz = g * y * _silu_slope(z)
    inner = dy[..., None] * C
    inner[tail] += s["grad_state"][full]
    later = torch.cat([cut[1:], cut.new_zeros(1, *cut.shape[1:])])  # the next row's decay, nothing past a segment
    dh = _scan(later.flip(0), inner.flip(0)).flip(0)
    before = torch.cat([h.new_zeros(1, *h.shape[1:]), h[:-1]])
    before[head] = start
    through = dh * a * before
    q = (dh * B).sum(-1)
    ddelta = q * u + (through * s["A"]).sum(-1)
    draw_ = ddelta * torch.sigmoid(raw)
    first_grad = s["grad_state"].clone()
    first_grad[full] = a[head] * dh[head]
    sums = lambda v: v.unflatten(1, (groups, ch // groups)).sum(2)  # noqa: E731
    shaped = lambda v: v.to(kind).view(*shape[:-1], *v.shape[1:])  # noqa: E731
    grads = {"u": shaped(q * delta + s["D"] * dy), "dt": shaped(draw_), "A": (through * delta[..., None]).sum(0),
             "B": shaped(sums(dh * (delta * u)[..., None])), "C": shaped(sums(dy[..., None] * h)), "D": (dy * u).sum(0),
             "z": shaped(dz), "dt_bias": draw_.sum(0), "initial_state": first_grad}
    return {"out": out, "final_state": final, "grads": grads}


def _plain_scan_step(s):
    kind, slots, state = s["u"].dtype, s["slots"].long(), s["state"]
    u, z = s["u"].float(), s["z"].float()
    B, C = (_spread(s[k].float(), u.shape[1]) for k in ("B", "C"))
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    old = state[slots.clamp(min=0)]
    new = torch.exp(delta[..., None] * s["A"]) * old + (delta * u)[..., None] * B
    y = ((new * C).sum(-1) + s["D"] * u) * _silu(z)
    _store(state, new, slots)
    return {"out": torch.where(slots[:, None] >= 0, y, y.new_zeros(())).to(kind), "state": state}


def _plain_norm(s):
    x = s["x"].float()
    v = s["residual"] + s["scale"] * x if s["residual"] is not None else x
    t = v * _silu(s["gate"].float()) if s["form"] == "gate" else v
    by = t.unflatten(1, (s["groups"], -1))
    y = (by * torch.rsqrt((by * by).mean(-1, keepdim=True) + 1e-5)).flatten(1) * s["weight"]
    if s["form"] == "gate_after":
        y = y * _silu(s["gate"].float())
    out = {"out": y.to(s["x"].dtype)}
    if s["residual"] is not None:
        out["sum"] = v
    return out


def _plain_norm_grad(s):
    kind, form = s["x"].dtype, s["form"]
    v = s["sum"] if form == "residual" else s["x"].float()
    g, z = s["grad"].float(), s["gate"].float() if s["gate"] is not None else None
    t = v * _silu(z) if form == "gate" else v
    by = t.unflatten(1, (s["groups"], -1))
    r = torch.rsqrt((by * by).mean(-1, keepdim=True) + 1e-5)
    hat = by * r
    grads = {}
    if form == "gate_after":
        grads["gate"] = (g * hat.flatten(1) * s["weight"] * _silu_slope(z)).to(kind)
        g = g * _silu(z)
    grads["weight"] = (g * hat.flatten(1)).sum(0)
    gw = (g * s["weight"]).unflatten(1, (s["groups"], -1))
    dt = (r * (gw - hat * (gw * hat).mean(-1, keepdim=True))).flatten(1)
    if form == "gate":
        grads["gate"] = (dt * v * _silu_slope(z)).to(kind)
        dt = dt * _silu(z)
    if form == "residual":
        dt = dt + s["grad_residual"]
        grads.update(residual=dt, x=(dt * s["scale"]).to(kind), scale=(dt * s["x"].float()).sum(0))
    else:
        grads["x"] = dt.to(kind)
    return grads


# ---------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op in ("norm", "norm_grad"):
        cells = case["rows"] * case["channels"]
        gated, resid = case["form"].startswith("gate"), case["form"] == "residual"
        if op == "norm":
            return {"bytes": cells * (2 * e + e * gated + 8 * resid) + 4 * case["channels"] * (1 + resid),
                    "flops": cells * (4 + 5 * gated + 2 * resid)}
        return {"bytes": cells * (3 * e + 2 * e * gated + (12 if resid else 0)) + 8 * case["channels"],
                "flops": cells * (10 + 12 * gated + 4 * resid)}
    ch = case["channels"]
    rows = case["batch"] * case.get("rows", 1)
    count = case.get("segments") or case["batch"]
    cells = rows * ch
    if op.startswith("conv"):
        w = case["width"]
        states = count * (w - 1) * ch * e * 2
        if op == "conv_grad":
            return {"bytes": cells * 3 * e + 2 * states + 8 * ch * (w + 1), "flops": cells * (6 * w + 12)}
        return {"bytes": cells * 2 * e + states + 4 * ch * (w + 1), "flops": cells * (2 * w + 5)}
    n, groups = case["states"], case["groups"]
    states = count * ch * n * 4 * 2
    small = 2 * rows * groups * n * e
    fixed = 4 * ch * (n + 2)
    if op == "scan_train":  # forward and backward: the inputs twice, the output's gradient, the output, the gradients
        return {"bytes": cells * e * (4 + 3 + 4) + 3 * small + 3 * states // 2 + 2 * fixed,
                "flops": cells * (7 * n + 10) + cells * (24 * n + 30)}
    return {"bytes": cells * 4 * e + small + states + fixed, "flops": cells * (7 * n + 10)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one segment and one row after another


def _spans(s):
    if s["offsets"] is not None:
        off = s["offsets"].tolist()
        return list(zip(off[:-1], off[1:]))
    batch, length = (s["x"] if "x" in s else s["u"]).shape[:2]
    return [(b * length, (b + 1) * length) for b in range(batch)]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op.startswith("norm"):
        return _exact_norm(s)
    if op.endswith("step"):
        return _exact_step(s)
    return _exact_conv(s) if op.startswith("conv") else _exact_scan(s)


def _exact_conv(s):
    w = s["weight"].double()
    ch, width = w.shape
    x = _rows(s, s["x"]).double()
    out, dx, dw, db = torch.empty_like(x), torch.empty_like(x), torch.zeros_like(w), w.new_zeros(ch)
    final, first = (torch.empty(s["state"].shape, dtype=torch.float64, device=x.device) for _ in range(2))
    for i, (lo, hi) in enumerate(_spans(s)):
        seq = torch.cat([s["state"][i].double(), x[lo:hi]])
        final[i] = seq[seq.shape[0] - (width - 1):]
        n = hi - lo
        p = s["bias"].double().expand(n, ch).clone()
        for k in range(width):
            p += w[:, k] * seq[k:k + n]
        if s["op"] == "conv":
            out[lo:hi] = p / (1 + torch.exp(-p))
            continue
        sig = 1 / (1 + torch.exp(-p))
        g = _rows(s, s["grad"])[lo:hi].double() * (sig + p * sig * (1 - sig))
        dseq = torch.zeros_like(seq)
        for k in range(width):
            dseq[k:k + n] += w[:, k] * g
            dw[:, k] += (g * seq[k:k + n]).sum(0)
        db += g.sum(0)
        dseq[seq.shape[0] - (width - 1):] += s["grad_state"][i].double()
        first[i], dx[lo:hi] = dseq[:width - 1], dseq[width - 1:]
    if s["op"] == "conv":
        return {"out": out.view(s["x"].shape), "final_state": final}
    return {"x": dx.view(s["x"].shape), "weight": dw, "bias": db, "initial_state": first}


def _exact_scan(s):
    train = s["op"] == "scan_train"
    u, raw, z, B, C = (_rows(s, s[k]).double() for k in ("u", "dt", "z", "B", "C"))
    A, D, bias = s["A"].double(), s["D"].double(), s["dt_bias"].double()
    rows, ch = u.shape
    groups, n = B.shape[1:]
    delta = torch.logaddexp(raw + bias, torch.zeros_like(raw))
    gate = z / (1 + torch.exp(-z))
    y = torch.empty_like(u)
    final = s["state"].double().clone()
    kept = torch.empty(rows, ch, n, dtype=torch.float64, device=u.device) if train else None
    wide = lambda v: v.repeat_interleave(ch // groups, 0)  # (groups, n) -> (channels, n)  # noqa: E731
    spans = _spans(s)
    equal = s["offsets"] is None  # equal sequences go side by side
    walk = [(torch.arange(len(spans), device=u.device), [lo for lo, _ in spans], spans[0][1] - spans[0][0])] if equal else [
        (torch.tensor([i], device=u.device), [lo], hi - lo) for i, (lo, hi) in enumerate(spans)]
    many = lambda v: v.repeat_interleave(ch // groups, 1)  # (segments, groups, n) -> (segments, channels, n)  # noqa: E731
    for which, lows, length in walk:
        lo = torch.tensor(lows, device=u.device)
        h = final[which]
        for t in range(length):
            r = lo + t
            if kept is not None:
                kept[r] = h
            h = torch.exp(delta[r][..., None] * A) * h + (delta[r] * u[r])[..., None] * many(B[r])
            y[r] = (h * many(C[r])).sum(-1)
        if length:
            final[which] = h
    y += D * u
    out = (y * gate).view(s["u"].shape)
    if not train:
        return {"out": out, "final_state": final}
    go = _rows(s, s["grad"]).double()
    sig = 1 / (1 + torch.exp(-z))
    dy = go * gate
    dz = go * y * (sig + z * sig * (1 - sig))
    du, ddelta = D * dy, torch.zeros_like(u)
    dA, dB, dC = torch.zeros_like(A), torch.zeros_like(B), torch.zeros_like(C)
    start = s["grad_state"].double().clone()
    together = lambda v: v.unflatten(1, (groups, ch // groups)).sum(2)  # noqa: E731
    for which, lows, length in walk:
        lo = torch.tensor(lows, device=u.device)
        carry = start[which]
        for t in reversed(range(length)):
            r = lo + t
            Bt, Ct, prev = many(B[r]), many(C[r]), kept[r]
            a = torch.exp(delta[r][..., None] * A)
            x = (delta[r] * u[r])[..., None]
            dh = carry + dy[r][..., None] * Ct
            dC[r] = together(dy[r][..., None] * (a * prev + x * Bt))
            dB[r] = together(dh * x)
            q = (dh * Bt).sum(-1)
            du[r] += q * delta[r]
            ddelta[r] = q * u[r] + (dh * a * prev * A).sum(-1)
            dA += (dh * a * prev * delta[r][..., None]).sum(0)
            carry = dh * a
        if length:
            start[which] = carry
    draw_ = ddelta / (1 + torch.exp(-(raw + bias)))
    lead = s["u"].shape[:-1]
    shaped = lambda v: v.reshape(*lead, *v.shape[1:])  # noqa: E731
    grads = {"u": shaped(du), "dt": shaped(draw_), "A": dA, "B": shaped(dB), "C": shaped(dC), "D": (dy * u).sum(0),
             "z": shaped(dz), "dt_bias": draw_.sum(0), "initial_state": start}
    return {"out": out, "final_state": final, "grads": grads}


def _exact_step(s):
    state = s["state"].double()
    rows = [(i, slot) for i, slot in enumerate(s["slots"].tolist()) if slot >= 0]
    row, slot = ([r[k] for r in rows] for k in (0, 1))
    if s["op"] == "conv_step":
        x, w = s["x"].double(), s["weight"].double()
        out = torch.zeros_like(x)
        p = s["bias"].double() + w[:, -1] * x[row]
        for k in range(w.shape[1] - 1):
            p = p + w[:, k] * state[slot, k]
        out[row] = p / (1 + torch.exp(-p))
        state[slot] = torch.cat([state[slot, 1:], x[row][:, None]], 1)
        return {"out": out, "state": state}
    u, z, B, C = (s[k].double() for k in ("u", "z", "B", "C"))
    out = torch.zeros_like(u)
    per = u.shape[1] // B.shape[1]
    delta = torch.logaddexp(s["dt"].double() + s["dt_bias"].double(), u.new_zeros(()))[row]
    h = torch.exp(delta[..., None] * s["A"].double()) * state[slot]
    h += (delta * u[row])[..., None] * B[row].repeat_interleave(per, 1)
    y = torch.einsum("bdn,bdn->bd", h, C[row].repeat_interleave(per, 1)) + s["D"].double() * u[row]
    out[row] = y * z[row] / (1 + torch.exp(-z[row]))
    state[slot] = h
    return {"out": out, "state": state}


def _exact_norm(s):
    x, w, form = s["x"].double(), s["weight"].double(), s["form"]
    leaves = {"x": x.requires_grad_()} if form != "residual" else {}
    if form == "residual":
        v = (s["sum"].double() if "sum" in s else s["residual"].double() + s["scale"].double() * x)
        leaves["residual"] = v.requires_grad_()
    else:
        v = x
    if s["gate"] is not None:
        z = leaves["gate"] = s["gate"].double().requires_grad_()
        gate = z / (1 + torch.exp(-z))
    leaves["weight"] = w.requires_grad_()
    t = v * gate if form == "gate" else v
    parts = [p / (p.square().sum(1, keepdim=True) / p.shape[1] + 1e-5).sqrt() for p in t.chunk(s["groups"], 1)]
    y = torch.cat(parts, 1) * w
    if form == "gate_after":
        y = y * gate
    if s["op"] == "norm":
        return {"out": y.detach(), "sum": v.detach()} if form == "residual" else {"out": y.detach()}
    grads = dict(zip(leaves, torch.autograd.grad(y, list(leaves.values()), s["grad"].double())))
    if form == "residual":
        dv = grads["residual"] + s["grad_residual"].double()
        grads.update(residual=dv, x=dv * s["scale"].double(), scale=(dv * x.detach()).sum(0))
    return grads
