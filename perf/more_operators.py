"""The gated delta rule and layer norm, as cases to measure.

Each case is one operator: the gated delta rule over prompts (batches and
packed requests), its training step (forward, then every gradient) and its
token form on a cache of states; layer norm with or without the residual
before it, over rows or over groups of a row, and its gradient.  `run`
computes it in elementary torch operations in 32 bits (own = False) or through
device_wide_prefix_gb300 (own = True).
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # an ordinary batch of prompts: query and key heads shared by two value heads
        {"name": "delta_prompt", "op": "delta", "dtype": "bf16", "batch": 4, "rows": 2048, "segments": 0, "key_heads": 16,
         "heads": 32, "keys": 128, "values": 128},
        # one very long prompt
        {"name": "delta_long", "op": "delta", "dtype": "bf16", "batch": 1, "rows": 32768, "segments": 0, "key_heads": 16,
         "heads": 32, "keys": 128, "values": 128},
        # packed requests of uneven length (some empty), each continuing its own state, sizes that no tile divides, in 32 bits
        {"name": "delta_packed_f32", "op": "delta", "dtype": "f32", "batch": 1, "rows": 4099, "segments": 23, "key_heads": 3,
         "heads": 6, "keys": 96, "values": 72},
        # one short prompt of a small layer: latency counts
        {"name": "delta_short", "op": "delta", "dtype": "bf16", "batch": 1, "rows": 100, "segments": 0, "key_heads": 8,
         "heads": 8, "keys": 64, "values": 64},
        # a training step: forward, then every gradient
        {"name": "delta_train", "op": "delta_train", "dtype": "bf16", "batch": 4, "rows": 2048, "segments": 0, "key_heads": 16,
         "heads": 16, "keys": 128, "values": 128},
        # a training step over packed documents, small heads, shared keys
        {"name": "delta_train_packed", "op": "delta_train", "dtype": "f16", "batch": 1, "rows": 3001, "segments": 9,
         "key_heads": 4, "heads": 8, "keys": 64, "values": 96},
        # generation at a full batch: the state cache is read and written
        {"name": "delta_token", "op": "delta_step", "dtype": "bf16", "batch": 64, "key_heads": 16, "heads": 32, "keys": 128,
         "values": 128},
        # generation for one request: latency counts
        {"name": "delta_token_one", "op": "delta_step", "dtype": "bf16", "batch": 1, "key_heads": 8, "heads": 16, "keys": 128,
         "values": 128},
        # before a block: residual stream in 32 bits
        {"name": "layer_norm_residual", "op": "norm", "dtype": "bf16", "rows": 8192, "channels": 4096, "groups": 1,
         "residual": True},
        # the same for one token of a few requests: latency counts
        {"name": "layer_norm_token", "op": "norm", "dtype": "bf16", "rows": 8, "channels": 4096, "groups": 1,
         "residual": True},
        # before a block, training: the gradient, with the sums of weight and bias over all rows
        {"name": "layer_norm_gradient", "op": "norm_grad", "dtype": "bf16", "rows": 8192, "channels": 4096, "groups": 1,
         "residual": True},
        # after the recurrence, training: each head normed by itself
        {"name": "layer_norm_heads_gradient", "op": "norm_grad", "dtype": "f16", "rows": 4099, "channels": 4096,
         "groups": 32, "residual": False},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of its range; odd values as often as not."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta_train", "delta_train", "delta_step", "norm", "norm_grad"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if op in ("norm", "norm_grad"):
        groups = rng.choice([1, 1, 2, 8, 32])
        c.update(rows=_size(rng, 1, 8192), channels=groups * _size(rng, max(1, 64 // groups), 8192 // groups),
                 groups=groups, residual=rng.random() < 0.5)
        return c
    key_heads = _size(rng, 1, 16)
    heads = key_heads * rng.choice([1, 1, 2, 3] if key_heads <= 10 else [1, 2])
    keys, values = (rng.choice([128, 128, 64, _size(rng, 16, 128)]) for _ in range(2))
    c.update(key_heads=key_heads, heads=heads, keys=keys, values=values)
    if op == "delta_step":
        c["batch"] = _size(rng, 1, 64)
        return c
    batch = rng.choice([1, 1, 2, 4])
    most = (32768 if op == "delta" else 4096) * 32 * 128 * 128
    rows = _size(rng, 1, max(1, min(16384 if op == "delta" else 4096, most // (batch * heads * keys * values))))
    c.update(batch=batch, rows=rows, segments=_size(rng, 1, 40) if batch == 1 and rng.random() < 0.6 else 0)
    return c


# ---------------------------------------------------------------------------
# inputs


def _cuts(count, rows, seed):
    """First rows of `count` uneven segments over `rows` rows, and the end; every seventh is empty."""
    r = random.Random(seed * 7919 + count)
    weight = [0.0 if i % 7 == 3 and count > 1 else math.exp(r.gauss(0.0, 1.0)) for i in range(count)]
    total, acc, off = sum(weight), 0.0, [0]
    for w in weight:
        acc += w
        off.append(min(rows, int(round(rows * acc / total))))
    off[-1] = rows
    return off


CHUNK = 64


def _plan(cuts):
    """Rows (chunks, CHUNK) of the packed stream that each chunk holds, -1 past a sequence's end; and for each step
    along the sequences the chunks that are at it, with their sequences."""
    rows, steps = [], []
    for i, (lo, hi) in enumerate(zip(cuts[:-1], cuts[1:])):
        for c, at in enumerate(range(lo, hi, CHUNK)):
            if c == len(steps):
                steps.append(([], []))
            steps[c][0].append(len(rows))
            steps[c][1].append(i)
            rows.append([t if t < hi else -1 for t in range(at, at + CHUNK)])
    place = torch.tensor(rows, dtype=torch.long).reshape(-1, CHUNK)
    return place.to("cuda"), [tuple(torch.tensor(v).to("cuda") for v in step) for step in steps]


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
        rows, ch = case["rows"], case["channels"]
        s.update(groups=case["groups"], weight=uniform(ch, lo=0.5, hi=1.5), bias=normal(ch, scale=0.1))
        x = normal(rows, ch, scale=1.5, dtype=dt) + 0.3
        if op == "norm":
            s["x"], s["residual"] = x, normal(rows, ch, scale=3.0) if case["residual"] else None
        else:
            s["v"] = normal(rows, ch, scale=3.0) + x.float() if case["residual"] else x
            s["grad"] = normal(rows, ch, dtype=dt)
            s["grad_residual"] = normal(rows, ch) if case["residual"] else None
        return s

    key_heads, heads, keys, values = (case[k] for k in ("key_heads", "heads", "keys", "values"))
    if op == "delta_step":
        batch = case["batch"]
        slots = batch + 8
        perm = torch.randperm(slots, generator=g, device="cuda")[:batch].to(torch.int32)
        if batch > 4:
            perm[batch // 2] = -1  # a padding row of the batch
        s["slots"], lead, count = perm, (batch,), slots
    else:
        batch, rows = case["batch"], case["rows"]
        cuts = _cuts(case["segments"], rows, seed) if case["segments"] else [i * rows for i in range(batch + 1)]
        s["cuts"], s["plan"] = cuts, _plan(cuts)  # the batch's shape, on the host and as the plain form walks it
        s["offsets"] = torch.tensor(cuts, dtype=torch.int32, device="cuda") if case["segments"] else None
        lead, count = (rows,) if case["segments"] else (batch, rows), len(cuts) - 1
    # queries and keys of length one; the values lie in the projection's output
    unit = lambda *shape: torch.nn.functional.normalize(normal(*shape), dim=-1).to(dt)  # noqa: E731
    s["q"], s["k"] = unit(*lead, key_heads, keys), unit(*lead, key_heads, keys)
    s["v"] = normal(*lead, 2 * heads * values, dtype=dt)[..., :heads * values].unflatten(-1, (heads, values))
    # a head's rate times the softplus of a projection: decays from almost none to almost all
    rate, step = uniform(heads, lo=1.0, hi=16.0), uniform(heads, lo=math.log(1e-3), hi=math.log(1e-1)).exp()
    s["g"] = -rate * torch.nn.functional.softplus(normal(*lead, heads, scale=0.5) + torch.log(torch.expm1(step)))
    s["beta"] = torch.sigmoid(normal(*lead, heads))
    s["scale"] = keys ** -0.5
    s["state"] = normal(count, heads, keys, values, scale=0.3)
    if op == "delta_train":
        s["grad"] = normal(*lead, heads, values, dtype=dt)
        s["grad_state"] = normal(count, heads, keys, values, scale=0.1)
    return s


# ---------------------------------------------------------------------------
# one pass


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import device_wide_prefix_gb300 as dwp
    op = s["op"]
    if op == "norm":
        out, total = dwp.layer_norm(s["x"], s["weight"], s["bias"], residual=s["residual"], groups=s["groups"], eps=1e-5)
        return {"out": out, "sum": total} if s["residual"] is not None else {"out": out}
    if op == "norm_grad":
        return dwp.layer_norm_backward(s["grad"], s["v"], s["weight"], bias=s["bias"], grad_residual=s["grad_residual"],
                                       groups=s["groups"], eps=1e-5)
    args = (s["q"], s["k"], s["v"], s["g"], s["beta"])
    if op == "delta_step":
        out = dwp.gated_delta_rule_step(*args, s["state"], scale=s["scale"], slots=s["slots"])
        return {"out": out, "state": s["state"]}
    if op == "delta":
        out, final = dwp.gated_delta_rule(*args, scale=s["scale"], offsets=s["offsets"], initial_state=s["state"],
                                          return_state=True)
        return {"out": out, "final_state": final}
    out, final, points = dwp.gated_delta_rule(*args, scale=s["scale"], offsets=s["offsets"], initial_state=s["state"],
                                              return_state=True, return_checkpoints=True)
    grads = dwp.gated_delta_rule_backward(s["grad"], *args, points, scale=s["scale"], offsets=s["offsets"],
                                          initial_state=s["state"], grad_final_state=s["grad_state"])
    return {"out": out, "final_state": final, "grads": grads}


def _run_plain(s):
    op = s["op"]
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_grad":
        return _plain_norm_grad(s)
    return _plain_step(s) if op == "delta_step" else _plain_delta(s)


# The plain forms: 32 bits throughout (sums of log decays in 64), rounded once at the end.

def _plain_delta(s):
    kind, heads, scale = s["q"].dtype, s["v"].shape[-2], s["scale"]
    flat = (lambda t: t) if s["offsets"] is not None else (lambda t: t.flatten(0, 1))
    place, steps = s["plan"]
    here = place >= 0

    def cut(t):  # (rows, heads or key heads, ...) -> (chunks, heads, CHUNK, ...), zero past the ends
        t = flat(t)[place.clamp(min=0)]
        t = torch.where(here.view(*here.shape, *(1,) * (t.dim() - 2)), t, t.new_zeros(())).float().transpose(1, 2)
        return t.repeat_interleave(heads // t.shape[1], 1) if t.shape[1] != heads else t

    q, k, v, beta = (cut(s[n]) for n in ("q", "k", "v", "beta"))
    sums = cut(s["g"]).double().cumsum(-1)
    last = sums[..., -1:]
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    decay = torch.where(lower, sums[..., :, None] - sums[..., None, :], -math.inf).exp().float()
    first, rest, whole = sums.exp().float()[..., None], (last - sums).exp().float()[..., None], last.exp().float()[..., None]
    products = k @ k.transpose(-1, -2)
    system = (beta[..., None] * decay * products).tril(-1)
    solve = torch.eye(CHUNK, device=q.device).expand_as(system).clone()  # (1 + system)^-1, row by row
    for i in range(1, CHUNK):
        solve[..., i, :i] = -(system[..., i, None, :i] @ solve[..., :i, :i]).squeeze(-2)
    weigh = decay * (q @ k.transpose(-1, -2))
    state = s["state"].clone()
    starts, u = q.new_empty(*q.shape[:2], *state.shape[2:]), torch.empty_like(v)
    for at, seqs in steps:
        now = state[seqs]
        starts[at] = now
        u[at] = solve[at] @ (beta[at][..., None] * (v[at] - first[at] * (k[at] @ now)))
        state[seqs] = whole[at] * now + k[at].transpose(-1, -2) @ (rest[at] * u[at])
    out = scale * (first * (q @ starts) + weigh @ u)

    def join(t, like):  # back to rows, shared heads summed
        t = t.transpose(1, 2)
        t = t.unflatten(2, (like.shape[-2], -1)).sum(3) if t.dim() == 4 else t
        return t[here].to(like.dtype).view(like.shape)

    result = {"out": join(out, s["v"]).to(kind), "final_state": state}
    if s["op"] == "delta":
        return result
    dout = cut(s["grad"])
    dstate = s["grad_state"].clone()
    ends, dr, inner = torch.empty_like(starts), torch.empty_like(v), scale * weigh.transpose(-1, -2) @ dout
    dq_state = scale * q.transpose(-1, -2) @ (first * dout)
    for at, seqs in reversed(steps):
        now = dstate[seqs]
        ends[at] = now
        dr[at] = solve[at].transpose(-1, -2) @ (inner[at] + rest[at] * (k[at] @ now))
        dstate[seqs] = whole[at] * now + dq_state[at] - k[at].transpose(-1, -2) @ (beta[at][..., None] * first[at] * dr[at])
    dweigh = scale * decay * (dout @ u.transpose(-1, -2))
    dq = scale * first * (dout @ starts.transpose(-1, -2)) + dweigh @ k
    cross = -(decay * (dr @ u.transpose(-1, -2))).tril(-1)
    z = cross @ k - first * (dr @ starts.transpose(-1, -2))
    y = rest * (u @ ends.transpose(-1, -2)) + dweigh.transpose(-1, -2) @ q + (beta[..., None] * cross).transpose(-1, -2) @ k
    kz = (k * z).sum(-1)
    dbeta = (dr * v).sum(-1) + kz
    dsum = (q * dq).sum(-1) + beta * kz - (k * y).sum(-1)
    after = whole * starts + k.transpose(-1, -2) @ (rest * u)
    dsum[..., -1] += (after * ends).sum((-1, -2))
    dg = dsum.double().flip(-1).cumsum(-1).flip(-1)
    result["grads"] = {"q": join(dq, s["q"]), "k": join(beta[..., None] * z + y, s["k"]),
                       "v": join(beta[..., None] * dr, s["v"]), "g": join(dg, s["g"]), "beta": join(dbeta, s["beta"]),
                       "initial_state": dstate}
    return result


def _plain_step(s):
    kind, slots, state = s["q"].dtype, s["slots"].long(), s["state"]
    heads = s["v"].shape[1]
    q, k = (s[n].float().repeat_interleave(heads // s[n].shape[1], 1) for n in ("q", "k"))
    old = s["g"].exp()[..., None, None] * state[slots.clamp(min=0)]
    u = s["beta"][..., None] * (s["v"].float() - (old * k[..., None]).sum(-2))
    new = old + k[..., None] * u[..., None, :]
    out = s["scale"] * (new * q[..., None]).sum(-2)
    # padding rows go to a row behind the cache
    room = torch.cat([state, state.new_empty(1, *state.shape[1:])])
    room[torch.where(slots >= 0, slots, state.shape[0])] = new
    state.copy_(room[:-1])
    return {"out": torch.where(slots[:, None, None] >= 0, out, out.new_zeros(())).to(kind), "state": state}


def _plain_norm(s):
    v = s["x"].float() if s["residual"] is None else s["residual"] + s["x"].float()
    by = v.unflatten(1, (s["groups"], -1))
    by = by - by.mean(-1, keepdim=True)
    hat = (by * torch.rsqrt((by * by).mean(-1, keepdim=True) + 1e-5)).flatten(1)
    out = {"out": (hat * s["weight"] + s["bias"]).to(s["x"].dtype)}
    if s["residual"] is not None:
        out["sum"] = v
    return out


def _plain_norm_grad(s):
    kind, groups = s["grad"].dtype, s["groups"]
    grad, by = s["grad"].float(), s["v"].float().unflatten(1, (groups, -1))
    by = by - by.mean(-1, keepdim=True)
    r = torch.rsqrt((by * by).mean(-1, keepdim=True) + 1e-5)
    hat = by * r
    gw = (grad * s["weight"]).unflatten(1, (groups, -1))
    dv = (r * (gw - gw.mean(-1, keepdim=True) - hat * (gw * hat).mean(-1, keepdim=True))).flatten(1)
    grads = {"weight": (grad * hat.flatten(1)).sum(0), "bias": grad.sum(0)}
    if s["grad_residual"] is not None:
        dv = dv + s["grad_residual"]
        grads["residual"] = dv
    grads["x"] = dv.to(kind)
    return grads


# ---------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op in ("norm", "norm_grad"):
        cells, resid = case["rows"] * case["channels"], case["residual"]
        if op == "norm":
            return {"bytes": cells * (2 * e + 8 * resid) + 8 * case["channels"], "flops": cells * (8 + resid)}
        return {"bytes": cells * (2 * e + (12 if resid else e)) + 12 * case["channels"], "flops": cells * (16 + resid)}
    rows = case["batch"] * case.get("rows", 1)
    count = case.get("segments") or case["batch"]
    key_cells, cells = rows * case["key_heads"] * case["keys"], rows * case["heads"] * case["values"]
    entries = case["heads"] * case["keys"] * case["values"]
    gates = 8 * rows * case["heads"]
    one = (2 * key_cells + 2 * cells) * e + gates
    if op == "delta_train":  # forward; then its inputs again with the output's gradient, and the gradients
        return {"bytes": one + (4 * key_cells + 3 * cells) * e + 2 * gates + 16 * count * entries,
                "flops": 24 * rows * entries}
    return {"bytes": one + 8 * count * entries, "flops": 7 * rows * entries}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one row after another


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"].startswith("norm"):
        return _exact_norm(s)
    if s["op"] == "delta_step":
        return _exact_step(s)
    if max(b - a for a, b in zip(s["cuts"][:-1], s["cuts"][1:])) * (3 if s["op"] == "delta_train" else 1) > 40000:
        return None
    return _exact_delta(s)


def _row_of(a, k, q, v, beta, scale, state):
    """One row of some sequences: the output, the state before it decayed, the state after it, the corrections."""
    old = a[..., None, None] * state
    hat = v - torch.einsum("nhk,nhkv->nhv", k, old)
    new = old + k[..., :, None] * (beta[..., None] * hat)[..., None, :]
    return scale * torch.einsum("nhk,nhkv->nhv", q, new), old, new, hat


def _exact_delta(s):
    heads, scale = s["v"].shape[-2], s["scale"]
    flat = lambda t: (t if s["offsets"] is not None else t.flatten(0, 1)).double()  # noqa: E731
    q, k = (flat(s[n]).repeat_interleave(heads // s[n].shape[-2], 1) for n in ("q", "k"))
    v, beta, a = flat(s["v"]), flat(s["beta"]), torch.exp(flat(s["g"]))
    lows, lengths = s["cuts"][:-1], [b - a_ for a_, b in zip(s["cuts"][:-1], s["cuts"][1:])]
    longest = max(lengths)
    state, out = s["state"].double(), torch.empty_like(v)
    train = s["op"] == "delta_train"
    walk, kept = [], []
    for t in range(longest):
        live = [i for i, n in enumerate(lengths) if n > t]
        if t == 0 or len(live) != len(walk[-1][0]):
            which = torch.tensor(live, device=q.device)
            base = torch.tensor([lows[i] for i in live], device=q.device)
        walk.append((live, which, base + t))
    for live, which, at in walk:
        now = state if len(live) == len(lengths) else state[which]
        out[at], old, new, hat = _row_of(a[at], k[at], q[at], v[at], beta[at], scale, now)
        if train:
            kept.append((old, new, hat))
        if len(live) == len(lengths):
            state = new
        else:
            state[which] = new
    result = {"out": out.view(s["v"].shape), "final_state": state}
    if not train:
        return result
    dout, dstate = flat(s["grad"]), s["grad_state"].double()
    dq, dk, dv, dbeta, dg = (torch.zeros_like(t) for t in (q, k, v, beta, a))
    for (live, which, at), (old, new, hat) in zip(reversed(walk), reversed(kept)):
        d = dstate[which] + scale * q[at][..., :, None] * dout[at][..., None, :]
        dq[at] = scale * torch.einsum("nhkv,nhv->nhk", new, dout[at])
        du = torch.einsum("nhkv,nhk->nhv", d, k[at])
        dbeta[at] = (du * hat).sum(-1)
        dv[at] = beta[at][..., None] * du
        dk[at] = (torch.einsum("nhkv,nhv->nhk", d, beta[at][..., None] * hat)
                  - torch.einsum("nhkv,nhv->nhk", old, dv[at]))
        d = d - k[at][..., :, None] * dv[at][..., None, :]
        dg[at] = (d * old).sum((-1, -2))
        dstate[which] = a[at][..., None, None] * d
    share = lambda t, like: t.unflatten(1, (like.shape[-2], -1)).sum(2).view(like.shape)  # noqa: E731
    result["grads"] = {"q": share(dq, s["q"]), "k": share(dk, s["k"]), "v": dv.view(s["v"].shape),
                       "g": dg.view(s["g"].shape), "beta": dbeta.view(s["beta"].shape), "initial_state": dstate}
    return result


def _exact_step(s):
    state, heads = s["state"].double(), s["v"].shape[1]
    q, k = (s[n].double().repeat_interleave(heads // s[n].shape[1], 1) for n in ("q", "k"))
    out = torch.zeros(s["v"].shape, dtype=torch.float64, device=state.device)
    live = [(i, slot) for i, slot in enumerate(s["slots"].tolist()) if slot >= 0]
    row, slot = ([r[n] for r in live] for n in (0, 1))
    out[row], _, state[slot], _ = _row_of(torch.exp(s["g"].double())[row], k[row], q[row], s["v"].double()[row],
                                          s["beta"].double()[row], s["scale"], state[slot])
    return {"out": out, "state": state}


def _exact_norm(s):
    if s["op"] == "norm":
        v = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
    else:
        v = s["v"].double()
    leaves = [v.requires_grad_(), s["weight"].double().requires_grad_(), s["bias"].double().requires_grad_()]
    parts = []
    for p in v.chunk(s["groups"], 1):
        p = p - p.sum(1, keepdim=True) / p.shape[1]
        parts.append(p / (p.square().sum(1, keepdim=True) / p.shape[1] + 1e-5).sqrt())
    y = torch.cat(parts, 1) * leaves[1] + leaves[2]
    if s["op"] == "norm":
        return {"out": y.detach(), "sum": v.detach()} if s["residual"] is not None else {"out": y.detach()}
    dv, dw, db = torch.autograd.grad(y, leaves, s["grad"].double())
    if s["grad_residual"] is None:
        return {"weight": dw, "bias": db, "x": dv}
    dv = dv + s["grad_residual"].double()
    return {"weight": dw, "bias": db, "residual": dv, "x": dv}
