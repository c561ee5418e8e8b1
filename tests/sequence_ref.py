"""Plain 64-bit definitions of the sequence operators, one sequence and one
row after another (numpy), for the tests.

Every result comes with the sum of its terms' magnitudes: an f32 evaluation
differs from the exact one by at most (roundings on the longest path) * 2^-24
times that sum, whatever its order.
"""
import numpy as np


def sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def silu(x):
    return x * sigmoid(x)


def silu_slope(x):
    s = sigmoid(x)
    return s * (1 + x * (1 - s))


# --- causal convolution ----------------------------------------------------


def conv_pre(x, w, b, init):
    """p before the activation, and the inputs with the state rows in front."""
    width = w.shape[1]
    seq = np.concatenate([init, x])
    p = np.tile(b, (x.shape[0], 1)).astype(np.float64)
    for t in range(x.shape[0]):
        for k in range(width):
            p[t] += w[:, k] * seq[t + k]
    return p, seq


def conv(x, w, b, init, act):
    p, seq = conv_pre(x, w, b, init)
    mag, _ = conv_pre(abs(x), abs(w), abs(b), abs(init))
    halo = w.shape[1] - 1
    # |act'| <= 1.1: an error of p carries over by at most that
    return (silu(p) if act else p), seq[seq.shape[0] - halo:], mag


def conv_grad(dy, x, w, b, init, act, dfinal):
    p, seq = conv_pre(x, w, b, init)
    width = w.shape[1]

    def sums(g, w, seq, dfinal):
        dseq = np.zeros_like(seq)
        dw = np.zeros_like(w)
        for t in range(g.shape[0]):
            for k in range(width):
                dseq[t + k] += w[:, k] * g[t]
                dw[:, k] += g[t] * seq[t + k]
        if width > 1:
            dseq[seq.shape[0] - (width - 1):] += dfinal
        return dseq[width - 1:], dw, g.sum(0), dseq[:width - 1]

    g = dy * silu_slope(p) if act else dy
    # the activation's slope is itself computed from p, whose error is a few
    # roundings of its magnitude (|act''| <= 1)
    pm, _ = conv_pre(abs(x), abs(w), abs(b), abs(init))
    gm = abs(dy) * (1 + pm) * 1.2 if act else abs(dy)
    return sums(g, w, seq, dfinal), sums(gm, abs(w), abs(seq), abs(dfinal))


# --- selective scan --------------------------------------------------------


def delta_of(dt, bias, softplus):
    raw = dt + bias
    return np.logaddexp(raw, 0.0) if softplus else raw


def _expand(v, ch):
    """(rows, groups, n) -> (rows, channels, n)."""
    return np.repeat(v, ch // v.shape[1], axis=1)


def scan_states(u, delta, a, B, C, D, init):
    """y before the gate, the states before each row, and the last state."""
    rows, ch = u.shape
    Bx, Cx = _expand(B, ch), _expand(C, ch)
    h = init.copy()
    before = np.zeros((rows,) + h.shape)
    y = np.zeros((rows, ch))
    for t in range(rows):
        before[t] = h
        h = a[t] * h + (delta[t] * u[t])[:, None] * Bx[t]
        y[t] = (h * Cx[t]).sum(-1) + D * u[t]
    return y, before, h


def scan(u, dt, A, B, C, D, z, bias, softplus, init):
    """((out, final), (their magnitudes)); z None for no gate."""
    delta = delta_of(dt, bias, softplus)
    a = np.exp(delta[..., None] * A)
    y, _, last = scan_states(u, delta, a, B, C, D, init)
    ym, _, lastm = scan_states(abs(u), abs(delta), a, abs(B), abs(C), abs(D), abs(init))
    g = 1.0 if z is None else silu(z)
    return (y * g, last), (ym * abs(g), lastm)


def scan_grad(dout, u, dt, A, B, C, D, z, bias, softplus, init, dfinal):
    """Two dicts: the gradients and their terms' magnitudes."""
    raw = dt + bias
    delta = delta_of(dt, bias, softplus)
    a = np.exp(delta[..., None] * A)
    slope = sigmoid(raw) if softplus else np.ones_like(raw)

    def sums(dout, u, delta, A, B, C, D, init, dfinal, gate, gate_slope):
        rows, ch = u.shape
        groups, n = B.shape[1:]
        Bx, Cx = _expand(B, ch), _expand(C, ch)
        y, before, _ = scan_states(u, delta, a, B, C, D, init)
        dy = dout * gate
        g = {"z": dout * y * gate_slope, "u": D * dy, "dt": np.zeros_like(u), "A": np.zeros_like(A),
             "B": np.zeros_like(B), "C": np.zeros_like(C), "D": (dy * u).sum(0)}
        e = dfinal.copy()
        for t in reversed(range(rows)):
            dh = e + dy[t][:, None] * Cx[t]
            x = (delta[t] * u[t])[:, None]
            h = a[t] * before[t] + x * Bx[t]
            g["C"][t] = (dy[t][:, None] * h).reshape(groups, ch // groups, n).sum(1)
            g["B"][t] = (dh * x).reshape(groups, ch // groups, n).sum(1)
            q = (dh * Bx[t]).sum(-1)
            e = dh * a[t]
            w = e * before[t]
            g["u"][t] += q * delta[t]
            g["dt"][t] = (q * u[t] + (w * A).sum(-1)) * slope[t]
            g["A"] += w * delta[t][:, None]
        g["dt_bias"] = g["dt"].sum(0)
        g["initial_state"] = e
        return g

    one, zero = np.ones_like(u), np.zeros_like(u)
    gate, gate_slope = (one, zero) if z is None else (silu(z), silu_slope(z))
    return (sums(dout, u, delta, A, B, C, D, init, dfinal, gate, gate_slope),
            sums(*(abs(v) for v in (dout, u, delta, A, B, C, D, init, dfinal, gate)),
                 one if z is not None else zero))


# --- block norm ------------------------------------------------------------


def norm(v, w, gate, after, groups, eps):
    t = v * silu(gate) if gate is not None and not after else v
    by = t.reshape(t.shape[0], groups, t.shape[1] // groups)
    y = (by / np.sqrt((by ** 2).mean(-1, keepdims=True) + eps)).reshape(t.shape) * w
    return y * silu(gate) if gate is not None and after else y


def norm_grad(dy, v, w, gate, after, groups, eps, dsum):
    """Gradients of x * w / rms through `sum`: dict of v, weight, gate."""
    shape = v.shape
    g = silu(gate) if gate is not None else 1.0
    t = v * g if gate is not None and not after else v
    r = 1 / np.sqrt((t.reshape(shape[0], groups, shape[1] // groups) ** 2).mean(-1, keepdims=True) + eps)
    h = (t.reshape(shape[0], groups, shape[1] // groups) * r).reshape(shape)
    out = {}
    if gate is not None and after:
        out["gate"] = dy * h * w * silu_slope(gate)
        dy = dy * g
    out["weight"] = (dy * h).sum(0)
    gw = (dy * w).reshape(shape[0], groups, shape[1] // groups)
    hh = h.reshape(shape[0], groups, shape[1] // groups)
    dt = (r * (gw - hh * (gw * hh).mean(-1, keepdims=True))).reshape(shape)
    if gate is not None and not after:
        out["gate"] = dt * v * silu_slope(gate)
        dt = dt * g
    out["v"] = dt + dsum
    return out
