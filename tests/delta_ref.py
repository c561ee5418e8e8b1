"""Plain 64-bit definitions of the gated delta rule and the layer norm, one
sequence and one row after another (numpy), for the tests.

With lengths of keys of at most 1, beta in [0, 1] and g <= 0 a step never
lengthens a difference of two states, so an error made at one row reaches a
later state at most decayed.  Each result therefore comes with the decayed sum
of the sizes of what the rows compute: an error of e times its size at every
row gives a state that is off by at most e times that sum, in the 2-norm.
"""
import numpy as np


def norm(x):
    return np.sqrt((x * x).sum(-1))


def delta(q, k, v, g, beta, scale, s0):
    """One head: out (rows, values), last state, and the sizes of each row's
    output and of the last state; `kept` for the gradient."""
    rows = v.shape[0]
    S, size = s0.copy(), np.sqrt((s0 * s0).sum())
    out, sizes, kept = np.zeros_like(v), np.zeros(rows), []
    for t in range(rows):
        a = np.exp(g[t])
        old = a * S
        hat = v[t] - old.T @ k[t]
        S = old + np.outer(k[t], beta[t] * hat)
        out[t] = scale * (S.T @ q[t])
        add = norm(k[t]) * beta[t] * (norm(v[t]) + norm(k[t]) * np.sqrt((old * old).sum()))
        size = a * size + add
        sizes[t] = scale * norm(q[t]) * size
        kept.append((old, S, hat, size))
    return out, S, sizes, size, kept


def delta_grad(dout, q, k, v, g, beta, scale, s0, dlast):
    """Dicts of one head's gradients and of their sizes: q, k, v a row's
    2-norm, g and beta each its own, initial_state the whole's."""
    rows, keys = k.shape
    _, _, _, _, kept = delta(q, k, v, g, beta, scale, s0)
    d, size = dlast.copy(), np.sqrt((dlast * dlast).sum())
    G = {"q": np.zeros_like(q), "k": np.zeros_like(k), "v": np.zeros_like(v), "g": np.zeros(rows), "beta": np.zeros(rows)}
    Z = {n: np.zeros(rows) for n in G}
    above = 0.0  # sizes of the later rows' terms of g's gradient, a sum over them
    for t in reversed(range(rows)):
        old, S, hat, ssize = kept[t]
        d = d + scale * np.outer(q[t], dout[t])
        size = size + scale * norm(q[t]) * norm(dout[t])
        du = d.T @ k[t]
        G["q"][t] = scale * (S @ dout[t])
        Z["q"][t] = scale * norm(dout[t]) * ssize
        G["beta"][t] = du @ hat
        dhat = beta[t] * du
        G["v"][t] = dhat
        G["k"][t] = d @ (beta[t] * hat) - old @ dhat
        nk, nu = norm(k[t]), beta[t] * (norm(v[t]) + norm(k[t]) * ssize)
        Z["v"][t] = beta[t] * nk * size
        Z["beta"][t] = nk * size * (norm(v[t]) + nk * ssize)
        Z["k"][t] = size * nu + ssize * beta[t] * nk * size
        d = d - np.outer(k[t], dhat)
        G["g"][t] = (d * old).sum()
        # dg is a sum over rows from t to the chunk's end of terms of q, k and the states
        above = above + norm(q[t]) * Z["q"][t] + 2 * nk * Z["k"][t]
        Z["g"][t] = above + size * ssize
        a = np.exp(g[t])
        d, size = a * d, a * size + beta[t] * nk * nk * np.sqrt((d * d).sum())
    G["initial_state"], Z["initial_state"] = d, size
    return G, Z


def layer_norm(v, w, b, groups, eps):
    by = v.reshape(v.shape[0], groups, v.shape[1] // groups)
    by = by - by.mean(-1, keepdims=True)
    return (by / np.sqrt((by ** 2).mean(-1, keepdims=True) + eps)).reshape(v.shape) * w + b


def layer_norm_grad(dy, v, w, groups, eps, dsum):
    """Dicts of gradients and of the sums of their terms' magnitudes."""
    shape = (v.shape[0], groups, v.shape[1] // groups)
    by = v.reshape(shape)
    by = by - by.mean(-1, keepdims=True)
    r = 1 / np.sqrt((by ** 2).mean(-1, keepdims=True) + eps)
    h = by * r
    gw = (dy * w).reshape(shape)
    dv = r * (gw - gw.mean(-1, keepdims=True) - h * (gw * h).mean(-1, keepdims=True))
    mag = r * (abs(gw) + abs(gw).mean(-1, keepdims=True) + abs(h) * abs(gw * h).mean(-1, keepdims=True))
    hh = h.reshape(v.shape)
    return ({"v": dv.reshape(v.shape) + dsum, "weight": (dy * hh).sum(0), "bias": dy.sum(0)},
            {"v": mag.reshape(v.shape) + abs(dsum), "weight": (abs(dy) * (1 + abs(hh))).sum(0), "bias": abs(dy).sum(0)})
