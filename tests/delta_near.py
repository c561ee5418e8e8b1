"""How near the gated delta rule's results are to be to the 64-bit definition,
head by head in the relative 2-norm.

An f32 in two pieces of bf16 keeps 17 bits, its sign's among them: at most
2^-17 of a number is lost, 2.4e-6 in the mean square.  Two such numbers in a
product, and four products one after another (the chunk's inverse, the
corrections, the state, the read), whose errors add as squares, leave 7e-6 of
the terms; sums of terms that cancel to about half their size 2^-16.  The
gradients of g and beta are sums of such sums with both signs: twice that.

A result w + e, |e| small, rounded to a type is off by at most what w rounded
to it would be and 2 |e| (where e moves it past a middle, both neighbours are
within |e| of equally far).  So a 16-bit result is off by its own rounding,
computed from the exact one, and twice the above.
"""
import numpy as np

NEAR = {"out": 2.0 ** -16, "final": 2.0 ** -16, "q": 2.0 ** -16, "k": 2.0 ** -16, "v": 2.0 ** -16, "initial_state": 2.0 ** -16,
        "g": 2.0 ** -15, "beta": 2.0 ** -15}
CHUNK = 64


def far(got, want):
    """The 2-norm of the difference over that of what is wanted."""
    return np.sqrt(((got - want) ** 2).sum() / (want ** 2).sum())


def windows(rows):
    """The whole, and each chunk of rows: those after a part's first row among them."""
    return [slice(0, rows), *(slice(r, min(r + CHUNK, rows)) for r in range(0, rows, CHUNK))]


def check(name, got, want, rounded, by_rows=True):
    """`got`, `want` and `rounded` (want in the output's type), float64 arrays of rows; the whole within its bound, each
    chunk within four times it (fewer terms, and a share of the whole's size each)."""
    for i, w in enumerate(windows(len(want)) if by_rows else [...]):
        x = want[w]
        own = far(rounded[w], x)
        limit = own + (2 if own else 1) * (4 if i else 1) * NEAR[name]
        assert far(got[w], x) <= limit, "%s, rows %s: %.3g against %.3g" % (name, w, far(got[w], x), limit)
