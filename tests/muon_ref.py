"""Newton-Schulz steps in 64 bits, from the definition in the header."""
import torch

COEFS = (3.4445, -4.7750, 2.0315)


def steps_of(u, steps=5, coefs=COEFS):
    """The steps of one matrix, in its device's 64-bit products."""
    each = [coefs] * steps if not hasattr(coefs[0], "__len__") else coefs
    x = u.double()
    norm = x.norm()
    x = x / norm if norm != 0 else x
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t().contiguous()
    for a, b, c in each:
        s = x @ x.t().contiguous()
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.t().contiguous() if tall else x


def bound(steps, rows, cols):
    """How far results may be off, in the 2-norm relative to sqrt(min(rows, cols)), the norm of an orthogonal matrix.

    A step's operands are held to 2^-22 and its fp32 sums add about as much: less than 2^-20 of |X| in all.  A step
    multiplies an earlier perturbation by at most 4 (the largest slope of a s + b s^3 + c s^5 on [0, 1.21], 3.95, which bounds
    its divided differences too), and lifts |X|, which starts at 1, by at most 3.45."""
    short = min(rows, cols) ** 0.5
    return sum(4.0 ** (steps - 1 - k) * 2.0 ** -20 * min(3.45 ** (k + 1), 1.21 * short) for k in range(steps)) / short
