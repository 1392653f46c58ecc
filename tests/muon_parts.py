"""Matrices that show whether a product of the Newton-Schulz steps keeps both fp16 parts of its operands.

A matrix of 0 and +-1 whose norm is no power of two: its entries over the norm are one magnitude, so their lo parts are the
same share of their hi parts everywhere, and a lost part moves sums by that share instead of averaging out.  A row has few
entries, so sums have few terms and fp32 adds little to them.  The diagonal of S and the places that share one column
are powers of two times each other, with one share for their lo parts too."""
import math

import torch


def share(v):
    """The lo part of a held value over its hi part."""
    hi = torch.tensor(v, dtype=torch.float64).half().double().item()
    return abs(v - hi) / v


def entries(rows, cols):
    """(entries a row, of the short side; share of X's lo parts, of S's)."""
    m, n = sorted((rows, cols))
    best = None
    # about 64 other rows share a column with one; the power of two that shows most
    at = max(1, min(n // 2, round(math.sqrt(64 * n / m))))
    for p in {2 ** max(0, int(math.log2(at)) + d) for d in (0, 1)}:
        got = (min(share(4096 / math.sqrt(m * p)), share(4096 / m)), p)
        best = max(best, got) if best else got
    p = best[1]
    return p, share(4096 / math.sqrt(m * p)), share(4096 / m)


def sparse_signs(rows, cols, seed, device):
    m, n = sorted((rows, cols))
    p, _, _ = entries(rows, cols)
    gen = torch.Generator().manual_seed(seed)
    u = torch.zeros(m, n)
    for row in u:
        row[torch.randperm(n, generator=gen)[:p]] = 2.0 * torch.randint(0, 2, (p,), generator=gen).float() - 1.0
    return (u if rows <= cols else u.t().contiguous()).to(device)


def coefficients(rows, cols):
    """(a, b, c) of one step each, fp32 values: X again, by its two parts; b S X with a diagonal of b S of 1 + 1.9 / 4096, whose lo
    part is 1.9 where its hi part is 4096; c S^2 X with a diagonal of about 2."""
    m = float(min(rows, cols))  # the diagonal of S is entries a row / all entries: 1 / m
    fp32 = lambda v: torch.tensor(v, dtype=torch.float64).float().item()  # noqa: E731
    return (1.0, 0.0, 0.0), (0.0, fp32(m * (1 + 1.9 / 4096)), 0.0), (0.0, 0.0, m * m)


def expected(u, coefs):
    """One step in 64 bits, and how far each value may be off.

    A held value is within 2^-22 of itself (1.25 of it: X is rounded to fp32 before), or within 2^-25 where its lo part is
    subnormal; the product of two lo parts, left out, is 2^-22 of a term.  A sum of t terms, three products of parts
    each, is off by 3 t 2^-23 of the sum of their sizes (terms that cancel included); zeros add nothing."""
    x = u.double()
    if x.shape[0] > x.shape[1]:
        x = x.t().contiguous()
    nonzero = x != 0
    count = float(nonzero.sum())
    x = x / math.sqrt(count)
    a, b, c = coefs
    s = x @ x.t().contiguous()
    sizes = x.abs() @ x.abs().t().contiguous()
    t_gram, t_apply = int(nonzero.sum(1).max()), int(nonzero.sum(0).max())
    t_poly = int((sizes > 0).sum(1).max())
    rep = max(1.25 * 2.0 ** -22, 2.0 ** -25 * count / 4096)
    gram = 2 * rep + 2.0 ** -22 + 3 * t_gram * 2.0 ** -23
    poly = (2 * (gram + rep) + 2.0 ** -22 + 3 * t_poly * 2.0 ** -23) if c else gram + rep
    apply_ = poly + 2 * rep + 2.0 ** -22 + 3 * t_apply * 2.0 ** -23
    want = a * x + (b * s + c * (s @ s)) @ x
    size = abs(a) * x.abs() * rep + apply_ * ((abs(b) * sizes + abs(c) * (sizes @ sizes)) @ x.abs())
    most = size + 2.0 ** -23 * want.abs()
    return (want, most) if u.shape[0] <= u.shape[1] else (want.t().contiguous(), most.t().contiguous())


def emulated(u, coefs, lost=None):
    """One step on parts in 64-bit sums, without the parts named in `lost`: a set of "x lo gram", "x lo apply", "x lo add", "s lo
    poly", "s lo add", "b lo apply"."""
    lost = lost or set()
    x = u.double()
    if x.shape[0] > x.shape[1]:
        x = x.t().contiguous()

    def parts(v):
        held = (v * 4096).float()
        hi = held.half()
        return hi.double() / 4096, (held - hi.float()).half().double() / 4096

    def times(l, r, without_l, without_r):
        (lh, ll), (rh, rl) = l, r
        return lh @ rh + (0 if without_l else ll @ rh) + (0 if without_r else lh @ rl)

    a, b, c = coefs
    x = parts(x / x.norm())
    t = tuple(v.t().contiguous() for v in x)
    gone = "x lo gram" in lost
    s = parts(times(x, t, gone, gone))
    gone = "s lo poly" in lost
    poly = parts(c * times(s, tuple(v.t().contiguous() for v in s), gone, gone) + b * (s[0] + (0 if "s lo add" in lost else s[1])))
    out = times(poly, x, "b lo apply" in lost, "x lo apply" in lost) + a * (x[0] + (0 if "x lo add" in lost else x[1]))
    return out if u.shape[0] <= u.shape[1] else out.t().contiguous()


def off_by(got, want, most):
    """The worst place's error over what it may be."""
    return ((got.double() - want).abs() / most.clamp(min=1e-300)).max().item()


# (batch, rows, cols): matrices of one workgroup, of S and the rest, small tiles; tiles of 128, 192 and 256 in each product, whole
# and with their sums split; tall ones, whose last step is turned, in tiles of 192 and 256
SIZES = [(1, 96, 120), (1, 60, 4000), (1, 300, 200), (1, 1000, 1030), (1, 672, 11424), (1, 1194, 11424), (1, 1774, 9504), (1, 2006, 2006),
         (1, 2006, 9504), (1, 2818, 2818), (2, 2818, 2818), (3, 2702, 2702), (1, 4090, 4096), (1, 11424, 672), (3, 5288, 2644),
         (1, 11008, 4090)]
