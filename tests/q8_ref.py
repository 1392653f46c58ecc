"""Plain 64-bit forms of the 8-bit training operators, on the CPU."""
import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# a rounding to the type is off by at most half a step, relative to the value
HALF_STEP = {k: torch.finfo(v).eps / 2 for k, v in DT.items()}
U32 = 2.0 ** -24


def save(x, rule, col_scale=None):
    """Codes (int8) and scales (float32) of a CPU tensor's rows, each code by exact comparison in 64 bits."""
    v = x.to(torch.float32)
    if col_scale is not None:
        v = v * col_scale  # one fp32 rounding
    v = v.numpy()
    rows, cols = v.shape
    codes = np.zeros((rows, cols), dtype=np.int8)
    scales = np.empty(rows, dtype=np.float32)
    for t in range(rows):
        top = np.abs(v[t]).max() if cols else np.float32(0)
        if not np.isfinite(top):
            scales[t] = np.nan
            continue
        if rule == "amax":
            s = max(np.float32(top / np.float32(127)), np.float32(2.0 ** -126))
        else:
            e = -126
            while 127.0 * 2.0 ** e < float(top):
                e += 1
            s = np.float32(2.0 ** e)
        scales[t] = s
        codes[t] = np.rint(v[t].astype(np.float64) / np.float64(s)).astype(np.int8)
    return torch.from_numpy(codes), torch.from_numpy(scales)


def load(codes, scales, kind):
    """q * s in fp32, rounded to the type: the operator's own two roundings."""
    return (codes.to(torch.float32) * scales[:, None]).to(DT[kind])


def product(xq, sx, wq, sw, trans_w):
    """The exact product in 64 bits (sums of code products are below 2^53)."""
    w = wq.double()
    y = xq.double() @ (w.t() if trans_w else w)
    y = y * sx.double()[:, None]
    return y if sw is None else y * sw.double()


def product_tolerance(y, kind):
    """f32(S), times one scale, times the other: three fp32 roundings, then the output's; and the least step where it
    falls among the type's subnormals (whose half step is absolute)."""
    return y.abs() * ((1 + U32) ** 3 * (1 + HALF_STEP[kind]) - 1) + torch.finfo(DT[kind]).smallest_normal * HALF_STEP[kind] * 2


def weight_grad(dy, xq, sx, add=None):
    dw = dy.double().t() @ (xq.double() * sx.double()[:, None])
    return dw if add is None else dw + add.double()


def weight_grad_tolerance(dy, xq, sx, kind, add=None, exact_scale=True):
    """T additions in fp32, each off by at most one step (2^-23) of the largest partial sum, which is at most the sum
    of magnitudes; bf16 operands add half a bf16 step for each term when the scale is not a power of two; one more
    addition for `add`; then the output's rounding."""
    mags = dy.double().abs().t() @ (xq.double().abs() * sx.double()[:, None])
    if add is not None:
        mags = mags + add.double().abs()
    dw = weight_grad(dy, xq, sx, add)
    t = mags * (dy.shape[0] + 2) * 2.0 ** -23
    if not exact_scale:
        t = t + mags * HALF_STEP["bf16"]
    return t + (dw.abs() + t) * HALF_STEP[kind] + torch.finfo(DT[kind]).smallest_normal * HALF_STEP[kind] * 2


def outside(got, want, tolerance, kind):
    """Where a result is off by more than its tolerance.  Above 2^(emax + 1) (1 - eps / 4), half a step past the largest
    value, rounding to nearest gives an infinity: there the result has to be that infinity (within the tolerance of
    that border, either)."""
    info = torch.finfo(DT[kind])
    border = 2.0 ** (np.floor(np.log2(info.max)) + 1) * (1 - info.eps / 4)
    got, tolerance = got.cpu().double(), tolerance.clamp(max=border)
    off = (got - want).abs()
    good = torch.where(want.abs() + tolerance < border, off <= tolerance, torch.isinf(got) & (got.sign() == want.sign()))
    near = (want.abs() - tolerance <= border) & (want.abs() + tolerance >= border) & (got.sign() == want.sign())
    return ~(good | (near & (got.abs() >= border * (1 - 2 * info.eps))))
