"""The gated feed-forward block against 64-bit forms (tests/glu_ref.py).

Sums are tested with whole numbers, which every order of fp32 additions adds exactly below 2^24: results are equal bit
for bit, whatever the tile.  Activations are tested value by value, with derived tolerances.  Matrices are views into
wider buffers filled with a pattern, which has to survive around the outputs, and with NaN around the operands."""
import math

import numpy as np
import pytest
import torch

from tests import glu_ref as ref

pytestmark = pytest.mark.gpu

DT = ref.DT


@pytest.fixture(scope="module")
def zs():
    import sharded_mixed_precision_rank_amd as zs

    return zs


class Buf:
    """A rows x cols view with `gap` elements between rows and `lead` before the first.  Around it: NaN for an operand, a
    pattern for an output."""

    def __init__(self, rows, cols, dtype, gap=0, lead=0, values=None):
        n = lead + (rows + 1) * (cols + gap) + 64
        if values is None:
            self.flat = (torch.arange(n) % 89 + 1).to(dtype).cuda()
        else:
            self.flat = torch.full((n,), math.nan, dtype=dtype, device="cuda")
        self.t = self.flat.as_strided((rows, cols), (cols + gap, 1), lead)
        if values is not None:
            self.t.copy_(values.to(dtype))
        self.before = self.flat.clone()

    def untouched_outside(self):
        a, b = self.flat.clone(), self.before.clone()
        for x in (a, b):
            x.as_strided(self.t.shape, self.t.stride(), self.t.storage_offset()).zero_()
        return torch.equal(torch.nan_to_num(a, nan=77.0), torch.nan_to_num(b, nan=77.0))


def whole(rng, rows, cols, most=3):
    return torch.from_numpy(rng.integers(-most, most + 1, (rows, cols)).astype(np.float32))


def same(got, want, dtype):
    """Equal after one rounding to the output's type."""
    return torch.equal(got.cpu(), want.to(dtype))


def near(got, want, kind, sums=0.0):
    """Within one rounding of `kind` of a value that is `sums` off at most."""
    off = (got.cpu().double() - want).abs()
    most = sums + ref.half_step(kind) * (want.abs() + sums) + ref.least(kind)
    worst = (off / most).max().item() if off.numel() else 0.0
    assert worst <= 1.0, worst
    return True


# (gap, lead) of every matrix: rows on 16-byte boundaries, on 4-byte ones (where the columns are even), and anywhere
LAYOUTS = [(0, 0), (8, 16), (6, 2), (5, 3)]
SHAPES = [(1, 1, 1), (1, 8, 8), (1, 300, 520), (3, 7, 5), (2, 33, 64), (16, 64, 128), (17, 130, 72), (64, 32, 64), (65, 96, 200),
          (100, 264, 136), (129, 257, 65), (300, 200, 328)]
# tiles of 128 and of 256, ragged at every side, and a summed axis that ends inside a stage
LARGE = [(520, 1400, 200), (700, 2100, 1000), (2100, 2600, 136), (2304, 3600, 72)]


# one more for each kernel that the sizes above do not reach: forward in tiles of 64 x 32, 64 x 64, 128 x 128, 192 x 128 and
# 256 x 256; input gradient in 32 x 64, 64 x 128 and 128 x 128 in two forms; weight gradients in 128 x 128 in two forms
FORWARD_TILES = [(61, 3924, 322), (67, 2141, 194), (262, 3362, 346), (333, 5504, 200), (2700, 2300, 136)]
INPUT_TILES = [(2301, 70, 65), (292, 3345, 193), (2298, 2870, 72), (3379, 533, 72)]
WEIGHT_TILES = [(457, 3823, 326), (739, 2766, 33), (1600, 2300, 520)]


def buf(rows, cols, dtype, gap, lead, values=None):
    """Rows whose distance is a multiple of 8 elements, unless the gap is odd."""
    return Buf(rows, cols, dtype, gap + (-cols % 8 if gap % 8 == 0 else 0), lead, values)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES + LARGE + FORWARD_TILES)
def test_forward_of_whole_numbers(zs, shape, kind):
    T, N, K = shape
    rng = np.random.default_rng(T * 31 + N * 7 + K)
    x, wg, wu = whole(rng, T, K), whole(rng, N, K), whole(rng, N, K, 1)
    h, gate, up = ref.forward(x, wg, wu, "relu")
    for gap, lead in LAYOUTS:
        bx, bg, bu = (buf(*v.shape, DT[kind], gap, lead, v) for v in (x, wg, wu))
        bh, kg, ku = (buf(T, N, DT[kind], gap, lead) for _ in range(3))
        zs.glu_forward(bx.t, bg.t, bu.t, bh.t, gate=kg.t, up=ku.t, act="relu")
        torch.cuda.synchronize()
        assert same(kg.t, gate, DT[kind]) and same(ku.t, up, DT[kind])
        # h: the product of two sums, rounded to fp32 and then to 16 bits: exact below 2^24 before the second
        assert same(bh.t, h.float(), DT[kind])
        only = buf(T, N, DT[kind], gap, lead)
        zs.glu_forward(bx.t, bg.t, bu.t, only.t, act="relu")
        torch.cuda.synchronize()
        assert torch.equal(only.t, bh.t)
        assert all(b.untouched_outside() for b in (bh, kg, ku, only))


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES + LARGE + INPUT_TILES)
def test_input_grad_of_whole_numbers(zs, shape, kind):
    T, K, N = shape
    rng = np.random.default_rng(T * 31 + N * 7 + K)
    dg, du, wg, wu = whole(rng, T, N), whole(rng, T, N), whole(rng, N, K), whole(rng, N, K)
    want = dg.double() @ wg.double() + du.double() @ wu.double()
    for gap, lead in LAYOUTS:
        a, b, c, d = (buf(*v.shape, DT[kind], gap, lead, v) for v in (dg, du, wg, wu))
        dx = buf(T, K, DT[kind], gap, lead)
        zs.glu_input_grad(a.t, b.t, c.t, d.t, dx.t)
        torch.cuda.synchronize()
        assert same(dx.t, want, DT[kind])
        assert dx.untouched_outside()


@pytest.mark.parametrize("out", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES + LARGE + WEIGHT_TILES)
def test_weight_grad_of_whole_numbers(zs, shape, kind, out):
    N, K, T = shape
    rng = np.random.default_rng(T * 31 + N * 7 + K)
    dg, du, x = whole(rng, T, N), whole(rng, T, N), whole(rng, T, K)
    want = [v.double().t() @ x.double() for v in (dg, du)]
    add = [whole(rng, N, K, 9).to(DT[out]) for _ in range(2)]
    for gap, lead in LAYOUTS:
        a, b, c = (buf(*v.shape, DT[kind], gap, lead, v) for v in (dg, du, x))
        og, ou = (buf(N, K, DT[out], gap, lead) for _ in range(2))
        zs.glu_weight_grad(a.t, b.t, c.t, og.t, ou.t)
        torch.cuda.synchronize()
        assert same(og.t, want[0], DT[out]) and same(ou.t, want[1], DT[out])
        ag, au = (buf(N, K, DT[out], gap, lead, v) for v in add)
        zs.glu_weight_grad(a.t, b.t, c.t, og.t, ou.t, add_gate=ag.t, add_up=au.t)
        zs.glu_weight_grad(a.t, b.t, c.t, ag.t, au.t, add_gate=ag.t, add_up=au.t)  # onto themselves
        torch.cuda.synchronize()
        for got in (og, ag):
            assert same(got.t, want[0] + add[0].double(), DT[out])
        for got in (ou, au):
            assert same(got.t, want[1] + add[1].double(), DT[out])
        assert all(v.untouched_outside() for v in (og, ou, ag, au))


def spread(kind, n):
    """Values over the type's range: small and large ones, both signs, zero, the ends."""
    rng = np.random.default_rng(n)
    v = rng.standard_normal(n) * np.exp(rng.uniform(-9, 4, n))
    v[:12] = [0.0, -0.0, 1.0, -1.0, 30.0, -30.0, 88.0, -88.0, 100.0, -100.0, 200.0, -6.0]
    return torch.from_numpy(v.astype(np.float32)).to(DT[kind])


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_activations_of_the_forward(zs, kind, act):
    """One token of 1 through weights of one column: gate and up are the weights themselves."""
    n = 5000
    wg, wu = spread(kind, n), spread(kind, n + 1)[:n]
    x = torch.ones(1, 1, dtype=DT[kind], device="cuda")
    h = torch.empty(1, n, dtype=DT[kind], device="cuda")
    zs.glu_forward(x, wg[:, None].cuda(), wu[:, None].cuda(), h, act=act)
    want = ref.act(wg.double(), act)[0] * wu.double()
    # fp32 activations: a few roundings of 2^-24 each, and (1 + |z|) of them in an exponent (|z| below 104 where the
    # result is not zero): 2^-16 relative.  A logistic function below 2^-126 may become 0, which is off by 2^-126, and
    # times gate and up by 2^-126 |gate up|
    near(h[0], want, kind, want.abs() * 2.0 ** -16 + 2.0 ** -126 * (wg.double() * wu.double()).abs())


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4099), (7, 64), (33, 1000), (5, 13)])
def test_backward(zs, rows, cols, kind, act):
    n = rows * cols
    gate, up, dh = (spread(kind, max(n, 12) + k)[:n].reshape(rows, cols) for k in range(3))
    dg, du, h = ref.backward(dh, gate, up, act)
    value, slope = ref.act(gate.double(), act)
    # the slope is a sum of two terms of at most 1.2: 2^-16 of that, and the products
    # (|v s (1 - s) z'| is at most 1.2 too)
    off_slope = 2.0 ** -16 * 2.4 * torch.ones_like(slope) if act != "relu" else 0 * slope
    # (a logistic function below 2^-126 may become 0: off by 2^-126 |gate|)
    off_value = 2.0 ** -16 * value.abs() + 2.0 ** -126 * gate.double().abs()
    tol_dg = (dh.double() * up.double()).abs() * (off_slope + 2.0 ** -22 * slope.abs())
    tol_du = dh.double().abs() * off_value
    tol_h = up.double().abs() * off_value
    for gap, lead in LAYOUTS:
        bd, bg, bu = (Buf(rows, cols, DT[kind], gap, lead, v) for v in (dh, gate, up))
        og, ou, oh = (Buf(rows, cols, DT[kind], gap, lead) for _ in range(3))
        zs.glu_backward(bd.t, bg.t, bu.t, og.t, ou.t, h=oh.t, act=act)
        torch.cuda.synchronize()
        near(og.t, dg, kind, tol_dg)
        near(ou.t, du, kind, tol_du)
        near(oh.t, h, kind, tol_h)
        assert all(b.untouched_outside() for b in (og, ou, oh))
        # onto its inputs, and without h: the same
        zs.glu_backward(bd.t, bg.t, bu.t, bg.t, bu.t, h=bd.t, act=act)
        torch.cuda.synchronize()
        assert torch.equal(bg.t, og.t) and torch.equal(bu.t, ou.t) and torch.equal(bd.t, oh.t)
        assert all(b.untouched_outside() for b in (bd, bg, bu))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_backward_against_differences(zs, act):
    """Central differences of h in 64 bits: off by step^2 / 6 times the third derivative (below 2 for these)."""
    gate, up = torch.linspace(-6, 6, 1024).to(torch.float16), torch.linspace(-2, 3, 1024).to(torch.float16)
    dh = torch.ones(1, 1024, dtype=torch.float16)
    og, ou = (torch.empty(1, 1024, dtype=torch.float16, device="cuda") for _ in range(2))
    zs.glu_backward(dh.cuda(), gate[None].cuda(), up[None].cuda(), og, ou, act=act)
    e = 1e-4
    f = lambda v: ref.act(v, act)[0]  # noqa: E731
    slope = (f(gate.double() + e) - f(gate.double() - e)) / (2 * e) * up.double()
    near(og[0], slope, "fp16", up.double().abs() * (2 * e * e / 6 + 2.0 ** -14))
    near(ou[0], f(gate.double()), "fp16", 2.0 ** -16 * f(gate.double()).abs())


def test_ends_of_the_range(zs):
    """Far values have finite activations and slopes; a result past fp16's range is an infinity; NaN stays NaN."""
    for kind, far in (("fp16", 65504.0), ("bf16", 3e38)):
        gate = torch.tensor([[far, -far, far, -far, math.nan]], dtype=DT[kind], device="cuda")
        up = torch.tensor([[1.0, 1.0, 0.0, 0.0, 1.0]], dtype=DT[kind], device="cuda")
        dh = torch.ones_like(gate)
        for act in ref.ACTS:
            dg, du, h = (torch.empty_like(gate) for _ in range(3))
            zs.glu_backward(dh, gate, up, dg, du, h=h, act=act)
            f = gate[0, 0].item()
            assert dg[0, :4].tolist() == [1.0, 0.0, 0.0, 0.0]
            assert du[0, :4].tolist() == [f, 0.0, f, 0.0]
            assert h[0, :4].tolist() == [f, 0.0, 0.0, 0.0]
            assert torch.isnan(du[0, 4]) and torch.isnan(h[0, 4])
    x = torch.full((2, 64), 100.0, dtype=torch.float16, device="cuda")
    w = torch.full((3, 64), 100.0, dtype=torch.float16, device="cuda")
    h = torch.empty(2, 3, dtype=torch.float16, device="cuda")
    zs.glu_forward(x, w, w, h, act="relu")
    assert torch.isinf(h).all()


def test_non_finite_values_stay_in_their_rows(zs):
    """A token with a NaN, a weight row with an infinity: nothing else changes, in every kernel's tiles."""
    for T, N, K in ((5, 40, 72), (130, 200, 264), (600, 1300, 200)):
        rng = np.random.default_rng(T)
        x, wg, wu = (v.bfloat16().cuda() for v in (whole(rng, T, K), whole(rng, N, K), whole(rng, N, K)))
        h, h2 = (torch.empty(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        zs.glu_forward(x, wg, wu, h, act="relu")
        x[T // 2, K - 1] = math.nan
        wu[N - 2, 0] = math.inf
        zs.glu_forward(x, wg, wu, h2, act="relu")
        assert torch.isnan(h2[T // 2]).all()
        keep_t, keep_n = torch.arange(T, device="cuda") != T // 2, torch.arange(N, device="cuda") != N - 2
        assert torch.equal(h[keep_t][:, keep_n], h2[keep_t][:, keep_n])
        assert not torch.isfinite(h2[keep_t][:, N - 2]).all()
        dg, du = (whole(rng, T, N).bfloat16().cuda() for _ in range(2))
        xx = whole(rng, T, K).bfloat16().cuda()
        o, o2 = ([torch.empty(N, K, device="cuda") for _ in range(2)] for _ in range(2))
        zs.glu_weight_grad(dg, du, xx, *o)
        du[T - 1, 3] = math.nan
        zs.glu_weight_grad(dg, du, xx, *o2)
        assert torch.equal(o[0], o2[0]) and torch.isnan(o2[1][3]).all()
        rows = torch.arange(N, device="cuda") != 3
        assert torch.equal(o[1][rows], o2[1][rows])


def test_sums_of_nothing_and_empty_calls(zs):
    for kind in ("bf16", "fp16"):
        new = lambda r, c, v=5.0: torch.full((r, c), v, dtype=DT[kind], device="cuda")  # noqa: E731
        h, g, u = new(3, 4), new(3, 4), new(3, 4)
        zs.glu_forward(new(3, 0), new(4, 0), new(4, 0), h, gate=g, up=u, act="gelu")
        assert (h == 0).all() and (g == 0).all() and (u == 0).all()
        dx = new(3, 4)
        zs.glu_input_grad(new(3, 0), new(3, 0), new(0, 4), new(0, 4), dx)
        assert (dx == 0).all()
        dw, dv = torch.full((4, 5), 7.0, device="cuda"), torch.full((4, 5), 8.0, device="cuda")
        zs.glu_weight_grad(new(0, 4), new(0, 4), new(0, 5), dw, dv, add_gate=dw, add_up=dv)
        assert (dw == 7).all() and (dv == 8).all()
        zs.glu_weight_grad(new(0, 4), new(0, 4), new(0, 5), dw, dv)
        assert (dw == 0).all() and (dv == 0).all()
        zs.glu_forward(new(0, 6), new(4, 6), new(4, 6), new(0, 4))
        zs.glu_forward(new(3, 6), new(0, 6), new(0, 6), new(3, 0))
        zs.glu_backward(new(0, 4), new(0, 4), new(0, 4), new(0, 4), new(0, 4))
        zs.glu_input_grad(new(0, 4), new(0, 4), new(4, 6), new(4, 6), new(0, 6))
        torch.cuda.synchronize()


@pytest.mark.parametrize("T,N,K", [(40, 130, 96), (700, 1500, 520)])
def test_graphs_and_streams(zs, T, N, K):
    """The whole block captured into a graph, replayed with new inputs in between; and on another stream."""
    rng = np.random.default_rng(5)
    new = lambda r, c, t=torch.bfloat16: torch.zeros(r, c, dtype=t, device="cuda")  # noqa: E731
    x, wg, wu, dh = new(T, K), new(N, K), new(N, K), new(T, N)
    outs = [new(T, N) for _ in range(5)] + [new(T, K)] + [new(N, K, torch.float32) for _ in range(2)]

    def fill(k):
        r = np.random.default_rng(k)
        for t in (x, wg, wu, dh):
            t.copy_(whole(r, *t.shape))

    def step(o):
        zs.glu_forward(x, wg, wu, o[0], gate=o[1], up=o[2], act="silu")
        zs.glu_backward(dh, o[1], o[2], o[3], o[4], act="silu")
        zs.glu_input_grad(o[3], o[4], wg, wu, o[5])
        zs.glu_weight_grad(o[3], o[4], x, o[6], o[7])

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(outs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(outs)
    for k in range(1, 4):
        fill(k)
        eager = [torch.empty_like(t) for t in outs]
        step(eager)
        for t in outs:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager))
        other = [torch.zeros_like(t) for t in outs]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(other)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(other, eager))


def test_rows_past_32_bit_offsets(zs):
    """Tokens whose elements lie past 2^31: the last rows are right, forward and back."""
    T, N, K = 70000, 32768, 64
    new = lambda r, c: torch.zeros(r, c, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    x, wg, wu = new(T, K), new(N, K), new(N, K)
    rng = np.random.default_rng(1)
    last = slice(T - 3, T)
    x[last] = whole(rng, 3, K).bfloat16().cuda()
    wg.copy_(whole(rng, N, K))
    wu.copy_(whole(rng, N, K))
    h, gate, up = new(T, N), new(T, N), new(T, N)
    zs.glu_forward(x, wg, wu, h, gate=gate, up=up, act="relu")
    torch.cuda.synchronize()
    want = ref.forward(x[last].cpu(), wg.cpu(), wu.cpu(), "relu")
    assert same(h[last], want[0].float(), torch.bfloat16) and same(gate[last], want[1], torch.bfloat16)
    assert not h[: T - 3].any()
    h[last] = 1  # dh, in place
    zs.glu_backward(h, gate, up, gate, up, act="relu")
    dx = new(T, K)
    zs.glu_input_grad(gate, up, wg, wu, dx)
    dg, du, _ = ref.backward(torch.ones(3, N), want[1], want[2], "relu")
    torch.cuda.synchronize()
    assert same(gate[last], dg, torch.bfloat16) and same(up[last], du, torch.bfloat16)
    dx_want = dg.bfloat16().double() @ wg.cpu().double() + du.bfloat16().double() @ wu.cpu().double()
    assert same(dx[last], dx_want, torch.bfloat16)
    dwg, dwu = (torch.empty(N, K, device="cuda") for _ in range(2))
    zs.glu_weight_grad(gate, up, x, dwg, dwu)
    torch.cuda.synchronize()
    assert same(dwu, du.bfloat16().double().t() @ x[last].cpu().double(), torch.float32)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("T,N,K", [(1, 11008, 4096), (333, 1376, 4096), (2048, 4096, 1024)])
def test_real_sizes(zs, T, N, K, kind):
    """Every value is rounded once from a sum that is off by far less: the 2-norm of all roundings is below half a
    step of the result's.  dx and the weight gradients carry the rounding of dgate and dup too."""
    g = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda r, c, s: (s * torch.randn(r, c, generator=g, device="cuda")).to(DT[kind])  # noqa: E731
    x, wg, wu, dh = rand(T, K, 1), rand(N, K, 0.02), rand(N, K, 0.02), rand(T, N, 1)
    new = lambda r, c: torch.empty(r, c, dtype=DT[kind], device="cuda")  # noqa: E731
    h, gate, up, dg, du, dx = new(T, N), new(T, N), new(T, N), new(T, N), new(T, N), new(T, K)
    dwg, dwu = new(N, K), new(N, K)
    zs.glu_forward(x, wg, wu, h, gate=gate, up=up, act="silu")
    zs.glu_backward(dh, gate, up, dg, du, act="silu")
    zs.glu_input_grad(dg, du, wg, wu, dx)
    zs.glu_weight_grad(dg, du, x, dwg, dwu)
    gate64, up64 = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    s = torch.sigmoid(gate.double())
    dg64 = dh.double() * up.double() * (s + gate.double() * s * (1 - s))
    du64 = dh.double() * gate.double() * s
    checks = [(gate, gate64, 1), (up, up64, 1), (h, gate64 * torch.sigmoid(gate64) * up64, 1), (dg, dg64, 1), (du, du64, 1),
              (dx, dg64 @ wg.double() + du64 @ wu.double(), 2), (dwg, dg64.t() @ x.double(), 2), (dwu, du64.t() @ x.double(), 2)]
    for got, want, roundings in checks:
        off = ((got.double() - want).norm() / want.norm()).item()
        assert off <= roundings * ref.half_step(kind) + 1e-5, off


# every bf16 value in a range where the activation falls from 2^-110 to below bf16's smallest
TAILS = {"silu": (-110.0, -76.0), "gelu": (-14.5, -12.0), "gelu_tanh": (-11.0, -9.0)}


@pytest.mark.parametrize("act", TAILS)
def test_tails_of_the_activations(zs, act):
    """Where act and its slope are far below 2^-100 they are still bf16 values, normal ones down to 2^-126."""
    lo, hi = (torch.tensor(v, dtype=torch.bfloat16).view(torch.int16).item() for v in TAILS[act])
    gate = torch.arange(hi, lo + 1, dtype=torch.int16).view(torch.bfloat16)  # (of negative values the larger bits are lower)
    n = gate.numel()
    rng = np.random.default_rng(n)
    up, dh = (torch.from_numpy(rng.uniform(0.3, 3.0, n) * rng.choice((-1, 1), n)).bfloat16() for _ in range(2))
    value, slope = ref.act(gate.double(), act)
    if act == "gelu_tanh":  # (1 - tanh^2 by the logistic function: 4 s(z) s(-z))
        c, v = 2 * math.sqrt(2 / math.pi), gate.double()
        z = c * (v + 0.044715 * v ** 3)
        slope = torch.sigmoid(z) * (1 + v * torch.sigmoid(-z) * c * (1 + 3 * 0.044715 * v * v))
    assert value.abs().max() > 2.0 ** -112 and 0 < value.abs().min() < 2.0 ** -133
    assert ((value.abs() < 2.0 ** -120) & (value.abs() > 2.0 ** -126)).sum() >= 2
    # fp32 steps: an exponent's argument of at most 160, off by 3 roundings of 2^-24 and 2^-18: below 2^-14 relative; where a
    # factor is subnormal by 2^-147 (a rounding of 2^-150 and its like for the error function), times gate in a product
    off_value = 2.0 ** -14 * value.abs() + 2.0 ** -147 * gate.double().abs()
    off_slope = 2.0 ** -14 * slope.abs() + 2.0 ** -147 * gate.double().abs() ** 2
    new = lambda: torch.empty(1, n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    h, dg, du, again = new(), new(), new(), new()
    x = torch.ones(1, 1, dtype=torch.bfloat16, device="cuda")
    zs.glu_forward(x, gate[:, None].cuda(), up[:, None].cuda(), h, act=act)
    zs.glu_backward(dh[None].cuda(), gate[None].cuda(), up[None].cuda(), dg, du, h=again, act=act)
    near(h[0], value * up.double(), "bf16", off_value * up.double().abs())
    near(again[0], value * up.double(), "bf16", off_value * up.double().abs())
    near(du[0], value * dh.double(), "bf16", off_value * dh.double().abs())
    near(dg[0], slope * up.double() * dh.double(), "bf16", off_slope * (up.double() * dh.double()).abs() + 2.0 ** -148)


def test_outputs_past_the_small_tiles_count(zs):
    """More outputs than 2^22 tiles of 64 x 32: the last rows are right and the others zeros, forward and back."""
    T, N, K = 800_000, 11008, 64
    new = lambda r, c: torch.zeros(r, c, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    rng = np.random.default_rng(2)
    last = slice(T - 3, T)
    for first in (True, False):
        out = torch.full((T, N), 5.0, dtype=torch.bfloat16, device="cuda")
        if first:
            x, wg, wu = new(T, K), whole(rng, N, K).bfloat16().cuda(), whole(rng, N, K).bfloat16().cuda()
            x[last] = whole(rng, 3, K).bfloat16().cuda()
            zs.glu_forward(x, wg, wu, out, act="relu")
            want = ref.forward(x[last].cpu(), wg.cpu(), wu.cpu(), "relu")[0].float()
        else:
            dg, du, wg, wu = new(T, K), new(T, K), whole(rng, K, N).bfloat16().cuda(), whole(rng, K, N).bfloat16().cuda()
            dg[last], du[last] = (whole(rng, 3, K).bfloat16().cuda() for _ in range(2))
            zs.glu_input_grad(dg, du, wg, wu, out)
            want = dg[last].cpu().double() @ wg.cpu().double() + du[last].cpu().double() @ wu.cpu().double()
        torch.cuda.synchronize()
        assert same(out[last], want, torch.bfloat16)
        assert not out[: T - 3].any()
        del out
