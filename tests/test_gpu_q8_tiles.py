"""The tiled kernels of the 8-bit weight gradient (128 x 128 and 256 x 256, operands loaded to LDS directly or through
registers) and the split one, at scales that are no power of two, non-finite values, values around the operands, long
sums that have to be exact, captured graphs and repeated calls.  Plain forms in 64 bits."""
import numpy as np
import pytest
import torch

from tests import q8_ref as ref
from tests.test_gpu_q8 import Buf, _layer, _layer_buffers, activations, random_codes, random_scales, same_bits

pytestmark = pytest.mark.gpu

DT = ref.DT
# (T, N, K): few weights, split over tokens; 12 x 12 tiles of 128; 17 x 13 tiles of 256 (rows anywhere: 128 x 128)
SHAPES = [(300, 130, 200), (200, 1500, 1530), (272, 4100, 3300)]


@pytest.fixture(scope="module")
def zs():
    import sharded_mixed_precision_rank_amd as zs

    return zs


def operands(dy, x, aligned):
    """Views of dy and x with rows on 16-byte boundaries, or anywhere."""
    (T, N), K = dy.shape, x.shape[1]
    gaps = (-N % 8, -K % 16, 16) if aligned else (3, 5, 1)
    return Buf(T, N, dy.dtype, gaps[0], 0 if aligned else 1, dy).t, Buf(T, K, torch.int8, gaps[1], gaps[2], x).t


def rounded_operand(x, sx):
    """A code times its scale as the contract has it: the fp32 product rounded to bf16."""
    return (x.to(torch.float32) * sx[:, None]).to(torch.bfloat16).double()


def gradient(dy, x, sx):
    """dw in 64 bits from the rounded operand, and the error of its fp32 sums: T additions (twice that for fp16's two
    parts), each off by at most one step, 2^-23, of the partial sums' bound."""
    w = rounded_operand(x, sx)
    dw = dy.double().t() @ w
    n = dy.shape[0] * (2 if dy.dtype == torch.float16 else 1) + 2
    return dw, (dy.double().abs().t() @ w.abs()) * n * 2.0 ** -23


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_scales_that_are_no_power_of_two(zs, T, N, K, kind, aligned):
    rng = np.random.default_rng(T + N)
    dy = activations(rng, T, N).mul(1e-2).to(DT[kind]).cuda()
    x, sx = random_codes(rng, T, K).cuda(), random_scales(rng, T, pow2=False).cuda()
    bdy, bx = operands(dy, x, aligned)
    dw = torch.empty(N, K, device="cuda")
    zs.q8_weight_grad(bdy, bx, sx, dw)
    want, slack = gradient(dy, x, sx)
    slack = slack + (want.abs() + slack) * ref.U32
    off = (dw.double() - want).abs()
    assert (off <= slack).all(), f"{int((off > slack).sum())} of {off.numel()} off, at most {float((off / slack).max())}"


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_non_finite(zs, T, N, K, kind, aligned):
    """A NaN scale makes every weight's gradient NaN; an infinite or NaN dy those of its output."""
    rng = np.random.default_rng(T * 3 + N)
    dy, x, sx = activations(rng, T, N).to(DT[kind]).cuda(), random_codes(rng, T, K).cuda(), random_scales(rng, T).cuda()
    dw = torch.empty(N, K, device="cuda")
    for row in (0, T // 2, T - 1):
        s2, x2 = sx.clone(), x.clone()
        s2[row] = float("nan")
        x2[row] = 0  # as a save leaves such a row
        bdy, bx = operands(dy, x2, aligned)
        zs.q8_weight_grad(bdy, bx, s2, dw)
        assert torch.isnan(dw).all(), row
    others = torch.ones(N, dtype=torch.bool, device="cuda")
    others[[2, N - 1]] = False
    for row in (0, T - 1):
        d2, x2 = dy.clone(), x.clone()
        d2[row, 2], d2[row, N - 1] = -float("inf"), float("nan")
        x2[row] = 7
        bdy, bx = operands(d2, x2, aligned)
        zs.q8_weight_grad(bdy, bx, sx, dw)
        assert (torch.isinf(dw[2]) & (dw[2] < 0)).all() and torch.isnan(dw[N - 1]).all(), row
        assert torch.isfinite(dw[others]).all(), row


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_what_lies_between_and_behind_rows_does_not_count(zs, T, N, K, kind):
    """NaN between dy's rows and behind its last, the least code around the codes, NaN behind the scales: the same
    bits as among zeros.  The products the same, among codes of both kinds."""
    rng = np.random.default_rng(T * 5 + K)
    dy, x, sx = activations(rng, T, N).to(DT[kind]), random_codes(rng, T, K), random_scales(rng, T)
    w, sw = random_codes(rng, N, K), random_scales(rng, N)
    results = []
    for around, code in ((float("nan"), -128), (0.0, 0)):
        def inside(v, fill, more):
            wide = torch.full((v.shape[0] + 1, v.shape[1] + more), fill, dtype=v.dtype, device="cuda")
            view = wide[:-1, :v.shape[1]]
            view.copy_(v)
            return view

        bdy, bx = inside(dy, around, 8 + -N % 8), inside(x, code, 16 + -K % 16)
        bw = inside(w, code, 16 + -K % 16)
        bs = torch.full((T + 9,), around, device="cuda")
        bs[:T] = sx
        dw = torch.empty(N, K, device="cuda")
        zs.q8_weight_grad(bdy, bx, bs[:T], dw)
        y = torch.empty(T, N, device="cuda")
        zs.q8_matmul(bx, bs[:T], bw, sw.cuda(), y)
        g = inside(random_codes(np.random.default_rng(N), T, N), code, 16 + -N % 16)
        dx = torch.empty(T, K, device="cuda")
        zs.q8_matmul(g, bs[:T], bw, None, dx, trans_w=False)
        results.append((dw, y, dx))
    for a, b in zip(*results):
        assert torch.isfinite(a).all() and same_bits(a, b)


# tokens split over waves, tiles of 64 at any address, tiles of 128 and of 256
LONG = [(3001, 256, 256), (4097, 70, 90), (5000, 1500, 1530), (8000, 1100, 1300), (4097, 3001, 3203)]


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("T,N,K", LONG)
def test_long_sums_of_small_integers_are_exact(zs, T, N, K, kind, aligned):
    """Whole numbers whose partial sums stay below 2^24 add up without rounding in fp32, in any order: every token
    counts once, and all of its bits do.  fp16: odd numbers of 11 bits, whose last three lie in the second bf16 part."""
    rng = np.random.default_rng(T + K)
    top = 2 ** 24 // (T * 1) - 1
    if kind == "fp16":
        dy = torch.from_numpy(rng.integers(1, min(1024, top // 2), (T, N)) * 2 + 1)
    else:
        dy = torch.from_numpy(rng.integers(1, 128, (T, N)))
    dy = dy * torch.from_numpy(rng.choice((-1, 1), (T, N)))
    most = max(1, top // (int(dy.abs().max()) + 4))
    x = torch.from_numpy(rng.integers(-min(most, 127), min(most, 127) + 1, (T, K), dtype=np.int8))
    assert (int(dy.abs().max()) + 4) * int(x.abs().max()) * T < 2 ** 24
    held = dy.to(DT[kind])
    assert torch.equal(held.double(), dy.double())
    bdy, bx = operands(held.cuda(), x.cuda(), aligned)
    dw = torch.empty(N, K, device="cuda")
    zs.q8_weight_grad(bdy, bx, torch.ones(T, device="cuda"), dw)
    want = dy.cuda().double().t() @ x.cuda().double()
    assert torch.equal(dw.double(), want), int((dw.double() != want).sum())


@pytest.mark.parametrize("T,N,K", [(1, 64, 64), (40, 33, 65), (200, 1500, 1530)])
def test_the_smallest_values_count(zs, T, N, K):
    """Subnormal bf16 gradients (2^-133 .. 2^-126) times codes: products and sums of normal size are not lost."""
    rng = np.random.default_rng(N)
    dy = torch.from_numpy(rng.integers(1, 128, (T, N))).double() * 2.0 ** -133
    held = dy.to(torch.bfloat16)
    assert torch.equal(held.double(), dy)
    x = torch.from_numpy(rng.integers(64, 128, (T, K), dtype=np.int8))
    sx = torch.full((T,), 1024.0)
    dw = torch.empty(N, K, device="cuda")
    zs.q8_weight_grad(held.cuda(), x.cuda(), sx.cuda(), dw)
    want = dy.t() @ (x.double() * 1024)
    assert torch.equal(dw.cpu().double(), want)  # whole numbers of 2^-123 below 2^24 of them


# ------------------------------------------------------------------ graphs and repeats at tiled sizes
@pytest.mark.parametrize("T,N,K", [(200, 1504, 1536), (300, 4104, 3312), (200, 1501, 1531)])
def test_tiled_layer_replays_and_repeats(zs, T, N, K):
    rng = np.random.default_rng(20)
    a = _layer_buffers(rng, T, N, K)
    e = {k: v.clone() for k, v in a.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _layer(zs, a)
    torch.cuda.current_stream().wait_stream(side)
    _layer(zs, e)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _layer(zs, a)
    for replay in range(4):
        x, dy = activations(rng, T, K).to(torch.bfloat16).cuda(), activations(rng, T, N).to(torch.bfloat16).cuda()
        for b in (a, e):
            b["x"].copy_(x)
            b["dy"].copy_(dy)
        graph.replay()
        _layer(zs, e)
        torch.cuda.synchronize()
        for k in a:
            assert same_bits(a[k], e[k]), (replay, k)


# ------------------------------------------------------------------ the end of a type's range
TOP = 127.0 * 2.0 ** 121
ROWS = {"fp16": [65024.0, 65056.0, 65088.0, 65504.0],
        "bf16": [TOP, float(torch.finfo(torch.bfloat16).max)],
        "fp32": [TOP, TOP * (1 + 2.0 ** -23), 2.0 ** 128 * (1 - 2.0 ** -23)]}


@pytest.mark.parametrize("kind", list(ROWS))
@pytest.mark.parametrize("cols", [6, 70, 5000])
def test_rows_at_the_end_of_the_range(zs, kind, cols):
    """Which finite values load as infinities: with powers of two those from 127 * 2^9 (fp16) or 127 * 2^121 (bf16, fp32)
    on, in rows that hold more than that; with the largest-magnitude rule none."""
    tops = torch.tensor(ROWS[kind], dtype=torch.float64)
    border = 65024.0 if kind == "fp16" else TOP
    shares = torch.linspace(0.5, 1.0, cols, dtype=torch.float64)
    shares[0] = 0.0
    x = (tops[:, None] * shares).to(DT[kind])
    x[:, cols - 1] = tops.to(DT[kind])
    x[:, 1] = -x[:, cols - 1]
    x[:, 2] = torch.tensor(border).to(DT[kind])
    assert torch.isfinite(x).all()
    rows = len(tops)
    q, s = torch.empty(rows, cols, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    out = torch.empty_like(x, device="cuda")
    for rule in ("pow2", "amax"):
        zs.q8_save(x.cuda(), q, s, rule=rule)
        wq, ws = ref.save(x, rule)
        assert torch.equal(q.cpu(), wq) and same_bits(s, ws)
        zs.q8_load(q, s, out)
        got, v = out.cpu().double(), x.double()
        past = (v.abs() >= border) & (tops[:, None] > border) if rule == "pow2" else torch.zeros_like(v, dtype=torch.bool)
        assert torch.equal(torch.isinf(got), past), rule
        assert (got.sign() == v.sign())[past].all()
        # elsewhere half a step of the scale, and the output's rounding
        off = (got - v).abs()[~past]
        assert (off <= (s.cpu().double()[:, None] / 2 + v.abs() * 2 * ref.HALF_STEP[kind])[~past]).all()
    if kind == "bf16":  # the weight gradient's operand: an infinity where the load gives one
        zs.q8_save(x.cuda(), q, s, rule="pow2")
        zs.q8_load(q, s, out)
        dy = torch.full((1, 1), 0.5, dtype=torch.bfloat16, device="cuda")
        for row in range(rows):
            dw = torch.empty(1, cols, device="cuda")
            zs.q8_weight_grad(dy, q[row:row + 1], s[row:row + 1], dw)
            assert torch.equal(torch.isinf(dw[0]), torch.isinf(out[row]))
            finite = torch.isfinite(out[row])
            assert torch.equal(dw[0][finite], out[row][finite].float() * 0.5)
