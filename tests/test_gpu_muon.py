"""Orthogonalised updates against 64-bit forms (tests/muon_ref.py).

Products are tested with matrices of 0 and +-1 whose norm is a power of two and with coefficients that leave values exact
in 22 bits and sums in fp32 up to sizes that the test counts: results are then right to their one rounding, whatever the
tiles and splits.  The default coefficients are tested within a derived bound."""
import math

import numpy as np
import pytest
import torch

from tests import muon_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def zs():
    import sharded_mixed_precision_rank_amd as zs

    return zs


def gradients(seed, *shape):
    """A few strong directions over noise."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, cols = shape[-2:]
    rank = max(1, min(rows, cols) // 16)
    left = torch.randn(*shape[:-2], rows, rank, generator=g, device="cuda") * torch.exp(-4 * torch.arange(rank, device="cuda") / rank)
    right = torch.randn(*shape[:-2], rank, cols, generator=g, device="cuda")
    return 1e-3 * (left @ right / rank ** 0.5 + torch.randn(*shape, generator=g, device="cuda"))


def signs(rng, rows, cols):
    """0 and +-1 with a power of four of nonzero values."""
    n = rows * cols
    count = 4 ** int(math.log(n, 4) + 1e-9)
    v = np.zeros(n, dtype=np.float32)
    v[rng.permutation(n)[:count]] = rng.choice((-1.0, 1.0), count)
    return torch.from_numpy(v.reshape(rows, cols))


class Guarded:
    """A workspace of exactly the needed size at an odd address, filled with NaN, in front of a pattern."""

    def __init__(self, zs, rows, cols, batch=1, lead=3):
        self.n = zs.orthogonalize_workspace_bytes(rows, cols, batch)
        self.flat = torch.full((lead + self.n + 64,), 255, dtype=torch.uint8, device="cuda")
        self.flat[:lead] = 77
        self.flat[lead + self.n:] = 77
        self.lead, self.t = lead, self.flat[lead:lead + self.n]

    def untouched_outside(self):
        return bool((self.flat[:self.lead] == 77).all() and (self.flat[self.lead + self.n:] == 77).all())


def most_off(u, coefs):
    """How far one step of `signs` may be off, value by value.  In units of the norm's powers X holds +-1, S and S^2 whole
    numbers.  Below 2^22 they are held exactly, and sums below 2^24 are exact; what passes that is rounded by 2^-22 of each
    operand and 2^-24 a sum.  a X and the last sum meet in one rounding to fp32."""
    x = u.double()
    if x.shape[0] > x.shape[1]:
        x = x.t().contiguous()
    n = x.norm()
    s = x @ x.t().contiguous()
    top = s @ s if coefs[2] else s
    size = (abs(coefs[1]) * s.abs() / n ** 2 + abs(coefs[2]) * (s.abs() @ s.abs()) / n ** 4) @ (x.abs() / n)
    rounded = 0.0
    if top.abs().max() >= 2.0 ** 22:
        rounded += 2 * 2.0 ** -22  # S and what is made of it
    if (top.abs() @ x.abs()).max() >= 2.0 ** 24 or (coefs[2] and (s.abs() @ s.abs()).max() >= 2.0 ** 24):
        rounded += (2 * x.shape[0] + x.shape[1]) * 2.0 ** -24
    want = ref.steps_of(u, 1, coefs)
    return want, 2.0 ** -24 * want.abs() + rounded * (size.t() if u.shape[0] > u.shape[1] else size)


# every tile, split sums and whole ones; wide and tall; one row, one column
SHAPES = [(1, 1), (1, 300), (5, 3), (31, 33), (32, 32), (64, 64), (100, 65), (128, 128), (33, 5000), (64, 4096), (9000, 70), (200, 2000),
          (517, 1001), (1001, 517), (1024, 1024), (700, 2600), (2048, 1500), (2100, 2100)]


@pytest.mark.parametrize("coefs", [(1.0, 1.0, 0.0), (1.0, 0.0, 1.0), (2.0, -1.0, 0.0)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_exact_products(zs, rows, cols, coefs):
    u = signs(np.random.default_rng(rows + cols), rows, cols).cuda()
    want, most = most_off(u, coefs)
    ws = Guarded(zs, rows, cols)
    out = torch.full((rows, cols), 3.0, device="cuda")
    zs.orthogonalize(u, out, ws.t, steps=1, coefs=coefs)
    torch.cuda.synchronize()
    assert ((out.double() - want).abs() <= most).all()
    assert ws.untouched_outside()


@pytest.mark.parametrize("rows,cols", [(4096, 4096), (3000, 5000)])
def test_exact_products_of_large_matrices(zs, rows, cols):
    u = signs(np.random.default_rng(rows), rows, cols).cuda()
    for coefs in ((1.0, 1.0, 0.0), (1.0, 0.0, 1.0)):
        out = torch.empty(rows, cols, device="cuda")
        zs.orthogonalize(u, out, steps=1, coefs=coefs)
        want, most = most_off(u, coefs)
        assert ((out.double() - want).abs() <= most).all()


# the tiles of 128, 192 and 256 in each product, whole and with their sums split
@pytest.mark.parametrize("batch,rows,cols", [(32, 96, 9664), (32, 192, 9504), (4, 992, 5344), (1, 2848, 2848), (8, 1344, 1344), (8, 1696, 1696),
                                             (4, 160, 11424), (1, 5100, 5150)])
def test_exact_products_of_stacks(zs, batch, rows, cols):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    count = 4 ** int(math.log(rows * cols, 4) + 1e-9)
    u = torch.zeros(batch, rows * cols, device="cuda")
    for v in u:
        at = torch.randperm(rows * cols, generator=gen, device="cuda")[:count]
        v[at] = 2.0 * torch.randint(0, 2, (count,), generator=gen, device="cuda").float() - 1.0
    u = u.view(batch, rows, cols)
    ws = Guarded(zs, rows, cols, batch)
    out = torch.empty_like(u)
    for coefs in ((1.0, 1.0, 0.0), (1.0, 0.0, 1.0)):
        out.fill_(math.nan)
        zs.orthogonalize(u, out, ws.t, steps=1, coefs=coefs)
        assert torch.isfinite(out).all()
        for i in sorted({0, batch // 2, batch - 1}):
            want, most = most_off(u[i], coefs)
            assert ((out[i].double() - want).abs() <= most).all()
    assert ws.untouched_outside()


def off(got, want):
    """The error's 2-norm relative to an orthogonal matrix's."""
    return ((got.double() - want).norm() / min(want.shape) ** 0.5).item()


@pytest.mark.parametrize("out", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 77), (64, 64), (100, 65), (517, 1001), (1001, 517), (64, 4096), (1024, 1024)])
def test_default_steps(zs, rows, cols, kind, out):
    x = gradients(rows, rows, cols).to(DT[kind])
    want = ref.steps_of(x)
    got = torch.empty(rows, cols, dtype=DT[out], device="cuda")
    zs.orthogonalize(x, got)
    half = torch.finfo(DT[out]).eps / 2
    limit = ref.bound(5, rows, cols)
    assert off(got, want) <= limit + half * (want.norm().item() / min(rows, cols) ** 0.5 + limit) + 1e-7


@pytest.mark.parametrize("steps,coefs", [(1, None), (2, (3.4445, -4.7750, 2.0315)), (3, [(1.5, -0.5, 0.0)] * 3),
                                         (4, [(3.4445, -4.7750, 2.0315), (2.5, -2.5, 0.9), (1.5, -0.5, 0.0), (1.5, -0.5, 0.0)]),
                                         (12, (1.5, -0.5, 0.0))])
def test_steps_and_coefficients(zs, steps, coefs):
    x = gradients(3, 96, 160)
    want = ref.steps_of(x, steps, coefs if coefs else ref.COEFS)
    got = torch.empty_like(x)
    zs.orthogonalize(x, got, steps=steps, coefs=coefs)
    # (1.5, -0.5) lifts a perturbation by 1.5 at most, which the bound's 4 covers up to 5 steps
    assert off(got, want) <= ref.bound(min(steps, 5), 96, 160) * (1.5 ** 7 if steps > 5 else 1)


def test_results_are_orthogonal(zs):
    """With steps that converge, O O^T is the identity."""
    x = torch.randn(200, 300, device="cuda") + 2 * torch.eye(200, 300, device="cuda") * 10
    out = torch.empty_like(x)
    zs.orthogonalize(x, out, steps=20, coefs=(1.5, -0.5, 0.0))
    one = out.double() @ out.double().t().contiguous()
    assert (one - torch.eye(200, device="cuda")).abs().max().item() < 1e-5


@pytest.mark.parametrize("rows,cols", [(20, 50), (130, 70), (300, 300)])
def test_views_and_batches(zs, rows, cols):
    """A stack with gaps between rows and matrices, NaN in them, at an odd address: the gaps of the output survive, every
    matrix comes out as it does alone, in place too."""
    batch, ld, gap = 3, cols + 5, 7
    each = rows * ld + gap
    flat = torch.full((batch * each + 9,), math.nan, device="cuda")
    x = flat.as_strided((batch, rows, cols), (each, ld, 1), 1)
    x.copy_(gradients(1, batch, rows, cols))
    for kind in DT:
        oflat = (torch.arange(batch * each + 9, device="cuda") % 89).to(DT[kind])
        before = oflat.clone()
        out = oflat.as_strided((batch, rows, cols), (each, ld, 1), 1)
        ws = Guarded(zs, rows, cols, batch)
        zs.orthogonalize(x, out, ws.t)
        alone = torch.empty(batch, rows, cols, dtype=DT[kind], device="cuda")
        for i in range(batch):
            want = ref.steps_of(x[i])
            assert off(out[i], want) <= ref.bound(5, rows, cols) + torch.finfo(DT[kind]).eps
            zs.orthogonalize(x[i], alone[i])
        assert all(off(a, b.double()) <= 2 * ref.bound(5, rows, cols) + torch.finfo(DT[kind]).eps for a, b in zip(out, alone))
        got = out.clone()
        oflat.as_strided(out.shape, out.stride(), 1).copy_(before.as_strided(out.shape, out.stride(), 1))
        assert torch.equal(oflat, before) and ws.untouched_outside()
        if kind == "fp32":
            inside = flat.clone().as_strided(x.shape, x.stride(), 1)
            zs.orthogonalize(inside, inside)
            assert torch.equal(inside, got)


def test_zeros_and_non_finite_values(zs):
    """A matrix of zeros stays one; one with a NaN or an infinity is NaN throughout; the others of the batch keep their bits."""
    for rows, cols in ((40, 90), (90, 40), (1, 5), (300, 200)):
        x = gradients(2, 5, rows, cols)
        out, again = torch.empty_like(x), torch.empty_like(x)
        zs.orthogonalize(x, out)
        x[1] = 0
        x[2, rows // 2, 0] = math.nan
        x[3, 0, cols - 1] = -math.inf
        zs.orthogonalize(x, again)
        assert torch.equal(again[0], out[0]) and torch.equal(again[4], out[4])
        assert (again[1] == 0).all()
        assert torch.isnan(again[2]).all() and torch.isnan(again[3]).all()


def test_the_ends_of_the_range(zs):
    """Squares are summed in 64 bits: the scale of a matrix does not matter, down to subnormals and up to fp32's end."""
    x = gradients(7, 48, 80)
    x = torch.where(x == 0, x, x / 2.0 ** torch.floor(torch.log2(x.abs().max())))
    out, again = torch.empty_like(x), torch.empty_like(x)
    zs.orthogonalize(x, out)
    for e in (-100, 100, 126):
        zs.orthogonalize(x * 2.0 ** e, again)
        assert torch.equal(out, again), e
    zs.orthogonalize(torch.full((8, 8), 2.0 ** -149, device="cuda"), again[:8, :8])
    assert off(again[:8, :8].cpu(), ref.steps_of(torch.ones(8, 8))) <= ref.bound(5, 8, 8)


def folded(mean_of, hp, master, momentum, param, zs, coefs=None):
    """The step in its own order of fp32 operations, with the library's own steps in the middle."""
    f32 = lambda v: torch.tensor(v, dtype=torch.float64).float().item()  # noqa: E731
    mu, dk, ss = f32(hp["momentum"]), f32(1 - hp["lr"] * hp["weight_decay"]), f32(hp["lr"] * hp["scale"])
    g = mean_of
    m1 = momentum * mu + g
    u = g + m1 * mu if hp["nesterov"] else m1
    o = torch.empty_like(u)
    zs.orthogonalize(u.contiguous(), o, steps=hp["steps"], coefs=coefs)
    p1 = master * dk - o * ss
    return p1, m1, p1.bfloat16()


@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("shape,N", [((1, 1), 1), ((3, 5), 2), ((64, 64), 3), ((130, 70), 8), ((70, 130), 5), ((4, 96, 160), 4),
                                     ((517, 1001), 64), ((2, 300, 90), 256), ((1024, 1024), 2)])
def test_reduce_muon(zs, shape, N, nesterov):
    """Mean, momentum and update bit for bit, around the library's own Newton-Schulz steps."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    base = gradients(N, *shape)
    grads = [(base + 1e-3 * torch.randn(*shape, generator=gen, device="cuda")).bfloat16() for _ in range(N)]
    master = 0.02 * torch.randn(*shape, generator=gen, device="cuda")
    momentum = gradients(N + 1, *shape)
    param = torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")
    s = grads[0].float()
    for g in grads[1:]:
        s = s + g.float()
    # the mean as the flat step has it: a correctly rounded quotient (torch's own may be a product with the reciprocal)
    mean = torch.from_numpy(s.cpu().numpy() / np.float32(N)).cuda()
    hp = dict(lr=0.02, momentum=0.95, weight_decay=0.1, scale=0.7, nesterov=nesterov, steps=3)
    want = folded(mean, hp, master, momentum, param, zs)
    ws = Guarded(zs, shape[-2], shape[-1], shape[0] if len(shape) == 3 else 1)
    zs.reduce_muon(grads, master, momentum, param, zs.MuonHP(**hp), ws.t)
    torch.cuda.synchronize()
    for got, w in zip((master, momentum, param), want):
        assert torch.equal(got, w)
    assert ws.untouched_outside()


def test_reduce_muon_at_odd_addresses(zs):
    """Arrays that start anywhere inside a flat shard: the neighbours survive and the values are the aligned ones."""
    rows, cols, n = 45, 67, 45 * 67
    make = lambda dtype, lead: torch.arange(n + 40, device="cuda").remainder(50).to(dtype)[lead:lead + n].view(rows, cols)  # noqa: E731
    results = []
    for lead in (8, 3):
        gen = torch.Generator(device="cuda").manual_seed(4)
        arrays = [make(torch.float32, lead), make(torch.float32, lead + 2), make(torch.bfloat16, lead + 4)]
        grads = [make(torch.bfloat16, lead + 2 * r) for r in range(3)]
        for t in arrays + grads:
            t.copy_(torch.randn(rows, cols, generator=gen, device="cuda"))
        whole = [t._base.clone() for t in arrays]
        zs.reduce_muon(grads, *arrays, dict(lr=0.1, scale=0.5))
        torch.cuda.synchronize()
        for t, w in zip(arrays, whole):
            k = t.storage_offset()
            assert torch.equal(t._base[:k], w[:k]) and torch.equal(t._base[k + n:], w[k + n:])
        results.append([t.clone() for t in arrays])
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("rows,cols", [(96, 128), (128, 96), (97, 128), (128, 97), (128, 128), (65, 33), (33, 65), (128, 1)])
def test_matrices_of_one_workgroup(zs, rows, cols):
    """Both sides at most 128, by either count of waves: products to their one rounding, default steps, the update."""
    for coefs in ((1.0, 1.0, 0.0), (1.0, 0.0, 1.0)):
        test_exact_products(zs, rows, cols, coefs)
    test_default_steps(zs, rows, cols, "bf16", "fp32")
    test_reduce_muon(zs, (3, rows, cols), 2, True)


@pytest.mark.parametrize("shape", [(96, 200), (2, 64, 64), (700, 520)])
def test_graph_replays_and_streams(zs, shape):
    """Captured with its own workspace, replayed between eager steps on another: both walk the same path of states."""
    rows, cols, batch = shape[-2], shape[-1], shape[0] if len(shape) == 3 else 1
    need = zs.orthogonalize_workspace_bytes(rows, cols, batch)
    spaces = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    grads = [torch.zeros(*shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    state = [[0.02 * torch.ones(*shape, device="cuda"), torch.zeros(*shape, device="cuda"),
              torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")] for _ in range(2)]
    hp = zs.MuonHP(lr=0.05, weight_decay=0.1, scale=0.3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        keep = [t.clone() for t in state[0]]
        zs.reduce_muon(grads, *state[0], hp, spaces[0])
        for t, k in zip(state[0], keep):
            t.copy_(k)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        zs.reduce_muon(grads, *state[0], hp, spaces[0])
    for k in range(4):
        for r, g in enumerate(grads):
            g.copy_(gradients(10 * k + r, *shape))
        # the replay and, beside it on another stream, the eager step with a workspace of its own
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            zs.reduce_muon(grads, *state[1], hp, spaces[1])
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(*state))


def test_other_stream_with_a_workspace_of_the_call(zs):
    """workspace=None on a stream that is not the current one: the allocator does not hand it out before the call is done."""
    x = gradients(5, 300, 400)
    want = torch.empty_like(x)
    zs.orthogonalize(x, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(6):
        out = torch.empty_like(x)
        zs.orthogonalize(x, out, stream=side)
        junk = [torch.full((zs.orthogonalize_workspace_bytes(300, 400),), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
        outs.append((out, junk))
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o, _ in outs)


@pytest.mark.parametrize("handle", (False, True))
def test_other_stream_beside_work_on_memory_just_freed(zs, handle):
    """workspace=None on a stream that does not wait for the current one, whose queue still writes a block that was freed
    there: the call's workspace is not that block."""
    x = gradients(6, 300, 400)
    want, out = torch.empty_like(x), torch.empty_like(x)
    zs.orthogonalize(x, want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    block = torch.empty(zs.orthogonalize_workspace_bytes(300, 400), dtype=torch.uint8, device="cuda")
    for _ in range(400):
        block.fill_(255)
    del block
    zs.orthogonalize(x, out, stream=side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_a_layers_training_steps(zs):
    """The gated block with the step of its weights, as a training loop has them: two replicas' forward and backward passes,
    their weight gradients as chunks, both weights (a stack of two) reduced, orthogonalised and updated, and the working
    copy back in the forward pass.  Against the same loop in 64 bits, from the same working copy each time."""
    T, N, K, R = 160, 136, 200, 2
    gen = torch.Generator(device="cuda").manual_seed(11)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    master = 0.05 * rand(2, N, K)
    momentum = torch.zeros_like(master)
    param = master.bfloat16()
    m64, v64 = master.double(), momentum.double()
    hp = dict(lr=0.02, momentum=0.9, weight_decay=0.1, scale=0.2 * max(N, K) ** 0.5, nesterov=True, steps=5)
    for _ in range(3):
        chunks, exact = [], []
        for _ in range(R):
            x, dh = rand(T, K).bfloat16(), rand(T, N).bfloat16()
            h, gate, up, dg, du = (torch.empty(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(5))
            dw = torch.empty(2, N, K, dtype=torch.bfloat16, device="cuda")
            zs.glu_forward(x, param[0], param[1], h, gate=gate, up=up)
            zs.glu_backward(dh, gate, up, dg, du)
            zs.glu_weight_grad(dg, du, x, dw[0], dw[1])
            chunks.append(dw)
            w = param.double()
            g64, u64 = x.double() @ w[0].t(), x.double() @ w[1].t()
            s = torch.sigmoid(g64)
            d = (dh.double() * u64 * (s + g64 * s * (1 - s)), dh.double() * g64 * s)
            exact.append(torch.stack([v.t() @ x.double() for v in d]))
            # three roundings of gate and up, of dgate and dup, and of the result
            assert ((dw.double() - exact[-1]).norm() / exact[-1].norm()).item() <= 3 * 2.0 ** -8
        zs.reduce_muon(chunks, master, momentum, param, hp)
        mean = sum(c.double() for c in chunks) / R
        v64 = hp["momentum"] * v64 + mean
        o = torch.stack([ref.steps_of(u) for u in mean + hp["momentum"] * v64])
        m64 = m64 * (1 - hp["lr"] * hp["weight_decay"]) - hp["lr"] * hp["scale"] * o
        # the update's own error, its share of the master's roundings of 2^-24 each, three steps
        off_by = (master.double() - m64).norm().item()
        most = 3 * (hp["lr"] * hp["scale"] * ref.bound(5, N, K) * (2 * min(N, K)) ** 0.5 + 2.0 ** -22 * m64.norm().item())
        assert off_by <= most
        assert torch.equal(param, master.bfloat16())


@pytest.mark.parametrize("batch,rows,cols", [(5, 40, 700), (3, 9000, 20), (7, 129, 8), (6, 90, 140), (2, 300, 1100)])
def test_stacks_in_workspaces_of_the_exact_size(zs, batch, rows, cols):
    """Every matrix of a stack within the bound, and the same bits beside one of NaN; nothing outside the workspace is written."""
    x = gradients(batch, batch, rows, cols)
    ws = Guarded(zs, rows, cols, batch)
    out, again = torch.empty_like(x), torch.empty_like(x)
    zs.orthogonalize(x, out, ws.t)
    for i in range(batch):
        assert off(out[i], ref.steps_of(x[i])) <= ref.bound(5, rows, cols)
    x[1] = math.nan
    zs.orthogonalize(x, again, ws.t)
    torch.cuda.synchronize()
    keep = [i for i in range(batch) if i != 1]
    assert torch.equal(again[keep], out[keep]) and torch.isnan(again[1]).all()
    assert ws.untouched_outside()
