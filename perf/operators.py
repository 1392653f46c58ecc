"""The measured cases of the 8-bit training operators: checkpoints in 8 bits (save, load), the 8-bit matrix product
with a scale for each token and channel (forward and input gradient) and the weight gradient that reads a checkpoint.

`own` False: their plain forms in elementary torch operations.  `own` True: the calls a user makes of the library."""
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
# the largest listed product; drawn ones cost no more
MOST = 8192 * 11008 * 4096
MOST_VALUES = 16384 * 11008


def listed():
    return [
        # a decoder's single new token, hidden size 4096: latency
        {"name": "checkpoint one token", "kind": "checkpoint", "rows": 1, "cols": 4096, "type": "bf16", "rule": "pow2", "gap": 0},
        # fp32 activations of a ragged batch, an odd width, cut out of a wider buffer
        {"name": "checkpoint odd view", "kind": "checkpoint", "rows": 1237, "cols": 4099, "type": "fp32", "rule": "amax", "gap": 13},
        # the feed-forward activations of a long training batch
        {"name": "checkpoint long batch", "kind": "checkpoint", "rows": 16384, "cols": 11008, "type": "bf16", "rule": "pow2", "gap": 0},
        # a single token through the wide feed-forward layer: the weight's bytes
        {"name": "product one token", "kind": "product", "T": 1, "N": 11008, "K": 4096, "type": "bf16"},
        # a prompt of a few hundred tokens through the layer that comes back to the hidden size
        {"name": "product prompt", "kind": "product", "T": 333, "N": 4096, "K": 11008, "type": "fp16"},
        # an odd slice of a vocabulary, logits kept in 32 bits, an inner size that ends inside a 16-byte piece
        {"name": "product odd", "kind": "product", "T": 1000, "N": 5003, "K": 1000, "type": "fp32"},
        # a training batch
        {"name": "product batch", "kind": "product", "T": 8192, "N": 11008, "K": 4096, "type": "bf16"},
        # a short fp16 sequence back through an attention projection
        {"name": "input gradient short", "kind": "input_grad", "T": 61, "N": 4096, "K": 4096, "type": "fp16"},
        # a training batch back through the feed-forward layer
        {"name": "input gradient batch", "kind": "input_grad", "T": 8192, "N": 11008, "K": 4096, "type": "bf16"},
        # one of eight shards of the feed-forward weight, added to the fp32 sums of earlier micro-batches
        {"name": "weight gradient shard", "kind": "weight_grad", "T": 1025, "N": 1376, "K": 4096, "type": "bf16", "out": "fp32", "add": True},
        # a few tokens of an fp16 model, nothing a multiple of anything
        {"name": "weight gradient odd", "kind": "weight_grad", "T": 77, "N": 1001, "K": 517, "type": "fp16", "out": "fp16", "add": False},
        # a training batch, written as the bf16 chunk that the reduce reads
        {"name": "weight gradient batch", "kind": "weight_grad", "T": 8192, "N": 11008, "K": 4096, "type": "bf16", "out": "bf16", "add": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def _width(rng):
    """A feature size: most are multiples of 128 or 16, some of nothing."""
    n = _log(rng, 64, 11008)
    step = rng.choice((128, 128, 16, 1))
    return max(step, n // step * step) if n >= step else n


def draw(rng):
    kind = rng.choice(("checkpoint", "product", "product", "input_grad", "weight_grad", "weight_grad"))
    t = _log(rng, 1, 16384)
    if kind == "checkpoint":
        cols = _width(rng)
        return {"kind": kind, "rows": min(t, MOST_VALUES // cols), "cols": cols, "type": rng.choice(("bf16", "bf16", "fp16", "fp32")),
                "rule": rng.choice(("pow2", "amax")), "gap": rng.choice((0, 0, rng.randrange(1, 65)))}
    n, k = _width(rng), _width(rng)
    c = {"kind": kind, "T": max(1, min(t, MOST // (n * k))), "N": n, "K": k, "type": rng.choice(("bf16", "bf16", "fp16", "fp32"))}
    if kind != "product":
        c["type"] = rng.choice(("bf16", "bf16", "fp16"))
    if kind == "weight_grad":
        c["out"] = rng.choice((c["type"], "fp32"))
        c["add"] = rng.random() < 0.5
    return c


def _activations(g, rows, cols):
    """Activations as norms leave them: a few wide channels, tokens of different size, a padding token here and there."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    wide = torch.rand(cols, generator=g, device="cuda") < 0.01
    x *= torch.where(wide, 6.0, 1.0)
    size = torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    size[torch.rand(rows, 1, generator=g, device="cuda") < 0.02] = 0.0
    return x * size


def _rows16(rows, cols, dtype):
    """Rows that start on 16-byte boundaries."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.zeros(rows, -(-cols // per) * per, dtype=dtype, device="cuda")[:, :cols]


def _coded(values, rule):
    """Codes (int8 rows on 16-byte boundaries) and scales of given values, as a user's program has them from earlier calls."""
    codes, scales = _plain_save(values, rule)
    q = _rows16(*values.shape, torch.int8)
    q.copy_(codes)
    return q, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = case["kind"]
    if kind == "checkpoint":
        rows, cols, dtype = case["rows"], case["cols"], TYPES[case["type"]]
        x = torch.empty(rows, cols + case["gap"], dtype=dtype, device="cuda")[:, :cols]
        x.copy_(_activations(g, rows, cols))
        return {"case": case, "x": x, "codes": _rows16(rows, cols, torch.int8),
                "scales": torch.empty(rows, device="cuda"), "out": torch.empty(rows, cols, dtype=dtype, device="cuda")}
    T, N, K, dtype = case["T"], case["N"], case["K"], TYPES[case["type"]]
    if kind == "weight_grad":
        dy = _rows16(T, N, dtype)
        dy.copy_(1e-3 * _activations(g, T, N))
        x, sx = _coded(_activations(g, T, K).to(dtype), "pow2")
        out = TYPES[case["out"]]
        add = (1e-2 * torch.randn(N, K, generator=g, device="cuda")).to(out) if case["add"] else None
        return {"case": case, "dy": dy, "x": x, "sx": sx, "add": add, "dw": torch.empty(N, K, dtype=out, device="cuda")}
    w, sw = _coded(0.02 * torch.randn(N, K, generator=g, device="cuda"), "amax")
    if kind == "product":
        x, sx = _coded(_activations(g, T, K), "pow2")
        return {"case": case, "x": x, "sx": sx, "w": w, "sw": sw, "y": torch.empty(T, N, dtype=dtype, device="cuda")}
    dy = _rows16(T, N, dtype)
    dy.copy_(1e-3 * _activations(g, T, N))
    return {"case": case, "dy": dy, "w": w, "sw": sw, "g": _rows16(T, N, torch.int8),
            "sg": torch.empty(T, device="cuda"), "dx": torch.empty(T, K, dtype=dtype, device="cuda")}


def _plain_save(v, rule):
    """Codes and scales of the rows of v: values next to a border between two codes need the quotient in 64 bits."""
    v = v.float()
    top = v.abs().amax(dim=1)
    if rule == "pow2":
        m, e = torch.frexp(top.clamp(min=127.0 * 2.0 ** -126))
        e = torch.where(m > 127.0 / 128.0, e - 6, e - 7).clamp(max=127)
        s = ((e + 127) << 23).to(torch.int32).view(torch.float32)
    else:
        s = (top.double() / torch.full_like(top, 127.0, dtype=torch.float64)).float()
    s = s.clamp(min=2.0 ** -126)
    s = torch.where(torch.isfinite(top), s, torch.nan)
    q = torch.round(v.double() / s.double()[:, None])
    return torch.where(torch.isnan(s)[:, None], 0.0, q).to(torch.int8), s


def _plain(state):
    case = state["case"]
    kind = case["kind"]
    if kind == "checkpoint":
        q, s = _plain_save(state["x"], case["rule"])
        return {"restored": (q.float() * s[:, None]).to(TYPES[case["type"]]), "scales": s}
    if kind == "product":
        y = state["x"].float() @ state["w"].float().t()
        return {"y": (y * state["sx"][:, None] * state["sw"]).to(TYPES[case["type"]])}
    if kind == "input_grad":
        g, sg = _plain_save(state["dy"].float() * state["sw"], "amax")
        return {"dx": ((g.float() @ state["w"].float()) * sg[:, None]).to(TYPES[case["type"]])}
    dw = state["dy"].float().t() @ (state["x"].float() * state["sx"][:, None])
    if state["add"] is not None:
        dw = state["add"].float() + dw
    return {"dw": dw.to(TYPES[case["out"]])}


def _own(state):
    import sharded_mixed_precision_rank_amd as zs

    case = state["case"]
    kind = case["kind"]
    if kind == "checkpoint":
        zs.q8_save(state["x"], state["codes"], state["scales"], rule=case["rule"])
        zs.q8_load(state["codes"], state["scales"], state["out"])
        return {"restored": state["out"], "scales": state["scales"]}
    if kind == "product":
        zs.q8_matmul(state["x"], state["sx"], state["w"], state["sw"], state["y"])
        return {"y": state["y"]}
    if kind == "input_grad":
        zs.q8_save(state["dy"], state["g"], state["sg"], col_scale=state["sw"], rule="amax")
        zs.q8_matmul(state["g"], state["sg"], state["w"], None, state["dx"], trans_w=False)
        return {"dx": state["dx"]}
    zs.q8_weight_grad(state["dy"], state["x"], state["sx"], state["dw"], add=state["add"])
    return {"dw": state["dw"]}


def run(state):
    if own:
        return _own(state)
    return _plain(state)


def work(case):
    kind = case["kind"]
    if kind == "checkpoint":
        # values read, codes written and read again, values written; a maximum, a quotient and a product for each
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 * SIZE[case["type"]] + 2) + 8 * case["rows"], "flops": 3 * n}
    T, N, K = case["T"], case["N"], case["K"]
    if kind == "product":
        moved = T * K + N * K + 4 * (T + N) + T * N * SIZE[case["type"]]
    elif kind == "input_grad":
        # the gradient's codes are there in whole before the product begins: written and read
        moved = T * N * (SIZE[case["type"]] + 2) + 8 * T + 4 * N + N * K + T * K * SIZE[case["type"]]
    else:
        moved = T * N * SIZE[case["type"]] + T * K + 4 * T + N * K * SIZE[case["out"]] * (2 if case["add"] else 1)
    return {"bytes": moved, "flops": 2 * T * N * K}


def _exact_codes(v, rule):
    """(codes, scales) in 64 bits from the definition: the least scale that keeps a row's codes within 127."""
    top = v.double().abs().max(dim=1).values
    unit = top / torch.tensor(127.0, dtype=torch.float64, device=top.device)
    if rule == "pow2":
        unit = unit.clamp(min=2.0 ** -126)
        below = (unit.view(torch.int64) >> 52 << 52).view(torch.float64)  # the power of two at or below
        scale = torch.where(below < unit, 2 * below, below)
    else:
        scale = unit.clamp(min=2.0 ** -126).float().double()  # the 32 bits that it is kept in
    near = torch.floor(v.double() / scale[:, None] + 0.5)
    tie = (v.double() / scale[:, None] + 0.5 == near) & (torch.remainder(near, 2) != 0)
    return near - tie.double(), scale


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "checkpoint":
        q, scale = _exact_codes(s["x"], case["rule"])
        return {"restored": q * scale[:, None], "scales": scale}
    if kind == "product":
        return {"y": torch.matmul(s["x"].double() * s["sx"].double()[:, None], (s["w"].double() * s["sw"].double()[:, None]).t())}
    if kind == "input_grad":
        q, scale = _exact_codes(s["dy"].float() * s["sw"], "amax")  # the folded gradient is held in 32 bits
        return {"dx": torch.matmul(q * scale[:, None], s["w"].double())}
    dw = torch.matmul((s["dy"].double() * s["sx"].double()[:, None]).t(), s["x"].double())
    return {"dw": dw if s["add"] is None else dw + s["add"].double()}
