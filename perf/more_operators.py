"""The measured cases of two sets of training operators: the gated feed-forward block (both projections, the activation
and the product, with its backward pass), and the step of a weight matrix by an orthogonalised update (Newton-Schulz
products, alone and within the reduce-and-update step of a shard).

`own` False: their plain forms in elementary torch operations.  `own` True: the calls a user makes of the library."""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
COEFS = (3.4445, -4.7750, 2.0315)
STEPS = 5
# the largest listed product and matrix; drawn ones cost no more
MOST = 8192 * 11008 * 4096
MOST_MATRIX = 4096 * 4096 * (3 * 11008 + 4096)


def listed():
    return [
        # a decoder's single new token: the bytes of both weights
        {"name": "gate one token", "kind": "forward", "T": 1, "N": 11008, "K": 4096, "type": "bf16", "act": "silu", "save": False, "packed": True},
        # a prompt of a few hundred tokens, nothing kept
        {"name": "gate prompt", "kind": "forward", "T": 333, "N": 11008, "K": 4096, "type": "fp16", "act": "silu", "save": False, "packed": True},
        # a tensor-parallel slice of odd width, gate and up kept for the backward pass
        {"name": "gate odd", "kind": "forward", "T": 1000, "N": 1371, "K": 1000, "type": "bf16", "act": "gelu_tanh", "save": True, "packed": True},
        # a training batch
        {"name": "gate batch", "kind": "forward", "T": 8192, "N": 11008, "K": 4096, "type": "bf16", "act": "silu", "save": True, "packed": True},
        # a short fp16 sequence back through the block: gradients of gate, up, input and both weights
        {"name": "gate back short", "kind": "backward", "T": 61, "N": 4096, "K": 4096, "type": "fp16", "act": "gelu", "packed": True},
        # a training batch back through the block
        {"name": "gate back batch", "kind": "backward", "T": 8192, "N": 11008, "K": 4096, "type": "bf16", "act": "silu", "packed": True},
        # one of eight shards of both weights, added to the fp32 sums of earlier micro-batches
        {"name": "gate weights shard", "kind": "weight_grad", "T": 1025, "N": 1376, "K": 4096, "type": "bf16", "out": "fp32", "add": True, "packed": True},
        # a layer's heads, each a matrix of its own
        {"name": "orthogonalise heads", "kind": "orthogonalise", "batch": 32, "rows": 128, "cols": 128, "type": "fp32", "out": "bf16"},
        # a tall matrix, nothing a multiple of anything
        {"name": "orthogonalise odd", "kind": "orthogonalise", "batch": 1, "rows": 1001, "cols": 517, "type": "bf16", "out": "fp32"},
        # an attention projection
        {"name": "orthogonalise square", "kind": "orthogonalise", "batch": 1, "rows": 4096, "cols": 4096, "type": "fp32", "out": "bf16"},
        # a small model's stacked projections, two replicas
        {"name": "muon small", "kind": "muon", "batch": 4, "rows": 512, "cols": 512, "replicas": 2, "nesterov": False},
        # a feed-forward weight, eight replicas
        {"name": "muon feed-forward", "kind": "muon", "batch": 1, "rows": 11008, "cols": 4096, "replicas": 8, "nesterov": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def _width(rng, lo=64):
    """A feature size: most are multiples of 128 or 16, some of nothing."""
    n = _log(rng, lo, 11008)
    step = rng.choice((128, 128, 16, 1))
    return max(step, n // step * step) if n >= step else n


def draw(rng):
    kind = rng.choice(("forward", "forward", "backward", "weight_grad", "orthogonalise", "muon"))
    if kind in ("orthogonalise", "muon"):
        rows, cols = _width(rng), _width(rng)
        small, large = min(rows, cols), max(rows, cols)
        one = small * small * (3 * large + small)
        if one > MOST_MATRIX:  # the long side shrinks until it costs no more
            large = max(small, (MOST_MATRIX // (small * small) - small) // 3)
            if small * small * (3 * large + small) > MOST_MATRIX:
                small = large = 4096
            rows, cols = (small, large) if rows <= cols else (large, small)
            one = small * small * (3 * large + small)
        batch = max(1, min(rng.choice((1, 1, _log(rng, 2, 64))), MOST_MATRIX // one, (11008 * 4096) // (rows * cols)))
        c = {"kind": kind, "batch": batch, "rows": rows, "cols": cols}
        if kind == "muon":
            return {**c, "replicas": _log(rng, 1, 16), "nesterov": rng.random() < 0.5}
        return {**c, "type": rng.choice(("bf16", "fp16", "fp32")), "out": rng.choice(("bf16", "fp16", "fp32"))}
    n, k = _width(rng, 256), _width(rng, 256)
    t = _log(rng, 1 if kind == "forward" else 16, 16384)
    c = {"kind": kind, "T": min(t, MOST // (n * k)), "N": n, "K": k, "type": rng.choice(("bf16", "bf16", "fp16")),
         "packed": rng.random() < 0.25}
    if kind == "weight_grad":
        return {**c, "out": rng.choice((c["type"], "fp32")), "add": rng.random() < 0.5}
    c["act"] = rng.choice(("silu", "silu", "gelu", "gelu_tanh", "relu"))
    if kind == "forward":
        c["save"] = rng.random() < 0.5
    return c


def _activations(g, rows, cols):
    """Activations as norms leave them: a few wide channels, tokens of different size, a padding token here and there."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    wide = torch.rand(cols, generator=g, device="cuda") < 0.01
    x *= torch.where(wide, 3.0, 1.0)
    size = torch.exp(0.3 * torch.randn(rows, 1, generator=g, device="cuda"))
    if rows > 16:
        size[torch.rand(rows, 1, generator=g, device="cuda") < 0.02] = 0.0
    return x * size


def _new(rows, cols, dtype, packed):
    """Rows back to back, or starting on 16-byte boundaries."""
    per = 1 if packed else 16 // torch.empty((), dtype=dtype).element_size()
    return torch.zeros(rows, -(-cols // per) * per, dtype=dtype, device="cuda")[:, :cols]


def _gradients(g, batch, rows, cols):
    """A weight's gradients: a few strong directions, whose sizes fall off, over noise."""
    rank = max(1, min(rows, cols) // 16)
    fall = torch.exp(-4.0 * torch.arange(rank, device="cuda") / rank)
    left = torch.randn(batch, rows, rank, generator=g, device="cuda") * fall
    right = torch.randn(batch, rank, cols, generator=g, device="cuda")
    return 1e-3 * (left @ right / math.sqrt(rank) + torch.randn(batch, rows, cols, generator=g, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = case["kind"]
    if kind == "orthogonalise":
        b, m, n = case["batch"], case["rows"], case["cols"]
        return {"case": case, "x": _gradients(g, b, m, n).to(TYPES[case["type"]]),
                "out": torch.empty(b, m, n, dtype=TYPES[case["out"]], device="cuda")}
    if kind == "muon":
        b, m, n, r = case["batch"], case["rows"], case["cols"], case["replicas"]
        mean = _gradients(g, b, m, n)
        return {"case": case,
                "grads": [(mean + 1e-3 * torch.randn(b, m, n, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(r)],
                "master": 0.02 * torch.randn(b, m, n, generator=g, device="cuda"),
                "momentum": 8.0 * (mean + 1e-4 * torch.randn(b, m, n, generator=g, device="cuda")),
                "param": torch.zeros(b, m, n, dtype=torch.bfloat16, device="cuda"),
                "hp": {"lr": 2e-4, "momentum": 0.95, "weight_decay": 0.1, "nesterov": case["nesterov"],
                       "scale": 0.2 * math.sqrt(max(m, n)), "steps": STEPS}}
    T, N, K, dtype, packed = case["T"], case["N"], case["K"], TYPES[case["type"]], case["packed"]

    def matrix(rows, cols, values):
        t = _new(rows, cols, dtype, packed)
        t.copy_(values)
        return t

    state = {"case": case}
    if kind != "weight_grad":
        for name in ("w_gate", "w_up"):
            state[name] = matrix(N, K, 0.02 * torch.randn(N, K, generator=g, device="cuda"))
    state["x"] = matrix(T, K, _activations(g, T, K))
    if kind == "forward":
        state["h"] = _new(T, N, dtype, packed)
        if case["save"]:
            state["gate"], state["up"] = _new(T, N, dtype, packed), _new(T, N, dtype, packed)
        return state
    size = 0.02 * math.sqrt(K)
    state["dgate"], state["dup"] = _new(T, N, dtype, packed), _new(T, N, dtype, packed)
    if kind == "weight_grad":
        state["dgate"].copy_(1e-2 * _activations(g, T, N))
        state["dup"].copy_(1e-2 * _activations(g, T, N))
        out = TYPES[case["out"]]
        for name in ("gate", "up"):
            state["dw_" + name] = torch.empty(N, K, dtype=out, device="cuda")
            state["add_" + name] = torch.randn(N, K, generator=g, device="cuda").to(out) if case["add"] else None
        return state
    state["gate"] = matrix(T, N, size * _activations(g, T, N))
    state["up"] = matrix(T, N, size * _activations(g, T, N))
    state["dh"] = matrix(T, N, 1e-2 * _activations(g, T, N))
    state["dx"] = torch.empty(T, K, dtype=dtype, device="cuda")
    for name in ("gate", "up"):
        state["dw_" + name] = torch.empty(N, K, dtype=dtype, device="cuda")
    return state


def _act(v, name):
    """The activation of fp32 values, and its derivative."""
    if name == "relu":
        on = (v > 0).float()
        return v * on, on
    if name == "gelu":
        # the distribution function where it is small is a difference of numbers near one: in 64 bits
        w = v.double()
        below = (0.5 * torch.special.erfc(w * -math.sqrt(0.5))).float()
        return v * below, below + v * torch.exp(-0.5 * v * v) * (1.0 / math.sqrt(2.0 * math.pi))
    if name == "silu":
        z, dz = v, torch.ones_like(v)
    else:  # gelu_tanh: v times the logistic function of 2 sqrt(2 / pi) (v + 0.044715 v^3)
        c = 2.0 * math.sqrt(2.0 / math.pi)
        z, dz = c * (v + 0.044715 * v * v * v), c * (1.0 + 3.0 * 0.044715 * v * v)
    s = 1.0 / (1.0 + torch.exp(-z))
    return v * s, s + v * s * (1.0 - s) * dz


def _plain_orthogonalise(u, wide=False):
    """The Newton-Schulz steps on matrices (batch, rows, cols), in 32 bits; in 64 where a 32-bit result is kept."""
    x = u.double() if wide else u.float()
    norm = x.double().square().sum(dim=(1, 2), keepdim=True).sqrt()
    x = (x.double() / norm.clamp(min=1e-300)).to(x.dtype)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    a, b, c = COEFS
    for _ in range(STEPS):
        s = x @ x.transpose(1, 2).contiguous()
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.transpose(1, 2).contiguous() if tall else x


def _plain(state):
    case = state["case"]
    kind = case["kind"]
    if kind == "orthogonalise":
        return {"out": _plain_orthogonalise(state["x"], case["out"] == "fp32").to(TYPES[case["out"]])}
    if kind == "muon":
        hp = state["hp"]
        mean = torch.stack([g.float() for g in state["grads"]]).sum(dim=0) / len(state["grads"])
        state["momentum"].copy_(hp["momentum"] * state["momentum"] + mean)
        u = mean + hp["momentum"] * state["momentum"] if hp["nesterov"] else state["momentum"]
        o = _plain_orthogonalise(u)
        state["master"].copy_((1.0 - hp["lr"] * hp["weight_decay"]) * state["master"] - hp["lr"] * hp["scale"] * o)
        state["param"].copy_(state["master"])
        return {"master": state["master"], "momentum": state["momentum"], "param": state["param"]}
    dtype = TYPES[case["type"]]
    if kind == "forward":
        x = state["x"].float()
        gate, up = x @ state["w_gate"].float().t(), x @ state["w_up"].float().t()
        out = {"h": (_act(gate, case["act"])[0] * up).to(dtype)}
        if case["save"]:
            out.update(gate=gate.to(dtype), up=up.to(dtype))
        return out
    x = state["x"].float()
    if kind == "weight_grad":
        out = {}
        for name in ("gate", "up"):
            dw = state["d" + name].float().t() @ x
            if case["add"]:
                dw = state["add_" + name].float() + dw
            out["dw_" + name] = dw.to(TYPES[case["out"]])
        return out
    gate, up, dh = state["gate"].float(), state["up"].float(), state["dh"].float()
    value, slope = _act(gate, case["act"])
    dgate, dup = dh * up * slope, dh * value
    dx = dgate @ state["w_gate"].float() + dup @ state["w_up"].float()
    return {"dgate": dgate.to(dtype), "dup": dup.to(dtype), "dx": dx.to(dtype), "dw_gate": (dgate.t() @ x).to(dtype),
            "dw_up": (dup.t() @ x).to(dtype)}


def _own(state):
    import sharded_mixed_precision_rank_amd as zs

    case = state["case"]
    kind = case["kind"]
    if kind == "orthogonalise":
        zs.orthogonalize(state["x"], state["out"], steps=STEPS, coefs=COEFS)
        return {"out": state["out"]}
    if kind == "muon":
        zs.reduce_muon(state["grads"], state["master"], state["momentum"], state["param"], zs.MuonHP(**state["hp"], coefs=COEFS))
        return {"master": state["master"], "momentum": state["momentum"], "param": state["param"]}
    if kind == "forward":
        zs.glu_forward(state["x"], state["w_gate"], state["w_up"], state["h"], gate=state.get("gate"), up=state.get("up"), act=case["act"])
        return {k: state[k] for k in ("h", "gate", "up") if k in state}
    if kind == "backward":
        zs.glu_backward(state["dh"], state["gate"], state["up"], state["dgate"], state["dup"], act=case["act"])
        zs.glu_input_grad(state["dgate"], state["dup"], state["w_gate"], state["w_up"], state["dx"])
    zs.glu_weight_grad(state["dgate"], state["dup"], state["x"], state["dw_gate"], state["dw_up"],
                       add_gate=state.get("add_gate"), add_up=state.get("add_up"))
    names = ("dgate", "dup", "dx", "dw_gate", "dw_up") if kind == "backward" else ("dw_gate", "dw_up")
    return {k: state[k] for k in names}


def run(state):
    if own:
        return _own(state)
    return _plain(state)


def work(case):
    kind = case["kind"]
    if kind in ("orthogonalise", "muon"):
        n = case["batch"] * case["rows"] * case["cols"]
        small, large = min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        # a step: X X^T and its square are symmetric, half of each; the last product is whole
        flops = case["batch"] * STEPS * small * small * (3 * large + small)
        if kind == "muon":
            return {"bytes": n * (2 * case["replicas"] + 4 + 4 + 4 + 4 + 2), "flops": flops}
        return {"bytes": n * (SIZE[case["type"]] + SIZE[case["out"]]), "flops": flops}
    T, N, K = case["T"], case["N"], case["K"]
    if kind == "forward":
        return {"bytes": 2 * (T * K + 2 * N * K + T * N * (3 if case["save"] else 1)), "flops": 4 * T * N * K}
    if kind == "weight_grad":
        return {"bytes": 2 * (2 * T * N + T * K) + 2 * N * K * SIZE[case["out"]] * (2 if case["add"] else 1), "flops": 4 * T * N * K}
    return {"bytes": 2 * (5 * T * N + 4 * N * K + 2 * T * K), "flops": 8 * T * N * K}


def _exact_orthogonal(u):
    """The polynomial of each matrix by its right factor, X p(X^T X), in 64 bits; matrices with more columns go by their transpose."""
    out = []
    for x in u.double():
        norm = torch.linalg.vector_norm(x)
        x = x / norm if norm > 0 else x
        y = x if x.shape[0] >= x.shape[1] else x.t().contiguous()
        one = torch.eye(y.shape[1], dtype=torch.float64, device=y.device)
        for _ in range(STEPS):
            s = torch.matmul(y.t().contiguous(), y)
            y = torch.matmul(y, COEFS[0] * one + torch.matmul(COEFS[1] * one + COEFS[2] * s, s))
        out.append(y if x.shape[0] >= x.shape[1] else y.t())
    return torch.stack(out)


def _exact_act(v, name):
    if name == "relu":
        return torch.relu(v)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2.0))
    return v * torch.sigmoid(math.sqrt(8.0 / math.pi) * (v + 0.044715 * v ** 3))


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "orthogonalise":
        return {"out": _exact_orthogonal(s["x"])}
    if kind == "muon":
        hp = s["hp"]
        mean = sum(g.double() for g in s["grads"]) / len(s["grads"])
        momentum = hp["momentum"] * s["momentum"].double() + mean
        o = _exact_orthogonal(hp["momentum"] * momentum + mean if hp["nesterov"] else momentum)
        master = s["master"].double() * (1.0 - hp["lr"] * hp["weight_decay"]) - o * (hp["lr"] * hp["scale"])
        return {"master": master, "momentum": momentum, "param": master}
    if kind == "forward":
        x = s["x"].double()
        gate, up = (torch.matmul(s[n].double(), x.t().contiguous()).t() for n in ("w_gate", "w_up"))
        out = {"h": _exact_act(gate, case["act"]) * up}
        if case["save"]:
            out.update(gate=gate, up=up)
        return out
    x = s["x"].double()
    if kind == "weight_grad":
        out = {}
        for name in ("gate", "up"):
            dw = torch.matmul(x.t().contiguous(), s["d" + name].double()).t()
            out["dw_" + name] = dw if s["add_" + name] is None else dw + s["add_" + name].double()
        return out
    gate, up = s["gate"].double().requires_grad_(), s["up"].double().requires_grad_()
    dgate, dup = torch.autograd.grad(_exact_act(gate, case["act"]) * up, (gate, up), s["dh"].double())
    dx = torch.matmul(torch.cat([dgate, dup], 1), torch.cat([s["w_gate"], s["w_up"]], 0).double())
    return {"dgate": dgate, "dup": dup, "dx": dx, "dw_gate": torch.matmul(x.t().contiguous(), dgate).t(),
            "dw_up": torch.matmul(x.t().contiguous(), dup).t()}
