"""The gated feed-forward block in 64 bits on the CPU, from the definitions in the header."""
import math

import torch

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = ("silu", "gelu", "gelu_tanh", "relu")


def act(v, name):
    """The activation and its slope."""
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v)), (v > 0).double()
    if name == "gelu":
        p = 0.5 * torch.special.erfc(-v / math.sqrt(2))
        return v * p, p + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        s = torch.sigmoid(v)
        return v * s, s * (1 + v * torch.sigmoid(-v))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (v + 0.044715 * v ** 3))
    # 1 + t where t is near -1: twice the logistic function
    one_t = 2 * torch.sigmoid(2 * c * (v + 0.044715 * v ** 3))
    return 0.5 * v * one_t, 0.5 * one_t + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)


def forward(x, wg, wu, name):
    gate, up = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    return act(gate, name)[0] * up, gate, up


def backward(dh, gate, up, name):
    value, slope = act(gate.double(), name)
    return dh.double() * up.double() * slope, dh.double() * value, value * up.double()


def half_step(kind):
    return torch.finfo(DT[kind]).eps / 2


def least(kind):
    """Half of the smallest subnormal."""
    return torch.finfo(DT[kind]).smallest_normal * torch.finfo(DT[kind]).eps / 2
