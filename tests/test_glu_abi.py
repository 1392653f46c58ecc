"""Refusals of the gated feed-forward block, through the C ABI with addresses that are never dereferenced (every call
fails before any HIP call) and through the Python binding with host tensors."""
import pytest
import torch

import sharded_mixed_precision_rank_amd as zs

LIB = zs.library()
A = 0x7F0000000000  # fake; arrays 1 MiB apart
MB = 1 << 20


def at(k):
    return A + k * MB


def forward(x=at(0), ld_x=32, wg=at(1), wu=at(2), ld_w=32, fmt=0, T=8, N=16, K=32, act=0, h=at(3), ld_h=16, gate=None, up=None,
            ld_gu=16):
    return LIB.zs_glu_forward(x, ld_x, wg, wu, ld_w, fmt, T, N, K, act, h, ld_h, gate, up, ld_gu, None)


def backward(dh=at(0), ld_dh=16, gate=at(1), up=at(2), ld_gu=16, fmt=0, T=8, N=16, act=0, dgate=at(3), dup=at(4), ld_d=16,
             h=None, ld_h=16):
    return LIB.zs_glu_backward(dh, ld_dh, gate, up, ld_gu, fmt, T, N, act, dgate, dup, ld_d, h, ld_h, None)


def input_grad(dgate=at(0), dup=at(1), ld_d=16, wg=at(2), wu=at(3), ld_w=32, fmt=0, T=8, N=16, K=32, dx=at(4), ld_dx=32):
    return LIB.zs_glu_input_grad(dgate, dup, ld_d, wg, wu, ld_w, fmt, T, N, K, dx, ld_dx, None)


def weight_grad(dgate=at(0), dup=at(1), ld_d=16, x=at(2), ld_x=32, fmt=0, T=8, N=16, K=32, ag=None, au=None, dwg=at(3),
                dwu=at(4), dfmt=0, ld_dw=32):
    return LIB.zs_glu_weight_grad(dgate, dup, ld_d, x, ld_x, fmt, T, N, K, ag, au, dwg, dwu, dfmt, ld_dw, None)


R, Z, G, S = "ZS_ERR_RANGE", "ZS_ERR_NULL", "ZS_ERR_ALIGN", "ZS_ERR_ALIAS"
CASES = [
    (forward, [
        (dict(T=-1), R), (dict(N=-1), R), (dict(K=-1), R), (dict(T=1 << 31), R), (dict(N=1 << 31), R), (dict(K=1 << 31), R),
        (dict(fmt=2), R), (dict(fmt=-1), R), (dict(act=4), R), (dict(act=-1), R), (dict(ld_x=31), R), (dict(ld_w=31), R),
        (dict(ld_h=15), R), (dict(gate=at(4), up=at(5), ld_gu=15), R), (dict(ld_x=1 << 62), R), (dict(ld_h=(1 << 63) - 1), R),
        (dict(x=None), Z), (dict(wg=None), Z), (dict(wu=None), Z), (dict(h=None), Z), (dict(gate=at(4)), Z), (dict(up=at(4)), Z),
        (dict(x=at(0) + 1), G), (dict(wu=at(2) + 1), G), (dict(h=at(3) + 1), G), (dict(gate=at(4) + 1, up=at(5)), G),
        (dict(h=at(0)), S), (dict(h=at(1)), S), (dict(h=at(2)), S), (dict(gate=at(3), up=at(5)), S), (dict(gate=at(4), up=at(4)), S),
        (dict(gate=at(4), up=at(3)), S), (dict(gate=at(0), up=at(5)), S), (dict(gate=at(4), up=at(2)), S),
        (dict(h=at(0) + 8 * 32 * 2 - 2), S),
    ]),
    (backward, [
        (dict(T=-1), R), (dict(N=1 << 31), R), (dict(fmt=2), R), (dict(act=4), R), (dict(ld_dh=15), R), (dict(ld_gu=15), R),
        (dict(ld_d=15), R), (dict(h=at(5), ld_h=15), R),
        (dict(dh=None), Z), (dict(gate=None), Z), (dict(up=None), Z), (dict(dgate=None), Z), (dict(dup=None), Z),
        (dict(dh=at(0) + 1), G), (dict(dup=at(4) + 1), G), (dict(h=at(5) + 1), G),
        (dict(dgate=at(0)), S), (dict(dgate=at(2)), S), (dict(dup=at(1)), S), (dict(dup=at(3)), S), (dict(h=at(1)), S),
        (dict(h=at(2)), S), (dict(h=at(3)), S), (dict(h=at(4)), S), (dict(dgate=at(1) + 2), S), (dict(h=at(0) + 32), S),
        # on the input's own place, but with rows at another distance
        (dict(dgate=at(1), ld_d=24), S), (dict(h=at(0), ld_h=17), S),
    ]),
    (input_grad, [
        (dict(T=-1), R), (dict(K=1 << 31), R), (dict(fmt=2), R), (dict(ld_d=15), R), (dict(ld_w=31), R), (dict(ld_dx=31), R),
        (dict(dgate=None), Z), (dict(dup=None), Z), (dict(wg=None), Z), (dict(wu=None), Z), (dict(dx=None), Z),
        (dict(dx=at(4) + 1), G), (dict(dup=at(1) + 1), G),
        (dict(dx=at(0)), S), (dict(dx=at(1)), S), (dict(dx=at(2)), S), (dict(dx=at(3)), S),
    ]),
    (weight_grad, [
        (dict(T=-1), R), (dict(N=1 << 31), R), (dict(fmt=2), R), (dict(dfmt=3), R), (dict(ld_d=15), R), (dict(ld_x=31), R),
        (dict(ld_dw=31), R),
        (dict(dgate=None), Z), (dict(dup=None), Z), (dict(x=None), Z), (dict(dwg=None), Z), (dict(dwu=None), Z), (dict(ag=at(5)), Z),
        (dict(au=at(5)), Z),
        (dict(x=at(2) + 1), G), (dict(dwg=at(3) + 2, dfmt=2), G), (dict(ag=at(5) + 1, au=at(6)), G),
        (dict(dwg=at(0)), S), (dict(dwu=at(2)), S), (dict(dwu=at(3)), S), (dict(ag=at(4), au=at(5)), S), (dict(ag=at(5), au=at(3)), S),
        (dict(ag=at(3) + 64, au=at(6)), S),
    ]),
]


@pytest.mark.parametrize("call,kw,want", [(c, kw, w) for c, cases in CASES for kw, w in cases])
def test_refuses(call, kw, want):
    got = zs.STATUS[call(**kw)]
    assert got == want and LIB.zs_last_error(), (kw, LIB.zs_last_error())


def test_empty_calls_do_nothing():
    assert forward(T=0) == 0 and forward(N=0) == 0 and backward(T=0) == 0 and backward(N=0) == 0
    assert input_grad(T=0) == 0 and input_grad(K=0) == 0 and weight_grad(N=0) == 0 and weight_grad(K=0) == 0


def t(r, c, dtype=torch.bfloat16):
    return torch.zeros(r, c, dtype=dtype)


def test_binding_refuses():
    x, w, h = t(4, 8), t(6, 8), t(4, 6)
    with pytest.raises(ValueError, match="device tensor"):
        zs.glu_forward(x, w, w.clone(), h)
    with pytest.raises(TypeError):
        zs.glu_forward(x.float(), w, w, h)
    with pytest.raises(TypeError):
        zs.glu_forward(x, w.half(), w, h)
    with pytest.raises(TypeError):
        zs.glu_forward(x, None, w, h)
    with pytest.raises(ValueError):
        zs.glu_forward(x, t(6, 9), w, h)
    with pytest.raises(ValueError):
        zs.glu_forward(x, w, t(5, 8), h)
    with pytest.raises(ValueError):
        zs.glu_forward(x, w, w, t(4, 7))
    with pytest.raises(ValueError, match="act"):
        zs.glu_forward(x, w, w, h, act="tanh")
    with pytest.raises(ValueError, match="together"):
        zs.glu_forward(x, w, w, h, gate=t(4, 6))
    with pytest.raises(ValueError, match="row stride"):
        zs.glu_forward(x, w, t(6, 16)[:, :8], h)
    with pytest.raises(ValueError, match="contiguous rows"):
        zs.glu_forward(x, t(8, 6).t(), t(8, 6).t(), h)
    with pytest.raises(ValueError):
        zs.glu_forward(x[0], w, w, h)
    with pytest.raises(ValueError):
        zs.glu_backward(h, t(4, 5), h, h, h)
    with pytest.raises(ValueError, match="together"):
        zs.glu_weight_grad(h, h, x, t(6, 8), t(6, 8), add_gate=t(6, 8))
    with pytest.raises(TypeError):
        zs.glu_weight_grad(h, h, x, t(6, 8), t(6, 8), add_gate=t(6, 8, torch.float32), add_up=t(6, 8, torch.float32))
    with pytest.raises(ValueError, match="row stride"):
        zs.glu_weight_grad(h, h, x, t(6, 8), t(6, 8), add_gate=t(6, 9)[:, :8], add_up=t(6, 9)[:, :8])
    with pytest.raises(ValueError):
        zs.glu_input_grad(h, h, w, w, t(4, 9))
