"""Refusals of the 8-bit training operators, through the C ABI with addresses that are never dereferenced (every
call fails before any HIP call) and through the Python binding with host tensors."""
import ctypes

import pytest
import torch

import sharded_mixed_precision_rank_amd as zs

LIB = zs.library()
A = 0x7F0000000000  # fake; arrays 1 MiB apart
MB = 1 << 20


def status(fn, **kw):
    return zs.STATUS[fn(**kw)], LIB.zs_last_error().decode()


def save(x=A, fmt=0, ld_x=64, rows=8, cols=64, col=None, rule=0, codes=A + MB, ld_q=64, scales=A + 2 * MB):
    return LIB.zs_q8_save(x, fmt, ld_x, rows, cols, col, rule, codes, ld_q, scales, None)


def load(codes=A, ld_q=64, scales=A + MB, rows=8, cols=64, out=A + 2 * MB, fmt=0, ld_out=64):
    return LIB.zs_q8_load(codes, ld_q, scales, rows, cols, out, fmt, ld_out, None)


def matmul(x=A, ld_x=32, sx=A + MB, w=A + 2 * MB, ld_w=32, sw=A + 3 * MB, T=8, N=16, K=32, layout=0, y=A + 4 * MB,
           fmt=0, ld_y=32):
    return LIB.zs_q8_matmul(x, ld_x, sx, w, ld_w, sw, T, N, K, layout, y, fmt, ld_y, None)


def wgrad(dy=A, fmt=0, ld_dy=16, x=A + MB, ld_x=32, sx=A + 2 * MB, T=8, N=16, K=32, add=None, dw=A + 3 * MB, dfmt=0,
          ld_dw=32):
    return LIB.zs_q8_weight_grad(dy, fmt, ld_dy, x, ld_x, sx, T, N, K, add, dw, dfmt, ld_dw, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), "ZS_ERR_RANGE"), (dict(cols=-1), "ZS_ERR_RANGE"), (dict(rows=1 << 31), "ZS_ERR_RANGE"),
    (dict(fmt=3), "ZS_ERR_RANGE"), (dict(fmt=-1), "ZS_ERR_RANGE"), (dict(rule=2), "ZS_ERR_RANGE"),
    (dict(ld_x=63), "ZS_ERR_RANGE"), (dict(ld_q=0), "ZS_ERR_RANGE"), (dict(ld_q=-64), "ZS_ERR_RANGE"),
    (dict(ld_x=1 << 62), "ZS_ERR_RANGE"), (dict(ld_q=(1 << 63) - 1), "ZS_ERR_RANGE"),
    (dict(x=None), "ZS_ERR_NULL"), (dict(codes=None), "ZS_ERR_NULL"), (dict(scales=None), "ZS_ERR_NULL"),
    (dict(x=A + 1), "ZS_ERR_ALIGN"), (dict(x=A + 2, fmt=2), "ZS_ERR_ALIGN"), (dict(scales=A + 2 * MB + 2), "ZS_ERR_ALIGN"),
    (dict(col=A + 3 * MB + 1), "ZS_ERR_ALIGN"),
    (dict(codes=A), "ZS_ERR_ALIAS"), (dict(codes=A + 2 * 8 * 64 - 1), "ZS_ERR_ALIAS"),
    (dict(scales=A + 4), "ZS_ERR_ALIAS"), (dict(scales=A + MB), "ZS_ERR_ALIAS"),
    (dict(col=A + MB), "ZS_ERR_ALIAS"), (dict(col=A + 2 * MB), "ZS_ERR_ALIAS"),
    # codes in the gap of x's rows, but too wide for it (pitch 160 bytes: 128 of x, 32 free)
    (dict(ld_x=80, codes=A + 128, ld_q=160), "ZS_ERR_ALIAS"),
])
def test_save_refuses(kw, want):
    got, msg = status(save, **kw)
    assert got == want and msg, (kw, msg)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), "ZS_ERR_RANGE"), (dict(cols=1 << 31), "ZS_ERR_RANGE"), (dict(fmt=7), "ZS_ERR_RANGE"),
    (dict(ld_q=63), "ZS_ERR_RANGE"), (dict(ld_out=63), "ZS_ERR_RANGE"),
    (dict(codes=None), "ZS_ERR_NULL"), (dict(scales=None), "ZS_ERR_NULL"), (dict(out=None), "ZS_ERR_NULL"),
    (dict(out=A + 2 * MB + 1), "ZS_ERR_ALIGN"), (dict(scales=A + MB + 1), "ZS_ERR_ALIGN"),
    (dict(out=A), "ZS_ERR_ALIAS"), (dict(out=A + MB), "ZS_ERR_ALIAS"),
])
def test_load_refuses(kw, want):
    got, msg = status(load, **kw)
    assert got == want and msg, (kw, msg)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), "ZS_ERR_RANGE"), (dict(N=-1), "ZS_ERR_RANGE"), (dict(K=1 << 31), "ZS_ERR_RANGE"),
    (dict(fmt=3), "ZS_ERR_RANGE"), (dict(layout=2), "ZS_ERR_RANGE"),
    (dict(K=131072, ld_x=131072, ld_w=131072), "ZS_ERR_RANGE"), (dict(N=131072, ld_x=131072, layout=1), "ZS_ERR_RANGE"),
    (dict(ld_x=31), "ZS_ERR_RANGE"), (dict(ld_w=31), "ZS_ERR_RANGE"), (dict(ld_y=15), "ZS_ERR_RANGE"),
    (dict(layout=1, ld_x=15), "ZS_ERR_RANGE"), (dict(layout=1, ld_y=31), "ZS_ERR_RANGE"),
    (dict(x=None), "ZS_ERR_NULL"), (dict(w=None), "ZS_ERR_NULL"), (dict(sx=None), "ZS_ERR_NULL"), (dict(y=None), "ZS_ERR_NULL"),
    (dict(sx=A + MB + 1), "ZS_ERR_ALIGN"), (dict(sw=A + 3 * MB + 2), "ZS_ERR_ALIGN"), (dict(y=A + 4 * MB + 1), "ZS_ERR_ALIGN"),
    (dict(y=A), "ZS_ERR_ALIAS"), (dict(y=A + MB), "ZS_ERR_ALIAS"), (dict(y=A + 2 * MB), "ZS_ERR_ALIAS"),
    (dict(y=A + 3 * MB), "ZS_ERR_ALIAS"),
])
def test_matmul_refuses(kw, want):
    got, msg = status(matmul, **kw)
    assert got == want and msg, (kw, msg)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), "ZS_ERR_RANGE"), (dict(N=1 << 31), "ZS_ERR_RANGE"), (dict(fmt=2), "ZS_ERR_RANGE"),
    (dict(dfmt=3), "ZS_ERR_RANGE"), (dict(ld_dy=15), "ZS_ERR_RANGE"), (dict(ld_x=31), "ZS_ERR_RANGE"),
    (dict(ld_dw=31), "ZS_ERR_RANGE"),
    (dict(dy=None), "ZS_ERR_NULL"), (dict(x=None), "ZS_ERR_NULL"), (dict(sx=None), "ZS_ERR_NULL"), (dict(dw=None), "ZS_ERR_NULL"),
    (dict(dy=A + 1), "ZS_ERR_ALIGN"), (dict(sx=A + 2 * MB + 1), "ZS_ERR_ALIGN"), (dict(dw=A + 3 * MB + 2, dfmt=2), "ZS_ERR_ALIGN"),
    (dict(add=A + 4 * MB + 1), "ZS_ERR_ALIGN"),
    (dict(dw=A), "ZS_ERR_ALIAS"), (dict(dw=A + MB), "ZS_ERR_ALIAS"), (dict(dw=A + 2 * MB), "ZS_ERR_ALIAS"),
    # add may be dw itself, not a part of it
    (dict(add=A + 3 * MB + 2), "ZS_ERR_ALIAS"), (dict(add=A + 3 * MB - 64), "ZS_ERR_ALIAS"),
])
def test_weight_grad_refuses(kw, want):
    got, msg = status(wgrad, **kw)
    assert got == want and msg, (kw, msg)


def test_two_pass_form_keeps_to_16_bits():
    """The fp32 format is for the 8-bit calls only."""
    tab = (ctypes.c_void_p * 1)(A)
    assert LIB.zs_reduce_grads_flat(tab, 1, 64, 2, 1.0, A + MB, 1 << 20, A + 2 * MB, None) == 2


def test_empty_calls_are_no_ops():
    assert save(rows=0, x=None, codes=None, scales=None) == 0
    assert load(rows=0, codes=None, out=None) == 0
    assert load(cols=0, codes=None, out=None) == 0
    assert matmul(T=0, x=None, y=None) == 0
    assert matmul(N=0, w=None, y=None) == 0
    assert matmul(K=0, layout=1, w=None, y=None) == 0
    assert wgrad(N=0, dw=None) == 0
    assert wgrad(K=0, dw=None) == 0


def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros(4, 8)
    q = torch.zeros(4, 8, dtype=torch.int8)
    s = torch.zeros(4)
    with pytest.raises(ValueError, match="device tensor"):
        zs.q8_save(x, q, s)
    with pytest.raises(TypeError, match="dtype"):
        zs.q8_save(x.double(), q, s)
    with pytest.raises(TypeError, match="torch.Tensor"):
        zs.q8_load(q.numpy(), s, x)
    with pytest.raises(TypeError, match="dtype"):
        zs.q8_weight_grad(x, q, s, x)
    with pytest.raises(TypeError, match="dtype"):
        zs.q8_matmul(q.to(torch.int16), s, q, None, x)
