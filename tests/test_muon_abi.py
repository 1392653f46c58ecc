"""Refusals of the orthogonalised updates, through the C ABI with addresses that are never dereferenced (every call fails
before any HIP call) and through the Python binding with host tensors."""
import ctypes
import math

import pytest
import torch

import sharded_mixed_precision_rank_amd as zs

LIB = zs.library()
A = 0x7F0000000000  # fake; arrays 1 MiB apart, the workspace last
MB = 1 << 20
NEED = zs.orthogonalize_workspace_bytes(8, 16, 2)


def at(k):
    return A + k * MB


def coefs(*v):
    return (ctypes.c_double * len(v))(*v)


def orth(x=at(0), xf=2, ld_x=16, bs_x=128, batch=2, rows=8, cols=16, steps=5, co=None, out=at(1), of=2, ld_o=16, bs_o=128, ws=at(9),
         n=NEED):
    return LIB.zs_orthogonalize(x, xf, ld_x, bs_x, batch, rows, cols, steps, co, out, of, ld_o, bs_o, ws, n, None)


def muon(grads=(at(0), at(1)), N=None, batch=2, rows=8, cols=16, master=at(2), mom=at(3), param=at(4), ws=at(9), n=NEED,
         table=True, **hp):
    h = zs.MuonHP(**{k: v for k, v in hp.items() if k != "raw_steps"})._c()
    if "raw_steps" in hp:
        h.steps = hp["raw_steps"]
    tab = (ctypes.c_void_p * max(len(grads), 1))(*grads) if table else None
    return LIB.zs_reduce_muon(tab, len(grads) if N is None else N, batch, rows, cols, master, mom, param, ctypes.byref(h), ws, n,
                              None)


R, Z, G, S = "ZS_ERR_RANGE", "ZS_ERR_NULL", "ZS_ERR_ALIGN", "ZS_ERR_ALIAS"


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), R), (dict(batch=65536), R), (dict(rows=-1), R), (dict(cols=(1 << 20) + 1), R),
    (dict(rows=65537, cols=65537), R), (dict(xf=3), R), (dict(of=-1), R), (dict(steps=0), R), (dict(steps=33), R),
    (dict(steps=1, co=coefs(1, math.nan, 0)), R), (dict(steps=1, co=coefs(1, 0, 1e300)), R),
    (dict(ld_x=15), R), (dict(ld_o=15), R), (dict(bs_x=127), R), (dict(bs_o=127), R), (dict(ld_x=1 << 62), R), (dict(bs_o=1 << 62), R),
    (dict(ld_x=-16), R), (dict(bs_x=-128), R),
    (dict(n=NEED - 1), R), (dict(n=0), R),
    (dict(x=None), Z), (dict(out=None), Z), (dict(ws=None), Z),
    (dict(x=at(0) + 2), G), (dict(out=at(1) + 1, of=0), G), (dict(x=at(0) + 1, xf=1), G),
    (dict(out=at(0) + 4), S), (dict(out=at(0), of=0), S), (dict(out=at(0), ld_o=17, bs_o=200), S), (dict(ws=at(0)), S),
    (dict(ws=at(1) + 128 * 8 - 1), S), (dict(out=at(0) - 4), S),
])
def test_orthogonalize_refuses(kw, want):
    got = zs.STATUS[orth(**kw)]
    assert got == want and LIB.zs_last_error(), (kw, LIB.zs_last_error())


@pytest.mark.parametrize("kw,want", [
    (dict(N=0), R), (dict(N=-1), R), (dict(N=257), R), (dict(batch=-1), R), (dict(rows=1 << 21), R), (dict(n=NEED - 1), R),
    (dict(lr=-1.0), R), (dict(lr=math.nan), R), (dict(momentum=1.0), R), (dict(momentum=-0.1), R), (dict(weight_decay=-1.0), R),
    (dict(scale=math.inf), R), (dict(raw_steps=0), R), (dict(raw_steps=99), R), (dict(coefs=(1.0, math.inf, 0.0)), R),
    (dict(table=False, N=2), Z), (dict(grads=(at(0), None)), Z), (dict(master=None), Z), (dict(param=None), Z), (dict(ws=None), Z),
    (dict(grads=(at(0), at(1) + 1)), G), (dict(master=at(2) + 2), G), (dict(param=at(4) + 1), G),
    (dict(mom=at(2)), S), (dict(param=at(2) + 1022), S), (dict(grads=(at(0), at(4))), S), (dict(grads=(at(3) + 510, at(1))), S),
    (dict(ws=at(1) - NEED + 1), S), (dict(ws=at(3) + 4), S),
])
def test_reduce_muon_refuses(kw, want):
    got = zs.STATUS[muon(**kw)]
    assert got == want and LIB.zs_last_error(), (kw, LIB.zs_last_error())


def test_hp_is_required():
    assert zs.STATUS[LIB.zs_reduce_muon(None, 1, 1, 1, 1, None, None, None, None, None, 0, None)] == Z


def test_empty_calls_do_nothing():
    for kw in (dict(batch=0), dict(rows=0), dict(cols=0)):
        assert orth(x=None, out=None, ws=None, n=0, **kw) == 0
        assert muon(master=None, ws=None, n=0, **kw) == 0


def test_workspace_bytes():
    assert zs.orthogonalize_workspace_bytes(0, 4) == zs.orthogonalize_workspace_bytes(4, 4, 0) == 0
    assert zs.orthogonalize_workspace_bytes(-1, 4) == zs.orthogonalize_workspace_bytes(1 << 21, 4) == 0
    # the transpose needs as much; two matrices more than one
    assert zs.orthogonalize_workspace_bytes(100, 300) == zs.orthogonalize_workspace_bytes(300, 100)
    assert zs.orthogonalize_workspace_bytes(100, 300, 2) > zs.orthogonalize_workspace_bytes(100, 300)
    # X twice, S and the polynomial, 4 bytes a value each, and no more than 200 MB for sums beside them
    for rows, cols, batch in ((4096, 4096, 1), (11008, 4096, 1), (128, 128, 32), (1, 1 << 20, 1), (65536, 65536, 1)):
        short, long = sorted(-(-n // 32) * 32 for n in (rows, cols))
        least = batch * 8 * short * (short + long)
        assert least <= zs.orthogonalize_workspace_bytes(rows, cols, batch) <= least + batch * 70_000 + 200_000_000


def test_binding_refuses():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device tensor"):
        zs.orthogonalize(x, torch.zeros(4, 8))
    with pytest.raises(ValueError):
        zs.orthogonalize(x, torch.zeros(4, 9))
    with pytest.raises(ValueError):
        zs.orthogonalize(torch.zeros(2, 4, 8), x)
    with pytest.raises(TypeError):
        zs.orthogonalize(x.double(), x)
    with pytest.raises(ValueError, match="contiguous rows"):
        zs.orthogonalize(torch.zeros(8, 4).t(), x)
    with pytest.raises(ValueError, match="coefs"):
        zs.orthogonalize(x, x.clone(), steps=2, coefs=[(1, 2, 3)])
    with pytest.raises(ValueError, match="coefs"):
        zs.orthogonalize(x, x.clone(), coefs=(1, 2))
    with pytest.raises(ValueError, match="device tensor"):
        zs.reduce_muon([x.bfloat16()], x, x.clone(), x.bfloat16(), zs.MuonHP())


@pytest.mark.parametrize("hp", [dict(lr=1e30, scale=1e30), dict(lr=1e30, scale=-1e30), dict(lr=1e30, weight_decay=1e30),
                                dict(lr=1e200, weight_decay=1e200, scale=0.0), dict(lr=1e200, scale=1e200)])
def test_reduce_muon_refuses_what_leaves_fp32_when_folded(hp):
    """lr * scale and 1 - lr * weight_decay are fp32 values of the step: past that range, inf * 0 would be NaN in the master."""
    assert zs.STATUS[muon(**hp)] == R and b"fp32" in LIB.zs_last_error(), LIB.zs_last_error()


def test_workspace_of_stacks_is_what_they_need():
    """No room for sums that are not made, for padding of matrices that a workgroup keeps to itself, or for a polynomial that
    lies nowhere."""
    many = 65535
    for rows, cols in ((8, 8), (1, 128), (100, 30), (128, 128)):
        assert zs.orthogonalize_workspace_bytes(rows, cols, many) <= many * 8 * min(rows, cols) * (rows + cols) + 256
    # 32 x 160 padded: X twice and S; a partial sum and a counter
    assert zs.orthogonalize_workspace_bytes(129, 8, many) <= many * (8 * 32 * 160 + 4 * 32 * 32 + 16) + 2048
    # 96 x 160: the polynomial too; 9 partial sums, at most 6 counters
    assert zs.orthogonalize_workspace_bytes(90, 140, many) <= many * (8 * 96 * (160 + 96) + 9 * 8 + 6 * 4) + 2048
