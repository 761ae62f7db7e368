"""Refusals of the gated recurrence and the residual RMS-Norm: every bad
argument is turned down on the host, before anything is enqueued."""
import ctypes

import pytest
import torch

import sparse_state_linear_gb300 as sdm
from sparse_state_linear_gb300 import build_ext

FAKE = ctypes.c_void_p(1 << 20)        # aligned, never dereferenced
MISALIGNED = ctypes.c_void_p((1 << 20) + 8)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    build_ext.build()
    return sdm.lib()


def rec(**kw):
    base = dict(n_seq=2, rows=8, D=64, dtype=sdm.SDM_F32)
    base.update(kw)
    return sdm.make_recurrence(**base)


def forward(L, sh, over=None, ws=BIG):
    # za zb v A bias offsets h0 y hT states workspace
    p = [FAKE] * 11
    for i, x in (over or {}).items():
        p[i] = x
    return L.sdm_recurrence_forward(ctypes.byref(sh), *p, ws, None)


def backward(L, sh, over=None, ws=BIG):
    # za zb v A bias offsets states dy dhT dza dzb dv dA dbias dh0 workspace
    p = [FAKE] * 16
    for i, x in (over or {}).items():
        p[i] = x
    return L.sdm_recurrence_backward(ctypes.byref(sh), *p, ws, None)


def step(L, sh, over=None, n_slots=16):
    # za zb v A bias state | slots y
    p = [FAKE] * 8
    for i, x in (over or {}).items():
        p[i] = x
    return L.sdm_recurrence_step(ctypes.byref(sh), *p[:6], n_slots, *p[6:], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seq=-1), 1), (dict(rows=-1), 1), (dict(D=0), 1), (dict(ld=-8), 1), (dict(ld_grad=-8), 1),
    (dict(dtype=2), 1), (dict(dtype=9), 1), (dict(ld=56), 1), (dict(ld_grad=56), 1),
    (dict(n_seq=65536), 2), (dict(D=65544), 2), (dict(rows=(1 << 31) - 1, D=65536, n_seq=1), 2), (dict(D=60), 2), (dict(ld=66), 2), (dict(ld_grad=68), 2),
])
def test_recurrence_rejects_bad_shapes(L, kw, code):
    sh = rec(**kw)
    assert forward(L, sh) == code
    assert backward(L, sh) == code
    assert step(L, sh) == code
    assert L.sdm_recurrence_workspace_size(ctypes.byref(sh)) == 0
    assert L.sdm_recurrence_states_size(ctypes.byref(sh)) == 0


def test_recurrence_rejects_bad_pointers(L):
    sh = rec()
    for i in (0, 1, 2, 7, 10):                       # required
        assert forward(L, sh, {i: None}) == 1, i
    for i in range(11):
        assert forward(L, sh, {i: MISALIGNED}) == 1, i
    for i in (0, 1, 2, 6, 7, 9, 10, 11, 15):
        assert backward(L, sh, {i: None}) == 1, i
    for i in range(16):
        assert backward(L, sh, {i: MISALIGNED}) == 1, i
    for i in (0, 1, 2, 5, 7):
        assert step(L, sh, {i: None}) == 1, i
    for i in range(8):
        assert step(L, sh, {i: MISALIGNED}) == 1, i
    need = L.sdm_recurrence_workspace_size(ctypes.byref(sh))
    assert need > 0
    assert forward(L, sh, ws=need - 1) == 1
    assert backward(L, sh, ws=need - 1) == 1
    # Without offsets the rows have to divide into equal sequences.
    assert forward(L, rec(rows=9), {5: None}) == 1
    assert backward(L, rec(rows=9), {5: None}) == 1
    # Without slots row i is state row i.
    assert step(L, sh, {6: None}, n_slots=7) == 1
    assert step(L, sh, n_slots=-1) == 1
    assert L.sdm_recurrence_forward(None, *([FAKE] * 11), BIG, None) == 1


def test_recurrence_without_work(L):
    sh = rec(n_seq=0)
    assert forward(L, sh, {i: None for i in range(11)}) == 0
    assert backward(L, sh, {i: None for i in range(16)}) == 0
    assert step(L, rec(rows=0), {i: None for i in range(8)}) == 0


def norm(**kw):
    base = dict(rows=8, D=256, dtype=sdm.SDM_BF16)
    base.update(kw)
    return sdm.make_norm(**base)


def norm_forward(L, sh, over=None, eps=1e-6, out_dtype=sdm.SDM_BF16, group=0):
    p = [FAKE] * 6                                   # x residual gamma | s out | scale
    for i, x in (over or {}).items():
        p[i] = x
    return L.sdm_add_rmsnorm(ctypes.byref(sh), *p[:3], eps, *p[3:5], out_dtype, group, p[5], None)


def norm_backward(L, sh, over=None, eps=1e-6, ws=BIG):
    p = [FAKE] * 7                                   # s dout gamma ds | dx dgamma workspace
    for i, x in (over or {}).items():
        p[i] = x
    return L.sdm_add_rmsnorm_backward(ctypes.byref(sh), *p[:4], eps, *p[4:], ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(D=0), 1), (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(D=252), 2),
    (dict(D=16392), 2),
])
def test_norm_rejects_bad_shapes(L, kw, code):
    assert norm_forward(L, norm(**kw)) == code
    assert norm_backward(L, norm(**kw)) == code
    assert L.sdm_add_rmsnorm_workspace_size(ctypes.byref(norm(**kw))) == 0


def test_norm_rejects_bad_arguments(L):
    sh = norm()
    for eps in (0.0, -1.0, float("inf"), float("nan")):
        assert norm_forward(L, sh, eps=eps) == 1
        assert norm_backward(L, sh, eps=eps) == 1
    assert norm_forward(L, sh, out_dtype=3) == 1
    assert norm_forward(L, sh, group=64) == 1                                  # group without 8 bits
    assert norm_forward(L, sh, out_dtype=sdm.SDM_E4M3, group=-32) == 1
    assert norm_forward(L, sh, out_dtype=sdm.SDM_E4M3, group=96) == 1          # does not divide D
    assert norm_forward(L, sh, out_dtype=sdm.SDM_E4M3, group=16) == 2
    assert norm_forward(L, sh, {5: None}, out_dtype=sdm.SDM_E4M3) == 1
    for i in (0, 4):
        assert norm_forward(L, sh, {i: None}) == 1, i
    for i in range(5):
        assert norm_forward(L, sh, {i: MISALIGNED}) == 1, i
    for i in (0, 1, 4, 6):
        assert norm_backward(L, sh, {i: None}) == 1, i
    for i in range(7):
        assert norm_backward(L, sh, {i: MISALIGNED}) == 1, i
    need = L.sdm_add_rmsnorm_workspace_size(ctypes.byref(sh))
    assert need > 0 and norm_backward(L, sh, ws=need - 1) == 1
    assert norm_forward(L, norm(rows=0), {i: None for i in range(6)}) == 0
    assert norm_backward(L, norm(rows=0), {i: None for i in range(7)}) == 0


def test_binding_refuses_cpu_tensors():
    t = torch.zeros(8, 64)
    for call in (lambda: sdm.sdm_recurrence_forward(rec(), t, t, t),
                 lambda: sdm.sdm_recurrence_backward(rec(), t, t, t, t, t),
                 lambda: sdm.sdm_recurrence_step(rec(), t, t, t, t),
                 lambda: sdm.sdm_add_rmsnorm(norm(), t),
                 lambda: sdm.sdm_add_rmsnorm_backward(norm(), t, t)):
        with pytest.raises(ValueError):
            call()
