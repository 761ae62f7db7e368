"""Refusals of the layer norm, the short convolution and the selective scan:
every bad argument is turned down on the host, before anything is enqueued; the
plain forms that the GPU tests compare with agree with differences; and every
kernel waits for the stream before it touches memory."""
import ctypes

import pytest
import torch

import sparse_state_linear_gb300 as sdm
from sparse_state_linear_gb300 import build_ext
from tests import _more_layers as R
from tests.test_stream_order_cpu import kernels

FAKE = ctypes.c_void_p(1 << 20)        # aligned, never dereferenced
MISALIGNED = ctypes.c_void_p((1 << 20) + 8)
BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    build_ext.build()
    return sdm.lib()


def pointers(n, over):
    p = [FAKE] * n
    for i, x in (over or {}).items():
        p[i] = x
    return p


# ---------------------------------------------------------------- layer norm

def norm(**kw):
    return sdm.make_norm(**{**dict(rows=8, D=256, dtype=sdm.SDM_BF16), **kw})


def ln_forward(L, sh, over=None, eps=1e-5, out_dtype=sdm.SDM_BF16, group=0):
    p = pointers(7, over)                            # x residual gamma beta | s out | scale
    return L.sdm_add_layernorm(ctypes.byref(sh), *p[:4], eps, *p[4:6], out_dtype, group, p[6], None)


def ln_backward(L, sh, over=None, eps=1e-5, ws=BIG):
    p = pointers(8, over)                            # s dout gamma ds | dx dgamma dbeta workspace
    return L.sdm_add_layernorm_backward(ctypes.byref(sh), *p[:4], eps, *p[4:], ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(D=0), 1), (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(D=252), 2), (dict(D=16392), 2),
])
def test_layernorm_rejects_bad_shapes(L, kw, code):
    assert ln_forward(L, norm(**kw)) == code
    assert ln_backward(L, norm(**kw)) == code
    assert L.sdm_add_layernorm_workspace_size(ctypes.byref(norm(**kw))) == 0


def test_layernorm_rejects_bad_arguments(L):
    sh = norm()
    for eps in (0.0, -1.0, float("inf"), float("nan")):
        assert ln_forward(L, sh, eps=eps) == 1
        assert ln_backward(L, sh, eps=eps) == 1
    assert ln_forward(L, sh, out_dtype=3) == 1
    assert ln_forward(L, sh, group=64) == 1                                  # group without 8 bits
    assert ln_forward(L, sh, out_dtype=sdm.SDM_E4M3, group=-32) == 1
    assert ln_forward(L, sh, out_dtype=sdm.SDM_E4M3, group=96) == 1          # does not divide D
    assert ln_forward(L, sh, out_dtype=sdm.SDM_E4M3, group=16) == 2
    assert ln_forward(L, sh, {6: None}, out_dtype=sdm.SDM_E4M3) == 1
    for i in (0, 5):
        assert ln_forward(L, sh, {i: None}) == 1, i
    for i in range(6):
        assert ln_forward(L, sh, {i: MISALIGNED}) == 1, i
    for i in (0, 1, 4, 7):
        assert ln_backward(L, sh, {i: None}) == 1, i
    for i in range(8):
        assert ln_backward(L, sh, {i: MISALIGNED}) == 1, i
    for keep in (5, 6):                              # one sum wanted: the workspace is needed
        assert ln_backward(L, sh, {11 - keep: None, 7: None}) == 1
    need = L.sdm_add_layernorm_workspace_size(ctypes.byref(sh))
    assert need > 0 and ln_backward(L, sh, ws=need - 1) == 1
    assert ln_forward(L, norm(rows=0), {i: None for i in range(7)}) == 0
    assert ln_backward(L, norm(rows=0), {i: None for i in range(8)}) == 0


# --------------------------------------------------------------- convolution

def conv(**kw):
    return sdm.make_conv(**{**dict(n_seq=2, rows=8, D=64, taps=4, dtype=sdm.SDM_F32), **kw})


def conv_forward(L, sh, over=None):
    return L.sdm_short_conv_forward(ctypes.byref(sh), *pointers(7, over), None)        # x w bias offsets x0 y xT


def conv_backward(L, sh, over=None, ws=BIG):
    # x w bias offsets x0 dy dxT dx dw dbias dx0 workspace
    return L.sdm_short_conv_backward(ctypes.byref(sh), *pointers(12, over), ws, None)


def conv_step(L, sh, over=None, n_slots=16):
    p = pointers(6, over)                            # x w bias state | slots y
    return L.sdm_short_conv_step(ctypes.byref(sh), *p[:4], n_slots, *p[4:], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seq=-1), 1), (dict(rows=-1), 1), (dict(D=0), 1), (dict(taps=0), 1), (dict(act=2), 1), (dict(act=-1), 1),
    (dict(ld=-8), 1), (dict(ld_grad=-8), 1), (dict(dtype=2), 1), (dict(ld=56), 1), (dict(ld_grad=56), 1),
    (dict(n_seq=65536), 2), (dict(D=65544), 2), (dict(taps=1), 2), (dict(taps=5), 2), (dict(D=60), 2), (dict(ld=66), 2),
    (dict(ld_grad=68), 2), (dict(rows=(1 << 30) + 8, n_seq=1), 2), (dict(rows=1 << 30, n_seq=1, D=65536), 2),
])
def test_conv_rejects_bad_shapes(L, kw, code):
    sh = conv(**kw)
    assert conv_forward(L, sh) == code
    assert conv_backward(L, sh) == code
    assert conv_step(L, sh) == code
    assert L.sdm_short_conv_workspace_size(ctypes.byref(sh)) == 0


def test_conv_rejects_bad_pointers(L):
    sh = conv()
    for i in (0, 1, 5):
        assert conv_forward(L, sh, {i: None}) == 1, i
    for i in range(7):
        assert conv_forward(L, sh, {i: MISALIGNED}) == 1, i
    for i in (0, 1, 5, 7, 11):
        assert conv_backward(L, sh, {i: None}) == 1, i
    for i in range(12):
        assert conv_backward(L, sh, {i: MISALIGNED}) == 1, i
    for i in (0, 1, 3, 5):
        assert conv_step(L, sh, {i: None}) == 1, i
    for i in range(6):
        assert conv_step(L, sh, {i: MISALIGNED}) == 1, i
    need = L.sdm_short_conv_workspace_size(ctypes.byref(sh))
    assert need > 0 and conv_backward(L, sh, ws=need - 1) == 1
    assert conv_forward(L, conv(rows=9), {3: None}) == 1                     # equal parts of 9 rows
    assert conv_backward(L, conv(rows=9), {3: None}) == 1
    assert conv_step(L, sh, {4: None}, n_slots=7) == 1                       # row i is window i
    assert conv_step(L, sh, n_slots=-1) == 1
    assert conv_step(L, conv(rows=(1 << 22) + 8), n_slots=1 << 23) == 2
    assert L.sdm_short_conv_forward(None, *([FAKE] * 7), None) == 1


def test_conv_without_work(L):
    sh = conv(n_seq=0)
    assert conv_forward(L, sh, {i: None for i in range(7)}) == 0
    assert conv_backward(L, sh, {i: None for i in range(12)}) == 0
    assert conv_step(L, conv(rows=0), {i: None for i in range(6)}) == 0


# ---------------------------------------------------------------------- scan

def sel(**kw):
    return sdm.make_selective(**{**dict(n_seq=2, rows=8, D=64, N=16, dtype=sdm.SDM_F32), **kw})


def scan_forward(L, sh, over=None, ws=BIG):
    # x dt A B C skip bias z offsets h0 y hT states workspace
    return L.sdm_selective_scan_forward(ctypes.byref(sh), *pointers(14, over), ws, None)


def scan_backward(L, sh, over=None, ws=BIG):
    # x dt A B C skip bias z offsets states dy dhT dx ddt dA dB dC dskip dbias dz dh0 workspace
    return L.sdm_selective_scan_backward(ctypes.byref(sh), *pointers(22, over), ws, None)


def scan_step(L, sh, over=None, n_slots=16):
    p = pointers(11, over)                           # x dt A B C skip bias z state | slots y
    return L.sdm_selective_scan_step(ctypes.byref(sh), *p[:9], n_slots, *p[9:], None)


STRIDES = ("ld", "ld_z", "ld_bc", "ld_grad", "ld_z_grad", "ld_bc_grad")


@pytest.mark.parametrize("kw,code", [
    (dict(n_seq=-1), 1), (dict(rows=-1), 1), (dict(D=0), 1), (dict(N=0), 1), (dict(groups=0), 1), (dict(groups=3), 1),
    (dict(dtype=2), 1), (dict(n_seq=65536), 2), (dict(D=65544), 2), (dict(N=12), 2), (dict(N=128), 2), (dict(D=60), 2),
    (dict(D=64, groups=16), 2), (dict(rows=(1 << 30) + 8, n_seq=1), 2), (dict(rows=1 << 30, n_seq=1, D=4096), 2),
] + [({k: -8}, 1) for k in STRIDES] + [({k: 8}, 1) for k in STRIDES] + [({k: 68}, 2) for k in STRIDES])
def test_scan_rejects_bad_shapes(L, kw, code):
    sh = sel(**kw)
    assert scan_forward(L, sh) == code
    assert scan_backward(L, sh) == code
    assert scan_step(L, sh) == code
    for size in (L.sdm_selective_scan_workspace_size, L.sdm_selective_scan_backward_workspace_size, L.sdm_selective_scan_states_size):
        assert size(ctypes.byref(sh)) == 0


def test_scan_rejects_bad_pointers(L):
    sh = sel()
    for i in (0, 1, 2, 3, 4, 10, 13):
        assert scan_forward(L, sh, {i: None}) == 1, i
    for i in range(14):
        assert scan_forward(L, sh, {i: MISALIGNED}) == 1, i
    for i in (0, 1, 2, 3, 4, 9, 10, 12, 13, 15, 16, 19, 21):
        assert scan_backward(L, sh, {i: None}) == 1, i
    for i in range(22):
        assert scan_backward(L, sh, {i: MISALIGNED}) == 1, i
    for i in (0, 1, 2, 3, 4, 8, 10):
        assert scan_step(L, sh, {i: None}) == 1, i
    for i in range(11):
        assert scan_step(L, sh, {i: MISALIGNED}) == 1, i
    need = L.sdm_selective_scan_workspace_size(ctypes.byref(sh))
    assert need > 0 and scan_forward(L, sh, ws=need - 1) == 1
    need = L.sdm_selective_scan_backward_workspace_size(ctypes.byref(sh))
    assert need > 0 and scan_backward(L, sh, ws=need - 1) == 1
    assert scan_forward(L, sel(rows=9), {8: None}) == 1                      # equal parts of 9 rows
    assert scan_backward(L, sel(rows=9), {8: None}) == 1
    assert scan_step(L, sh, {9: None}, n_slots=7) == 1                       # row i is state row i
    assert scan_step(L, sh, n_slots=-1) == 1
    assert scan_step(L, sel(rows=(1 << 22) + 8), n_slots=1 << 23) == 2
    assert L.sdm_selective_scan_forward(None, *([FAKE] * 14), BIG, None) == 1


def test_scan_without_work(L):
    sh = sel(n_seq=0)
    assert scan_forward(L, sh, {i: None for i in range(14)}) == 0
    assert scan_backward(L, sh, {i: None for i in range(22)}) == 0
    assert scan_step(L, sel(rows=0), {i: None for i in range(11)}) == 0


def test_binding_refuses_cpu_tensors():
    t, w = torch.zeros(8, 64), torch.zeros(64, 16)
    for call in (lambda: sdm.sdm_add_layernorm(norm(), t), lambda: sdm.sdm_add_layernorm_backward(norm(), t, t),
                 lambda: sdm.sdm_short_conv_forward(conv(), t, w), lambda: sdm.sdm_short_conv_backward(conv(), t, w, t),
                 lambda: sdm.sdm_short_conv_step(conv(), t, w, t), lambda: sdm.sdm_selective_scan_forward(sel(), t, t, w, t, t),
                 lambda: sdm.sdm_selective_scan_backward(sel(), t, t, w, t, t, t, t),
                 lambda: sdm.sdm_selective_scan_step(sel(), t, t, w, t, t, t)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------ the plain forms

def differences(loss, p, name, grad, picks, h=(1e-3, 5e-4)):
    """A gradient of a 64-bit form against central differences, the h^2 term
    taken out by the two step sizes."""
    t = p[name]
    for i in picks:
        i %= t.numel()
        est = []
        for step in h:
            e = torch.zeros(t.numel(), dtype=torch.float64)
            e[i] = step
            e = e.reshape(t.shape)
            est.append((loss({**p, name: t + e}) - loss({**p, name: t - e})) / (2 * step))
        best = est[1] + (est[1] - est[0]) / 3
        assert abs(float(grad.flatten()[i]) - best) <= abs(est[1] - est[0]) + 1e-9 * (1 + abs(best)), (name, i)


def test_plain_layernorm_against_differences():
    g = torch.Generator().manual_seed(0)
    p = {"s": torch.randn(4, 24, generator=g, dtype=torch.float64) + 0.5, "gamma": torch.rand(24, generator=g, dtype=torch.float64),
         "beta": torch.randn(24, generator=g, dtype=torch.float64)}
    dout, ds = torch.randn(4, 24, generator=g, dtype=torch.float64), torch.randn(4, 24, generator=g, dtype=torch.float64)
    loss = lambda q: float((R.layernorm(q["s"], q["gamma"], q["beta"], 1e-3)[0] * dout).sum() + (q["s"] * ds).sum())
    b = R.layernorm_backward(p["s"], dout, p["gamma"], ds, 1e-3)
    for name, grad in (("s", "dx"), ("gamma", "dgamma"), ("beta", "dbeta")):
        differences(loss, p, name, b[grad][0], (0, 13, 77))


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_plain_conv_against_differences(K, act):
    g = torch.Generator().manual_seed(K)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    off, D = [0, 1, 1, 3, 12], 8
    p = {"x": n(12, D), "w": n(D, K), "bias": n(D), "x0": n(4, K - 1, D)}
    dy, dxT = n(12, D), n(4, K - 1, D)

    def loss(q):
        r = R.conv(q["x"], q["w"], q["bias"], off, act, q["x0"])
        return float((r["y"][0] * dy).sum() + (r["xT"][0] * dxT).sum())

    b = R.conv(p["x"], p["w"], p["bias"], off, act, p["x0"], dy, dxT)
    for name, grad in (("x", "dx"), ("w", "dw"), ("bias", "dbias"), ("x0", "dx0")):
        differences(loss, p, name, b[grad][0], (0, 3, 11, 25, 50, 95))


def test_plain_scan_against_differences():
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    off, D, G, N = [0, 1, 1, 14], 16, 2, 8
    p = {"x": n(14, D), "dt": n(14, D), "A": torch.rand(D, N, generator=g, dtype=torch.float64), "B": n(14, G, N), "C": n(14, G, N),
         "skip": n(D), "bias": n(D), "z": n(14, D), "h0": n(3, D, N)}
    dy, dhT = n(14, D), n(3, D, N)

    def loss(q):
        r = R.scan(q["x"], q["dt"], q["A"], q["B"], q["C"], off, q["skip"], q["bias"], q["z"], q["h0"])
        return float((r["y"][0] * dy).sum() + (r["hT"][0] * dhT).sum())

    b = R.scan(*(p[k] for k in ("x", "dt", "A", "B", "C")), off, p["skip"], p["bias"], p["z"], p["h0"], dy, dhT)
    for name in p:
        differences(loss, p, name, b["d" + name][0], (0, 5, 33, 100))


@pytest.mark.parametrize("name", ["short_conv.cu", "selective_scan.cu"])
def test_waits_for_the_stream_first(name):
    found = list(kernels(name))
    assert len(found) >= 4
    for kernel, body in found:
        at = body.find("wait_for_stream()")
        assert at >= 0, kernel
        for taken in ("tmem_alloc", "__ldg", "offsets_ok", "record_status", "load_states", "raw4", "raw_at"):
            assert taken not in body[:at], (kernel, taken)
