"""Residual addition and RMS-Norm on the GPU against the plain 64-bit form
(tests/_layers.py), and the layer that it makes with the recurrence."""
import pytest
import torch

from tests import _layers as R

pytestmark = pytest.mark.gpu

sdm = pytest.importorskip("sparse_state_linear_gb300")
DEV = "cuda:0"
DT = {sdm.SDM_F32: torch.float32, sdm.SDM_BF16: torch.bfloat16}
BOTH = pytest.mark.parametrize("dtype", [sdm.SDM_F32, sdm.SDM_BF16], ids=["f32", "bf16"])
# Enough rows to fill the GPU (at 8 an SM another form takes over), and fewer.
MANY = [(1301, 512), (1217, 1000), (1300, 2056), (1216, 4104), (1217, 256), (1220, 8200)]
SIZES = [(1, 8), (3, 32), (7, 64), (64, 1920), (5, 1000), (33, 128), (2, 16384), (301, 520), (4, 8200), (9, 4096), (11, 2048)]


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sdm.lib()
    assert sdm.sdm_get_device_status() == 0


def draw(rows, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + rows * 7 + D)
    n = lambda std: (torch.randn(rows, D, generator=g) * std).to(DT[dtype]).to(DEV)
    return dict(x=n(1.0), residual=n(3.0), gamma=(torch.rand(D, generator=g) + 0.5).to(DEV), dout=n(1.0), ds=n(0.5))


@BOTH
@pytest.mark.parametrize("rows,D", SIZES + MANY)
def test_forward(rows, D, dtype):
    x = draw(rows, D, dtype)
    sh = sdm.make_norm(rows, D, dtype=dtype)
    for residual, gamma, out_dtype in ((True, True, dtype), (False, True, sdm.SDM_F32), (True, False, sdm.SDM_BF16), (False, False, dtype)):
        res, gm = x["residual"] if residual else None, x["gamma"] if gamma else None
        r = sdm.sdm_add_rmsnorm(sh, x["x"], res, gm, eps=1e-5, out_dtype=out_dtype)
        s = R.norm_sum(x["x"], res)
        assert r["scale"] is None and r["out"].dtype == DT[out_dtype]
        if residual:
            assert torch.equal(r["s"], s)
        else:
            assert r["s"] is None
        y, E, _ = R.rmsnorm(s, gm, 1e-5)
        R.within(r["out"], y, E, "out")


def check_quantised(r, y, E, group):
    rows, D = y.shape
    per = y.reshape(rows, -1, group or D)
    Eper = E.reshape(per.shape)
    scale = r["scale"].cpu().double().reshape(rows, -1)
    want = torch.clamp(per.abs().amax(2) / 448, min=2.0 ** -126)
    lim = Eper.amax(2) / 448 + 4 * R.U * want
    assert ((scale - want).abs() <= lim).all()
    # Half a step of e4m3 (2^-4 of the value; 2^-10 of a scale below 2^-6 of one).
    q = r["out"].cpu().float().double().reshape(per.shape) * scale[:, :, None]
    off = (q - per).abs()
    lim = 2.0 ** -4 * (per.abs() + Eper) + 2.0 ** -10 * scale[:, :, None] + 2 * Eper + 8 * R.U * per.abs()
    assert (off <= lim).all(), float((off - lim).max())
    # The largest of each group is 448 (its scale's rounding apart).
    top = r["out"].cpu().float().abs().reshape(per.shape).amax(2)
    assert ((top == 448) | (want <= 2.0 ** -126)).all()


@BOTH
@pytest.mark.parametrize("rows,D,group", [(1, 8, 0), (64, 1920, 0), (64, 1920, 128), (5, 1000, 0), (33, 96, 32), (7, 4160, 64),
                                          (2, 16384, 128), (301, 512, 32), (9, 8200, 0), (3, 128, 128), (6, 2112, 64),
                                          (1217, 1000, 0), (1301, 512, 128), (1300, 2112, 32), (1216, 4096, 64), (1217, 8200, 0)])
def test_eight_bits(rows, D, group, dtype):
    x = draw(rows, D, dtype)
    x["x"][0] *= 1e-3
    if rows > 2:
        x["x"][2], x["residual"][2] = 0, 0           # a row of zeros
    r = sdm.sdm_add_rmsnorm(sdm.make_norm(rows, D, dtype=dtype), x["x"], x["residual"], x["gamma"], out_dtype=sdm.SDM_E4M3, group=group)
    s = R.norm_sum(x["x"], x["residual"])
    assert torch.equal(r["s"], s)
    y, E, _ = R.rmsnorm(s, x["gamma"], 1e-6)
    check_quantised(r, y, E, group)
    if rows > 2:
        assert (r["out"][2].float() == 0).all() and (r["scale"][2] == 2.0 ** -126).all()


def test_extreme_rows():
    # A row with a NaN is NaN throughout; huge and tiny rows; gamma zero in a group.
    D = 256
    x = torch.randn(6, D, device=DEV)
    x[1, 17] = float("nan")
    x[2] *= 1e18
    x[3] *= 1e-30
    x[4, 200] = float("inf")
    gamma = torch.ones(D, device=DEV)
    gamma[128:] = 0
    sh = sdm.make_norm(6, D, dtype=sdm.SDM_F32)
    r = sdm.sdm_add_rmsnorm(sh, x, None, gamma, out_dtype=sdm.SDM_F32)
    q = sdm.sdm_add_rmsnorm(sh, x, None, gamma, out_dtype=sdm.SDM_E4M3, group=128)
    ok = [0, 2, 3, 5]
    y, E, _ = R.rmsnorm(x[ok], gamma, 1e-6)
    R.within(r["out"][ok], y, E, "out")
    check_quantised({"out": q["out"][ok], "scale": q["scale"][ok]}, y, E, 128)
    assert torch.isnan(r["out"][1]).all() and torch.isnan(q["scale"][1]).all() and torch.isnan(q["out"][1].float()).all()
    assert (r["out"][4, :128] == 0).all() and torch.isnan(r["out"][4, 200])       # 1/inf, and inf/inf
    assert torch.isnan(q["scale"][4, 1]) and (q["out"][4, :128].float() == 0).all()


@BOTH
def test_residual_stream_in_place(dtype):
    x = draw(50, 264, dtype)
    sh = sdm.make_norm(50, 264, dtype=dtype)
    want = sdm.sdm_add_rmsnorm(sh, x["x"], x["residual"], x["gamma"], out_dtype=dtype)
    for k in ("residual", "x"):
        y = {n: t.clone() for n, t in x.items()}
        got = sdm.sdm_add_rmsnorm(sh, y["x"], y["residual"], y["gamma"], s=y[k], out_dtype=dtype)
        assert torch.equal(y[k], want["s"]) and torch.equal(got["out"], want["out"])


@BOTH
@pytest.mark.parametrize("rows,D", SIZES + MANY + [(2000, 136)])
def test_backward(rows, D, dtype):
    x = draw(rows, D, dtype, seed=1)
    sh = sdm.make_norm(rows, D, dtype=dtype)
    s = R.norm_sum(x["x"], x["residual"])
    for gamma, ds in ((True, True), (True, False), (False, True)):
        gm, d = x["gamma"] if gamma else None, x["ds"] if ds else None
        b = sdm.sdm_add_rmsnorm_backward(sh, s, x["dout"], gm, ds=d, eps=1e-5, dgamma=torch.empty(D, device=DEV))
        ref = R.rmsnorm_backward(s, x["dout"], gm, d, 1e-5)
        R.within(b["dx"], *ref["dx"], "dx")
        R.within(b["dgamma"], *ref["dgamma"], "dgamma")
    only = sdm.sdm_add_rmsnorm_backward(sh, s, x["dout"], None, ds=x["ds"], eps=1e-5)
    assert only["dgamma"] is None and torch.equal(only["dx"], b["dx"])
    # In place: dx is dout or ds.
    for k in ("dout", "ds"):
        y = {n: t.clone() for n, t in x.items()}
        got = sdm.sdm_add_rmsnorm_backward(sh, s, y["dout"], None, ds=y["ds"], eps=1e-5, dx=y[k], dgamma=torch.empty(D, device=DEV))
        assert torch.equal(y[k], b["dx"]) and torch.equal(got["dgamma"], b["dgamma"])


def test_backward_against_differences():
    rows, D, eps = 5, 24, 1e-3
    x = draw(rows, D, sdm.SDM_F32, seed=3)
    s = R.norm_sum(x["x"], x["residual"]) * 0.1
    b = sdm.sdm_add_rmsnorm_backward(sdm.make_norm(rows, D, dtype=sdm.SDM_F32), s, x["dout"], x["gamma"], ds=x["ds"], eps=eps)
    p = {"s": R.double(s), "gamma": R.double(x["gamma"])}
    dout, ds = R.double(x["dout"]), R.double(x["ds"])
    ref = R.rmsnorm_backward(s, x["dout"], x["gamma"], x["ds"], eps)

    def loss(**over):
        q = {**p, **over}
        return float((R.rmsnorm(q["s"], q["gamma"], eps)[0] * dout).sum() + (q["s"] * ds).sum())

    for name, grad in (("s", "dx"), ("gamma", "dgamma")):
        for i in (0, 13, p[name].numel() - 1):
            est = []
            for h in (1e-3, 5e-4):
                e = torch.zeros(p[name].numel(), dtype=torch.float64)
                e[i] = h
                e = e.reshape(p[name].shape)
                est.append((loss(**{name: p[name] + e}) - loss(**{name: p[name] - e})) / (2 * h))
            best = est[1] + (est[1] - est[0]) / 3
            lim = float(ref[grad][1].flatten()[i]) + abs(est[1] - est[0]) + 1e-9 * (1 + abs(best)) + R.U * abs(best)
            assert abs(float(b[grad].flatten()[i]) - best) <= lim, (name, i)


def test_no_rows():
    sh = sdm.make_norm(0, 64)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    r = sdm.sdm_add_rmsnorm(sh, e, e, None)
    assert r["out"].shape == (0, 64)
    g = sdm.sdm_add_rmsnorm_backward(sh, e, e, torch.ones(64, device=DEV))["dgamma"]
    assert (g == 0).all()


def test_repeats_streams_and_graph():
    x = draw(3001, 1160, sdm.SDM_BF16)
    sh = sdm.make_norm(3001, 1160)

    def run(**kw):
        f = sdm.sdm_add_rmsnorm(sh, x["x"], x["residual"], x["gamma"], out_dtype=sdm.SDM_E4M3, **kw)
        b = sdm.sdm_add_rmsnorm_backward(sh, f["s"], x["dout"], x["gamma"], ds=x["ds"], **kw)
        return [f["s"], f["out"].view(torch.uint8), f["scale"], b["dx"], b["dgamma"]]

    want = run()
    for _ in range(5):
        assert all(torch.equal(p, q) for p, q in zip(want, run()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_binding_refuses_wrong_tensors():
    x = draw(8, 64, sdm.SDM_BF16)
    sh = sdm.make_norm(8, 64)
    with pytest.raises(ValueError):
        sdm.sdm_add_rmsnorm(sh, x["x"].T, x["residual"])
    with pytest.raises(ValueError):
        sdm.sdm_add_rmsnorm(sh, x["x"].float(), x["residual"])
    with pytest.raises(ValueError):
        sdm.sdm_add_rmsnorm(sh, x["x"][:7], x["residual"])
    with pytest.raises(ValueError):
        sdm.sdm_add_rmsnorm(sh, x["x"], x["residual"].cpu())
    with pytest.raises(sdm.SdmError):
        sdm.sdm_add_rmsnorm(sh, x["x"], out_dtype=sdm.SDM_E4M3, group=128)
    with pytest.raises(sdm.SdmError):
        sdm.sdm_add_rmsnorm(sh, x["x"], out_dtype=9)


# ------------------------------------------------------------------ together

def test_layer_forward_backward_and_decode():
    """A recurrent layer as a model stacks it: residual + norm, projections
    (library products), the recurrence, the per-head norm with its gate; its
    backward pass; and the same tokens one at a time."""
    T, n_seq, d, H, dv = 70, 3, 96, 2, 64
    D, rows, f32 = H * dv, 3 * 70, sdm.SDM_F32
    g = torch.Generator().manual_seed(0)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(DEV)
    x, res, gamma = rnd(rows, d), rnd(rows, d), torch.ones(d, device=DEV)
    Wp, A, bias, gate = rnd(d, 3 * D, std=d ** -0.5), torch.ones(D, device=DEV), rnd(D, std=0.1) - 2, rnd(rows, D)
    nsh, rsh = sdm.make_norm(rows, d, dtype=f32), sdm.make_recurrence(n_seq, rows, D, dtype=f32, ld=3 * D, ld_grad=3 * D)
    f = sdm.sdm_add_rmsnorm(nsh, x, res, gamma, out_dtype=f32)
    proj = (f["out"].double() @ Wp.double()).float()
    cols = lambda t: [t[:, i * D:(i + 1) * D] for i in range(3)]
    r = sdm.sdm_recurrence_forward(rsh, *cols(proj), A=A, bias=bias, save_states=True)
    esh = sdm.make_shape(rows, 1, 1, 16, 16, D, 8, 8, in_dtype=f32)
    out = sdm.sdm_rmsnorm_gate(esh, r["y"].view(rows, 1, 1, D), gate.view(rows, 1, 1, D), out_dtype=f32)
    ref = R.recurrence(*cols(proj), A, bias, [0, T, 2 * T, 3 * T], None, rnd(rows, D), None)
    R.within(r["y"], *ref["y"], "y")
    n = R.double(r["y"]) / torch.sqrt(R.double(r["y"]).square().mean(1, keepdim=True) + 1e-6) * R.double(gate)
    assert ((out.cpu().double().view(rows, D) - n).abs() <= 4e-6 * n.abs() + 1e-30).all()
    # Backward: the gradient of y, through the recurrence and the projection to the norm.
    dy, ds = rnd(rows, D), rnd(rows, d)
    dproj = torch.zeros(rows, 3 * D, device=DEV)
    b = sdm.sdm_recurrence_backward(rsh, *cols(proj), r["states"], dy, A=A, bias=bias, **dict(zip(("dza", "dzb", "dv"), cols(dproj))))
    dn = (dproj.double() @ Wp.double().T).float()
    nb = sdm.sdm_add_rmsnorm_backward(nsh, f["s"], dn, gamma, ds=ds)
    ref = R.recurrence(*cols(proj), A, bias, [0, T, 2 * T, 3 * T], None, dy, None)
    for k in ("dza", "dzb", "dv", "dA", "dbias", "dh0"):
        R.within(b[k], *ref[k], k)
    rb = R.rmsnorm_backward(f["s"], dn, gamma, ds, 1e-6)
    R.within(nb["dx"], *rb["dx"], "dx")
    R.within(nb["dgamma"], *rb["dgamma"], "dgamma")
    # Decode: one token of every sequence per call, states in a pool.
    pool = torch.zeros(5, D, device=DEV)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    ssh = sdm.make_recurrence(1, n_seq, D, dtype=f32)
    ys = []
    for t in range(T):
        at = [s * T + t for s in range(n_seq)]
        ft = sdm.sdm_add_rmsnorm(sdm.make_norm(n_seq, d, dtype=f32), x[at], res[at], gamma, out_dtype=f32)
        assert torch.equal(ft["s"], f["s"][at])
        one = [c.contiguous() for c in cols(proj[at])]
        ys.append(sdm.sdm_recurrence_step(ssh, *one, pool, A=A, bias=bias, slots=slots))
    assert sdm.sdm_get_device_status() == 0
    val, err = R.recurrence(*cols(proj), A, bias, [0, T, 2 * T, 3 * T])["y"]
    R.within(torch.stack(ys, 1).reshape(rows, D), val, err, "steps")
    assert (pool[[1, 3]] == 0).all()
