"""Residual addition and layer norm on the GPU against the plain 64-bit form
(tests/_more_layers.py, which also derives how far float32 may be off)."""
import pytest
import torch

from tests import _layers as P
from tests import _more_layers as R

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


def draw(rows, D, dtype, seed=0, mean=0.5):
    g = torch.Generator().manual_seed(seed + rows * 7 + D)
    n = lambda std, m=0.0: (torch.randn(rows, D, generator=g) * std + m).to(DT[dtype]).to(DEV)
    return dict(x=n(1.0), residual=n(3.0, mean), gamma=(torch.rand(D, generator=g) + 0.5).to(DEV),
                beta=(torch.randn(D, generator=g) * 0.3).to(DEV), dout=n(1.0), ds=n(0.5))


@BOTH
@pytest.mark.parametrize("rows,D", SIZES + MANY)
def test_forward(rows, D, dtype):
    x = draw(rows, D, dtype)
    sh = sdm.make_norm(rows, D, dtype=dtype)
    for residual, gamma, beta, out_dtype in ((1, 1, 1, dtype), (0, 1, 0, sdm.SDM_F32), (1, 0, 1, sdm.SDM_BF16), (0, 0, 0, dtype)):
        res, gm, bt = x["residual"] if residual else None, x["gamma"] if gamma else None, x["beta"] if beta else None
        r = sdm.sdm_add_layernorm(sh, x["x"], res, gm, bt, eps=1e-5, out_dtype=out_dtype)
        s = P.norm_sum(x["x"], res)
        assert r["scale"] is None and r["out"].dtype == DT[out_dtype]
        assert torch.equal(r["s"], s) if residual else r["s"] is None
        R.within(r["out"], *R.layernorm(s, gm, bt, 1e-5), "out")


def test_large_means():
    # A mean 1e4 times what differs from it, and one element far from the others.
    x = draw(40, 1000, sdm.SDM_F32, seed=2)
    s = x["x"] * 0.1 + 1e3
    s[20:] = x["x"][20:]
    s[20:, 0] = 1e3
    r = sdm.sdm_add_layernorm(sdm.make_norm(40, 1000, dtype=sdm.SDM_F32), s, None, x["gamma"], x["beta"], out_dtype=sdm.SDM_F32)
    y, E = R.layernorm(s, x["gamma"], x["beta"], 1e-5)
    assert (E[:20] < 1).all()                        # of numbers up to 4: (87 U 1e3 / 0.1) (1 + 1.7 |hat|), so it says something
    R.within(r["out"], y, E, "out")
    b = sdm.sdm_add_layernorm_backward(sdm.make_norm(40, 1000, dtype=sdm.SDM_F32), s, x["dout"], x["gamma"], ds=x["ds"])
    ref = R.layernorm_backward(s, x["dout"], x["gamma"], x["ds"], 1e-5)
    for k in ref:
        R.within(b[k], *ref[k], k)


@BOTH
@pytest.mark.parametrize("rows,D,group", [(1, 8, 0), (64, 1920, 128), (5, 1000, 0), (33, 96, 32), (7, 4160, 64), (2, 16384, 128),
                                          (9, 8200, 0), (3, 128, 128), (1217, 1000, 0), (1301, 512, 128), (1216, 4096, 64)])
def test_eight_bits(rows, D, group, dtype):
    x = draw(rows, D, dtype)
    if rows > 2:
        x["x"][2], x["residual"][2] = 1, 2           # a row of one number: n is beta
    r = sdm.sdm_add_layernorm(sdm.make_norm(rows, D, dtype=dtype), x["x"], x["residual"], x["gamma"], x["beta"], out_dtype=sdm.SDM_E4M3, group=group)
    s = P.norm_sum(x["x"], x["residual"])
    assert torch.equal(r["s"], s)
    y, E = R.layernorm(s, x["gamma"], x["beta"], 1e-5)
    per, Eper = y.reshape(rows, -1, group or D), E.reshape(rows, -1, group or D)
    scale = r["scale"].cpu().double().reshape(rows, -1)
    want = torch.clamp(per.abs().amax(2) / 448, min=2.0 ** -126)
    assert ((scale - want).abs() <= Eper.amax(2) / 448 + 4 * R.U * want).all()
    q = r["out"].cpu().float().double().reshape(per.shape) * scale[:, :, None]
    # Half a step of e4m3 (2^-4 of the value; 2^-10 of a scale below 2^-6 of one).
    lim = 2.0 ** -4 * (per.abs() + Eper) + 2.0 ** -10 * scale[:, :, None] + 2 * Eper + 8 * R.U * per.abs()
    assert ((q - per).abs() <= lim).all()
    assert (r["out"].cpu().float().abs().reshape(per.shape).amax(2) == 448).all()


def test_rows_that_are_not_finite():
    D = 256
    x = torch.randn(5, D, device=DEV)
    x[1, 17] = float("nan")
    x[2, 200] = float("inf")
    x[3] = 0
    sh = sdm.make_norm(5, D, dtype=sdm.SDM_F32)
    r = sdm.sdm_add_layernorm(sh, x, out_dtype=sdm.SDM_F32)
    q = sdm.sdm_add_layernorm(sh, x, out_dtype=sdm.SDM_E4M3, group=128)
    R.within(r["out"][[0, 3, 4]], *R.layernorm(x[[0, 3, 4]], None, None, 1e-5), "out")
    assert torch.isnan(r["out"][1:3]).all() and torch.isnan(q["scale"][1:3]).all() and torch.isnan(q["out"][1:3].float()).all()
    assert (r["out"][3] == 0).all() and (q["out"][3].float() == 0).all()


@BOTH
def test_residual_stream_in_place(dtype):
    x = draw(50, 264, dtype)
    sh = sdm.make_norm(50, 264, dtype=dtype)
    want = sdm.sdm_add_layernorm(sh, x["x"], x["residual"], x["gamma"], x["beta"], out_dtype=dtype)
    for k in ("residual", "x"):
        y = {n: t.clone() for n, t in x.items()}
        got = sdm.sdm_add_layernorm(sh, y["x"], y["residual"], y["gamma"], y["beta"], s=y[k], out_dtype=dtype)
        assert torch.equal(y[k], want["s"]) and torch.equal(got["out"], want["out"])


@BOTH
@pytest.mark.parametrize("rows,D", SIZES + MANY + [(2000, 136)])
def test_backward(rows, D, dtype):
    x = draw(rows, D, dtype, seed=1)
    sh = sdm.make_norm(rows, D, dtype=dtype)
    s = P.norm_sum(x["x"], x["residual"])
    sums = lambda: dict(dgamma=torch.empty(D, device=DEV), dbeta=torch.empty(D, device=DEV))
    for gamma, ds in ((True, True), (True, False), (False, True)):
        gm, d = x["gamma"] if gamma else None, x["ds"] if ds else None
        b = sdm.sdm_add_layernorm_backward(sh, s, x["dout"], gm, ds=d, **sums())
        ref = R.layernorm_backward(s, x["dout"], gm, d, 1e-5)
        for k in ref:
            R.within(b[k], *ref[k], k)
    only = sdm.sdm_add_layernorm_backward(sh, s, x["dout"], None, ds=x["ds"])
    assert only["dgamma"] is None and only["dbeta"] is None and torch.equal(only["dx"], b["dx"])
    for k in ("dgamma", "dbeta"):                    # one of the sums
        one = sdm.sdm_add_layernorm_backward(sh, s, x["dout"], None, ds=x["ds"], **{k: torch.empty(D, device=DEV)})
        assert torch.equal(one[k], b[k]) and torch.equal(one["dx"], b["dx"])
    for k in ("dout", "ds"):                         # in place: dx is dout or ds
        y = {n: t.clone() for n, t in x.items()}
        got = sdm.sdm_add_layernorm_backward(sh, s, y["dout"], None, ds=y["ds"], dx=y[k], **sums())
        assert torch.equal(y[k], b["dx"]) and torch.equal(got["dgamma"], b["dgamma"]) and torch.equal(got["dbeta"], b["dbeta"])


def test_no_rows():
    sh = sdm.make_norm(0, 64)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    assert sdm.sdm_add_layernorm(sh, e, e)["out"].shape == (0, 64)
    b = sdm.sdm_add_layernorm_backward(sh, e, e, torch.ones(64, device=DEV))
    assert (b["dgamma"] == 0).all() and (b["dbeta"] == 0).all()


def test_repeats_streams_and_graph():
    x = draw(3001, 1160, sdm.SDM_BF16)
    sh = sdm.make_norm(3001, 1160)

    def run(**kw):
        f = sdm.sdm_add_layernorm(sh, x["x"], x["residual"], x["gamma"], x["beta"], out_dtype=sdm.SDM_E4M3, **kw)
        b = sdm.sdm_add_layernorm_backward(sh, f["s"], x["dout"], x["gamma"], ds=x["ds"], **kw)
        return [f["s"], f["out"].view(torch.uint8), f["scale"], b["dx"], b["dgamma"], b["dbeta"]]

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
    for bad in (lambda: sdm.sdm_add_layernorm(sh, x["x"].T, x["residual"]), lambda: sdm.sdm_add_layernorm(sh, x["x"].float()),
                lambda: sdm.sdm_add_layernorm(sh, x["x"][:7]), lambda: sdm.sdm_add_layernorm(sh, x["x"], beta=x["beta"][:8]),
                lambda: sdm.sdm_add_layernorm_backward(sh, x["x"], x["dout"], x["gamma"].double())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sdm.SdmError):
        sdm.sdm_add_layernorm(sh, x["x"], out_dtype=sdm.SDM_E4M3, group=128)
