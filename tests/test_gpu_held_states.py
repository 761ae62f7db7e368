"""States that are held for long: the gate a = (1 - beta) alpha of closed write
gates (zb far below zero) and slow decays, and logits that cancel their bias.

The bounds, from those of the operations (2^x instruction 4 U, reciprocal 2 U,
each float32 operation U, the logarithm 6.5 U), count what each step is
sensitive to:
  x = za + bias, one sum, then log2(e) (rounded) times it:   3 U |x|
  softplus(x):      (3 |x| + 13) U, relative
  alpha:            (l (3 |x| + 14) + 4) U with l = A softplus(x)
  2^-z, z = zb log2(e):  (2 |zb| + 4) U, of which 1 / (1 + 2^-z) takes the
  part 1 - beta and two operations more:
  beta:             ((1 - beta) (2 |zb| + 4) + 3) U
  1 - beta, zb < 0: beta (2 |zb| + 4) U + 4 U: beta's error is as small as beta
  1 - beta, zb >= 0: beta's error, and an exponent that is rounded twice and
                    summed with l once: ((1 - beta) (2 |zb| + 4) + 3 + 3 |zb| + l) U
So nothing grows with |zb| where the gate is closed.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

sdm = pytest.importorskip("sparse_state_linear_gb300")
DEV = "cuda:0"
U = 2.0 ** -24
DT = {sdm.SDM_F32: torch.float32, sdm.SDM_BF16: torch.bfloat16}
BOTH = pytest.mark.parametrize("dtype", [sdm.SDM_F32, sdm.SDM_BF16], ids=["f32", "bf16"])
CLOSED = [-4.0, -12.0, -16.0, -23.0, -30.0, -40.0, -55.0, -63.0, -80.0, -86.0, -120.0]


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sdm.lib()
    assert sdm.sdm_get_device_status() == 0


def gates(za, zb, A, bias):
    """alpha, beta, a, softplus, sigmoid(za + bias) in 64 bits and the relative errors of a, beta, softplus, sigmoid."""
    x = za.double() + bias.double()
    zb, A = zb.double(), A.double()
    sp = torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))
    lam = A * sp
    alpha, beta, keep = torch.exp(-lam), torch.sigmoid(zb), torch.sigmoid(-zb)
    e_alpha = (lam * (3 * x.abs() + 14) + 4) * U
    e_beta = (keep * (2 * zb.abs() + 4) + 3) * U
    e_keep = torch.where(zb < 0, (beta * (2 * zb.abs() + 4) + 4) * U, e_beta + (3 * zb.abs() + lam) * U)
    return (alpha, beta, keep * alpha, sp, torch.sigmoid(x),
            e_keep + e_alpha + U, e_beta, (3 * x.abs() + 13) * U, (6 * x.abs() + 12) * U)


def slow(D, seed=0):
    """za, A and bias of D channels: decays l of 1e-6 to 0.5 a row."""
    g = torch.Generator().manual_seed(seed)
    r = lambda: torch.rand(D, generator=g)
    step = torch.exp(r() * 11.0 - 13.8)
    return torch.randn(D, generator=g).bfloat16().float() * 0.5, r() * 15 + 1, torch.log(torch.expm1(step))


def cancelling(D, seed=0):
    """x = za + bias of a few units from za and bias of some hundreds, exactly."""
    g = torch.Generator().manual_seed(seed)
    x = torch.round((torch.rand(D, generator=g) * 10 - 6) * 1024) / 1024
    bias = torch.round((torch.rand(D, generator=g) - 0.5) * 1500)
    return x - bias, torch.rand(D, generator=g) * 7 + 1, bias


def near(got, want, rel, what):
    got, want = got.detach().cpu().double(), want.double()
    lim = rel * want.abs() + torch.finfo(torch.float32).tiny
    bad = ~((got - want).abs() <= lim)
    assert not bad.any(), (what, int(bad.sum()), float(((got - want).abs() / lim)[bad].max()), torch.nonzero(bad)[:4].tolist())


@pytest.mark.parametrize("inputs", [slow, cancelling])
def test_one_row_is_its_gate(inputs):
    # No input, one row: the state behind it, and the gradient in front of it, is
    # a times what it was.
    D, rows = 2048, len(CLOSED) + 3
    za, A, bias = inputs(D)
    za = za.repeat(rows, 1)
    zb = torch.tensor(CLOSED + [0.0, 2.0, 9.0])[:, None].repeat(1, D)
    alpha, beta, a, sp, sig, e_a, e_beta, e_sp, e_sig = gates(za, zb, A, bias)
    g = torch.Generator().manual_seed(5)
    h0, dhT = torch.randn(rows, D, generator=g), torch.randn(rows, D, generator=g)
    t = [z.to(DEV) for z in (za, zb, torch.zeros(rows, D))]
    kw = dict(A=A.to(DEV), bias=bias.to(DEV))
    sh = sdm.make_recurrence(rows, rows, D, dtype=sdm.SDM_F32)
    f = sdm.sdm_recurrence_forward(sh, *t, h0=h0.to(DEV), save_states=True, **kw)
    near(f["y"], a * h0.double(), e_a + U, "y")
    assert torch.equal(f["y"], f["hT"])
    b = sdm.sdm_recurrence_backward(sh, *t, f["states"], torch.zeros(rows, D, device=DEV), dhT=dhT.to(DEV), **kw)
    near(b["dh0"], a * dhT.double(), e_a + U, "dh0")
    state = h0.to(DEV)
    y = sdm.sdm_recurrence_step(sh, *t, state, **kw)
    near(y, a * h0.double(), e_a + U, "step")
    assert torch.equal(y, state)
    # One row alone: its share of the gradients of A and bias.
    one = sdm.make_recurrence(1, 1, D, dtype=sdm.SDM_F32)
    for i in (0, 5, rows - 2):
        r = [z[i:i + 1].contiguous() for z in t]
        s = sdm.sdm_recurrence_forward(one, *r, h0=h0[i:i + 1].to(DEV), save_states=True, **kw)["states"]
        b = sdm.sdm_recurrence_backward(one, *r, s, torch.zeros(1, D, device=DEV), dhT=dhT[i:i + 1].to(DEV), **kw)
        dlog = a[i] * h0[i].double() * dhT[i].double()
        near(b["dA"], -sp[i] * dlog, e_a[i] + e_sp[i] + 5 * U, "dA")
        near(b["dbias"], -A.double() * sig[i] * dlog, e_a[i] + e_sig[i] + 5 * U, "dbias")
    assert sdm.sdm_get_device_status() == 0


@BOTH
def test_held_for_thousands_of_rows(dtype):
    # Closed gates in steady state: an error of a is the same every row and adds up.
    T, D = 6001, 64 * len(CLOSED)
    za, A, bias = slow(D, seed=3)
    A = A.clamp(max=2.0)
    bias = bias - 5.0                                # l of 1e-8 to 1e-2
    za, bias, A = za.to(DT[dtype]).float(), bias, A
    zb = torch.tensor(CLOSED).repeat(64)
    alpha, beta, a, *_, e_a, e_beta, _, _ = gates(za, zb, A, bias)
    g = torch.Generator().manual_seed(9)
    v = torch.randn(T, D, generator=g).to(DT[dtype])
    h = torch.randn(D, generator=g).double()
    h0, M, E = h.float(), h.float().abs().double(), torch.zeros(D, dtype=torch.float64)
    h = h0.double()
    y, Ey = torch.empty(T, D, dtype=torch.float64), torch.empty(T, D, dtype=torch.float64)
    for t in range(T):
        b = beta * v[t].double()
        # A product, a sum, and the composition of pairs: four roundings a row at most.
        E = a * E + (e_a + 4 * U) * a * M + (e_beta + 4 * U) * b.abs()
        h, M = a * h + b, a * M + b.abs()
        y[t], Ey[t] = h, E
    t = [za.to(DT[dtype]).repeat(T, 1).to(DEV), zb.to(DT[dtype]).repeat(T, 1).to(DEV), v.to(DEV)]
    kw = dict(A=A.to(DEV), bias=bias.to(DEV))
    sh = sdm.make_recurrence(1, T, D, dtype=dtype)
    f = sdm.sdm_recurrence_forward(sh, *t, h0=h0[None].to(DEV), save_states=True, **kw)
    tiny = 1e-37 * T                                 # a beta below float32's range counts as zero
    assert ((f["hT"][0].cpu().double() - y[-1]).abs() <= Ey[-1] + tiny).all()
    half = torch.finfo(DT[dtype]).eps / 2
    assert ((f["y"].cpu().double() - y).abs() <= Ey + half * (y.abs() + Ey) + tiny).all()
    # The gradient of the initial state is the product of all the gates.
    b = sdm.sdm_recurrence_backward(sh, *t, f["states"], torch.zeros(T, D, dtype=DT[dtype], device=DEV), dhT=torch.ones(1, D, device=DEV), **kw)
    want = torch.exp(T * torch.log(a))
    assert ((b["dh0"][0].cpu().double() - want).abs() <= T * (e_a + 4 * U) * want + tiny).all()
    # And token by token.
    state, one = h0[None].to(DEV), sdm.make_recurrence(1, 1, D, dtype=dtype)
    for k in range(2000):
        sdm.sdm_recurrence_step(one, *(z[k:k + 1] for z in t), state, **kw)
    assert ((state[0].cpu().double() - y[1999]).abs() <= Ey[1999] + tiny).all()
    assert sdm.sdm_get_device_status() == 0


def test_gates_at_the_ends_of_the_range():
    # Logits at which 2^-z is infinite or zero: beta is 0 or 1 and nothing is NaN.
    vals = [-float("inf"), -3e38, -200.0, -128.0, -88.0, 88.0, 128.0, 200.0, 3e38, float("inf")]
    zb = torch.tensor(vals)[:, None].repeat(1, 64).to(DEV)
    rows = len(vals)
    za, v, h0 = torch.full((rows, 64), -2.0, device=DEV), torch.full((rows, 64), 3.0, device=DEV), torch.full((rows, 64), 5.0, device=DEV)
    sh = sdm.make_recurrence(rows, rows, 64, dtype=sdm.SDM_F32)
    f = sdm.sdm_recurrence_forward(sh, za, zb, v, h0=h0, save_states=True)
    alpha = torch.exp(-torch.nn.functional.softplus(torch.tensor(-2.0, dtype=torch.float64)))
    for y in (f["y"], sdm.sdm_recurrence_step(sh, za, zb, v, h0.clone())):
        near(y[:5], torch.full((5, 64), float(alpha) * 5), torch.tensor(40 * U), "closed")
        assert (y[5:] == 3).all()
    one = torch.ones(rows, 64, device=DEV)
    b = sdm.sdm_recurrence_backward(sh, za, zb, v, f["states"], one, **{})
    near(b["dh0"][:5], torch.full((5, 64), float(alpha)), torch.tensor(40 * U), "dh0")
    assert (b["dv"][5:] == 1).all() and (b["dv"][:5].abs() < 1e-37).all()
    for k in ("dza", "dzb", "dv", "dh0"):
        assert torch.isfinite(b[k]).all(), k
    assert (b["dh0"][6:] < 1e-37).all() and (b["dzb"].abs() < 1e-36).all()
