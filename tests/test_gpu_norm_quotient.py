"""The 8-bit output of the residual RMS-Norm is the quotient that the header
names, rounded once to float32 and once to e4m3: the same norm in float32 gives
n bit for bit, and from it scale and output follow without a tolerance."""
import pytest
import torch

pytestmark = pytest.mark.gpu

sdm = pytest.importorskip("sparse_state_linear_gb300")
DEV = "cuda:0"
DT = {sdm.SDM_F32: torch.float32, sdm.SDM_BF16: torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sdm.lib()
    assert sdm.sdm_get_device_status() == 0


def both(rows, D, dtype, x, residual, gamma, group):
    sh = sdm.make_norm(rows, D, dtype=dtype)
    n = sdm.sdm_add_rmsnorm(sh, x, residual, gamma, out_dtype=sdm.SDM_F32)["out"].cpu()
    r = sdm.sdm_add_rmsnorm(sh, x, residual, gamma, out_dtype=sdm.SDM_E4M3, group=group)
    return n, r["out"].cpu(), r["scale"].cpu()


def quotient(n, group):
    per = n.view(n.shape[0], -1, group or n.shape[1])
    scale = torch.clamp(per.abs().amax(2) / torch.tensor(448.0), min=2.0 ** -126)     # float32 throughout
    return (per / scale[:, :, None]).to(torch.float8_e4m3fn).view(n.shape), scale


@pytest.mark.parametrize("dtype", [sdm.SDM_F32, sdm.SDM_BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,D,group", [(2000, 3840, 128), (900, 1000, 0), (1500, 2080, 32), (64, 1920, 64), (1300, 8200, 0)])
def test_quotient(rows, D, group, dtype):
    g = torch.Generator().manual_seed(rows + D)
    t = lambda std: (torch.randn(rows, D, generator=g) * std).to(DT[dtype]).to(DEV)
    x, residual = t(1.0), t(3.0)
    x[1] *= 1e-4
    gamma = (torch.rand(D, generator=g) + 0.5).to(DEV)
    n, q, scale = both(rows, D, dtype, x, residual, gamma, group)
    want, want_scale = quotient(n, group)
    assert torch.equal(scale.view(want_scale.shape), want_scale)
    assert torch.equal(q.view(torch.uint8), want.view(torch.uint8))


def test_ties_go_to_even():
    # Rows of +-1 with gamma = multiples of a scale that land exactly between two
    # neighbours of e4m3.  n is gamma times one number per row.
    D, rows = 256, 64
    sign = torch.where(torch.rand(rows, D, generator=torch.Generator().manual_seed(1)) < 0.5, -1.0, 1.0)
    mids = torch.tensor([1 + (2 * k + 1) / 16 for k in range(7)])
    for scale in (3.0, 7.0, 11.0, 43.0, 641.0, 1637.0):
        gamma = (mids.repeat(37)[:D] * scale).float()
        gamma[0] = 448 * scale
        n, q, s = both(rows, D, sdm.SDM_F32, sign.to(DEV), None, gamma.to(DEV), 0)
        want, want_scale = quotient(n, 0)
        assert torch.equal(s.view(want_scale.shape), want_scale)
        assert torch.equal(q.view(torch.uint8), want.view(torch.uint8))


def test_scales_at_the_ends_of_the_range():
    # The smallest scale, infinite maxima and NaN.
    D = 128
    x = torch.ones(4, D, device=DEV)
    gamma = torch.ones(D, device=DEV)
    sh = sdm.make_norm(4, D, dtype=sdm.SDM_F32)
    tiny = sdm.sdm_add_rmsnorm(sh, x, None, gamma * 2.0 ** -130, out_dtype=sdm.SDM_E4M3)
    assert (tiny["scale"] == 2.0 ** -126).all()
    assert (tiny["out"].float() == 2.0 ** -4).all()
    gamma[5] = float("inf")                          # n / inf is 0, inf / inf NaN
    r = sdm.sdm_add_rmsnorm(sh, x, None, gamma, out_dtype=sdm.SDM_E4M3)
    assert torch.isinf(r["scale"]).all()
    out = r["out"].float()
    assert torch.isnan(out[:, 5]).all() and (out[:, :5] == 0).all() and (out[:, 6:] == 0).all()
    gamma[5] = float("nan")
    r = sdm.sdm_add_rmsnorm(sh, x, None, gamma, out_dtype=sdm.SDM_E4M3)
    assert torch.isnan(r["scale"]).all() and torch.isnan(r["out"].float()).all()
