"""A last row that is not finite: what the scan's backward pass sums over the rows in front
of it (dA, the gradient of the initial state) does not hold the state behind that row, and
is finite by its formula, whatever part of a turn of rows the sequence ends in."""
import pytest
import torch

from tests import _more_layers as R

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


@pytest.mark.parametrize("dtype", [sdm.SDM_F32, sdm.SDM_BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("T", [1, 2, 5, 15, 16, 17, 18, 32, 47])
def test_sums_over_rows_in_front(T, gate, N, dtype):
    D, bad = 16, 3                                   # channel 3's last x
    for value in (float("inf"), float("nan")):
        g = torch.Generator().manual_seed(T + N)
        n = lambda *s, std=1.0, mean=0.0: torch.randn(*s, generator=g) * std + mean
        x, dt, z, B, C, dy = (n(T, D), n(T, D, std=0.7), n(T, D), n(T, 1, N), n(T, 1, N), n(T, D))
        x, dt, z, B, C, dy = (t.to(DT[dtype]) for t in (x, dt, z, B, C, dy))
        x[T - 1, bad] = value
        A, h0, dhT = torch.rand(D, N, generator=g) + 0.5, n(1, D, N), n(1, D, N)
        bias = n(D)
        d = lambda t: t.to(DEV)
        sh = sdm.make_selective(1, T, D, N, dtype=dtype)
        ins, kw = [d(t) for t in (x, dt, A, B, C)], dict(bias=d(bias), z=d(z) if gate else None)
        f = sdm.sdm_selective_scan_forward(sh, *ins, h0=d(h0), save_states=True, **kw)
        b = sdm.sdm_selective_scan_backward(sh, *ins, f["states"], d(dy), dhT=d(dhT), **kw)
        assert sdm.sdm_get_device_status() == 0
        ref = R.scan(x, dt, A, B, C, [0, T], None, bias, z if gate else None, h0, dy, dhT)
        assert not torch.isfinite(ref["hT"][0][0, bad]).any() and not torch.isfinite(f["hT"][0, bad]).any()
        for k in ("dA", "dh0"):
            assert torch.isfinite(ref[k][0]).all() and torch.isfinite(ref[k][1]).all()
            R.within(b[k], *ref[k], k)
