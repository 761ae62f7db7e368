"""The layer norm's gradients of a gain and an offset: each is made where it, or what it
belongs to, was given."""
import pytest
import torch

from tests import _more_layers as R

pytestmark = pytest.mark.gpu

sdm = pytest.importorskip("sparse_state_linear_gb300")
DEV = "cuda:0"
DT = {sdm.SDM_F32: torch.float32, sdm.SDM_BF16: torch.bfloat16}
BOTH = pytest.mark.parametrize("dtype", [sdm.SDM_F32, sdm.SDM_BF16], ids=["f32", "bf16"])


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sdm.lib()
    assert sdm.sdm_get_device_status() == 0


@BOTH
@pytest.mark.parametrize("rows,D", [(1, 8), (33, 264), (2000, 136)])
def test_gradients_are_made_for_what_was_given(rows, D, dtype):
    g = torch.Generator().manual_seed(rows + D)
    n = lambda *s: torch.randn(*s, generator=g)
    s, dout = n(rows, D).to(DT[dtype]).to(DEV), n(rows, D).to(DT[dtype]).to(DEV)
    gamma, beta = (n(D) + 1).to(DEV), n(D).to(DEV)
    sh = sdm.make_norm(rows, D, dtype=dtype)
    f = sdm.sdm_add_layernorm(sh, s, beta=beta, out_dtype=dtype)
    R.within(f["out"], *R.layernorm(s, None, beta, 1e-5), "out")
    call = lambda gm, **kw: sdm.sdm_add_layernorm_backward(sh, s, dout, gm, **kw)
    for gm in (None, gamma):
        ref = R.layernorm_backward(s, dout, gm, None, 1e-5)
        b = call(gm, beta=beta)
        R.within(b["dx"], *ref["dx"], "dx")
        R.within(b["dbeta"], *ref["dbeta"], "dbeta")
        assert (b["dgamma"] is None) == (gm is None)
        if gm is not None:
            R.within(b["dgamma"], *ref["dgamma"], "dgamma")
            both = call(gm)
            assert all(torch.equal(both[k], b[k]) for k in b)
    given = torch.full((D,), 3.0, device=DEV)
    b = call(None, beta=beta, dbeta=given)
    assert b["dbeta"] is given
    R.within(given, *R.layernorm_backward(s, dout, None, None, 1e-5)["dbeta"], "dbeta")
    none = call(None)
    assert none["dgamma"] is None and none["dbeta"] is None and torch.equal(none["dx"], b["dx"])
