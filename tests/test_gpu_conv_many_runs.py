"""The short convolution where there are more runs of rows than warps: a run has 65536
rows at most, so that a warp of the backward pass takes a second one only where rows are
many and channels so many that a block walks all rows of its 128.  x and dy are one
tensor of 7.8 G elements whose channels repeat, so that eight of them stand for all."""
import pytest
import torch

from tests import _more_layers as R

pytestmark = pytest.mark.gpu

sdm = pytest.importorskip("sparse_state_linear_gb300")
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("too little device memory")
    sdm.lib()
    assert sdm.sdm_get_device_status() == 0


def same_channels(t, width):
    """Whether every `width` channels of t [rows, D] hold the same."""
    for a in range(0, t.shape[0], 16384):
        part = t[a:a + 16384].unflatten(1, (-1, width))
        if not torch.equal(part, part[:, :1].expand_as(part)):
            return False
    return True


def test_a_warp_takes_a_second_run():
    K, width, most = 4, 8, 65536
    lens = [100000, 1, 0, 2 * most - 3, 30000, 2, 7000]
    off = [3]
    for n in lens:
        off.append(off[-1] + n)
    rows, n_seq = off[-1] + 2, len(lens)
    D = 128 * (3 * torch.cuda.get_device_properties(0).multi_processor_count // 2 + 1)
    assert rows > 4 * most                           # four warps a block, one block for 128 channels
    g = torch.Generator().manual_seed(1)
    n = lambda *s, std=1.0, mean=0.0: torch.randn(*s, generator=g) * std + mean
    # The rows of second runs are larger, so that without them the sums would be others.
    x, x0, dxT = (t.bfloat16() for t in (n(rows, width, mean=0.5), n(n_seq, K - 1, width), n(n_seq, K - 1, width)))
    x[4 * most:] += 16
    w, bias = n(width, K, std=0.6), n(width, std=0.3)
    wide = lambda t, dim: t.to(DEV).repeat(*[D // width if i == dim else 1 for i in range(t.dim())])
    sh = sdm.make_conv(n_seq, rows, D, taps=K)
    at = dict(bias=wide(bias, 0), offsets=torch.tensor(off, dtype=torch.int32, device=DEV), x0=wide(x0, 2))
    big, ws = wide(x, 1), wide(w, 0)
    ref = R.conv(x, w, bias, off, sdm.SDM_ACT_SILU, x0, x, dxT)
    inside = slice(off[0], off[-1])
    out = torch.full((rows, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    f = sdm.sdm_short_conv_forward(sh, big, ws, y=out, **at)
    assert same_channels(out[inside], width)
    R.within(out[inside, :width], ref["y"][0][inside], ref["y"][1][inside], "y")
    assert torch.isnan(out[:off[0]]).all() and torch.isnan(out[off[-1]:]).all()
    assert torch.equal(f["xT"][:, :, :width].cpu().double(), ref["xT"][0]) and same_channels(f["xT"].flatten(0, 1), width)
    out.fill_(float("nan"))
    b = sdm.sdm_short_conv_backward(sh, big, ws, big, dxT=wide(dxT, 2), dx=out, **at)
    assert sdm.sdm_get_device_status() == 0
    assert same_channels(out[inside], width)
    R.within(out[inside, :width], ref["dx"][0][inside], ref["dx"][1][inside], "dx")
    assert torch.isnan(out[:off[0]]).all() and torch.isnan(out[off[-1]:]).all()
    assert same_channels(b["dx0"].flatten(0, 1), width)
    R.within(b["dx0"][:, :, :width], *ref["dx0"], "dx0")
    second = R.conv(x[4 * most:off[-1]], w, bias, [0, off[-1] - 4 * most], sdm.SDM_ACT_SILU, None, x[4 * most:off[-1]])
    for k in ("dw", "dbias"):
        t = b[k].view(-1, width, *b[k].shape[1:])
        assert torch.equal(t, t[:1].expand_as(t)), k
        assert (second[k][0].abs() > 2 * ref[k][1]).float().mean() >= 0.5, k
        R.within(t[0], *ref[k], k)
