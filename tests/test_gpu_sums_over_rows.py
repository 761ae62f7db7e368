"""Gradients that are sums over many rows (dw, dbias of the convolution, dA, dskip, dbias
of the scan, dgamma, dbeta of the layer norm) against bounds that a few missing rows
break: see tests/_pieces.py."""
import pytest
import torch

from tests import _more_layers as R
from tests._pieces import summed, told_apart, tree

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


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def starts(lens, first=0):
    off = [first]
    for n in lens:
        off.append(off[-1] + n)
    return off


def device(x):
    return {k: t.to(DEV) for k, t in x.items()}


def check(got, pieces, depth, names):
    for k in names:
        p = [(*r[k], n) for r, n in pieces]
        assert told_apart(p, depth) > 0.98, (k, told_apart(p, depth))
        R.within(got[k], *summed(p, depth), k)


# --------------------------------------------------------------- convolution

def conv_case(lens, D, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
    rows, m = sum(lens), len(lens)
    x = dict(x=n(rows, D), w=n(D, K, std=0.6), bias=n(D, std=0.3), x0=n(m, K - 1, D), dy=n(rows, D))
    return {k: t if k in ("w", "bias") else t.to(DT[dtype]) for k, t in x.items()}


def conv_pieces(x, lens, act):
    off, out = starts(lens), []
    for s, n in enumerate(lens):
        r = slice(off[s], off[s + 1])
        if n:
            out.append((R.conv(x["x"][r], x["w"], x["bias"], [0, n], act, x["x0"][s:s + 1], x["dy"][r]), n))
    return out


def conv_depth(rows, D, n_sms):
    # A run of rows a warp, four a block, and on a multiprocessor one block at least.
    return tree(-(-rows // (4 * max(1, n_sms // -(-D // 128)))))


@BOTH
@pytest.mark.parametrize("lens,D,K,act", [([31, 0, 40, 1, 33, 64, 2, 57, 3, 100] * 180, 8, 4, sdm.SDM_ACT_SILU),
                                          ([47, 50, 1, 0, 61] * 40, 520, 3, sdm.SDM_ACT_SILU),
                                          ([47, 50, 1, 0, 61] * 80, 136, 2, sdm.SDM_ACT_NONE)])
def test_convolution(lens, D, K, act, dtype):
    x = conv_case(lens, D, K, dtype, D + K)
    d, rows = device(x), sum(lens)
    sh = sdm.make_conv(len(lens), rows, D, taps=K, act=act, dtype=dtype)
    off = torch.tensor(starts(lens), dtype=torch.int32, device=DEV)
    got = sdm.sdm_short_conv_backward(sh, d["x"], d["w"], d["dy"], bias=d["bias"], offsets=off, x0=d["x0"])
    assert sdm.sdm_get_device_status() == 0
    check(got, conv_pieces(x, lens, act), conv_depth(rows, D, sms()), ("dw", "dbias"))


# ---------------------------------------------------------------------- scan

def scan_case(lens, per, N, dtype, seed):
    """One group of `per` channels."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0, mean=0.0: torch.randn(*s, generator=g) * std + mean
    rows, m = sum(lens), len(lens)
    step = torch.exp(torch.rand(per, generator=g) * 4.6 - 6.9)
    x = dict(x=n(rows, per), dt=n(rows, per, std=0.7), z=n(rows, per), B=n(rows, 1, N), C=n(rows, 1, N), dy=n(rows, per))
    x = {k: t.to(DT[dtype]) for k, t in x.items()}
    x.update(A=torch.arange(1, N + 1) * torch.exp(n(per, N, std=0.1)), skip=n(per, mean=1.0, std=0.1), bias=torch.log(torch.expm1(step)),
             h0=n(m, per, N, std=0.5))
    return x


def scan_pieces(x, lens):
    off, out = starts(lens), []
    for s, n in enumerate(lens):
        r = slice(off[s], off[s + 1])
        if n:
            out.append((R.scan(x["x"][r], x["dt"][r], x["A"], x["B"][r], x["C"][r], [0, n], x["skip"], x["bias"], x["z"][r], x["h0"][s:s + 1],
                               x["dy"][r]), n))
    return out


def scan_depth(lens, tiles, n_sms):
    # A block takes its share of the chunks of a tile, whole sequences at most, each of
    # whole turns of 16 rows; on a multiprocessor there is one block at least.
    turns = sum(-(-n // 16) * 16 for n in lens)
    return tree(-(-turns // max(1, n_sms // tiles)) + -(-max(lens) // 16) * 16)


def scan_sums(x, lens, groups, dtype):
    d, rows, (per, N) = device(x), sum(lens), x["A"].shape
    wide = lambda t, dim: torch.cat([t] * groups, dim)
    d = {k: wide(t, 0 if k in ("A", "skip", "bias") else 1) for k, t in d.items()}
    sh = sdm.make_selective(len(lens), rows, per * groups, N, groups=groups, dtype=dtype)
    ins = [d[k] for k in ("x", "dt", "A", "B", "C")]
    kw = dict(skip=d["skip"], bias=d["bias"], z=d["z"], offsets=torch.tensor(starts(lens), dtype=torch.int32, device=DEV))
    f = sdm.sdm_selective_scan_forward(sh, *ins, h0=d["h0"], save_states=True, **kw)
    b = sdm.sdm_selective_scan_backward(sh, *ins, f["states"], d["dy"], **kw)
    assert sdm.sdm_get_device_status() == 0
    # Groups of the same inputs have the same sums.
    for k in ("dA", "dskip", "dbias"):
        t = b[k].view(groups, per, -1)
        assert torch.equal(t, t[:1].expand_as(t)), k
        b[k] = t[0].reshape(x["A" if k == "dA" else "skip"].shape)
    return b


@BOTH
@pytest.mark.parametrize("lens,per,N,groups", [([40, 0, 33, 1, 48, 17] * 60, 24, 16, 1), ([40, 33, 25] * 30, 40, 8, 2),
                                               ([31, 0, 64, 100] * 6, 40, 64, 20), ([100, 77, 0, 16] * 6, 8, 16, 321)])
def test_scan(lens, per, N, groups, dtype):
    x = scan_case(lens, per, N, dtype, per + N)
    tiles = groups * -(-per // (2048 // N))
    check(scan_sums(x, lens, groups, dtype), scan_pieces(x, lens), scan_depth(lens, tiles, sms()), ("dA", "dskip", "dbias"))


# ---------------------------------------------------------------- layer norm

def norm_case(rows, D, dtype):
    g = torch.Generator().manual_seed(rows + D)
    n = lambda *s, mean=0.0: torch.randn(*s, generator=g) + mean
    return dict(s=n(rows, D, mean=0.5).to(DT[dtype]), dout=n(rows, D).to(DT[dtype]), gamma=n(D, mean=1.0))


def norm_pieces(x, size=50):
    rows = x["s"].shape[0]
    cut = [slice(a, min(a + size, rows)) for a in range(0, rows, size)]
    return [(R.layernorm_backward(x["s"][c], x["dout"][c], x["gamma"], None, 1e-5), c.stop - c.start) for c in cut]


def norm_depth(rows, n_sms):
    return tree(-(-rows // n_sms))                   # a row a block at a time, one on a multiprocessor at least


@BOTH
@pytest.mark.parametrize("rows,D", [(20001, 136), (3001, 1160), (2500, 4104)])
def test_layernorm(rows, D, dtype):
    x = norm_case(rows, D, dtype)
    d = device(x)
    got = sdm.sdm_add_layernorm_backward(sdm.make_norm(rows, D, dtype=dtype), d["s"], d["dout"], d["gamma"])
    check(got, norm_pieces(x), norm_depth(rows, sms()), ("dgamma", "dbeta"))
