"""The selective scan where its chunks are of several turns of rows: inputs for the next
rows asked for during a turn, the state (the gradient) handed from turn to turn, states
saved in the middle of a chunk, and chunks that the last rows fill in part.

A chunk is as long as the GPU's places divided by the tiles of channels ask for, so that
long ones need many tiles.  A group of few channels is a tile, or a few, and here groups
repeat: what is compared with the 64-bit form is the first of them, and the others have
to equal it bit for bit.  How long chunks are at least is read off the workspace's size."""
import pytest
import torch

from tests import _layers as P
from tests import _more_layers as R

pytestmark = pytest.mark.gpu

sdm = pytest.importorskip("sparse_state_linear_gb300")
DEV = "cuda:0"
DT = {sdm.SDM_F32: torch.float32, sdm.SDM_BF16: torch.bfloat16}
BOTH = pytest.mark.parametrize("dtype", [sdm.SDM_F32, sdm.SDM_BF16], ids=["f32", "bf16"])
ROWS = ("y", "dx", "ddt", "dz", "dB", "dC")


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sdm.lib()
    assert sdm.sdm_get_device_status() == 0


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def starts(lens, first=0):
    return [first + sum(lens[:i]) for i in range(len(lens) + 1)]


def tiles_of(sh):
    return sh.groups * -(-sh.D // sh.groups // (2048 // sh.N))


def chunks_have(sh, L, backward, places=2):
    """Whether both passes, or the forward pass alone, cut chunks of L rows or more: the
    workspace holds a state and a sum for rows / (rows of a chunk) + n_seq of them.  L is
    a multiple of 16; `places`: blocks of the backward kernel a multiprocessor."""
    up = lambda n: (n + 255) // 256 * 256
    carry = lambda n: up(n * sh.D * sh.N * 4) + up(n * sh.D * 4)
    most = carry(sh.rows // L + sh.n_seq)
    assert most < carry(sh.rows // (L - 16) + sh.n_seq), "rows too few to tell"
    tiles = tiles_of(sh)
    sums = up(max(1, places * sms() // tiles) * sh.D * (sh.N + 2) * 4) + sh.rows * tiles * 2 * sh.N * 4
    if sdm.sdm_selective_scan_workspace_size(sh) > 256 + most:
        return False
    return not backward or sdm.sdm_selective_scan_backward_workspace_size(sh) <= 256 + most + sums


def draw(rows, per, n_seq, N, dtype, seed, pace=1.0):
    """One group: memories from a few to about a thousand rows (`pace` times as fast)."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0, mean=0.0: torch.randn(*s, generator=g) * std + mean
    step = torch.exp(torch.rand(per, generator=g) * 4.6 - 6.9) * pace
    x = dict(x=n(rows, per), dt=n(rows, per, std=0.7), z=n(rows, per), B=n(rows, 1, N), C=n(rows, 1, N), dy=n(rows, per))
    x = {k: t.to(DT[dtype]) for k, t in x.items()}
    x.update(A=torch.arange(1, N + 1) * torch.exp(n(per, N, std=0.1)), skip=n(per, mean=1.0, std=0.1), bias=torch.log(torch.expm1(step)),
             h0=n(n_seq, per, N, std=0.5), dhT=n(n_seq, per, N))
    return x


def repeated(x, groups):
    return {k: torch.cat([t] * groups, 0 if k in ("A", "skip", "bias") else 1).to(DEV) for k, t in x.items()}


def run(x, off, n_seq, N, groups, dtype, **kw):
    rows, D = x["x"].shape
    sh = sdm.make_selective(n_seq, rows, D, N, groups=groups, dtype=dtype)
    ins = [x[k] for k in ("x", "dt", "A", "B", "C")]
    more = dict(skip=x["skip"], bias=x["bias"], z=x.get("z"), offsets=off)
    f = sdm.sdm_selective_scan_forward(sh, *ins, h0=x.get("h0"), save_states=True, **more, **kw)
    b = sdm.sdm_selective_scan_backward(sh, *ins, f["states"], x["dy"], dhT=x.get("dhT"), **more, **kw)
    assert sdm.sdm_get_device_status() == 0
    return sh, {k: t for k, t in {**f, **b}.items() if k != "states" and t is not None}


def check(x, off, n_seq, groups, dtype, L):
    rows, per = x["x"].shape
    N = x["A"].shape[1]
    o = None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV)
    sh, got = run(repeated(x, groups), o, n_seq, N, groups, dtype)
    assert chunks_have(sh, L, True)
    bounds = P.bounds_of(o, n_seq, rows)
    inside = torch.zeros(rows, dtype=torch.bool)
    inside[bounds[0]:bounds[-1]] = True
    ref = R.scan(*(x[k] for k in ("x", "dt", "A", "B", "C")), bounds, x["skip"], x["bias"], x.get("z"), x.get("h0"), x["dy"], x.get("dhT"))
    assert set(ref) == set(got)
    for k, t in got.items():
        t = t[bounds[0]:bounds[-1]] if k in ROWS else t
        if k in ("dA", "dskip", "dbias"):
            t = t.unflatten(0, (groups, -1)).unsqueeze(0)
        else:
            t = t.unflatten(1, (groups, -1))
        assert torch.equal(t, t[:, :1].expand_as(t)), k          # a group like the others
        one = t[:, 0]
        value, bound = ref[k]
        if k in ROWS:
            value, bound = value[inside], bound[inside]
        R.within(one, value, bound, k)
    return got


# Lengths around chunks of 48 to 176 rows and their turns of 8 and 16; rows in front of
# the first sequence and behind the last.
LENS = [0, 1, 47, 48, 49, 0, 520, 16, 333, 106, 8, 95]


@BOTH
@pytest.mark.parametrize("per,N,groups,L", [(8, 16, 63, 48), (8, 8, 129, 80), (8, 64, 129, 80), (8, 32, 321, 176),
                                            (264, 8, 33, 48), (136, 16, 33, 48), (72, 32, 33, 48), (40, 64, 33, 48)])
def test_packed_sequences(per, N, groups, L, dtype):
    # (More groups than places: a block sums every chunk of its tile.)
    rows = sum(LENS) + 8
    off = starts(LENS, 3)
    check(draw(rows, per, len(LENS), N, dtype, seed=per + N), off, len(LENS), groups, dtype, L)


@BOTH
@pytest.mark.parametrize("n_seq,T,per,N,groups,Lf,Lb", [(3, 701, 8, 16, 63, 64, 32), (1, 1300, 8, 16, 129, 80, 32), (5, 333, 8, 64, 160, 112, 64),
                                                        (1, 1003, 136, 16, 65, 64, 32), (20, 100, 8, 16, 321, 112, 112)])
def test_equal_sequences(n_seq, T, per, N, groups, Lf, Lb, dtype):
    x = draw(n_seq * T, per, n_seq, N, dtype, seed=T)
    check(x, None, n_seq, groups, dtype, Lb)
    assert chunks_have(sdm.make_selective(n_seq, n_seq * T, per * groups, N, groups=groups, dtype=dtype), Lf, False)
    # The same sequences packed: chunks of another length.
    check(x, starts([T] * n_seq), n_seq, groups, dtype, Lb)


@BOTH
def test_many_sequences_of_several_turns(dtype):
    # From 32 sequences on the offsets are checked by a kernel of its own.
    lens = [0, 70, 3, 100, 33, 17, 0, 129] * 5
    check(draw(sum(lens) + 5, 8, len(lens), 16, dtype, seed=9), starts(lens, 2), len(lens), 129, dtype, 80)


@BOTH
@pytest.mark.parametrize("off", [None, (0, 500, 1301)])
def test_fast_and_slow_decay(off, dtype):
    n_seq, rows = (2, 1301) if off else (1, 1301)
    for pace in (0.05, 30.0):
        check(draw(rows, 8, n_seq, 16, dtype, seed=21, pace=pace), list(off) if off else None, n_seq, 129, dtype, 32)


@BOTH
def test_without_gate_and_states(dtype):
    x = draw(sum(LENS) + 8, 8, len(LENS), 16, dtype, seed=22)
    for k in ("z", "h0", "dhT"):
        del x[k]
    got = check(x, starts(LENS, 3), len(LENS), 129, dtype, 80)
    assert "dz" not in got


@BOTH
def test_rows_outside_and_repeats(dtype):
    rows, groups = sum(LENS) + 8, 129
    off = torch.tensor(starts(LENS, 3), dtype=torch.int32, device=DEV)
    x = repeated(draw(rows, 8, len(LENS), 16, dtype, seed=23), groups)
    keep = lambda r: {k: t[3:-5] if k in ROWS else t for k, t in r.items()}
    call = lambda **kw: keep(run(x, off, len(LENS), 16, groups, dtype, **kw)[1])
    want = {k: t.clone() for k, t in call().items()}
    sh = sdm.make_selective(len(LENS), rows, 8 * groups, 16, groups=groups, dtype=dtype)
    ws = torch.full((sdm.sdm_selective_scan_backward_workspace_size(sh),), 255, dtype=torch.uint8, device=DEV)
    for k, bad in zip(("x", "dt", "z", "B", "C", "dy"), (float("nan"), float("inf"), float("nan"), float("-inf"), float("nan"), float("inf"))):
        x[k][:3] = bad
        x[k][-5:] = bad
    for kw in ({}, {}, {"workspace": ws}):
        got = call(**kw)
        assert all(torch.equal(want[k], got[k]) for k in want)
