"""Calls of the selective scan and the short convolution at the ends of what they take:
the widest rows, the most sequences, outputs that are left out, inputs that are one
tensor, and captured calls replayed on other offsets."""
import ctypes

import pytest
import torch

from tests import _more_layers as R

pytestmark = pytest.mark.gpu

sdm = pytest.importorskip("sparse_state_linear_gb300")
DEV = "cuda:0"
DT = {sdm.SDM_F32: torch.float32, sdm.SDM_BF16: torch.bfloat16}
BOTH = pytest.mark.parametrize("dtype", [sdm.SDM_F32, sdm.SDM_BF16], ids=["f32", "bf16"])
ROWS = ("y", "dx", "ddt", "dz", "dB", "dC")
WIDEST, WIDTH = 65536, 8                             # channels, and how many of them differ


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sdm.lib()
    assert sdm.sdm_get_device_status() == 0


def offsets(off):
    return torch.tensor(off, dtype=torch.int32, device=DEV)


def starts(lens, first=0):
    off = [first]
    for n in lens:
        off.append(off[-1] + n)
    return off


def scan_inputs(rows, D, n_seq, N, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0, mean=0.0: torch.randn(*s, generator=g) * std + mean
    x = dict(x=n(rows, D), dt=n(rows, D, std=0.7, mean=-1.0), z=n(rows, D), B=n(rows, 1, N), C=n(rows, 1, N), dy=n(rows, D))
    x = {k: t.to(DT[dtype]) for k, t in x.items()}
    x.update(A=torch.arange(1, N + 1) * torch.exp(n(D, N, std=0.1)), skip=n(D, mean=1.0, std=0.1), bias=n(D, std=0.5),
             h0=n(n_seq, D, N, std=0.5), dhT=n(n_seq, D, N))
    return x


def conv_inputs(rows, D, n_seq, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
    x = dict(x=n(rows, D), x0=n(n_seq, K - 1, D), dy=n(rows, D), dxT=n(n_seq, K - 1, D))
    x = {k: t.to(DT[dtype]) for k, t in x.items()}
    x.update(w=n(D, K, std=0.6), bias=n(D, std=0.3))
    return x


AXIS = dict(x=1, dt=1, z=1, dy=1, A=0, skip=0, bias=0, h0=1, dhT=1, w=0, x0=2, dxT=2)


def widened(x, times):
    """Its channels, over and over; what the channels share as it is."""
    return {k: (torch.cat([t] * times, AXIS[k]) if k in AXIS else t).to(DEV) for k, t in x.items()}


def narrowed(t, axis):
    """The first channels of t, which all others have to equal."""
    u = t.unflatten(axis, (-1, WIDTH)).movedim(axis, 0)
    assert torch.equal(u, u[:1].expand_as(u))
    return u[0]


def run_scan(x, off, n_seq, N, dtype):
    rows, D = x["x"].shape
    sh = sdm.make_selective(n_seq, rows, D, N, dtype=dtype)
    ins, kw = [x[k] for k in ("x", "dt", "A", "B", "C")], dict(skip=x["skip"], bias=x["bias"], z=x["z"], offsets=off)
    f = sdm.sdm_selective_scan_forward(sh, *ins, h0=x["h0"], save_states=True, **kw)
    b = sdm.sdm_selective_scan_backward(sh, *ins, f["states"], x["dy"], dhT=x["dhT"], **kw)
    assert sdm.sdm_get_device_status() == 0
    return {k: t for k, t in {**f, **b}.items() if k != "states"}


def run_conv(x, off, n_seq, dtype):
    rows, D = x["x"].shape
    sh = sdm.make_conv(n_seq, rows, D, taps=x["w"].shape[1], dtype=dtype)
    kw = dict(bias=x["bias"], offsets=off, x0=x["x0"])
    f = sdm.sdm_short_conv_forward(sh, x["x"], x["w"], **kw)
    b = sdm.sdm_short_conv_backward(sh, x["x"], x["w"], x["dy"], dxT=x["dxT"], **kw)
    assert sdm.sdm_get_device_status() == 0
    return {**f, **b}


# ------------------------------------------------------------ the widest rows

@BOTH
@pytest.mark.parametrize("N", [8, 64])
def test_widest_scan(N, dtype):
    rows, off = 41, [2, 2, 20, 21, 39]
    x = scan_inputs(rows, WIDTH, 4, N, dtype, seed=N)
    times = WIDEST // WIDTH
    got = run_scan(widened(x, times), offsets(off), 4, N, dtype)
    ref = R.scan(*(x[k] for k in ("x", "dt", "A", "B", "C")), off, x["skip"], x["bias"], x["z"], x["h0"], x["dy"], x["dhT"])
    for k, (value, bound) in ref.items():
        t = got[k][off[0]:off[-1]] if k in ROWS else got[k]
        if k in ROWS:
            value, bound = value[off[0]:off[-1]], bound[off[0]:off[-1]]
        if k in ("dB", "dC"):
            # Sums over the channels: the form's bound counts WIDTH + 64 additions, of the tiles
            # of 2048 / N channels there are WIDEST N / 2048 added in order, and 64 before them.
            more = max(1.0, (WIDEST * N // 2048 + 64) / (WIDTH + 64))
            R.within(t, value * times, bound * times * more, k)
        else:
            R.within(narrowed(t, 0 if k in ("dA", "dskip", "dbias") else 1), value, bound, k)


@BOTH
def test_widest_scan_step(dtype):
    rows, N, times = 5, 64, WIDEST // WIDTH
    x = scan_inputs(rows, WIDTH, rows, N, dtype, seed=3)
    w = widened(x, times)
    slots = torch.tensor([4, 0, -1, 6, 2], dtype=torch.int32)
    ok = slots >= 0
    pool = torch.zeros(7, WIDEST, N, device=DEV)
    pool[slots[ok].long().to(DEV)] = w["h0"][ok.to(DEV)]
    y = torch.full((rows, WIDEST), 3.0, dtype=DT[dtype], device=DEV)
    sdm.sdm_selective_scan_step(sdm.make_selective(1, rows, WIDEST, N, dtype=dtype), *(w[k] for k in ("x", "dt", "A", "B", "C")), pool,
                                skip=w["skip"], bias=w["bias"], z=w["z"], slots=slots.to(DEV), y=y)
    assert sdm.sdm_get_device_status() == 0
    ref = R.scan(*(x[k] for k in ("x", "dt", "A", "B", "C")), list(range(rows + 1)), x["skip"], x["bias"], x["z"], x["h0"])
    R.within(narrowed(y, 1)[ok.to(DEV)], ref["y"][0][ok], ref["y"][1][ok], "y")
    R.within(narrowed(pool, 1)[slots[ok].long().to(DEV)], ref["hT"][0][ok], ref["hT"][1][ok], "state")
    assert (y[~ok.to(DEV)] == 3).all() and (pool[[1, 3, 5]] == 0).all()


@BOTH
def test_widest_convolution(dtype):
    rows, off, K = 41, [2, 2, 20, 21, 39], 4
    x = conv_inputs(rows, WIDTH, 4, K, dtype, seed=5)
    w = widened(x, WIDEST // WIDTH)
    got = run_conv(w, offsets(off), 4, dtype)
    ref = R.conv(x["x"], x["w"], x["bias"], off, 1, x["x0"], x["dy"], x["dxT"])
    axis = dict(y=1, dx=1, xT=2, dx0=2, dw=0, dbias=0)
    for k, (value, bound) in ref.items():
        t = narrowed(got[k][off[0]:off[-1]] if k in ROWS else got[k], axis[k])
        if k in ROWS:
            value, bound = value[off[0]:off[-1]], bound[off[0]:off[-1]]
        R.within(t, value, bound, k)
    # And its single tokens: the first row of every sequence that has one.
    at, has = [2, 20, 21], torch.tensor([1, 2, 3], device=DEV)
    state = w["x0"].clone()
    y = sdm.sdm_short_conv_step(sdm.make_conv(1, 3, WIDEST, dtype=dtype), w["x"][at].contiguous(), w["w"], state, bias=w["bias"], slots=has.int())
    assert sdm.sdm_get_device_status() == 0
    assert torch.equal(y, got["y"][at]) and torch.equal(state[0], w["x0"][0])
    assert torch.equal(state[1:, :-1], w["x0"][1:, 1:]) and torch.equal(state[1:, -1], w["x"][at])


# --------------------------------------------------------- the most sequences

@BOTH
def test_most_sequences_of_the_scan(dtype):
    n_seq, D, N = 65535, 8, 8
    lens = [1] * n_seq
    x = scan_inputs(n_seq, D, n_seq, N, dtype, seed=1)
    dev = {k: t.to(DEV) for k, t in x.items()}
    equal = run_scan(dev, None, n_seq, N, dtype)
    packed = run_scan(dev, offsets(starts(lens)), n_seq, N, dtype)
    for k in ROWS + ("hT", "dh0"):
        assert torch.equal(equal[k], packed[k]), k
    for part in (slice(0, 70), slice(32700, 32770), slice(n_seq - 70, n_seq)):
        ref = R.scan(x["x"][part], x["dt"][part], x["A"], x["B"][part], x["C"][part], list(range(71)), x["skip"], x["bias"], x["z"][part],
                     x["h0"][part], x["dy"][part], x["dhT"][part])
        for k in ROWS + ("hT", "dh0"):
            R.within(packed[k][part], *ref[k], k)
    # None, one or two rows each; those of 70 sequences in the middle.
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(0, 3, (n_seq,), generator=g)
    off = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)])
    rows = int(off[-1])
    x = scan_inputs(rows, D, n_seq, N, dtype, seed=4)
    got = run_scan({k: t.to(DEV) for k, t in x.items()}, off.int().to(DEV), n_seq, N, dtype)
    for a in (0, 40000, n_seq - 70):
        o = off[a:a + 71]
        part, seqs = slice(int(o[0]), int(o[-1])), slice(a, a + 70)
        ref = R.scan(x["x"][part], x["dt"][part], x["A"], x["B"][part], x["C"][part], (o - o[0]).tolist(), x["skip"], x["bias"], x["z"][part],
                     x["h0"][seqs], x["dy"][part], x["dhT"][seqs])
        for k in ROWS + ("hT", "dh0"):
            R.within(got[k][part if k in ROWS else seqs], *ref[k], k)


@BOTH
def test_most_sequences_of_the_convolution(dtype):
    n_seq, D, K = 65535, 8, 4
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(0, 6, (n_seq,), generator=g)
    off = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)])
    rows = int(off[-1])
    x = conv_inputs(rows, D, n_seq, K, dtype, seed=4)
    dev = {k: t.to(DEV) for k, t in x.items()}
    got = run_conv(dev, off.int().to(DEV), n_seq, dtype)
    for a in (0, 40000, n_seq - 200):
        o = off[a:a + 201]
        part, seqs = slice(int(o[0]), int(o[-1])), slice(a, a + 200)
        ref = R.conv(x["x"][part], x["w"], x["bias"], (o - o[0]).tolist(), 1, x["x0"][seqs], x["dy"][part], x["dxT"][seqs])
        for k in ("y", "dx", "xT", "dx0"):
            R.within(got[k][part if k in ROWS else seqs], *ref[k], k)


# ----------------------------------------------------- outputs that are left out

def call(name, sh, *args):
    p = [a if isinstance(a, int) or a is None else a.data_ptr() for a in args]
    rc = getattr(sdm.lib(), name)(ctypes.byref(sh), *p, torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and sdm.sdm_get_device_status() == 0


@pytest.mark.parametrize("n_seq,T,off", [(2, 100, None), (3, 7, None), (2, 100, (0, 30, 200))])
def test_scan_without_some_outputs(n_seq, T, off):
    rows, D, N = n_seq * T, 40, 16
    x = {k: t.to(DEV) for k, t in scan_inputs(rows, D, n_seq, N, sdm.SDM_F32, seed=6).items()}
    o = None if off is None else offsets(off)
    want = run_scan(x, o, n_seq, N, sdm.SDM_F32)
    sh = sdm.make_selective(n_seq, rows, D, N, dtype=sdm.SDM_F32)
    new = lambda t: torch.full_like(t, 3.0)
    buf = lambda n: torch.empty(n, dtype=torch.uint8, device=DEV)
    states, y = buf(sdm.sdm_selective_scan_states_size(sh)), new(x["x"])
    ws, wb = buf(sdm.sdm_selective_scan_workspace_size(sh)), buf(sdm.sdm_selective_scan_backward_workspace_size(sh))
    ins = [x[k] for k in ("x", "dt", "A", "B", "C", "skip", "bias", "z")] + [o]
    for st in (None, states):                        # no final states, with and without saved ones
        y.fill_(3)
        call("sdm_selective_scan_forward", sh, *ins, x["h0"], y, None, st, ws, ws.numel())
        assert torch.equal(y, want["y"])
    for keep in ((), ("dA",), ("dskip",), ("dbias", "dh0")):
        out = {k: new(want[k]) for k in ("dx", "ddt", "dB", "dC", "dz", *keep)}
        call("sdm_selective_scan_backward", sh, *ins, states, x["dy"], x["dhT"],
             *(out.get(k) for k in ("dx", "ddt", "dA", "dB", "dC", "dskip", "dbias", "dz", "dh0")), wb, wb.numel())
        for k, t in out.items():
            assert torch.equal(t, want[k]), (keep, k)


@pytest.mark.parametrize("n_seq,T,off", [(2, 100, None), (3, 2, None), (2, 100, (0, 2, 200))])
def test_convolution_without_some_outputs(n_seq, T, off):
    rows, D, K = n_seq * T, 40, 4
    x = {k: t.to(DEV) for k, t in conv_inputs(rows, D, n_seq, K, sdm.SDM_F32, seed=7).items()}
    o = None if off is None else offsets(off)
    want = run_conv(x, o, n_seq, sdm.SDM_F32)
    sh = sdm.make_conv(n_seq, rows, D, taps=K, dtype=sdm.SDM_F32)
    y = torch.full_like(x["x"], 3.0)
    call("sdm_short_conv_forward", sh, x["x"], x["w"], x["bias"], o, x["x0"], y, None)
    assert torch.equal(y, want["y"])
    ws = torch.empty(sdm.sdm_short_conv_workspace_size(sh), dtype=torch.uint8, device=DEV)
    for keep in ((), ("dw",), ("dbias",), ("dx0",)):
        out = {k: torch.full_like(want[k], 3.0) for k in ("dx", *keep)}
        scratch = (ws, ws.numel()) if {"dw", "dbias"} & set(keep) else (None, 0)
        call("sdm_short_conv_backward", sh, x["x"], x["w"], x["bias"], o, x["x0"], x["dy"], x["dxT"],
             *(out.get(k) for k in ("dx", "dw", "dbias", "dx0")), *scratch)
        for k, t in out.items():
            assert torch.equal(t, want[k]), (keep, k)


# ------------------------------------------------------------- shared inputs

@BOTH
def test_inputs_that_are_one_tensor(dtype):
    x = scan_inputs(150, 40, 2, 16, dtype, seed=8)
    dev = {k: t.to(DEV) for k, t in x.items()}
    one = {**dev, "dt": dev["x"], "z": dev["x"], "dy": dev["x"], "C": dev["B"], "dhT": dev["h0"], "skip": dev["bias"]}
    apart = {k: t.clone() for k, t in one.items()}
    a, b = run_scan(one, None, 2, 16, dtype), run_scan(apart, None, 2, 16, dtype)
    assert all(torch.equal(a[k], b[k]) for k in a)
    x = conv_inputs(150, 40, 2, 4, dtype, seed=9)
    dev = {k: t.to(DEV) for k, t in x.items()}
    one = {**dev, "dy": dev["x"], "dxT": dev["x0"]}
    apart = {k: t.clone() for k, t in one.items()}
    a, b = run_conv(one, None, 2, dtype), run_conv(apart, None, 2, dtype)
    assert all(torch.equal(a[k], b[k]) for k in a)


# ----------------------------------------------- replays on other offsets

@pytest.mark.parametrize("n_seq", [4, 40])
@pytest.mark.parametrize("kind", ["scan", "conv"])
def test_replays_on_other_offsets(kind, n_seq):
    rows, D, N, dtype = 700, 40, 16, sdm.SDM_BF16
    g = torch.Generator().manual_seed(n_seq)
    cut = lambda: torch.cat([torch.tensor([0]), torch.randint(0, rows + 1, (n_seq - 1,), generator=g).sort()[0], torch.tensor([rows])]).int()
    x = {k: t.to(DEV) for k, t in (scan_inputs(rows, D, n_seq, N, dtype, 1) if kind == "scan" else conv_inputs(rows, D, n_seq, 4, dtype, 1)).items()}
    off = cut().to(DEV)
    # (Workspaces and states of their own: what a captured call makes and drops is memory of
    # its graph that a later output of the capture may lie in.)
    if kind == "conv":
        sh = sdm.make_conv(n_seq, rows, D, dtype=dtype)
        sizes = (sdm.sdm_short_conv_workspace_size(sh),)
    else:
        sh = sdm.make_selective(n_seq, rows, D, N, dtype=dtype)
        sizes = (sdm.sdm_selective_scan_workspace_size(sh), sdm.sdm_selective_scan_backward_workspace_size(sh), sdm.sdm_selective_scan_states_size(sh))
    mem = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]

    def run():
        if kind == "conv":
            kw = dict(bias=x["bias"], offsets=off, x0=x["x0"])
            f = sdm.sdm_short_conv_forward(sh, x["x"], x["w"], **kw)
            return {**f, **sdm.sdm_short_conv_backward(sh, x["x"], x["w"], x["dy"], dxT=x["dxT"], workspace=mem[0], **kw)}
        ins, kw = [x[k] for k in ("x", "dt", "A", "B", "C")], dict(skip=x["skip"], bias=x["bias"], z=x["z"], offsets=off)
        states = mem[2].view(torch.float32)
        f = sdm.sdm_selective_scan_forward(sh, *ins, h0=x["h0"], states=states, workspace=mem[0], **kw)
        b = sdm.sdm_selective_scan_backward(sh, *ins, states, x["dy"], dhT=x["dhT"], workspace=mem[1], **kw)
        return {k: t for k, t in {**f, **b}.items() if k != "states"}

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    good = [cut() for _ in range(3)]
    bad = good[0].clone()
    bad[n_seq // 2] = rows + 1
    for o, code in ((good[0], 0), (bad, 5), (good[1], 0), (bad, 5), (good[2], 0)):
        off.copy_(o)
        for t in got.values():
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert sdm.sdm_get_device_status() == code
        if code:
            assert all((t == 3).all() for t in got.values())
        else:
            want = run()
            assert all(torch.equal(got[k], want[k]) for k in want)
