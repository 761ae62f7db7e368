"""The selective state space scan on the GPU against its plain 64-bit form
(tests/_more_layers.py, which also derives how far float32 may be off), and a
block of norm, convolution and scan."""
import pytest
import torch

from tests import _layers as P
from tests import _more_layers as R

pytestmark = pytest.mark.gpu

sdm = pytest.importorskip("sparse_state_linear_gb300")
DEV = "cuda:0"
DT = {sdm.SDM_F32: torch.float32, sdm.SDM_BF16: torch.bfloat16}
BOTH = pytest.mark.parametrize("dtype", [sdm.SDM_F32, sdm.SDM_BF16], ids=["f32", "bf16"])
ROWS = ("x", "dt", "z", "B", "C", "dy")


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sdm.lib()
    assert sdm.sdm_get_device_status() == 0


def offsets(*off):
    return torch.tensor(off, dtype=torch.int32, device=DEV)


def starts(lens, first=0):
    return [first + sum(lens[:i]) for i in range(len(lens) + 1)]


def draw(rows, D, n_seq, N, G, dtype, seed=0, pace=1.0):
    """Memories from a few to about a thousand rows (`pace` times as fast)."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0, mean=0.0: torch.randn(*s, generator=g) * std + mean
    step = torch.exp(torch.rand(D, generator=g) * 4.6 - 6.9) * pace
    x = dict(x=n(rows, D), dt=n(rows, D, std=0.7), z=n(rows, D), B=n(rows, G, N), C=n(rows, G, N), dy=n(rows, D))
    x = {k: t.to(DT[dtype]) for k, t in x.items()}
    x.update(A=torch.arange(1, N + 1) * torch.exp(n(D, N, std=0.1)), skip=n(D, mean=1.0, std=0.1), bias=torch.log(torch.expm1(step)),
             h0=n(n_seq, D, N, std=0.5), dhT=n(n_seq, D, N))
    return {k: t.to(DEV) for k, t in x.items()}


def run(x, off, n_seq, dtype, save=True, **kw):
    rows, D = x["x"].shape
    G, N = x["B"].shape[1:]
    sh = sdm.make_selective(n_seq, rows, D, N, groups=G, dtype=dtype)
    ins = [x[k] for k in ("x", "dt", "A", "B", "C")]
    more = dict(skip=x.get("skip"), bias=x.get("bias"), z=x.get("z"), offsets=off)
    f = sdm.sdm_selective_scan_forward(sh, *ins, h0=x.get("h0"), save_states=True, **more, **kw)
    b = sdm.sdm_selective_scan_backward(sh, *ins, f["states"], x["dy"], dhT=x.get("dhT"), **more, **kw)
    return {k: t for k, t in {**f, **b}.items() if k != "states" and t is not None}


def check(x, off, n_seq, dtype):
    rows = x["x"].shape[0]
    got = run(x, off, n_seq, dtype)
    assert sdm.sdm_get_device_status() == 0
    bounds = P.bounds_of(off, n_seq, rows)
    ref = R.scan(*(x[k] for k in ("x", "dt", "A", "B", "C")), bounds, x.get("skip"), x.get("bias"), x.get("z"), x.get("h0"), x["dy"], x.get("dhT"))
    inside = torch.zeros(rows, dtype=torch.bool)
    inside[bounds[0]:bounds[-1]] = True
    for k in ref:
        if k in got:
            R.within(got[k], *ref[k], k, inside if k in ("y", "dx", "ddt", "dz", "dB", "dC") else None)
    return got


@BOTH
@pytest.mark.parametrize("N,G", [(8, 1), (16, 1), (32, 1), (64, 1), (16, 2)])
@pytest.mark.parametrize("lens,D", [([1], 16), ([0, 1, 0], 80), ([15, 16, 17, 33], 144), ([5, 0, 300, 1, 0, 157], 48), ([0], 16)])
def test_packed_sequences(lens, D, N, G, dtype):
    check(draw(sum(lens), D, len(lens), N, G, dtype, seed=len(lens) * 100 + D + N), offsets(*starts(lens)), len(lens), dtype)


@BOTH
@pytest.mark.parametrize("n_seq,T,D,N,G", [(1, 1, 8, 16, 1), (3, 130, 40, 16, 1), (2, 300, 272, 8, 2), (4, 0, 8, 16, 1), (64, 1, 96, 32, 3),
                                           (2, 65, 1032, 16, 1), (1, 64, 64, 64, 8), (2, 96, 600, 16, 1)])
def test_equal_sequences(n_seq, T, D, N, G, dtype):
    check(draw(n_seq * T, D, n_seq, N, G, dtype, seed=T + D), None, n_seq, dtype)


def test_many_chunks_carry_the_state():
    # Long memories over many chunks.
    x = draw(3001, 24, 1, 16, 1, sdm.SDM_F32, seed=2, pace=0.1)
    check(x, None, 1, sdm.SDM_F32)
    check(draw(4001, 16, 2, 8, 1, sdm.SDM_BF16, seed=3), offsets(1, 1700, 4000), 2, sdm.SDM_BF16)


def test_sequences_that_need_no_cutting():
    # As many sequences as fill the GPU, each walked by one block; fast and slow decay.
    for dtype, pace in ((sdm.SDM_F32, 20.0), (sdm.SDM_BF16, 0.2)):
        check(draw(640 * 3, 8, 640, 16, 1, dtype, seed=4, pace=pace), None, 640, dtype)


def test_hundreds_of_short_sequences():
    g = torch.Generator().manual_seed(7)
    lens = torch.randint(0, 4, (701,), generator=g).tolist()
    lens[350] = 400                                  # and a long one among them
    check(draw(sum(lens), 40, 701, 16, 1, sdm.SDM_BF16, seed=61), offsets(*starts(lens)), 701, sdm.SDM_BF16)


@BOTH
def test_without_the_options(dtype):
    x = draw(200, 64, 2, 16, 1, dtype, seed=5)
    for k in ("z", "skip", "bias", "h0", "dhT"):
        del x[k]
    got = check(x, None, 2, dtype)
    assert not {"dz", "dskip", "dbias"} & set(got)


@BOTH
def test_columns_of_wider_tensors(dtype):
    # x beside z in one projection; B and C behind other columns of another.
    rows, D, N, G = 201, 48, 16, 2
    x = draw(rows, D, 2, N, G, dtype, seed=8)
    off = offsets(3, 90, 198)
    fill = lambda w, v: torch.full((rows, w), v, dtype=DT[dtype], device=DEV)
    xd, zz, bc = fill(2 * D + 8, 7.0), fill(2 * D, 7.0), fill(2 * G * N + 24, 7.0)
    xd[:, :D], xd[:, D:2 * D], zz[:, D:] = x["x"], x["dt"], x["z"]
    bc[:, 16:16 + G * N], bc[:, 16 + G * N:16 + 2 * G * N] = x["B"].flatten(1), x["C"].flatten(1)
    gxd, gzz, gbc, y = fill(2 * D + 16, 5.0), fill(3 * D, 5.0), fill(2 * G * N + 8, 5.0), fill(D, 9.0)
    sh = sdm.make_selective(2, rows, D, N, groups=G, dtype=dtype, ld=2 * D + 8, ld_z=2 * D, ld_bc=2 * G * N + 24, ld_grad=2 * D + 16,
                            ld_z_grad=3 * D, ld_bc_grad=2 * G * N + 8)
    B, C = bc[:, 16:16 + G * N], bc[:, 16 + G * N:16 + 2 * G * N].unflatten(1, (G, N))
    ins = (xd[:, :D], xd[:, D:2 * D], x["A"], B, C)
    kw = dict(skip=x["skip"], bias=x["bias"], z=zz[:, D:], offsets=off)
    f = sdm.sdm_selective_scan_forward(sh, *ins, h0=x["h0"], y=y, save_states=True, **kw)
    b = sdm.sdm_selective_scan_backward(sh, *ins, f["states"], x["dy"], dhT=x["dhT"], dx=gxd[:, :D], ddt=gxd[:, D:2 * D],
                                        dB=gbc[:, :G * N], dC=gbc[:, G * N:2 * G * N], dz=gzz[:, D:2 * D], **kw)
    assert sdm.sdm_get_device_status() == 0
    want = run(x, off, 2, dtype)
    for k in ("dx", "ddt", "dz", "dB", "dC"):
        assert torch.equal(b[k][3:198], want[k][3:198].flatten(1)), k
    for k in ("dA", "dskip", "dbias", "dh0"):
        assert torch.equal(b[k], want[k]), k
    assert torch.equal(y[3:198], want["y"][3:198]) and torch.equal(f["hT"], want["hT"])
    # Rows of no sequence and the columns beside stay as they were.
    for t, v, cols in ((y, 9, []), (gxd, 5, [slice(2 * D, None)]), (gzz, 5, [slice(0, D), slice(2 * D, None)]), (gbc, 5, [slice(2 * G * N, None)])):
        assert (t[:3] == v).all() and (t[198:] == v).all() and all((t[:, c] == v).all() for c in cols)


@BOTH
def test_rows_outside_hold_anything(dtype):
    rows, D = 320, 64
    off = offsets(7, 7, 135, 190, 311)
    x = draw(rows, D, 4, 16, 1, dtype, seed=3)
    keep = lambda r: [r[k][7:311] if k in ("y", "dx", "ddt", "dz", "dB", "dC") else r[k] for k in sorted(r)]
    clean = [t.clone() for t in keep(run(x, off, 4, dtype))]
    for k, bad in zip(ROWS, (float("nan"), float("inf"), float("nan"), float("-inf"), float("nan"), float("inf"))):
        x[k][:7] = bad
        x[k][311:] = bad
    for p, q in zip(clean, keep(run(x, off, 4, dtype))):
        assert torch.equal(p, q)


@BOTH
def test_extreme_steps_and_gates(dtype):
    # Time steps that are 0 or huge in float32, gates that are 0 or 1, no decay.
    vals = [-1e30, -120.0, -90.0, -30.0, -1.0, 0.0, 1.0, 30.0, 90.0]
    D = 16
    dt = torch.tensor([a for a in vals for _ in vals]).repeat(D, 1).T.contiguous()
    z = torch.tensor([b for _ in vals for b in vals]).repeat(D, 1).T.contiguous()
    x = draw(dt.shape[0], D, 1, 16, 1, dtype, seed=2)
    x["dt"], x["z"] = dt.to(DT[dtype]).to(DEV), z.to(DT[dtype]).to(DEV)
    x["bias"].zero_()
    x["A"][:, 3] = 0
    check(x, None, 1, dtype)


@BOTH
def test_segments_carry_on_in_place(dtype):
    # Calls with the state in place (hT = h0) are one call on all parts.
    x = draw(512, 64, 1, 16, 1, dtype, seed=11)
    ref = R.scan(*(x[k] for k in ("x", "dt", "A", "B", "C")), [0, 512], x["skip"], x["bias"], x["z"], x["h0"])
    state, ys = x["h0"].clone(), []
    for a, b in ((0, 1), (1, 1), (1, 256), (256, 300), (300, 512)):
        sh = sdm.make_selective(1, b - a, 64, 16, dtype=dtype)
        ys.append(sdm.sdm_selective_scan_forward(sh, x["x"][a:b], x["dt"][a:b], x["A"], x["B"][a:b], x["C"][a:b], skip=x["skip"], bias=x["bias"],
                                                 z=x["z"][a:b], h0=state, hT=state)["y"])
    R.within(torch.cat(ys), *ref["y"], "y")
    R.within(state, *ref["hT"], "hT")


def test_in_place_ends():
    # hT = h0 and dh0 = dhT, with and without chunks.
    for n_seq, T, off in ((2, 500, None), (3, 10, None), (3, 10, offsets(0, 3, 3, 30)), (2, 500, offsets(0, 900, 1000))):
        x = draw(n_seq * T, 40, n_seq, 16, 1, sdm.SDM_F32, seed=12)
        want = run(x, off, n_seq, sdm.SDM_F32)
        sh = sdm.make_selective(n_seq, n_seq * T, 40, 16, dtype=sdm.SDM_F32)
        ins, kw = [x[k] for k in ("x", "dt", "A", "B", "C")], dict(skip=x["skip"], bias=x["bias"], z=x["z"], offsets=off)
        h, d = x["h0"].clone(), x["dhT"].clone()
        f = sdm.sdm_selective_scan_forward(sh, *ins, h0=h, hT=h, save_states=True, **kw)
        b = sdm.sdm_selective_scan_backward(sh, *ins, f["states"], x["dy"], dhT=d, dh0=d, **kw)
        assert torch.equal(f["y"], want["y"]) and torch.equal(h, want["hT"])
        assert all(torch.equal(b[k], want[k]) for k in b)


@pytest.mark.parametrize("off", [(0, 50, 40, 100), (0, 50, 60, 101), (-1, 50, 60, 100), (0, 200, 60, 100)])
def test_bad_offsets_write_nothing(off):
    x = draw(100, 64, 3, 16, 1, sdm.SDM_F32)
    sh = sdm.make_selective(3, 100, 64, 16, dtype=sdm.SDM_F32)
    ins = [x[k] for k in ("x", "dt", "A", "B", "C")]
    states = sdm.sdm_selective_scan_forward(sh, *ins, offsets=offsets(0, 10, 10, 100), save_states=True)["states"]
    three = lambda *s: torch.full(s, 3.0, device=DEV)
    y, hT = three(100, 64), three(3, 64, 16)
    sdm.sdm_selective_scan_forward(sh, *ins, offsets=offsets(*off), y=y, hT=hT)
    assert sdm.sdm_get_device_status() == 5
    outs = dict(dx=three(100, 64), ddt=three(100, 64), dz=three(100, 64), dB=three(100, 1, 16), dC=three(100, 1, 16), dA=three(64, 16),
                dskip=three(64), dbias=three(64), dh0=three(3, 64, 16))
    sdm.sdm_selective_scan_backward(sh, *ins, states, x["dy"], z=x["z"], offsets=offsets(*off), **outs)
    assert sdm.sdm_get_device_status() == 5
    assert all((t == 3).all() for t in (y, hT, *outs.values()))
    check(x, offsets(0, 10, 10, 100), 3, sdm.SDM_F32)


@pytest.mark.parametrize("at,to", [(17, -1), (17, 101), (40, 101), (30, 5), (39, 100)])
def test_bad_offsets_of_many_sequences(at, to):
    good = sorted([0, 100] + [(7 * i) % 100 for i in range(1, 40)])
    off = list(good)
    off[at] = to
    x = draw(100, 64, 40, 16, 1, sdm.SDM_BF16)
    sh = sdm.make_selective(40, 100, 64, 16)
    ins = [x[k] for k in ("x", "dt", "A", "B", "C")]
    states = sdm.sdm_selective_scan_forward(sh, *ins, offsets=offsets(*good), save_states=True)["states"]
    three = lambda *s, dtype=torch.bfloat16: torch.full(s, 3.0, device=DEV, dtype=dtype)
    f32 = dict(dtype=torch.float32)
    y, hT = three(100, 64), three(40, 64, 16, **f32)
    sdm.sdm_selective_scan_forward(sh, *ins, offsets=offsets(*off), y=y, hT=hT)
    bad = off != sorted(off) or off[0] < 0 or off[-1] > 100
    assert bad == (at != 39)
    assert sdm.sdm_get_device_status() == (5 if bad else 0)
    outs = dict(dx=three(100, 64), ddt=three(100, 64), dz=three(100, 64), dB=three(100, 1, 16), dC=three(100, 1, 16), dA=three(64, 16, **f32),
                dskip=three(64, **f32), dbias=three(64, **f32), dh0=three(40, 64, 16, **f32))
    if bad:
        sdm.sdm_selective_scan_backward(sh, *ins, states, x["dy"], z=x["z"], offsets=offsets(*off), **outs)
        assert sdm.sdm_get_device_status() == 5
        assert all((t == 3).all() for t in (y, hT, *outs.values()))
    check(x, offsets(*good), 40, sdm.SDM_BF16)


def test_no_sequences_gives_zero_sums():
    x = draw(8, 64, 1, 16, 1, sdm.SDM_F32)
    sh = sdm.make_selective(0, 8, 64, 16, dtype=sdm.SDM_F32)
    three = lambda *s: torch.full(s, 3.0, device=DEV)
    sums = dict(dA=three(64, 16), dskip=three(64), dbias=three(64))
    dx = three(8, 64)
    sdm.sdm_selective_scan_backward(sh, *(x[k] for k in ("x", "dt", "A", "B", "C")), torch.zeros(16, device=DEV), x["dy"], dx=dx, **sums)
    assert all((t == 0).all() for t in sums.values()) and (dx == 3).all()


# ---------------------------------------------------------------------- step

STATE = ("x", "dt", "A", "B", "C")


@BOTH
@pytest.mark.parametrize("rows,D,N,G,n_slots,z", [(1, 8, 16, 1, 1, True), (5, 72, 8, 1, 9, False), (64, 1920, 16, 1, 96, True),
                                                  (33, 1000, 32, 1, 40, True), (7, 96, 64, 4, 7, True), (9, 272, 16, 2, 30, False)])
def test_step(rows, D, N, G, n_slots, z, dtype):
    x = draw(rows, D, 1, N, G, dtype, seed=rows)
    g = torch.Generator().manual_seed(rows)
    slots = torch.randperm(n_slots, generator=g)[:rows].to(torch.int32)
    state = torch.randn(n_slots, D, N, generator=g)
    dev = state.to(DEV)
    gate = x["z"] if z else None
    sh = sdm.make_selective(1, rows, D, N, groups=G, dtype=dtype)
    y = sdm.sdm_selective_scan_step(sh, *(x[k] for k in STATE), dev, skip=x["skip"], bias=x["bias"], z=gate, slots=slots.to(DEV))
    assert sdm.sdm_get_device_status() == 0
    ref = R.scan(*(x[k] for k in STATE), list(range(rows + 1)), x["skip"], x["bias"], gate, state[slots.long()])
    R.within(y, *ref["y"], "y")
    R.within(dev[slots.long().to(DEV)], *ref["hT"], "state")
    rest = torch.ones(n_slots, dtype=torch.bool)
    rest[slots.long()] = False
    assert torch.equal(dev.cpu()[rest], state[rest])


def step_skips(rows, n_slots, D, slots, code, skipped):
    """Tokens in `skipped` change nothing, the others are as alone."""
    x = draw(rows, D, 1, 8, 1, sdm.SDM_F32, seed=6)
    state0 = torch.randn(n_slots, D, 8, device=DEV)
    state, y = state0.clone(), torch.full((rows, D), 4.0, device=DEV)
    sdm.sdm_selective_scan_step(sdm.make_selective(1, rows, D, 8, dtype=sdm.SDM_F32), *(x[k] for k in STATE), state, z=x["z"], slots=slots, y=y)
    assert sdm.sdm_get_device_status() == code
    ok = torch.ones(rows, dtype=torch.bool, device=DEV)
    ok[skipped] = False
    of = slots[ok].long()
    alone = state0[of].contiguous()
    p = {k: x[k] if k == "A" else x[k][ok].contiguous() for k in (*STATE, "z")}
    want = sdm.sdm_selective_scan_step(sdm.make_selective(1, int(ok.sum()), D, 8, dtype=sdm.SDM_F32), *(p[k] for k in STATE), alone, z=p["z"])
    assert (y[~ok] == 4).all() and torch.equal(y[ok], want)
    expect = state0.clone()
    expect[of] = alone
    assert torch.equal(state, expect)


@pytest.mark.parametrize("slots,code,skipped", [([3, -1, 7, 0, -5, 2], 0, [1, 4]), ([3, 10, 7, 0, 9, 2], 5, [1]), ([3, 1, 3, 0, 9, 3], 6, [2, 5])])
def test_step_padding_bad_and_repeated_slots(slots, code, skipped):
    step_skips(6, 10, 64, torch.tensor(slots, dtype=torch.int32, device=DEV), code, skipped)


@pytest.mark.parametrize("rows", [1030, 140001])
def test_step_on_many_rows_with_repeats(rows):
    g = torch.Generator().manual_seed(rows)
    slots = torch.randperm(rows, generator=g).to(torch.int32)
    again = torch.randperm(rows - 1, generator=g)[:200] + 1
    slots[again] = slots[(again.double() * 0.7).long()]   # the slot of some earlier row
    slots[torch.randperm(rows, generator=g)[:50]] = -1
    seen, skipped = set(), []
    for i, s in enumerate(slots.tolist()):
        if s < 0 or s in seen:
            skipped.append(i)
        seen.add(s)
    assert len(skipped) > 100
    step_skips(rows, rows, 8, slots.to(DEV), 6, skipped)


# ------------------------------------------------- streams, graphs, addresses

def test_repeats_streams_and_graph():
    lens = [300, 0, 600, 3]
    x = draw(903, 72, 4, 16, 1, sdm.SDM_BF16, seed=41)
    off = offsets(*starts(lens))
    all_of = lambda **kw: [t for _, t in sorted(run(x, off, 4, sdm.SDM_BF16, **kw).items())]
    want = [t.clone() for t in all_of()]
    for _ in range(5):
        assert all(torch.equal(p, q) for p, q in zip(want, all_of()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = all_of(stream=stream)
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, got))
    sh = sdm.make_selective(4, 903, 72, 16)
    ws = torch.full((sdm.sdm_selective_scan_backward_workspace_size(sh),), 255, dtype=torch.uint8, device=DEV)
    assert all(torch.equal(p, q) for p, q in zip(want, all_of(workspace=ws)))     # whatever it held
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_of(workspace=ws)
    for seed in (41, 42):
        for k, t in draw(903, 72, 4, 16, 1, sdm.SDM_BF16, seed=seed).items():
            x[k].copy_(t)
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(all_of(), got))
    assert sdm.sdm_get_device_status() == 0


def test_two_calls_at_once():
    cases = [draw(3000, 264, 2, 16, 1, sdm.SDM_BF16, seed=s) for s in (1, 2)]
    want = [run(x, None, 2, sdm.SDM_BF16) for x in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [run(x, None, 2, sdm.SDM_BF16, stream=s) for x, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for p, q in zip(want, got):
            assert all(torch.equal(p[k], q[k]) for k in p)


def test_beside_the_recurrence():
    # Both take tensor memory: at once on two streams.
    x = draw(3000, 264, 2, 16, 1, sdm.SDM_BF16, seed=1)
    want = run(x, None, 2, sdm.SDM_BF16)
    rec = sdm.make_recurrence(2, 3000, 264)
    call = lambda **kw: sdm.sdm_recurrence_forward(rec, x["x"], x["dt"], x["z"], **kw)["y"]
    y = call()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        a, b = run(x, None, 2, sdm.SDM_BF16, stream=streams[0]), call(stream=streams[1])
        torch.cuda.synchronize()
        assert torch.equal(b, y) and all(torch.equal(a[k], want[k]) for k in a)
    assert sdm.sdm_get_device_status() == 0


def test_elements_beyond_32_bits():
    rows, D, N, ld = 66000, 8, 8, 65536
    wide = torch.empty(rows * ld, dtype=torch.bfloat16, device=DEV).view(rows, ld)
    x = draw(rows, D, 1, N, 1, sdm.SDM_BF16, seed=1)
    cols = lambda i: wide[:, i * 8:i * 8 + 8]
    for i, k in enumerate(("x", "dt", "z", "B", "C")):
        cols(i)[:] = x[k].flatten(1)
    want = run(x, None, 1, sdm.SDM_BF16)
    sh = sdm.make_selective(1, rows, D, N, **{k: ld for k in ("ld", "ld_z", "ld_bc", "ld_grad", "ld_z_grad", "ld_bc_grad")})
    ins, kw = (cols(0), cols(1), x["A"], cols(3), cols(4)), dict(skip=x["skip"], bias=x["bias"], z=cols(2))
    f = sdm.sdm_selective_scan_forward(sh, *ins, h0=x["h0"], save_states=True, **kw)
    b = sdm.sdm_selective_scan_backward(sh, *ins, f["states"], x["dy"], dhT=x["dhT"], dx=cols(5), ddt=cols(6), dz=cols(7), dB=cols(8), dC=cols(9), **kw)
    assert torch.equal(f["y"], want["y"]) and torch.equal(f["hT"], want["hT"])
    assert all(torch.equal(b[k].flatten(1), want[k].flatten(1)) for k in ("dx", "ddt", "dz", "dB", "dC", "dA"))


def test_binding_refuses_wrong_tensors():
    x = draw(16, 64, 2, 16, 1, sdm.SDM_BF16)
    sh = sdm.make_selective(2, 16, 64, 16)
    ins = [x[k] for k in STATE]
    swap = lambda i, t: [t if j == i else p for j, p in enumerate(ins)]
    for bad in (lambda: sdm.sdm_selective_scan_forward(sdm.make_selective(2, 16, 64, 16, ld=128), *ins),
                lambda: sdm.sdm_selective_scan_forward(sh, *swap(0, x["x"].float())),
                lambda: sdm.sdm_selective_scan_forward(sh, *swap(1, x["dt"][:15])),
                lambda: sdm.sdm_selective_scan_forward(sh, *swap(2, x["A"][:, :8].contiguous())),
                lambda: sdm.sdm_selective_scan_forward(sh, *swap(3, x["B"][:, :, :8].contiguous())),
                lambda: sdm.sdm_selective_scan_forward(sdm.make_selective(2, 16, 64, 16, ld_bc=32), *ins),
                lambda: sdm.sdm_selective_scan_step(sh, *ins, torch.zeros(16, 64, 8, device=DEV)),
                lambda: sdm.sdm_selective_scan_backward(sdm.make_selective(2, 16, 64, 16, ld_grad=128), *ins, torch.zeros(1 << 16, device=DEV), x["dy"])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sdm.SdmError):                # 16 rows on 15 states without slots
        sdm.sdm_selective_scan_step(sh, *ins, torch.zeros(15, 64, 16, device=DEV))


# ------------------------------------------------------------------ together

def test_block_forward_backward_and_decode():
    """A block as a model stacks it: residual + layer norm, projections (library
    products), the convolution, the scan with its gate; its backward pass; and
    the same tokens one at a time."""
    T, n_seq, d, D, N, f32 = 50, 3, 96, 128, 16, sdm.SDM_F32
    rows = T * n_seq
    g = torch.Generator().manual_seed(0)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(DEV)
    x, res, gamma, beta = rnd(rows, d), rnd(rows, d), rnd(d, std=0.1) + 1, rnd(d, std=0.1)
    Win, Wx = rnd(d, 2 * D, std=d ** -0.5), rnd(D, D + 2 * N, std=D ** -0.5)
    w, cb = rnd(D, 4, std=0.5), rnd(D, std=0.1)
    A, skip, bias = torch.arange(1, N + 1, device=DEV) * torch.ones(D, 1, device=DEV), torch.ones(D, device=DEV), rnd(D, std=0.5) - 3
    mm = lambda a, b: (a.double() @ b.double()).float()
    nsh = sdm.make_norm(rows, d, dtype=f32)
    csh = sdm.make_conv(n_seq, rows, D, dtype=f32, ld=2 * D, ld_grad=2 * D)
    ssh = sdm.make_selective(n_seq, rows, D, N, dtype=f32, ld_z=2 * D, ld_bc=D + 2 * N, ld_z_grad=2 * D, ld_bc_grad=D + 2 * N)
    off = [0, T, 2 * T, 3 * T]
    n = sdm.sdm_add_layernorm(nsh, x, res, gamma, beta, out_dtype=f32)
    R.within(n["out"], *R.layernorm(n["s"], gamma, beta, 1e-5), "norm")
    xz = mm(n["out"], Win)
    c = sdm.sdm_short_conv_forward(csh, xz[:, :D], w, bias=cb)
    R.within(c["y"], *R.conv(xz[:, :D], w, cb, off, 1)["y"], "conv")
    proj = mm(c["y"], Wx)
    dt, B, C = proj[:, :D].contiguous(), proj[:, D:D + N], proj[:, D + N:]
    kw = dict(skip=skip, bias=bias, z=xz[:, D:])
    s = sdm.sdm_selective_scan_forward(ssh, c["y"], dt, A, B, C, save_states=True, **kw)
    dy, ds = rnd(rows, D), rnd(rows, d)
    ref = R.scan(c["y"], dt, A, B[:, None], C[:, None], off, skip, bias, xz[:, D:], None, dy, None)
    R.within(s["y"], *ref["y"], "y")
    # Backward.
    dxz, dproj = torch.empty(rows, 2 * D, device=DEV), torch.empty(rows, D + 2 * N, device=DEV)
    b = sdm.sdm_selective_scan_backward(ssh, c["y"], dt, A, B, C, s["states"], dy, dB=dproj[:, D:D + N], dC=dproj[:, D + N:], dz=dxz[:, D:], **kw)
    for k in ("dx", "ddt", "dz", "dA", "dskip", "dbias", "dh0"):
        R.within(b[k], *ref[k], k)
    for k in ("dB", "dC"):
        R.within(b[k], ref[k][0][:, 0], ref[k][1][:, 0], k)
    dproj[:, :D] = b["ddt"]
    dc = b["dx"] + mm(dproj, Wx.T)
    cbk = sdm.sdm_short_conv_backward(csh, xz[:, :D], w, dc, bias=cb, dx=dxz[:, :D])
    cref = R.conv(xz[:, :D], w, cb, off, 1, None, dc, None)
    for k in ("dx", "dw", "dbias"):
        R.within(cbk[k], *cref[k], k)
    dn = mm(dxz, Win.T)
    nb = sdm.sdm_add_layernorm_backward(nsh, n["s"], dn, gamma, ds=ds)
    nref = R.layernorm_backward(n["s"], dn, gamma, ds, 1e-5)
    for k in nref:
        R.within(nb[k], *nref[k], k)
    assert sdm.sdm_get_device_status() == 0
    # Decode: one token of every sequence per call, windows and states in pools.
    window, pool = torch.zeros(5, 3, D, device=DEV), torch.zeros(5, D, N, device=DEV)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    ys = []
    for t in range(T):
        at = [q * T + t for q in range(n_seq)]
        nt = sdm.sdm_add_layernorm(sdm.make_norm(n_seq, d, dtype=f32), x[at], res[at], gamma, beta, out_dtype=f32)
        assert torch.equal(nt["s"], n["s"][at])
        xzt, pt = xz[at], proj[at]
        ct = sdm.sdm_short_conv_step(sdm.make_conv(1, n_seq, D, dtype=f32, ld=2 * D), xzt[:, :D], w, window, bias=cb, slots=slots)
        assert torch.equal(ct, c["y"][at])
        ys.append(sdm.sdm_selective_scan_step(sdm.make_selective(1, n_seq, D, N, dtype=f32, ld_z=2 * D, ld_bc=D + 2 * N), ct, pt[:, :D].contiguous(), A,
                                              pt[:, D:D + N], pt[:, D + N:], pool, skip=skip, bias=bias, z=xzt[:, D:], slots=slots))
    assert sdm.sdm_get_device_status() == 0
    R.within(torch.stack(ys, 1).reshape(rows, D), *ref["y"], "steps")
    R.within(pool[slots.long()], *ref["hT"], "states")
    assert (pool[[1, 3]] == 0).all() and (window[[1, 3]] == 0).all()
