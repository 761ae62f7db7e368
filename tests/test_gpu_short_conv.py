"""The short causal convolution on the GPU against its plain 64-bit form
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
TAPS = pytest.mark.parametrize("K", [2, 3, 4])


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


def draw(rows, D, n_seq, K, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
    x = dict(x=n(rows, D).to(DT[dtype]), w=n(D, K, std=0.6), bias=n(D, std=0.3), x0=n(n_seq, K - 1, D).to(DT[dtype]),
             dy=n(rows, D).to(DT[dtype]), dxT=n(n_seq, K - 1, D).to(DT[dtype]))
    return {k: t.to(DEV) for k, t in x.items()}


def run(x, off, n_seq, dtype, act=sdm.SDM_ACT_SILU, sums=True, **kw):
    rows, D = x["x"].shape
    sh = sdm.make_conv(n_seq, rows, D, taps=x["w"].shape[1], act=act, dtype=dtype)
    f = sdm.sdm_short_conv_forward(sh, x["x"], x["w"], bias=x.get("bias"), offsets=off, x0=x.get("x0"), **kw)
    b = sdm.sdm_short_conv_backward(sh, x["x"], x["w"], x["dy"], bias=x.get("bias"), offsets=off, x0=x.get("x0"), dxT=x.get("dxT"),
                                    dbias=torch.empty(D, device=DEV) if sums else None, **kw)
    return {**f, **b}


def check(x, off, n_seq, dtype, act=sdm.SDM_ACT_SILU):
    rows = x["x"].shape[0]
    got = run(x, off, n_seq, dtype, act)
    assert sdm.sdm_get_device_status() == 0
    bounds = P.bounds_of(off, n_seq, rows)
    ref = R.conv(x["x"], x["w"], x.get("bias"), bounds, act, x.get("x0"), x["dy"], x.get("dxT"))
    inside = torch.zeros(rows, dtype=torch.bool)
    inside[bounds[0]:bounds[-1]] = True
    for k in ref:
        if k == "xT":
            assert torch.equal(got[k].cpu().double(), ref[k][0])
        else:
            R.within(got[k], *ref[k], k, inside if k in ("y", "dx") else None)
    return got


@BOTH
@TAPS
@pytest.mark.parametrize("lens,D", [
    ([1], 8), ([2, 1], 8), ([0, 1, 0], 72), ([3, 2, 1, 0, 4, 5], 136), ([7, 8, 9, 31, 32, 33], 64), ([5, 0, 300, 1, 0, 257], 200),
    ([513], 8), ([0], 16), ([1] * 40, 24), ([0] * 5, 8), ([100, 0, 0, 0], 520),
])
def test_packed_sequences(lens, D, K, dtype):
    check(draw(sum(lens), D, len(lens), K, dtype, seed=len(lens) * 100 + D), offsets(*starts(lens)), len(lens), dtype)


@BOTH
@pytest.mark.parametrize("n_seq,T,D,K", [(1, 1, 8, 4), (3, 130, 40, 4), (2, 700, 64, 3), (4, 0, 8, 4), (64, 1, 96, 2), (2, 128, 1032, 4)])
def test_equal_sequences(n_seq, T, D, K, dtype):
    x = draw(n_seq * T, D, n_seq, K, dtype, seed=T + D)
    check(x, None, n_seq, dtype)
    del x["x0"], x["dxT"]                            # zeros
    check(x, None, n_seq, dtype)


@BOTH
def test_no_activation_and_no_bias(dtype):
    x = draw(300, 64, 3, 4, dtype, seed=5)
    check(x, None, 3, dtype, sdm.SDM_ACT_NONE)
    del x["bias"]
    check(x, offsets(0, 7, 7, 290), 3, dtype, sdm.SDM_ACT_NONE)
    check(x, offsets(0, 7, 7, 290), 3, dtype)
    assert run(x, None, 3, dtype, sums=False)["dbias"] is None


@BOTH
def test_many_runs_a_block(dtype):
    # More runs of rows than the grid has warps, narrow and wide.
    check(draw(60001, 8, 3, 4, dtype, seed=1), offsets(0, 20000, 20001, 59990), 3, dtype)
    check(draw(3000, 3000, 2, 4, dtype, seed=2), offsets(3, 1500, 3000), 2, dtype)


def test_thousands_of_short_sequences():
    g = torch.Generator().manual_seed(7)
    lens = torch.randint(0, 4, (3001,), generator=g).tolist()
    lens[1500] = 700                                 # and a long one among them
    check(draw(sum(lens), 72, 3001, 4, sdm.SDM_BF16, seed=61), offsets(*starts(lens)), 3001, sdm.SDM_BF16)


@BOTH
def test_columns_of_one_projection(dtype):
    rows, D, K = 401, 104, 4
    x = draw(rows, D, 2, K, dtype, seed=8)
    off = offsets(3, 150, 398)
    wide = torch.full((rows, 2 * D + 8), 7.0, dtype=DT[dtype], device=DEV)
    wide[:, 8:8 + D] = x["x"]
    grad = torch.full((rows, 2 * D + 16), 5.0, dtype=DT[dtype], device=DEV)
    sh = sdm.make_conv(2, rows, D, taps=K, dtype=dtype, ld=2 * D + 8, ld_grad=2 * D + 16)
    y = torch.full((rows, D), 9.0, dtype=DT[dtype], device=DEV)
    col, gcol = wide[:, 8:8 + D], grad[:, 16:16 + D]
    f = sdm.sdm_short_conv_forward(sh, col, x["w"], bias=x["bias"], offsets=off, x0=x["x0"], y=y)
    b = sdm.sdm_short_conv_backward(sh, col, x["w"], x["dy"], bias=x["bias"], offsets=off, x0=x["x0"], dxT=x["dxT"], dx=gcol)
    want = run(x, off, 2, dtype)
    assert torch.equal(f["y"][3:398], want["y"][3:398]) and torch.equal(f["xT"], want["xT"])
    for k in ("dw", "dbias", "dx0"):
        assert torch.equal(b[k], want[k]), k
    assert torch.equal(gcol[3:398], want["dx"][3:398])
    # Rows of no sequence and the columns beside stay as they were.
    assert (y[:3] == 9).all() and (y[398:] == 9).all()
    assert (grad[:, :16] == 5).all() and (grad[:, 16 + D:] == 5).all() and (grad[:3] == 5).all() and (grad[398:] == 5).all()


@BOTH
def test_rows_outside_hold_anything(dtype):
    rows, D = 420, 64
    off = offsets(7, 7, 135, 290, 411)
    x = draw(rows, D, 4, 4, dtype, seed=3)
    keep = lambda r: [r["y"][7:411], r["xT"], r["dx"][7:411], r["dw"], r["dbias"], r["dx0"]]
    clean = [t.clone() for t in keep(run(x, off, 4, dtype))]
    for k, bad in (("x", float("nan")), ("dy", float("-inf"))):
        x[k][:7] = bad
        x[k][411:] = bad
    for p, q in zip(clean, keep(run(x, off, 4, dtype))):
        assert torch.equal(p, q)


@BOTH
def test_large_values(dtype):
    # Arguments at which the sigmoid is 0 or 1 in float32.
    x = draw(64, 16, 1, 4, dtype, seed=4)
    x["x"] *= 60
    check(x, None, 1, dtype)
    x["x"] *= 1e3
    check(x, None, 1, dtype)


@BOTH
def test_segments_carry_on_in_place(dtype):
    # Calls with the start in place (xT = x0) are one call on all parts, bit for bit.
    x = draw(512, 264, 1, 4, dtype, seed=11)
    whole = run(x, None, 1, dtype)
    state, ys = x["x0"].clone(), []
    for a, b in ((0, 1), (1, 3), (3, 3), (3, 256), (256, 258), (258, 512)):
        sh = sdm.make_conv(1, b - a, 264, dtype=dtype)
        ys.append(sdm.sdm_short_conv_forward(sh, x["x"][a:b], x["w"], bias=x["bias"], x0=state, xT=state)["y"])
    assert torch.equal(torch.cat(ys), whole["y"]) and torch.equal(state, whole["xT"])
    # And of many sequences at once, of every length around the taps.
    lens = [0, 1, 2, 3, 4, 5, 30, 31, 32, 33, 0, 0, 200, 1, 64, 3] * 40
    x = draw(sum(lens), 72, len(lens), 4, dtype, seed=12)
    off = offsets(*starts(lens))
    want = run(x, off, len(lens), dtype)
    state = x["x0"].clone()
    got = sdm.sdm_short_conv_forward(sdm.make_conv(len(lens), sum(lens), 72, dtype=dtype), x["x"], x["w"], bias=x["bias"], offsets=off,
                                     x0=state, xT=state)
    assert torch.equal(got["y"], want["y"]) and torch.equal(state, want["xT"])


@pytest.mark.parametrize("off", [(0, 50, 40, 100), (0, 50, 60, 101), (-1, 50, 60, 100), (0, 200, 60, 100)])
def test_bad_offsets_write_nothing(off):
    x = draw(100, 64, 3, 4, sdm.SDM_F32)
    sh = sdm.make_conv(3, 100, 64, dtype=sdm.SDM_F32)
    three = lambda *s: torch.full(s, 3.0, device=DEV)
    y, xT = three(100, 64), three(3, 3, 64)
    sdm.sdm_short_conv_forward(sh, x["x"], x["w"], offsets=offsets(*off), x0=x["x0"], y=y, xT=xT)
    assert sdm.sdm_get_device_status() == 5
    outs = dict(dx=three(100, 64), dw=three(64, 4), dbias=three(64), dx0=three(3, 3, 64))
    sdm.sdm_short_conv_backward(sh, x["x"], x["w"], x["dy"], offsets=offsets(*off), x0=x["x0"], **outs)
    assert sdm.sdm_get_device_status() == 5
    assert all((t == 3).all() for t in (y, xT, *outs.values()))
    check(x, offsets(0, 10, 10, 100), 3, sdm.SDM_F32)


def test_no_sequences_gives_zero_sums():
    x = draw(8, 64, 1, 4, sdm.SDM_F32)
    three = lambda *s: torch.full(s, 3.0, device=DEV)
    dw, db, y = three(64, 4), three(64), three(8, 64)
    sh = sdm.make_conv(0, 8, 64, dtype=sdm.SDM_F32)
    sdm.sdm_short_conv_forward(sh, x["x"], x["w"], y=y)
    sdm.sdm_short_conv_backward(sh, x["x"], x["w"], x["dy"], dx=y, dw=dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all() and (y == 3).all()


# ---------------------------------------------------------------------- step

@BOTH
@TAPS
@pytest.mark.parametrize("rows,D,n_slots,act", [(1, 8, 1, 1), (5, 72, 9, 1), (64, 1920, 96, 1), (33, 1000, 40, 0)])
def test_step(rows, D, n_slots, act, K, dtype):
    x = draw(rows, D, rows, K, dtype, seed=rows)
    g = torch.Generator().manual_seed(rows)
    slots = torch.randperm(n_slots, generator=g)[:rows].to(torch.int32)
    state = torch.randn(n_slots, K - 1, D, generator=g).to(DT[dtype])
    dev = state.to(DEV)
    sh = sdm.make_conv(1, rows, D, taps=K, act=act, dtype=dtype)
    y = sdm.sdm_short_conv_step(sh, x["x"], x["w"], dev, bias=x["bias"], slots=slots.to(DEV))
    assert sdm.sdm_get_device_status() == 0
    ref = R.conv(x["x"], x["w"], x["bias"], list(range(rows + 1)), act, state[slots.long()])
    R.within(y, *ref["y"], "y")
    want = state.clone().double()
    want[slots.long()] = ref["xT"][0]
    assert torch.equal(dev.cpu().double(), want)


def test_steps_are_the_forward_pass():
    T, D = 9, 136
    x = draw(3 * T, D, 3, 4, sdm.SDM_BF16, seed=3)
    whole = run(x, None, 3, sdm.SDM_BF16)
    state, at = x["x0"].clone(), torch.arange(3) * T
    sh = sdm.make_conv(1, 3, D)
    ys = [sdm.sdm_short_conv_step(sh, x["x"][at + t].contiguous(), x["w"], state, bias=x["bias"]) for t in range(T)]
    assert torch.equal(torch.stack(ys, 1).reshape(3 * T, D), whole["y"]) and torch.equal(state, whole["xT"])


def step_skips(rows, n_slots, D, slots, code, skipped):
    """Tokens in `skipped` change nothing, the others are as alone."""
    x = draw(rows, D, 1, 4, sdm.SDM_F32, seed=6)
    sh = sdm.make_conv(1, rows, D, dtype=sdm.SDM_F32)
    state0 = torch.randn(n_slots, 3, D, device=DEV)
    state, y = state0.clone(), torch.full((rows, D), 4.0, device=DEV)
    sdm.sdm_short_conv_step(sh, x["x"], x["w"], state, bias=x["bias"], slots=slots, y=y)
    assert sdm.sdm_get_device_status() == code
    ok = torch.ones(rows, dtype=torch.bool, device=DEV)
    ok[skipped] = False
    of = slots[ok].long()
    want = sdm.sdm_short_conv_step(sdm.make_conv(1, int(ok.sum()), D, dtype=sdm.SDM_F32), x["x"][ok].contiguous(), x["w"],
                                   alone := state0[of].contiguous(), bias=x["bias"])
    assert (y[~ok] == 4).all() and torch.equal(y[ok], want)
    expect = state0.clone()
    expect[of] = alone
    assert torch.equal(state, expect)


@pytest.mark.parametrize("slots,code,skipped", [([3, -1, 7, 0, -5, 2], 0, [1, 4]), ([3, 10, 7, 0, 9, 2], 5, [1]), ([3, 1, 3, 0, 9, 3], 6, [2, 5])])
def test_step_padding_bad_and_repeated_slots(slots, code, skipped):
    step_skips(6, 10, 64, torch.tensor(slots, dtype=torch.int32, device=DEV), code, skipped)


@pytest.mark.parametrize("rows", [1030, 20001])
def test_step_on_many_rows_with_repeats(rows):
    g = torch.Generator().manual_seed(rows)
    slots = torch.randperm(rows, generator=g).to(torch.int32)
    again = torch.randperm(rows - 1, generator=g)[:200] + 1
    slots[again] = slots[(again.float() * 0.7).long()]   # the slot of some earlier row
    pad = torch.randperm(rows, generator=g)[:50]
    slots[pad] = -1
    seen, skipped = set(), []
    for i, s in enumerate(slots.tolist()):
        if s < 0 or s in seen:
            skipped.append(i)
        seen.add(s)
    assert len(skipped) > 100
    step_skips(rows, rows, 8, slots.to(DEV), 6, skipped)


def test_step_on_columns_and_without_slots():
    rows, D = 19, 40
    x = draw(rows, D, rows, 4, sdm.SDM_BF16, seed=14)
    wide = torch.cat([x["x"], x["x"]], 1)
    a, b = x["x0"].clone(), x["x0"].clone()
    y = sdm.sdm_short_conv_step(sdm.make_conv(1, rows, D, ld=2 * D), wide[:, D:], x["w"], a)
    z = sdm.sdm_short_conv_step(sdm.make_conv(1, rows, D), x["x"], x["w"], b, slots=torch.arange(rows, dtype=torch.int32, device=DEV))
    assert torch.equal(y, z) and torch.equal(a, b)


# ------------------------------------------------- streams, graphs, addresses

def test_repeats_streams_and_graph():
    lens = [300, 0, 600, 3]
    x = draw(903, 72, 4, 4, sdm.SDM_BF16, seed=41)
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
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_of()
    for seed in (41, 42):
        for k, t in draw(903, 72, 4, 4, sdm.SDM_BF16, seed=seed).items():
            x[k].copy_(t)
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(all_of(), got))
    assert sdm.sdm_get_device_status() == 0


def test_two_calls_at_once():
    cases = [draw(6000, 520, 2, 4, sdm.SDM_BF16, seed=s) for s in (1, 2)]
    want = [run(x, None, 2, sdm.SDM_BF16) for x in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [run(x, None, 2, sdm.SDM_BF16, stream=s) for x, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for p, q in zip(want, got):
            assert all(torch.equal(p[k], q[k]) for k in p if k != "dbias") and torch.equal(p["dbias"], q["dbias"])


def test_elements_beyond_32_bits():
    rows, D, ld = 66000, 8, 65536
    wide = torch.empty(rows * ld, dtype=torch.bfloat16, device=DEV).view(rows, ld)
    x = draw(rows, D, 1, 4, sdm.SDM_BF16, seed=1)
    wide[:, :D] = x["x"]
    want = run(x, None, 1, sdm.SDM_BF16)
    sh = sdm.make_conv(1, rows, D, ld=ld, ld_grad=ld)
    a = sdm.sdm_short_conv_forward(sh, wide[:, :D], x["w"], bias=x["bias"], x0=x["x0"])
    b = sdm.sdm_short_conv_backward(sh, wide[:, :D], x["w"], x["dy"], bias=x["bias"], x0=x["x0"], dxT=x["dxT"], dx=wide[:, 16:16 + D])
    assert torch.equal(a["y"], want["y"]) and torch.equal(wide[:, 16:16 + D], want["dx"]) and torch.equal(b["dw"], want["dw"])


def test_binding_refuses_wrong_tensors():
    x = draw(16, 64, 2, 4, sdm.SDM_BF16)
    sh = sdm.make_conv(2, 16, 64)
    for bad in (lambda: sdm.sdm_short_conv_forward(sdm.make_conv(2, 16, 64, ld=128), x["x"], x["w"]),
                lambda: sdm.sdm_short_conv_forward(sh, x["x"].float(), x["w"]), lambda: sdm.sdm_short_conv_forward(sh, x["x"][:15], x["w"]),
                lambda: sdm.sdm_short_conv_forward(sh, x["x"], x["w"][:, :3].contiguous()),
                lambda: sdm.sdm_short_conv_forward(sh, x["x"], x["w"], x0=x["x0"].float()),
                lambda: sdm.sdm_short_conv_step(sh, x["x"], x["w"], torch.zeros(16, 2, 64, dtype=torch.bfloat16, device=DEV)),
                lambda: sdm.sdm_short_conv_backward(sdm.make_conv(2, 16, 64, ld_grad=128), x["x"], x["w"], x["dy"])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sdm.SdmError):                # 16 rows on 15 windows without slots
        sdm.sdm_short_conv_step(sh, x["x"], x["w"], torch.zeros(15, 3, 64, dtype=torch.bfloat16, device=DEV))
