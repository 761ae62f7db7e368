"""The gated recurrence on the GPU against its plain 64-bit form
(tests/_layers.py, which also derives how far float32 may be off)."""
import pytest
import torch

from tests import _layers as R

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


def offsets(*off):
    return torch.tensor(off, dtype=torch.int32, device=DEV)


def draw(rows, D, n_seq, dtype, seed=0, long_memory=True, h0=True):
    """Inputs with memories from a few to about a thousand rows."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0, mean=0.0: torch.randn(*s, generator=g) * std + mean
    dt = DT[dtype]
    step = torch.exp(torch.rand(D, generator=g) * 4.6 - 6.9)
    x = dict(za=n(rows, D, std=0.7).to(dt), zb=n(rows, D, mean=-4.0 if long_memory else 0.0, std=2.0).to(dt),
             v=n(rows, D).to(dt), A=torch.rand(D, generator=g) * 15 + 1, bias=torch.log(torch.expm1(step)),
             h0=n(n_seq, D, std=0.5) if h0 else None, dy=n(rows, D).to(dt), dhT=n(n_seq, D))
    return {k: None if t is None else t.to(DEV) for k, t in x.items()}


def check(x, off, dtype, n_seq, where=None, A="A", bias="bias", **kw):
    """Forward and backward against the 64-bit form; returns both outputs."""
    rows, D = x["za"].shape
    sh = sdm.make_recurrence(n_seq, rows, D, dtype=dtype, **kw)
    A, bias = x.get(A), x.get(bias)
    f = sdm.sdm_recurrence_forward(sh, x["za"], x["zb"], x["v"], A=A, bias=bias, offsets=off, h0=x["h0"], save_states=True)
    b = sdm.sdm_recurrence_backward(sh, x["za"], x["zb"], x["v"], f["states"], x["dy"], A=A, bias=bias, offsets=off, dhT=x["dhT"],
                                    dA=torch.empty(D, device=DEV), dbias=torch.empty(D, device=DEV))
    assert sdm.sdm_get_device_status() == 0
    bounds = R.bounds_of(off, n_seq, rows)
    ref = R.recurrence(x["za"], x["zb"], x["v"], A, bias, bounds, x["h0"], x["dy"], x["dhT"])
    inside = torch.zeros(rows, dtype=torch.bool)
    inside[bounds[0]:bounds[-1]] = True
    for k in ("y", "hT"):
        R.within(f[k], *ref[k], k, inside if k == "y" else where)
    for k in ("dza", "dzb", "dv", "dA", "dbias", "dh0"):
        R.within(b[k], *ref[k], k, inside if k in ("dza", "dzb", "dv") else None)
    return f, b


@BOTH
@pytest.mark.parametrize("lens,D", [
    ([1], 8), ([2, 1], 8), ([0, 1, 0], 72), ([127, 128, 129], 64), ([64, 63, 65, 32, 33, 31], 136),
    ([5, 0, 300, 1, 0, 257], 200), ([513], 8), ([0], 16), ([1] * 40, 24), ([384, 256], 328),
])
def test_packed_sequences(lens, D, dtype):
    off = offsets(*[sum(lens[:i]) for i in range(len(lens) + 1)])
    x = draw(sum(lens), D, len(lens), dtype, seed=len(lens) * 100 + D)
    check(x, off, dtype, len(lens))


@BOTH
@pytest.mark.parametrize("n_seq,T,D", [(1, 1, 8), (3, 130, 40), (2, 700, 64), (4, 0, 8), (64, 1, 96), (2, 128, 1032)])
def test_equal_sequences(n_seq, T, D, dtype):
    x = draw(n_seq * T, D, n_seq, dtype, seed=T + D, h0=False)
    check(x, None, dtype, n_seq)


def test_many_chunks_carry_the_state():
    # Long memories over 90 chunks of one narrow and one wider sequence.
    for T, D, n_seq in ((11521, 8, 1), (4097, 72, 2)):
        x = draw(T * n_seq, D, n_seq, sdm.SDM_F32, seed=T)
        x["zb"] -= 4.0                               # beta about 1e-4 .. 1e-2
        x["bias"] -= 2.0
        check(x, None, sdm.SDM_F32, n_seq)


@BOTH
def test_many_tiles_per_block(dtype):
    # More tiles than the grid holds several times over, so that the blocks'
    # rings of stages and descriptions go round; packed and equal sequences.
    off = offsets(5, 1200, 1200, 1201, 2990)
    check(draw(3000, 2056, 4, dtype, seed=51), off, dtype, 4)
    check(draw(2400, 2056, 2, dtype, seed=52), None, dtype, 2)


@BOTH
def test_many_chains(dtype):
    # More chains (a sequence's 64 channels) than half the multiprocessors: the
    # backward pass then finishes each tile at once.  Empty, single and long ones.
    lens = [0, 1, 31, 32, 33, 63, 64, 65, 2, 300] * 8 + [1500, 0]
    off = offsets(*[3 + sum(lens[:i]) for i in range(len(lens) + 1)])
    x = draw(sum(lens) + 7, 200, len(lens), dtype, seed=53)
    check(x, off, dtype, len(lens))
    check(draw(40 * 330, 136, 40, dtype, seed=54), None, dtype, 40)


@BOTH
def test_one_long_sequence(dtype):
    # Few chains and many tiles of each in every block.
    check(draw(20011, 120, 1, dtype, seed=55), offsets(0, 20011), dtype, 1)
    check(draw(2 * 8000, 72, 2, dtype, seed=56), None, dtype, 2)


@BOTH
def test_thousands_of_short_sequences(dtype):
    g = torch.Generator().manual_seed(7)
    lens = torch.randint(0, 4, (3001,), generator=g)
    lens[1500] = 700                                 # and a long one among them
    off = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)]).to(torch.int32).to(DEV)
    check(draw(int(lens.sum()), 72, 3001, dtype, seed=61), off, dtype, 3001)


def test_widest_rows():
    check(draw(5, 65536, 2, sdm.SDM_BF16, seed=62), offsets(0, 2, 5), sdm.SDM_BF16, 2)


def test_no_rate_and_no_bias():
    x = draw(300, 64, 3, sdm.SDM_F32, seed=5, h0=False)
    check(x, None, sdm.SDM_F32, 3, A="none", bias="none")
    sh = sdm.make_recurrence(3, 300, 64, dtype=sdm.SDM_F32)
    f = sdm.sdm_recurrence_forward(sh, x["za"], x["zb"], x["v"], save_states=True)
    b = sdm.sdm_recurrence_backward(sh, x["za"], x["zb"], x["v"], f["states"], x["dy"])
    assert b["dA"] is None and b["dbias"] is None
    ref = R.recurrence(x["za"], x["zb"], x["v"], None, None, [0, 100, 200, 300], None, x["dy"], None)
    for k in ("dza", "dzb", "dv", "dh0"):
        R.within(b[k], *ref[k], k)


@BOTH
def test_columns_of_one_projection(dtype):
    # za, zb, v and their gradients as column ranges of [rows, 3 D] (+ padding).
    rows, D = 401, 104
    x = draw(rows, D, 2, dtype, seed=8)
    off = offsets(3, 150, 398)
    wide = torch.full((rows, 3 * D + 8), 7.0, dtype=DT[dtype], device=DEV)
    for i, k in enumerate(("za", "zb", "v")):
        wide[:, i * D:(i + 1) * D] = x[k]
    cols = [wide[:, i * D:(i + 1) * D] for i in range(3)]
    grad = torch.full((rows, 3 * D + 16), 5.0, dtype=DT[dtype], device=DEV)
    gcols = [grad[:, i * D:(i + 1) * D] for i in range(3)]
    sh = sdm.make_recurrence(2, rows, D, dtype=dtype, ld=3 * D + 8, ld_grad=3 * D + 16)
    y = torch.full((rows, D), 9.0, dtype=DT[dtype], device=DEV)
    f = sdm.sdm_recurrence_forward(sh, *cols, A=x["A"], bias=x["bias"], offsets=off, h0=x["h0"], y=y, save_states=True)
    b = sdm.sdm_recurrence_backward(sh, *cols, f["states"], x["dy"], A=x["A"], bias=x["bias"], offsets=off, dhT=x["dhT"],
                                    dza=gcols[0], dzb=gcols[1], dv=gcols[2])
    assert sdm.sdm_get_device_status() == 0
    dense = sdm.make_recurrence(2, rows, D, dtype=dtype)
    f2 = sdm.sdm_recurrence_forward(dense, x["za"], x["zb"], x["v"], A=x["A"], bias=x["bias"], offsets=off, h0=x["h0"],
                                    y=torch.full_like(y, 9.0), save_states=True)
    b2 = sdm.sdm_recurrence_backward(dense, x["za"], x["zb"], x["v"], f2["states"], x["dy"], A=x["A"], bias=x["bias"], offsets=off,
                                     dhT=x["dhT"], **{k: torch.full((rows, D), 5.0, dtype=DT[dtype], device=DEV)
                                                      for k in ("dza", "dzb", "dv")})
    assert torch.equal(f["y"], f2["y"]) and torch.equal(f["hT"], f2["hT"])
    for k, c in zip(("dza", "dzb", "dv"), gcols):
        assert torch.equal(c, b2[k]), k
    # Rows of no sequence and the columns behind the three stay as they were.
    assert (y[:3] == 9).all() and (y[398:] == 9).all()
    assert (grad[:, 3 * D:] == 5).all() and (grad[:3] == 5).all() and (grad[398:] == 5).all()


def test_binding_refuses_wrong_tensors():
    x = draw(16, 64, 2, sdm.SDM_BF16)
    sh = sdm.make_recurrence(2, 16, 64, ld=128)
    ok = sdm.make_recurrence(2, 16, 64)
    with pytest.raises(ValueError):                  # stride is not ld
        sdm.sdm_recurrence_forward(sh, x["za"], x["zb"], x["v"])
    with pytest.raises(ValueError):
        sdm.sdm_recurrence_forward(ok, x["za"].float(), x["zb"], x["v"])
    with pytest.raises(ValueError):
        sdm.sdm_recurrence_forward(ok, x["za"][:15], x["zb"], x["v"])
    with pytest.raises(ValueError):
        sdm.sdm_recurrence_forward(ok, x["za"], x["zb"], x["v"], A=x["A"].double())
    with pytest.raises(ValueError):
        sdm.sdm_recurrence_forward(ok, x["za"], x["zb"], x["v"], offsets=torch.zeros(3, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        sdm.sdm_recurrence_step(ok, x["za"], x["zb"], x["v"], torch.zeros(16, 32, device=DEV))
    with pytest.raises(sdm.SdmError):                # 16 rows on 15 states without slots
        sdm.sdm_recurrence_step(ok, x["za"], x["zb"], x["v"], torch.zeros(15, 64, device=DEV))
    with pytest.raises(ValueError):                  # gradients of another stride have to be given
        f = sdm.sdm_recurrence_forward(ok, x["za"], x["zb"], x["v"], save_states=True)
        sdm.sdm_recurrence_backward(sdm.make_recurrence(2, 16, 64, ld_grad=128), x["za"], x["zb"], x["v"], f["states"], x["dy"])


@BOTH
def test_rows_outside_hold_anything(dtype):
    # NaN and infinities in rows of no sequence reach nothing.
    rows, D = 420, 64
    off = offsets(7, 7, 135, 290, 411)
    x = draw(rows, D, 4, dtype, seed=3)
    sh = sdm.make_recurrence(4, rows, D, dtype=dtype)

    def run():
        f = sdm.sdm_recurrence_forward(sh, x["za"], x["zb"], x["v"], A=x["A"], bias=x["bias"], offsets=off, h0=x["h0"],
                                       y=torch.zeros(rows, D, dtype=DT[dtype], device=DEV), save_states=True)
        z = lambda: torch.zeros(rows, D, dtype=DT[dtype], device=DEV)
        b = sdm.sdm_recurrence_backward(sh, x["za"], x["zb"], x["v"], f["states"], x["dy"], A=x["A"], bias=x["bias"], offsets=off,
                                        dhT=x["dhT"], dza=z(), dzb=z(), dv=z())
        return [f["y"], f["hT"]] + [b[k] for k in ("dza", "dzb", "dv", "dA", "dbias", "dh0")]

    clean = run()
    for k, bad in (("za", float("nan")), ("zb", float("inf")), ("v", float("nan")), ("dy", float("-inf"))):
        x[k][:7] = bad
        x[k][411:] = bad
    for p, q in zip(clean, run()):
        assert torch.equal(p, q)
    assert sdm.sdm_get_device_status() == 0


@BOTH
def test_saturated_gates(dtype):
    # Logits at which the gates are 0 or 1 in float32, and infinite ones.
    D = 16
    vals = [-float("inf"), -1e30, -90.0, -30.0, -1.0, 0.0, 1.0, 30.0, 90.0, 1e30, float("inf")]
    za = torch.tensor([a for a in vals for _ in vals]).repeat(D, 1).T.contiguous()
    zb = torch.tensor([b for _ in vals for b in vals]).repeat(D, 1).T.contiguous()
    rows = za.shape[0]
    x = draw(rows, D, 1, dtype, seed=2)
    x["za"], x["zb"] = za.to(DT[dtype]).to(DEV), zb.to(DT[dtype]).to(DEV)
    sh = sdm.make_recurrence(1, rows, D, dtype=dtype)
    f = sdm.sdm_recurrence_forward(sh, x["za"], x["zb"], x["v"], A=x["A"], bias=x["bias"], h0=x["h0"], save_states=True)
    ref = R.recurrence(x["za"], x["zb"], x["v"], x["A"], x["bias"], [0, rows], x["h0"], x["dy"], x["dhT"])
    R.within(f["y"], *ref["y"], "y")
    R.within(f["hT"], *ref["hT"], "hT")
    # Gradients with finite logits only (softplus'(inf) * inf is NaN in the formula itself).
    fin = torch.isfinite(za[:, 0]) & torch.isfinite(zb[:, 0]) & (za[:, 0].abs() < 1e29) & (zb[:, 0].abs() < 1e29)
    y = {k: (t[fin.to(DEV)].contiguous() if k in ("za", "zb", "v", "dy") else t) for k, t in x.items()}
    check(y, None, dtype, 1)


def test_segments_carry_on_in_place():
    # Two calls with the state in place (hT = h0) are one call on both parts.
    x = draw(512, 64, 1, sdm.SDM_F32, seed=11)
    whole = sdm.sdm_recurrence_forward(sdm.make_recurrence(1, 512, 64, dtype=sdm.SDM_F32), x["za"], x["zb"], x["v"], A=x["A"],
                                       bias=x["bias"], h0=x["h0"])
    state, ys = x["h0"].clone(), []
    for a, b in ((0, 256), (256, 300), (300, 512)):
        sh = sdm.make_recurrence(1, b - a, 64, dtype=sdm.SDM_F32)
        ys.append(sdm.sdm_recurrence_forward(sh, x["za"][a:b], x["zb"][a:b], x["v"][a:b], A=x["A"], bias=x["bias"], h0=state,
                                             hT=state)["y"])
    ref = R.recurrence(x["za"], x["zb"], x["v"], x["A"], x["bias"], [0, 512], x["h0"])
    R.within(torch.cat(ys), *ref["y"], "y")
    R.within(state, *ref["hT"], "hT")
    R.within(whole["y"], *ref["y"], "y")


def test_gradients_in_place():
    # dh0 may be dhT itself.
    x = draw(700, 40, 2, sdm.SDM_F32, seed=12)
    sh = sdm.make_recurrence(2, 700, 40, dtype=sdm.SDM_F32)
    f = sdm.sdm_recurrence_forward(sh, x["za"], x["zb"], x["v"], A=x["A"], bias=x["bias"], h0=x["h0"], save_states=True)
    call = lambda d, o: sdm.sdm_recurrence_backward(sh, x["za"], x["zb"], x["v"], f["states"], x["dy"], A=x["A"], bias=x["bias"],
                                                    dhT=d, dh0=o)
    apart = call(x["dhT"], None)
    both = x["dhT"].clone()
    together = call(both, both)
    for k in apart:
        assert torch.equal(apart[k], together[k]), k


def test_gradients_against_differences():
    # Central differences of the 64-bit form, with the truncation taken out by
    # comparing two step sizes.
    rows, D, off = 150, 8, [0, 20, 150]
    x = draw(rows, D, 2, sdm.SDM_F32, seed=21, long_memory=False)
    f, b = check(x, offsets(*off), sdm.SDM_F32, 2)
    base = {k: R.double(t) for k, t in x.items()}
    ref = R.recurrence(x["za"], x["zb"], x["v"], x["A"], x["bias"], off, x["h0"], x["dy"], x["dhT"])

    def loss(**over):
        p = {**base, **over}
        r = R.recurrence(p["za"], p["zb"], p["v"], p["A"], p["bias"], off, p["h0"])
        return float((r["y"][0] * p["dy"]).sum() + (r["hT"][0] * p["dhT"]).sum())

    g = torch.Generator().manual_seed(1)
    for name, grad in (("za", "dza"), ("zb", "dzb"), ("v", "dv"), ("A", "dA"), ("bias", "dbias"), ("h0", "dh0")):
        for _ in range(2):
            t = base[name]
            i = int(torch.randint(t.numel(), (1,), generator=g))
            est = []
            for h in (1e-3, 5e-4):
                e = torch.zeros_like(t).flatten()
                e[i] = h
                e = e.reshape(t.shape)
                est.append((loss(**{name: t + e}) - loss(**{name: t - e})) / (2 * h))
            best = est[1] + (est[1] - est[0]) / 3        # the h^2 term removed
            got = float(b[grad].flatten()[i])
            lim = float(ref[grad][1].flatten()[i]) + abs(est[1] - est[0]) + 1e-9 * (1 + abs(best)) + R.U * abs(best)
            assert abs(got - best) <= lim, (name, i, got, best, lim)


@BOTH
def test_same_bits_every_time(dtype):
    off = offsets(0, 1000, 1001, 5000)
    x = draw(5000, 264, 3, dtype, seed=31)
    sh = sdm.make_recurrence(3, 5000, 264, dtype=dtype)

    def run():
        f = sdm.sdm_recurrence_forward(sh, x["za"], x["zb"], x["v"], A=x["A"], bias=x["bias"], offsets=off, h0=x["h0"],
                                       save_states=True)
        b = sdm.sdm_recurrence_backward(sh, x["za"], x["zb"], x["v"], f["states"], x["dy"], A=x["A"], bias=x["bias"], offsets=off,
                                        dhT=x["dhT"])
        return [f["y"], f["hT"]] + [b[k] for k in sorted(b)]

    first = run()
    for _ in range(10):
        for p, q in zip(first, run()):
            assert torch.equal(p, q)
    # A workspace of other contents does not matter.
    ws = torch.full((sdm.sdm_recurrence_workspace_size(sh),), 255, dtype=torch.uint8, device=DEV)
    f = sdm.sdm_recurrence_forward(sh, x["za"], x["zb"], x["v"], A=x["A"], bias=x["bias"], offsets=off, h0=x["h0"], workspace=ws)
    assert torch.equal(f["y"], first[0])


@pytest.mark.parametrize("off", [(0, 50, 40, 100), (0, 50, 60, 101), (-1, 50, 60, 100), (0, 200, 60, 100)])
def test_bad_offsets_write_nothing(off):
    x = draw(100, 64, 3, sdm.SDM_F32)
    sh = sdm.make_recurrence(3, 100, 64, dtype=sdm.SDM_F32)
    f = sdm.sdm_recurrence_forward(sh, x["za"], x["zb"], x["v"], offsets=offsets(0, 10, 10, 100), h0=x["h0"], save_states=True)
    assert sdm.sdm_get_device_status() == 0
    y, hT = torch.full((100, 64), 3.0, device=DEV), torch.full((3, 64), 3.0, device=DEV)
    sdm.sdm_recurrence_forward(sh, x["za"], x["zb"], x["v"], offsets=offsets(*off), h0=x["h0"], y=y, hT=hT)
    assert sdm.sdm_get_device_status() == 5
    assert (y == 3).all() and (hT == 3).all()
    outs = {k: torch.full((100, 64), 3.0, device=DEV) for k in ("dza", "dzb", "dv")}
    outs.update(dA=torch.full((64,), 3.0, device=DEV), dbias=torch.full((64,), 3.0, device=DEV),
                dh0=torch.full((3, 64), 3.0, device=DEV))
    sdm.sdm_recurrence_backward(sh, x["za"], x["zb"], x["v"], f["states"], x["dy"], offsets=offsets(*off), **outs)
    assert sdm.sdm_get_device_status() == 5
    assert all((t == 3).all() for t in outs.values())
    # And the next call works.
    g = sdm.sdm_recurrence_forward(sh, x["za"], x["zb"], x["v"], offsets=offsets(0, 10, 10, 100), h0=x["h0"])
    assert sdm.sdm_get_device_status() == 0
    assert torch.isfinite(g["y"]).all()


def test_no_sequences_gives_zero_sums():
    x = draw(8, 64, 1, sdm.SDM_F32)
    sh = sdm.make_recurrence(0, 8, 64, dtype=sdm.SDM_F32)
    dA, db = torch.full((64,), 3.0, device=DEV), torch.full((64,), 3.0, device=DEV)
    sdm.sdm_recurrence_backward(sh, x["za"], x["zb"], x["v"], torch.zeros(16, device=DEV), x["dy"], dA=dA, dbias=db,
                                dh0=torch.zeros(1, 64, device=DEV))
    assert sdm.sdm_get_device_status() == 0
    assert (dA == 0).all() and (db == 0).all()


# ---------------------------------------------------------------------- step

@BOTH
@pytest.mark.parametrize("rows,D,n_slots", [(1, 8, 1), (5, 72, 9), (64, 1920, 96), (33, 1000, 40)])
def test_step(rows, D, n_slots, dtype):
    x = draw(rows, D, rows, dtype, seed=rows)
    g = torch.Generator().manual_seed(rows)
    slots = torch.randperm(n_slots, generator=g)[:rows].to(torch.int32)
    state = torch.randn(n_slots, D, generator=g)
    dev = state.to(DEV)
    sh = sdm.make_recurrence(1, rows, D, dtype=dtype)
    y = sdm.sdm_recurrence_step(sh, x["za"], x["zb"], x["v"], dev, A=x["A"], bias=x["bias"], slots=slots.to(DEV))
    assert sdm.sdm_get_device_status() == 0
    ref = R.recurrence(x["za"], x["zb"], x["v"], x["A"], x["bias"], list(range(rows + 1)), state[slots.long()])
    R.within(y, *ref["y"], "y")
    R.within(dev[slots.long().to(DEV)], *ref["hT"], "state")
    rest = torch.ones(n_slots, dtype=torch.bool)
    rest[slots.long()] = False
    assert torch.equal(dev.cpu()[rest], state[rest])


def test_step_without_slots_equals_one_row_sequences():
    rows, D = 37, 136
    x = draw(rows, D, rows, sdm.SDM_F32, seed=4)
    state = x["h0"].clone()
    y = sdm.sdm_recurrence_step(sdm.make_recurrence(1, rows, D, dtype=sdm.SDM_F32), x["za"], x["zb"], x["v"], state)
    ref = R.recurrence(x["za"], x["zb"], x["v"], None, None, list(range(rows + 1)), x["h0"])
    R.within(y, *ref["y"], "y")
    assert torch.equal(y, state)


def test_step_padding_bad_and_repeated_slots():
    rows, D = 6, 64
    x = draw(rows, D, rows, sdm.SDM_F32, seed=6)
    sh = sdm.make_recurrence(1, rows, D, dtype=sdm.SDM_F32)
    state0 = torch.randn(10, D, device=DEV)
    clean = state0.clone()
    want = sdm.sdm_recurrence_step(sh, x["za"], x["zb"], x["v"], clean, slots=torch.tensor([3, 1, 7, 0, 9, 2], dtype=torch.int32, device=DEV))
    for slots, code, skipped in (([3, -1, 7, 0, -5, 2], 0, [1, 4]), ([3, 10, 7, 0, 9, 2], 5, [1]), ([3, 1, 3, 0, 9, 3], 6, [2, 5])):
        state, y = state0.clone(), torch.full((rows, D), 4.0, device=DEV)
        sdm.sdm_recurrence_step(sh, x["za"], x["zb"], x["v"], state, slots=torch.tensor(slots, dtype=torch.int32, device=DEV), y=y)
        assert sdm.sdm_get_device_status() == code
        for i in range(rows):
            assert (y[i] == 4).all() if i in skipped else torch.equal(y[i], want[i]), (slots, i)
        touched = {s for i, s in enumerate(slots) if i not in skipped}
        for s in range(10):
            assert torch.equal(state[s], clean[s] if s in touched else state0[s]), (slots, s)


@BOTH
def test_step_on_columns_of_one_projection(dtype):
    rows, D = 19, 40
    x = draw(rows, D, rows, dtype, seed=14)
    wide = torch.cat([x["za"], x["zb"], x["v"]], 1)
    cols = [wide[:, i * D:(i + 1) * D] for i in range(3)]
    a, b = x["h0"].clone(), x["h0"].clone()
    y = sdm.sdm_recurrence_step(sdm.make_recurrence(1, rows, D, dtype=dtype, ld=3 * D), *cols, a, A=x["A"], bias=x["bias"])
    z = sdm.sdm_recurrence_step(sdm.make_recurrence(1, rows, D, dtype=dtype), x["za"], x["zb"], x["v"], b, A=x["A"], bias=x["bias"])
    assert torch.equal(y, z) and torch.equal(a, b)


def test_step_on_many_rows():
    # More rows than a grid's second dimension has blocks.
    rows, D = 70001, 8
    x = draw(rows, D, 1, sdm.SDM_BF16, seed=9)
    state = torch.randn(rows, D, device=DEV)
    before = state.clone()
    y = sdm.sdm_recurrence_step(sdm.make_recurrence(1, rows, D), x["za"], x["zb"], x["v"], state, A=x["A"], bias=x["bias"])
    a = torch.exp(-x["A"].double() * torch.nn.functional.softplus(x["za"].double() + x["bias"].double(), threshold=100))
    zb = x["zb"].double()
    h = torch.sigmoid(-zb) * a * before.double() + torch.sigmoid(zb) * x["v"].double()
    assert (y.double() - h).abs().max() <= 2.0 ** -8 * h.abs().max()
    assert (state.double() - h).abs().max() <= 1e-5


# ------------------------------------------------- streams, graphs, addresses

def test_graph_replay_and_other_stream():
    off = offsets(0, 300, 300, 900)
    x = draw(900, 72, 3, sdm.SDM_BF16, seed=41)
    sh = sdm.make_recurrence(3, 900, 72)
    ws = torch.empty(sdm.sdm_recurrence_workspace_size(sh), dtype=torch.uint8, device=DEV)
    state = torch.randn(3, 72, device=DEV)

    def run(**kw):
        f = sdm.sdm_recurrence_forward(sh, x["za"], x["zb"], x["v"], A=x["A"], bias=x["bias"], offsets=off, h0=x["h0"],
                                       save_states=True, **kw)
        b = sdm.sdm_recurrence_backward(sh, x["za"], x["zb"], x["v"], f["states"], x["dy"], A=x["A"], bias=x["bias"], offsets=off,
                                        dhT=x["dhT"], **kw)
        return [f["y"], f["hT"]] + [b[k] for k in sorted(b)]

    want = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(stream=side)
    side.synchronize()
    for p, q in zip(want, got):
        assert torch.equal(p, q)
    got = run(stream=side.cuda_stream)                # a raw handle
    side.synchronize()
    for p, q in zip(want, got):
        assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(workspace=ws)
    for seed in (41, 42, 43):
        z = draw(900, 72, 3, sdm.SDM_BF16, seed=seed)
        for k in x:
            x[k].copy_(z[k])
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(run(), got):
            assert torch.equal(p, q)
    assert sdm.sdm_get_device_status() == 0


def test_two_calls_at_once():
    # Two streams, a workspace each.
    shapes = [(draw(6000, 520, 2, sdm.SDM_BF16, seed=s), sdm.make_recurrence(2, 6000, 520)) for s in (1, 2)]
    call = lambda x, sh, **kw: sdm.sdm_recurrence_forward(sh, x["za"], x["zb"], x["v"], A=x["A"], bias=x["bias"], h0=x["h0"], **kw)["y"]
    want = [call(*p) for p in shapes]
    streams = [torch.cuda.Stream() for _ in shapes]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [call(*p, stream=s) for p, s in zip(shapes, streams)]
        torch.cuda.synchronize()
        for p, q in zip(want, got):
            assert torch.equal(p, q)


def test_two_backward_calls_at_once():
    shapes = [(draw(6000, 520, 2, sdm.SDM_BF16, seed=s), sdm.make_recurrence(2, 6000, 520)) for s in (3, 4)]
    states = [sdm.sdm_recurrence_forward(sh, x["za"], x["zb"], x["v"], A=x["A"], bias=x["bias"], save_states=True)["states"]
              for x, sh in shapes]
    call = lambda i, **kw: sdm.sdm_recurrence_backward(shapes[i][1], *(shapes[i][0][k] for k in ("za", "zb", "v")), states[i],
                                                       shapes[i][0]["dy"], A=shapes[i][0]["A"], bias=shapes[i][0]["bias"], **kw)
    want = [call(i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in shapes]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [call(i, stream=streams[i]) for i in range(2)]
        torch.cuda.synchronize()
        for p, q in zip(want, got):
            assert all(torch.equal(p[k], q[k]) for k in p)
    assert sdm.sdm_get_device_status() == 0


def test_elements_beyond_32_bits():
    # Row offsets past 2^31 and 2^32 elements (a wide row stride).
    rows, D, ld = 66000, 8, 65536
    wide = torch.empty(rows * ld, dtype=torch.bfloat16, device=DEV)[:rows * ld].view(rows, ld)
    x = draw(rows, D, 1, sdm.SDM_BF16, seed=1)
    cols = []
    for i, k in enumerate(("za", "zb", "v")):
        wide[:, i * D:(i + 1) * D] = x[k]
        cols.append(wide[:, i * D:(i + 1) * D])
    a = sdm.sdm_recurrence_forward(sdm.make_recurrence(1, rows, D, ld=ld), *cols, A=x["A"], bias=x["bias"])
    b = sdm.sdm_recurrence_forward(sdm.make_recurrence(1, rows, D), x["za"], x["zb"], x["v"], A=x["A"], bias=x["bias"])
    assert torch.equal(a["y"], b["y"]) and torch.equal(a["hT"], b["hT"])
    assert sdm.sdm_get_device_status() == 0
