"""The single-token step with slots on thousands of rows: repeated, missing and
padding slots that lie far apart, and what looking for them costs."""
import ctypes

import pytest
import torch

sdm = pytest.importorskip("sparse_state_linear_gb300")
DEV = "cuda:0"
DT = {sdm.SDM_F32: torch.float32, sdm.SDM_BF16: torch.bfloat16}
gpu = pytest.mark.gpu


def test_most_rows_with_slots():
    from sparse_state_linear_gb300 import build_ext
    build_ext.build()
    L, p = sdm.lib(), ctypes.c_void_p(1 << 20)
    sh = sdm.make_recurrence(1, (1 << 22) + 1, 8)
    assert L.sdm_recurrence_step(ctypes.byref(sh), p, p, p, p, p, p, 1 << 23, p, p, None) == 2


def inputs(rows, D, n_slots, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)
    t = [n(rows, D).to(DT[dtype]) for _ in range(3)]
    return t, n(n_slots, D), torch.rand(D, generator=g, device=DEV) * 4, n(D)


@gpu
@pytest.mark.parametrize("dtype", [sdm.SDM_F32, sdm.SDM_BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,D", [(16383, 8), (16384, 8), (20003, 40), (4096, 1928), (5001, 2056), (300, 32776)])
def test_slots_of_many_rows(rows, D, dtype):
    n_slots = rows + 100
    t, state, A, bias = inputs(rows, D, n_slots, dtype, rows + D)
    g = torch.Generator().manual_seed(rows)
    slots = torch.randperm(n_slots, generator=g)[:rows].to(torch.int32)
    for code, plant in ((0, []), (0, [(5, -1), (rows // 2, -7), (rows - 1, -1 << 31)]), (5, [(3, n_slots), (rows - 2, (1 << 31) - 1)]),
                        (6, [(rows - 1, int(slots[0])), (rows // 2 + 1, int(slots[rows // 2])), (70, int(slots[1])), (71, int(slots[1])),
                             (rows - 5, int(slots[rows - 200]))])):
        s = slots.clone()
        for i, slot in plant:
            s[i] = slot
        skipped = torch.zeros(rows, dtype=torch.bool)
        skipped[[i for i, _ in plant]] = True
        # What the rows that are not skipped give, by a call without repeats.
        some = torch.nonzero(~skipped).flatten().to(DEV)
        at = s.to(DEV)[some].long()
        part, want_state = state[at].clone(), state.clone()
        want = sdm.sdm_recurrence_step(sdm.make_recurrence(1, len(some), D, dtype=dtype), *(z[some].contiguous() for z in t), part, A=A, bias=bias)
        want_state[at] = part
        assert sdm.sdm_get_device_status() == 0
        got_state, y = state.clone(), torch.full((rows, D), 4.0, dtype=DT[dtype], device=DEV)
        sdm.sdm_recurrence_step(sdm.make_recurrence(1, rows, D, dtype=dtype), *t, got_state, A=A, bias=bias, slots=s.to(DEV), y=y)
        assert sdm.sdm_get_device_status() == code
        assert torch.equal(got_state, want_state)
        assert torch.equal(y[some], want)
        assert (y[skipped.to(DEV)] == 4).all()


@gpu
def test_same_slot_in_every_row_and_strided_columns():
    rows, D = 16500, 24
    t, state, A, bias = inputs(rows, 3 * D, 4, sdm.SDM_F32, 3)
    cols = [t[0][:, i * D:(i + 1) * D] for i in range(3)]
    state = state[:, :D].contiguous()
    one = state[2:3].clone()
    want = sdm.sdm_recurrence_step(sdm.make_recurrence(1, 1, D, dtype=sdm.SDM_F32), *(c[:1].contiguous() for c in cols), one)
    y = torch.full((rows, D), 4.0, device=DEV)
    got = state.clone()
    sdm.sdm_recurrence_step(sdm.make_recurrence(1, rows, D, dtype=sdm.SDM_F32, ld=3 * D), *cols, got,
                            slots=torch.full((rows,), 2, dtype=torch.int32, device=DEV), y=y)
    assert sdm.sdm_get_device_status() == 6
    assert torch.equal(y[:1], want) and (y[1:] == 4).all()
    assert torch.equal(got[2:3], one) and torch.equal(got[[0, 1, 3]], state[[0, 1, 3]])


@gpu
def test_slots_do_not_rule_the_time():
    # 70000 rows of 1920 channels move 1.6 GB; comparing every row's slot with all
    # earlier ones by itself would take twice as long again.
    rows, D = 70000, 1920
    t, state, A, bias = inputs(rows, D, rows, sdm.SDM_BF16, 4)
    sh, y = sdm.make_recurrence(1, rows, D), torch.empty(rows, D, dtype=torch.bfloat16, device=DEV)
    slots = torch.randperm(rows, device=DEV).int()

    def best(**kw):
        times = []
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(3):
                sdm.sdm_recurrence_step(sh, *t, state, A=A, bias=bias, y=y, **kw)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times[2:])

    assert best(slots=slots) < 2.2 * best()
    assert sdm.sdm_get_device_status() == 0
