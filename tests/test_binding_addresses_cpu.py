"""Which address the bindings of the selective scan hand on for B, C, dB and dC: that of
the caller's tensor, or none at all.  The library is stood in for by one that notes its
arguments, so that tensors may lie on the CPU."""
import pytest
import torch

import sparse_state_linear_gb300 as sdm

B_FORWARD, C_FORWARD = 3, 4                          # places behind the shape: x dt A B C
DB_BACKWARD, DC_BACKWARD = 15, 16                    # ... dx ddt dA dB dC


class Notes:
    """Every call notes its arguments; sizes are 4096 bytes, calls return SDM_OK."""

    def __init__(self):
        self.calls = {}

    def __getattr__(self, name):
        def call(*args):
            self.calls[name] = args[1:]
            return 4096 if name.endswith("_size") else 0
        return call


@pytest.fixture
def notes(monkeypatch):
    n = Notes()
    monkeypatch.setattr(sdm, "lib", lambda: n)
    monkeypatch.setattr(sdm, "_where", lambda like, stream: (-1, 0, None))
    return n


def inputs(rows, D, N):
    return torch.zeros(rows, D), torch.zeros(rows, D), torch.zeros(D, N)


def forward(sh, B, C):
    x, dt, A = inputs(sh.rows, sh.D, sh.N)
    sdm.sdm_selective_scan_forward(sh, x, dt, A, B, C)


def step(sh, B, C):
    x, dt, A = inputs(sh.rows, sh.D, sh.N)
    sdm.sdm_selective_scan_step(sh, x, dt, A, B, C, torch.zeros(sh.rows, sh.D, sh.N))


def backward(sh, dB, dC):
    x, dt, A = inputs(sh.rows, sh.D, sh.N)
    dense = torch.zeros(sh.rows, sh.groups, sh.N)
    sdm.sdm_selective_scan_backward(sh, x, dt, A, dense, dense, torch.zeros(1024), x, dB=dB, dC=dC)


def make(rows, G, N, ld):
    return sdm.make_selective(1, rows, 16 * G, N, groups=G, dtype=sdm.SDM_F32, ld_bc=ld)


def make_grad(rows, G, N, ld):
    return sdm.make_selective(1, rows, 16 * G, N, groups=G, dtype=sdm.SDM_F32, ld_bc_grad=ld)


def strided(shape, strides):
    return torch.zeros(4096).as_strided(shape, strides)


# Tensors whose elements do not lie where the kernels look for them.
BAD = [
    ((1, 2, 8), (128, 8, 16), 128),                  # one row, states 16 elements apart
    ((1, 2, 8), (128, 8, 0), 128),                   # one row, a value for all states
    ((1, 2, 8), (128, 8, 2), 128),
    ((1, 1, 8), (128, 8, 2), 128),                   # one group
    ((1, 2, 8), (128, 16, 1), 128),                  # groups apart
    ((3, 2, 8), (128, 8, 16), 128),
    ((3, 2, 8), (128, 8, 1), 256),                   # another row stride
    ((3, 8, 2), (128, 2, 1), 128),                   # states in front of groups
    ((1, 8, 2), (128, 2, 1), 128),
    ((2, 2, 8), (128, 8, 1), 128),                   # too few rows of three
]
# Dense rows: of the right number of elements, in another order.
BAD_DENSE = [(3, 8, 2), (1, 8, 2), (3, 4, 4), (3, 16, 1)]
GOOD = [
    (3, (3, 2, 8), (128, 8, 1), 128),
    (3, (3, 16), (128, 1), 128),
    (3, (5, 2, 8), (128, 8, 1), 128),                # more rows than the call's
    (1, (1, 2, 8), (128, 8, 1), 128),
    (1, (1, 2, 8), (7, 8, 1), 128),                  # one row has no stride
    (3, (3, 2, 8), (16, 8, 1), 0),
    (3, (3, 16), (16, 1), 0),
    (3, (1, 3, 16), (48, 16, 1), 0),                 # batch and time are the rows
    (3, (1, 3, 2, 8), (48, 16, 8, 1), 0),
    (1, (2, 8), (8, 1), 0),                          # the one row itself
    (3, (48,), (1,), 0),
]


@pytest.mark.parametrize("shape,strides,ld", BAD)
def test_refuses_what_lies_elsewhere(notes, shape, strides, ld):
    rows = 1 if shape[0] == 1 else 3
    N, G = 8, shape[1] if shape[2] == 8 else shape[2]
    bad, good = strided(shape, strides), strided((rows, G, N), (ld, N, 1))
    for call, sh in ((forward, make(rows, G, N, ld)), (step, make(rows, G, N, ld)), (backward, make_grad(rows, G, N, ld))):
        for first, second in ((bad, good), (good, bad)):
            with pytest.raises(ValueError):
                call(sh, first, second)
    assert not [c for c in notes.calls if not c.endswith("_size")]


@pytest.mark.parametrize("shape", BAD_DENSE)
def test_refuses_other_orders_of_dense_rows(notes, shape):
    rows = 1 if shape[0] == 1 else 3
    bad, good = torch.zeros(shape), torch.zeros(rows, 2, 8)
    for call in (forward, step, backward):
        for first, second in ((bad, good), (good, bad)):
            with pytest.raises(ValueError):
                call(make(rows, 2, 8, 0), first, second)
    assert not [c for c in notes.calls if not c.endswith("_size")]


@pytest.mark.parametrize("rows,shape,strides,ld", GOOD)
def test_hands_on_the_tensors_own_address(notes, rows, shape, strides, ld):
    a, b = strided(shape, strides), strided(shape, strides)
    forward(make(rows, 2, 8, ld), a, b)
    step(make(rows, 2, 8, ld), a, b)
    backward(make_grad(rows, 2, 8, ld), a, b)
    for name, first, second in (("forward", B_FORWARD, C_FORWARD), ("step", B_FORWARD, C_FORWARD), ("backward", DB_BACKWARD, DC_BACKWARD)):
        args = notes.calls["sdm_selective_scan_" + name]
        assert (args[first], args[second]) == (a.data_ptr(), b.data_ptr()), name


def test_groups_of_one_take_batches_of_rows(notes):
    # [batch, time, N] with one group: what a projection over batches returns.
    B, C = torch.zeros(2, 3, 16), torch.zeros(2, 3, 16)
    forward(make(6, 1, 16, 0), B, C)
    assert notes.calls["sdm_selective_scan_forward"][B_FORWARD:C_FORWARD + 1] == (B.data_ptr(), C.data_ptr())
    # No rows: nothing is looked at.
    forward(make(0, 1, 16, 0), torch.zeros(0, 1, 16), torch.zeros(0, 16))
    forward(make(0, 2, 8, 128), torch.zeros(0, 2, 8), torch.zeros(0, 16))
