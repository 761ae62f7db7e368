"""Waits of the recurrence's kernels that run out: the call ends with the status
that the header names, and the next one is as good as any."""
import pytest
import torch

sdm = pytest.importorskip("sparse_state_linear_gb300")
DEV = "cuda:0"
DT = {sdm.SDM_F32: torch.float32, sdm.SDM_BF16: torch.bfloat16}


def test_limit_is_checked():
    from sparse_state_linear_gb300 import build_ext
    build_ext.build()
    L = sdm.lib()
    for bad in (-2, 10 ** 7 + 1):
        assert L.sdm_set_recurrence_wait(bad) == 1
        with pytest.raises(sdm.SdmError):
            sdm.sdm_set_recurrence_wait(bad)
    for good in (0, 1, 10 ** 7, -1):
        assert L.sdm_set_recurrence_wait(good) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [sdm.SDM_F32, sdm.SDM_BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n_seq,D", [(1, 64), (3, 200), (40, 264)])
def test_waits_that_run_out(n_seq, D, dtype):
    # Chains of hundreds of chunks, all at work at once: no chunk finds what the
    # one before it publishes at its first look.  (40 sequences of 264 channels
    # take the backward pass's form that finishes a tile at once.)
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    T = 40000 // n_seq
    rows = T * n_seq
    g = torch.Generator().manual_seed(D)
    dt = DT[dtype]
    t = [torch.randn(rows, D, generator=g).to(dt).to(DEV) for _ in range(4)]
    h0, dhT = torch.randn(n_seq, D, generator=g).to(DEV), torch.randn(n_seq, D, generator=g).to(DEV)
    off = torch.arange(n_seq + 1, dtype=torch.int32, device=DEV) * T
    sh = sdm.make_recurrence(n_seq, rows, D, dtype=dtype)

    def forward():
        return sdm.sdm_recurrence_forward(sh, *t[:3], offsets=off, h0=h0, save_states=True)

    def backward(states):
        return sdm.sdm_recurrence_backward(sh, *t[:3], states, t[3], offsets=off, dhT=dhT, dA=torch.empty(D, device=DEV))

    want = forward()
    grads = backward(want["states"])
    assert sdm.sdm_get_device_status() == 0
    try:
        for call in (forward, lambda: backward(want["states"])):
            for _ in range(3):
                sdm.sdm_set_recurrence_wait(0)
                call()
                assert sdm.sdm_get_device_status() == 4
                sdm.sdm_set_recurrence_wait(-1)
                f = forward()
                b = backward(f["states"])
                assert sdm.sdm_get_device_status() == 0
                assert torch.equal(f["y"], want["y"]) and torch.equal(f["hT"], want["hT"])
                assert all(torch.equal(b[k], grads[k]) for k in b if b[k] is not None)
    finally:
        sdm.sdm_set_recurrence_wait(-1)
