"""Failure path of the tree kernels' bounded waits, exercised on the GPU without hanging anything: every warp waits for half a
millisecond for what never comes, the copies under way are let land, the status is read, and the next call is right."""
import numpy as np
import pytest

from tests import _drafts as R

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 128, 64), ("bf16", 100, 36), ("f32", 64, 64)])
@pytest.mark.parametrize("N", [5, 40])
@pytest.mark.parametrize("t", [0, 1, 3000])
def test_a_wait_that_runs_out_is_reported(t, N, dtype, dk, dv):
    from log_linear_attention_gb300 import binding as lla
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    B, H, L = 2, 3, 13
    q, k = (torch.randn(B, H, N, dk, device="cuda").to(dt) for _ in range(2))
    v = torch.randn(B, H, N, dv, device="cuda").to(dt)
    la, lam = -torch.rand(B, H, N, device="cuda"), torch.rand(B, H, N, L, device="cuda")
    states, decay = torch.randn(B, H, L, dk, dv, device="cuda"), -torch.rand(H, device="cuda")
    pos = torch.full((B,), t, dtype=torch.int64, device="cuda")
    parent = torch.tensor(R.random_tree(np.random.default_rng(N), N), dtype=torch.int32, device="cuda")
    state = states[:, :, 0].contiguous()

    calls = (lambda: lla.decode_tree(q, k, v, la, lam, states, pos, parent),
             lambda: lla.linear_decode_tree(q, k, v, decay, state, parent))
    want = [call() for call in calls]
    assert lla.device_error() == lla.LLA_OK
    for call, ref in zip(calls, want):
        lla.debug_set_waits(1_000_000, hold=True)
        try:
            call()
            status = lla.device_error()
        finally:
            lla.debug_set_waits(0, hold=False)
        assert status == lla.LLA_ERR_TIMEOUT, lla.status_string(status)
        assert lla.device_error() == lla.LLA_OK
        assert torch.equal(call(), ref)
        assert lla.device_error() == lla.LLA_OK
