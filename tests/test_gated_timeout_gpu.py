"""Waits of the gated recurrence that run out in the middle of an exchange between blocks: the call ends, whatever was under way
lands in blocks that are still there, and the next call is right."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("B,T,D,dtype", [(1, 60000, 64, "bf16"), (2, 20000, 256, "f32"), (1, 30000, 65, "f32"), (40, 3000, 64, "bf16")])
def test_waits_of_one_cycle(B, T, D, dtype):
    """No wait that has to look twice gets what it waits for. Whether one has to is the GPU's affair: the status says."""
    from log_linear_attention_gb300 import binding as lla
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, a, s0 = torch.randn(B, T, D, device="cuda").to(dt), -torch.rand(B, T, D, device="cuda"), torch.randn(1, D, device="cuda")

    def calls():
        out = lla.gated_forward(x, a, state0=s0)
        return (out, *lla.gated_backward(a, x, x, state0=s0))

    want = calls()
    assert lla.device_error() == lla.LLA_OK
    for _ in range(5):
        lla.debug_set_waits(1, hold=False)
        try:
            got = calls()
            status = lla.device_error()
        finally:
            lla.debug_set_waits(0, hold=False)
        assert status in (lla.LLA_OK, lla.LLA_ERR_TIMEOUT)
        if status == lla.LLA_OK:
            assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert all(torch.equal(p, q) for p, q in zip(calls(), want))
        assert lla.device_error() == lla.LLA_OK
