"""GPU checks of commits behind gates that are not finite."""
import numpy as np
import pytest

from tests import _drafts as R

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture()
def lla():
    from log_linear_attention_gb300 import binding
    yield binding
    assert binding.device_error() == 0


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


@pytest.mark.parametrize("gate", [float("nan"), float("inf"), 200.0])
@pytest.mark.parametrize("t", [0, 1, 3, 8, 12])
def test_slots_of_new_tokens_alone(lla, t, gate):
    """The first token's gate weighs the old slots only: where it is not a number of any use, slots without an old one are as
    decode steps leave them."""
    H, N, L, dk, dv = 2, 5, 6, 16, 32
    r = np.random.default_rng(t)
    q, k = (torch.from_numpy(r.standard_normal((1, H, N, dk)).astype(np.float32)).cuda() for _ in range(2))
    v = torch.from_numpy(r.standard_normal((1, H, N, dv)).astype(np.float32)).cuda()
    la, lam = -torch.rand(1, H, N, device="cuda"), torch.rand(1, H, L, device="cuda")
    la[0, 1, 0] = gate
    states = torch.randn(1, H, L, dk, dv, device="cuda")
    for n in range(1, N + 1):
        got, steps = states.clone(), states.clone()
        lla.decode_commit(k, v, la, got, ints([t], torch.int64), ints([n]))
        for i in range(n):
            lla.decode_step(*(x[:, :, i].contiguous() for x in (q, k, v, la)), lam, steps, ints([t + i], torch.int64))
        for m, (lo, _) in R.held(t + n - 1).items():
            a, b = got[0, :, m], steps[0, :, m]
            if lo >= t:  # the slot's first token is a new one
                assert torch.isfinite(b).all()
            assert torch.equal(torch.isfinite(a), torch.isfinite(b)), (n, m)
            a, b = torch.nan_to_num(a, 0, 0, 0), torch.nan_to_num(b, 0, 0, 0)
            # sums in another order: (n + 1) products of five units each at most, of values of up to 16
            assert (a - b).abs().max() <= 16 * 5 * (n + 1) * R.U32 * b.abs().max().clamp(min=1), (n, m)
