"""GPU checks of the gates themselves: every path of the gated recurrence forms the gate that a single token's step forms (prompts
with gates of 16 bits come close to it), and a slow channel's long memory holds what 64 bits hold."""
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


def log_gates(n, dtype):
    """Gates from 1 down to 0, those that fp32 holds as subnormal numbers among them, and above 1."""
    r = np.random.default_rng(n)
    a = np.concatenate([-np.exp(r.uniform(-16, 4.7, n)), r.uniform(-104, -80, n // 8 + 1), r.uniform(0, 3, n // 8 + 1),
                        [0.0, -0.0, -np.inf, -3.4e38, -1e9, -87.4, -103.9, -104.1]])
    a = torch.from_numpy(r.permutation(a)[:n].astype(np.float32))
    return (a.bfloat16() if dtype == "bf16" else a).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,row,D", [(1, 0, 64), (1, 0, 65), (1, 0, 68), (128, 5, 64), (256, 100, 64), (700, 300, 96),
                                     (600, 257, 16), (64, 3, 68), (64, 40, 67), (2048, 1500, 32)])
def test_a_prompts_gate_is_a_steps_gate(lla, T, row, D, dtype):
    """A state of ones, inputs of zero and one row of gates that are not 1: every other factor is exactly 1, so the state
    that leaves is the gate itself, as the step forms it. A prompt's gates of 16 bits: the product of log_a with log2 e is rounded
    (|log_a| 2^-24 of the gate, and as much for log2 e's own rounding), its power of two and the step's expf are off by 4 x 2^-24
    each at most; subnormal gates are 0."""
    def check(got, want, la, fine):
        if fine:
            assert torch.equal(got, want)
        else:
            got, want, size = got.double(), want.double(), la.double().abs().nan_to_num(posinf=0)
            assert ((got - want).abs() <= (2 * size + 8) * R.U32 * want + 1.2e-38).all()

    for batch in (1, 3, 40):
        la = log_gates(batch * D, dtype).reshape(batch, D)
        one = torch.ones(batch, D, device="cuda")
        want = one.clone()
        lla.gated_decode_step(torch.zeros_like(one), la.float(), want)
        a = torch.zeros(batch, T, D, device="cuda", dtype=la.dtype)
        a[:, row] = la
        x = torch.zeros(batch, T, D, device="cuda", dtype=la.dtype)
        end = torch.empty_like(one)
        lla.gated_forward(x, a, state0=one, state_out=end)
        check(end, want, la, dtype == "f32")
        assert torch.equal(lla.gated_backward(a, x, x, state0=one, dstate_out=one)[2], want)
        # packed: the sequences one behind the other
        cu = torch.arange(0, batch * T + 1, T, dtype=torch.int32, device="cuda")
        x, a = x.reshape(-1, D), a.reshape(-1, D)
        lla.gated_forward_varlen(x, a, cu, state0=one, state_out=end.zero_())
        check(end, want, la, dtype == "f32")
        assert torch.equal(lla.gated_backward_varlen(a, x, x, cu, state0=one, dstate_out=one)[2], want)


@pytest.mark.parametrize("D", [64, 65])
def test_a_long_memory_of_one_sign(lla, D):
    """65536 rows of gates that forget a hundred-thousandth a row, inputs of one sign: nothing averages out."""
    T = 65536
    r = np.random.default_rng(D)
    a = (-1e-5 * (0.5 + r.random((T, D)))).astype(np.float32)
    x = r.random((T, D)).astype(np.float32)
    do = r.random((T, D)).astype(np.float32)
    at, xt, dot = (torch.from_numpy(y).cuda()[None] for y in (a, x, do))
    end = torch.empty(1, D, device="cuda")
    out = lla.gated_forward(xt, at, state_out=end)
    a, x, do = (y.astype(np.float64) for y in (a, x, do))
    e, h = np.exp(a), np.zeros(D)
    want = np.empty((T, D))
    for t in range(T):
        h = e[t] * h + x[t]
        want[t] = h
    # A row that is remembered for n rows takes n gates of expf (one unit in the last place of a value below 1, 2^-24) and n
    # roundings of a product or a sum: 2 x 2^-24 a row. The maps of a thread, a warp, a block and a cluster are composed on top of
    # that, up to 8 + 3 + 8 + 8 roundings for rows of the step at hand and one a block for each step before, of 64 rows at least.
    def close(got, ref, size, more=0):
        got = np.asarray(got)
        assert (np.abs(got - ref) <= (2 + 1 / 64) * R.U32 * size + (32 + more) * R.U32 * np.abs(ref)).all()

    size, _ = R.gated_size(x, a)
    kept = out[0].double().cpu().numpy()
    close(kept, want, size)
    close(end[0].double().cpu().numpy(), h, size[-1])
    dx, da, _ = (None if y is None else y[0].double().cpu().numpy() for y in lla.gated_backward(at, out, dot))
    g, k, w = np.zeros(D), np.zeros(D), np.zeros(D)
    rx, ra, sizes = np.empty((T, D)), np.zeros((T, D)), np.empty((T, D))
    for t in reversed(range(T)):
        g = g + do[t]
        w = w + np.abs(do[t])
        k = k + w
        rx[t], sizes[t] = g, k
        g, w, k = g * e[t], w * e[t], k * e[t]
        if t:
            ra[t] = g * kept[t - 1]
    before = np.concatenate([np.zeros((1, D)), kept[:-1]])
    close(dx, rx, sizes, 8)  # a row's own sum and product are two roundings where rows are walked one by one, 8 of them
    close(da, ra, sizes * before, 11)
