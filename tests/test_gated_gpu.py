"""GPU checks of the gated linear recurrence: forward, packed, gradients, single tokens, drafted trees and commits against
sums over rows in 64 bits."""
import numpy as np
import pytest

from tests import _drafts as R
from tests import _linear as L

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture()
def lla():
    from log_linear_attention_gb300 import binding
    yield binding
    assert binding.device_error() == 0


def gate(r, shape, dtype):
    """Log gates from hardly to strongly decaying, channel by channel."""
    rate = np.exp(-6 * r.random(shape[-1]))
    a = (-rate * 2 * r.random(shape)).astype(np.float32)
    t = torch.from_numpy(a)
    if dtype == "bf16":
        t = t.bfloat16()
    return t.double().numpy(), t.cuda()


def normal(r, shape, dtype):
    a, t = L.make(r, shape, dtype)
    return a, t.cuda()


def np64(t):
    return t.double().cpu().numpy()


def one(x, log_a, s0):
    """Reference and size of one sequence, by a loop where the sums would be large."""
    if len(x) > 200:
        h, out = (np.zeros(x.shape[1]) if s0 is None else s0.copy()), np.zeros_like(x)
        a = np.exp(log_a)
        for t in range(len(x)):
            h = a[t] * h + x[t]
            out[t] = h
        return out, out[-1]
    return R.gated(x, log_a, s0)


def one_back(log_a, h, do, s0, ds):
    if len(h) > 200:
        a, g = np.exp(log_a), (np.zeros(h.shape[1]) if ds is None else ds.copy())
        dx, da = np.zeros_like(h), np.zeros_like(h)
        for t in reversed(range(len(h))):
            g = g + do[t]
            dx[t] = g
            da[t] = g * a[t] * (h[t - 1] if t else (0 if s0 is None else s0))
            g = g * a[t]
        return dx, da, g
    return R.gated_grads(log_a, h, do, s0, ds)


def back_size(log_a, do, ds):
    """Sizes of F_{t+1} + dout_t, walked from the end, and of F_0."""
    a = np.exp(log_a)
    g = np.zeros(do.shape[1]) if ds is None else np.abs(ds)
    e = g.copy()
    out = np.zeros_like(do)
    for t in reversed(range(len(do))):
        g = g + np.abs(do[t])
        e = e + g
        out[t] = e
        g, e = a[t] * g, a[t] * e
    return out, e


SIZES = [(1, 1, 1), (2, 1, 64), (3, 2, 5), (1, 7, 4), (2, 8, 63), (1, 9, 66), (2, 127, 20), (1, 128, 65), (2, 129, 8),
         (1, 256, 130), (1, 1023, 12), (2, 1025, 68), (1, 2500, 515), (5, 300, 36)]


@pytest.mark.parametrize("dtype,gt", TYPES)
@pytest.mark.parametrize("B,T,D", SIZES)
def test_forward(lla, B, T, D, dtype, gt):
    r = np.random.default_rng(B * 1000 + T + D)
    (x, xt), (a, at) = normal(r, (B, T, D), dtype), gate(r, (B, T, D), gt)
    for n0 in sorted({0, 1, B}):
        s0, s0t = normal(r, (n0, D), "f32") if n0 else (None, None)
        end = torch.full((B, D), float("nan"), device="cuda")
        out = lla.gated_forward(xt, at, state0=s0t, state_out=end)
        again = lla.gated_forward(xt, at, state0=s0t)
        assert torch.equal(out, again)
        for b in range(B):
            s = None if s0 is None else s0[b if n0 > 1 else 0]
            ref, last = one(x[b], a[b], s)
            size, end_size = R.gated_size(x[b], a[b], s)
            R.gated_check(np64(out[b]), ref, size, dtype, ("out", n0, b))
            R.gated_check(np64(end[b]), last, end_size, "f32", ("state", n0, b))


@pytest.mark.parametrize("dtype,gt", TYPES)
@pytest.mark.parametrize("B,T,D", SIZES)
def test_backward(lla, B, T, D, dtype, gt):
    r = np.random.default_rng(B * 999 + T + D)
    (h, ht), (a, at) = normal(r, (B, T, D), dtype), gate(r, (B, T, D), gt)
    (do, dot) = normal(r, (B, T, D), dtype)
    for n0 in sorted({0, 1, B}):
        s0, s0t = normal(r, (n0, D), "f32") if n0 else (None, None)
        ds, dst = normal(r, (B, D), "f32") if n0 != 1 else (None, None)
        dx, da, dsg = lla.gated_backward(at, ht, dot, state0=s0t, dstate_out=dst)
        assert (dsg is None) == (n0 == 0)
        total, most = 0, 0
        for b in range(B):
            s = None if s0 is None else s0[b if n0 > 1 else 0]
            d = None if ds is None else ds[b]
            rx, ra, rs = one_back(a[b], h[b], do[b], s, d)
            size, s_size = back_size(a[b], do[b], d)
            R.gated_check(np64(dx[b]), rx, size, dtype, ("dx", n0, b))
            before = np.abs(np.concatenate([(np.zeros(D) if s is None else s)[None], h[b][:-1]]))
            R.gated_check(np64(da[b]), ra, size * np.exp(a[b]) * before, gt, ("dlog_a", n0, b), factors=3)
            if n0 > 1:
                R.gated_check(np64(dsg[b]), rs, s_size, "f32", ("dstate0", b))
            total, most = total + rs, most + s_size
        if n0 == 1:
            R.gated_check(np64(dsg[0]), total, most, "f32", "dstate0 of all", factors=B)


PACKS = [([5], 0, 0), ([0, 0], 0, 3), ([1, 1, 1], 0, 0), ([3, 0, 200, 1, 0, 128, 7], 2, 9), ([127, 1, 128, 129, 0], 0, 0),
         ([1100, 40, 1024], 5, 1), ([0] * 40 + [2] * 300, 0, 2), ([2600], 1, 1)]


@pytest.mark.parametrize("dtype,gt", TYPES)
@pytest.mark.parametrize("D", [1, 20, 65, 132])
@pytest.mark.parametrize("lens,lead,tail", PACKS)
def test_packed(lla, lens, lead, tail, D, dtype, gt):
    r = np.random.default_rng(sum(lens) + D)
    n, total = len(lens), max(1, lead + sum(lens) + tail)
    at_ = np.concatenate([[lead], lead + np.cumsum(lens)]).astype(np.int32)
    cu = torch.from_numpy(at_).cuda()
    (x, xt), (a, at), (do, dot) = normal(r, (total, D), dtype), gate(r, (total, D), gt), normal(r, (total, D), dtype)
    # rows of no sequence hold what must not come near the others
    real = np.zeros(total, bool)
    real[lead:lead + sum(lens)] = True
    dead = torch.from_numpy(~real).cuda()
    for t_ in (xt, at, dot):
        t_[dead] = float("nan")
    for n0 in sorted({0, 1, n}):
        s0, s0t = normal(r, (n0, D), "f32") if n0 else (None, None)
        ds, dst = normal(r, (n, D), "f32") if n0 != 1 else (None, None)
        out = torch.full((total, D), 7.0, device="cuda", dtype=xt.dtype)
        end = torch.full((n, D), float("nan"), device="cuda")
        lla.gated_forward_varlen(xt, at, cu, state0=s0t, state_out=end, out=out)
        dx, da, dsg = lla.gated_backward_varlen(at, xt, dot, cu, state0=s0t, dstate_out=dst)
        assert bool((out[dead] == 7).all()) and not dx[dead].any() and not da[dead].any()
        sum_s, sum_size = np.zeros(D), np.zeros(D)
        for b in range(n):
            w = slice(int(at_[b]), int(at_[b + 1]))
            s = None if s0 is None else s0[b if n0 > 1 else 0]
            d = None if ds is None else ds[b]
            if lens[b] == 0:
                assert np.array_equal(np64(end[b]), np.zeros(D) if s is None else s)
                ref_s, s_size = (np.zeros(D) if d is None else d), np.zeros(D)
                if n0 > 1:
                    assert np.array_equal(np64(dsg[b]), ref_s)
            else:
                ref, last = one(x[w], a[w], s)
                size, end_size = R.gated_size(x[w], a[w], s)
                R.gated_check(np64(out[w]), ref, size, dtype, ("out", n0, b))
                R.gated_check(np64(end[b]), last, end_size, "f32", ("state", n0, b))
                rx, ra, ref_s = one_back(a[w], x[w], do[w], s, d)
                size, s_size = back_size(a[w], do[w], d)
                R.gated_check(np64(dx[w]), rx, size, dtype, ("dx", n0, b))
                before = np.abs(np.concatenate([(np.zeros(D) if s is None else s)[None], x[w][:-1]]))
                R.gated_check(np64(da[w]), ra, size * np.exp(a[w]) * before, gt, ("dlog_a", n0, b), factors=3)
                if n0 > 1:
                    R.gated_check(np64(dsg[b]), ref_s, s_size, "f32", ("dstate0", b))
            sum_s, sum_size = sum_s + ref_s, sum_size + np.abs(ref_s) + s_size
        if n0 == 1:
            R.gated_check(np64(dsg[0]), sum_s, sum_size, "f32", "dstate0 of all", factors=0)


@pytest.mark.parametrize("dtype,gt", TYPES)
@pytest.mark.parametrize("B,T,D", [(4, 1100, 96), (40, 1100, 64), (3, 530, 24), (160, 140, 72), (1, 9000, 32)])
def test_every_cut_of_the_channels(lla, B, T, D, dtype, gt):
    """Columns of 64, 32 and 16 channels, clusters of one to eight blocks, several steps, rows of whole 16-byte pieces."""
    r = np.random.default_rng(B + T + D)
    (x, xt), (a, at), (do, dot) = normal(r, (B, T, D), dtype), gate(r, (B, T, D), gt), normal(r, (B, T, D), dtype)
    (s0, s0t), (ds, dst) = normal(r, (B, D), "f32"), normal(r, (B, D), "f32")
    end = torch.empty(B, D, device="cuda")
    out = lla.gated_forward(xt, at, state0=s0t, state_out=end)
    dx, da, dsg = lla.gated_backward(at, xt, dot, state0=s0t, dstate_out=dst)
    # all sequences at once, row by row
    e, h, g, w = np.exp(a), s0.copy(), ds.copy(), np.abs(ds)
    sizes, k = np.abs(s0), np.abs(s0)
    want, size = np.empty_like(x), np.empty_like(x)
    for t in range(T):
        h = e[:, t] * h + x[:, t]
        sizes = e[:, t] * sizes + np.abs(x[:, t])
        k = e[:, t] * k + sizes
        want[:, t], size[:, t] = h, k
    R.gated_check(np64(out), want, size, dtype, "out")
    R.gated_check(np64(end), h, k, "f32", "state")
    rx, ra, back = np.empty_like(x), np.empty_like(x), np.empty_like(x)
    k = w.copy()
    for t in reversed(range(T)):
        g = g + do[:, t]
        w = w + np.abs(do[:, t])
        k = k + w
        rx[:, t], back[:, t] = g, k
        ra[:, t] = g * e[:, t] * (x[:, t - 1] if t else s0)
        g, w, k = g * e[:, t], w * e[:, t], k * e[:, t]
    R.gated_check(np64(dx), rx, back, dtype, "dx")
    before = np.abs(np.concatenate([s0[:, None], x[:, :-1]], 1))
    R.gated_check(np64(da), ra, back * e * before, gt, "dlog_a", factors=3)
    R.gated_check(np64(dsg), g, k, "f32", "dstate0")


@pytest.mark.parametrize("D", [8, 40, 264])
@pytest.mark.parametrize("lens,lead,tail", PACKS + [([700, 0, 1, 900, 33, 0, 0, 5] * 3, 3, 2)])
def test_packed_rows_of_16_bytes(lla, lens, lead, tail, D):
    """Packed rows that come by TMA, in bf16 with gates of both types."""
    for gt in ("f32", "bf16"):
        r = np.random.default_rng(sum(lens) + D)
        n, total = len(lens), max(1, lead + sum(lens) + tail)
        at_ = np.concatenate([[lead], lead + np.cumsum(lens)])
        cu = torch.from_numpy(at_.astype(np.int32)).cuda()
        (x, xt), (a, at), (do, dot) = normal(r, (total, D), "bf16"), gate(r, (total, D), gt), normal(r, (total, D), "bf16")
        (s0, s0t), (ds, dst) = normal(r, (n, D), "f32"), normal(r, (n, D), "f32")
        end, out = torch.full((n, D), float("nan"), device="cuda"), torch.full((total, D), 7.0, device="cuda").bfloat16()
        lla.gated_forward_varlen(xt, at, cu, state0=s0t, state_out=end, out=out)
        dx, da, dsg = lla.gated_backward_varlen(at, xt, dot, cu, state0=s0t, dstate_out=dst)
        for b in range(n):
            w = slice(int(at_[b]), int(at_[b + 1]))
            s, d = s0[b], ds[b]
            if lens[b] == 0:
                assert np.array_equal(np64(end[b]), s) and np.array_equal(np64(dsg[b]), d)
                continue
            ref, last = one(x[w], a[w], s)
            size, end_size = R.gated_size(x[w], a[w], s)
            R.gated_check(np64(out[w]), ref, size, "bf16", ("out", b))
            R.gated_check(np64(end[b]), last, end_size, "f32", ("state", b))
            rx, ra, rs = one_back(a[w], x[w], do[w], s, d)
            size, s_size = back_size(a[w], do[w], d)
            R.gated_check(np64(dx[w]), rx, size, "bf16", ("dx", b))
            before = np.abs(np.concatenate([s[None], x[w][:-1]]))
            R.gated_check(np64(da[w]), ra, size * np.exp(a[w]) * before, gt, ("dlog_a", b), factors=3)
            R.gated_check(np64(dsg[b]), rs, s_size, "f32", ("dstate0", b))


def test_two_streams_at_once(lla):
    """Calls side by side on two streams, of clusters that fill the GPU together: as alone."""
    x = torch.randn(4, 4096, 512, device="cuda").bfloat16()
    a = -torch.rand(4, 4096, 512, device="cuda")
    s0 = torch.randn(1, 512, device="cuda")
    want = lla.gated_forward(x, a, state0=s0)
    grads = lla.gated_backward(a, want, x, state0=s0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream(priority=-1)]
    got = []
    for i in range(6):
        s = streams[i % 2]
        got.append((lla.gated_forward(x, a, state0=s0, stream=s), lla.gated_backward(a, want, x, state0=s0, stream=s)))
    torch.cuda.synchronize()
    for out, g in got:
        assert torch.equal(out, want) and all(torch.equal(p, q) for p, q in zip(g, grads))


def test_values_that_are_not_finite_stay_where_they_belong(lla):
    T, D = 700, 8
    r = np.random.default_rng(1)
    for dtype in ("bf16", "f32"):
        (_, x), (_, a) = normal(r, (T, D), dtype), gate(r, (T, D), "f32")
        cu = torch.tensor([0, 200, 200, 450, 700], dtype=torch.int32, device="cuda")
        clean = lla.gated_forward_varlen(x, a, cu)
        bad = x.clone()
        bad[210, 3] = float("inf")
        bad[300, 5] = float("nan")
        out = lla.gated_forward_varlen(bad, a, cu)
        hit = torch.zeros(T, D, dtype=torch.bool, device="cuda")
        hit[210:450, 3] = True
        hit[300:450, 5] = True
        assert torch.equal(out[~hit], clean[~hit]) and not torch.isfinite(out[hit]).any()
        # gradients: earlier rows of the same sequence and channel
        dx, da, _ = lla.gated_backward_varlen(a, clean, x, cu)
        bx, ba, _ = lla.gated_backward_varlen(a, clean, bad, cu)
        hit[:] = False
        hit[200:211, 3] = True
        hit[200:301, 5] = True
        assert torch.equal(bx[~hit], dx[~hit]) and torch.equal(ba[~hit], da[~hit])
        assert not torch.isfinite(bx[hit]).any()


def test_gates_of_zero(lla):
    """log_a = -inf forgets: rows from there on are those of a new sequence, and nothing flows back past it."""
    T, D = 300, 12
    r = np.random.default_rng(2)
    (_, x), (_, a) = normal(r, (1, T, D), "f32"), gate(r, (1, T, D), "f32")
    a[0, 140] = -float("inf")
    out = lla.gated_forward(x, a)
    tail = lla.gated_forward(x[:, 140:].contiguous(), a[:, 140:].contiguous())
    ref, _ = one(np64(x[0, 140:]), np.where(np.isinf(np64(a[0, 140:])), -800.0, np64(a[0, 140:])), None)
    size, _ = R.gated_size(np64(x[0, 140:]), np.where(np.isinf(np64(a[0, 140:])), -800.0, np64(a[0, 140:])))
    R.gated_check(np64(out[0, 140:]), ref, size, "f32", "after")
    R.gated_check(np64(tail[0]), ref, size, "f32", "alone")
    dx, da, _ = lla.gated_backward(a, out, x)
    hx, ha, _ = lla.gated_backward(a[:, :140].contiguous(), out[:, :140].contiguous(), x[:, :140].contiguous())
    assert not da[0, 140].any() and torch.isfinite(dx).all()
    for got, alone in ((dx, hx), (da, ha)):
        assert (got[:, :140] - alone).abs().max() <= 1e-5 * alone.abs().max()


@pytest.mark.parametrize("cu", [[0, 9, 5, 20], [-1, 5, 20, 20], [0, 5, 20, 51], [3, 2, 20, 50]])
def test_bad_bounds_write_nothing(lla, cu):
    x, a = torch.randn(50, 20, device="cuda"), -torch.rand(50, 20, device="cuda")
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    out, end = torch.full((50, 20), 7.0, device="cuda"), torch.full((3, 20), 7.0, device="cuda")
    lla.gated_forward_varlen(x, a, cu, state_out=end, out=out)
    assert lla.device_error() == lla.LLA_ERR_DEVICE
    assert bool((out == 7).all()) and bool((end == 7).all())
    lla.gated_backward_varlen(a, x, x, cu)
    assert lla.device_error() == lla.LLA_ERR_DEVICE


@pytest.mark.parametrize("cu", [[0, 9, 5, 20], [-1, 3, 9, 20], [0, 3, 9, 21]])
def test_bad_bounds_leave_the_shared_gradient(lla, cu):
    """The gradient of one shared state is a sum over the sequences, in a launch of its own."""
    x, a = torch.ones(20, 24, device="cuda"), torch.zeros(20, 24, device="cuda")
    s0, c = torch.zeros(1, 24, device="cuda"), torch.tensor(cu, dtype=torch.int32, device="cuda")
    dx, da, ds = torch.full_like(x, 7.0), torch.full_like(x, 7.0), torch.full_like(s0, 7.0)
    stream = torch.cuda.current_stream().cuda_stream
    status = lla.load().lla_gated_backward_varlen(
        a.data_ptr(), x.data_ptr(), s0.data_ptr(), x.data_ptr(), None, dx.data_ptr(), da.data_ptr(), ds.data_ptr(),
        c.data_ptr(), 3, 1, 20, 24, stream, lla.LLA_F32, lla.LLA_F32)
    assert status == lla.LLA_OK
    assert lla.device_error() == lla.LLA_ERR_DEVICE
    assert all(bool((t == 7.0).all()) for t in (dx, da, ds))


def test_prompts_go_on_from_states(lla):
    r = np.random.default_rng(3)
    for dtype, gt in TYPES:
        (_, x), (_, a) = normal(r, (2, 700, 68), dtype), gate(r, (2, 700, 68), gt)
        end, mid, last = (torch.empty(2, 68, device="cuda") for _ in range(3))
        whole = lla.gated_forward(x, a, state_out=end)
        p = lla.gated_forward(x[:, :333].contiguous(), a[:, :333].contiguous(), state_out=mid)
        q = lla.gated_forward(x[:, 333:].contiguous(), a[:, 333:].contiguous(), state0=mid, state_out=last)
        # Two fp32 results of one value v, each within 2^-21 of the size (gated_check), are 2^-20 of it apart at most;
        # rounded to bf16 each moves by half a step, 2^-8 |v|, so the outputs by 2 x 2^-8 |v| more.
        size, size_end = zip(*(R.gated_size(np64(x[b]), np64(a[b])) for b in range(2)))
        size, size_end = np.stack(size), np.stack(size_end)

        def close(got, want, size, rounded):
            got, want = np64(got), np64(want)
            bound = 2.0 ** -20 * size
            if rounded:
                bound = bound + 2 * R.UBF * (np.abs(want) * (1 + R.UBF) + bound)
            else:
                bound = bound + 2 * R.U32 * np.abs(want)
            assert (np.abs(got - want) <= bound).all()

        close(torch.cat([p, q], 1), whole, size, dtype == "bf16")
        close(last, end, size_end, False)
        # single tokens
        state = mid.clone()
        for t in range(333, 340):
            o = lla.gated_decode_step(x[:, t].contiguous(), a[:, t].contiguous(), state)
            close(o, whole[:, t], size[:, t], dtype == "bf16")


@pytest.mark.parametrize("dtype,gt", TYPES)
@pytest.mark.parametrize("B,D", [(1, 1), (3, 5), (2, 64), (64, 1024), (7, 515)])
def test_step(lla, B, D, dtype, gt):
    r = np.random.default_rng(B + D)
    (x, xt), (a, at), (s, st) = normal(r, (B, D), dtype), gate(r, (B, D), gt), normal(r, (B, D), "f32")
    out = lla.gated_decode_step(xt, at, st)
    ref = np.exp(a) * s + x
    size = 2 * (np.abs(np.exp(a) * s) + np.abs(x))
    R.gated_check(np64(st), ref, size, "f32", "state")
    R.gated_check(np64(out), ref, size, dtype, "out")


@pytest.mark.parametrize("dtype,gt", TYPES)
@pytest.mark.parametrize("B,N,D,one_tree", [(1, 1, 1, True), (3, 7, 5, False), (2, 32, 64, False), (5, 128, 70, True),
                                            (2, 128, 130, False), (4, 19, 515, True)])
def test_tree_and_commit(lla, B, N, D, one_tree, dtype, gt):
    r = np.random.default_rng(N + D)
    (x, xt), (a, at), (s, st) = normal(r, (B, N, D), dtype), gate(r, (B, N, D), gt), normal(r, (B, D), "f32")
    trees = [R.random_tree(r, N, int(r.integers(1, N + 1)), 0.7)] * B if one_tree else [
        R.random_tree(r, N, int(r.integers(1, N + 1))) for _ in range(B)]
    parent = torch.tensor(trees[0] if one_tree else trees, dtype=torch.int32, device="cuda")
    dead = torch.tensor(trees, device="cuda") == -2
    xt[dead], at[dead] = float("nan"), float("nan")
    out = torch.full((B, N, D), 7.0, device="cuda", dtype=xt.dtype)
    assert lla.gated_decode_tree(xt, at, st, parent, out=out) is out
    assert bool((out[dead] == 7).all())
    paths = []
    for b in range(B):
        live = [i for i in range(N) if trees[b][i] > -2]
        for i in live:
            way = R.branch(trees[b], i)
            ref, _ = R.gated(x[b][way], a[b][way], s[b])
            size, _ = R.gated_size(x[b][way], a[b][way], s[b])
            R.gated_check(np64(out[b, i]), ref[-1], size[-1], dtype, (b, i))
        paths.append(R.branch(trees[b], live[-1])[:int(r.integers(0, N + 1))])
    M = max(1, max(len(p) for p in paths))
    path = torch.tensor([p + [1 << 30] * (M - len(p)) for p in paths], dtype=torch.int32, device="cuda")
    count = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
    got = lla.gated_decode_commit(xt, at, st, count, path)
    assert got is st
    for b in range(B):
        if paths[b]:
            _, ref = R.gated(x[b][paths[b]], a[b][paths[b]], s[b])
            _, size = R.gated_size(x[b][paths[b]], a[b][paths[b]], s[b])
            R.gated_check(np64(st[b]), ref, size, "f32", ("state", b))
        else:
            assert np.array_equal(np64(st[b]), s[b])
    # without a path: the first tokens
    xt, at = (torch.nan_to_num(y) for y in (xt, at))
    first = torch.tensor([int(r.integers(0, N + 1)) for _ in range(B)], dtype=torch.int32, device="cuda")
    one_, two = st.clone(), st.clone()
    lla.gated_decode_commit(xt, at, one_, first)
    lla.gated_decode_commit(xt, at, two, first, torch.arange(N, dtype=torch.int32, device="cuda").repeat(B, 1))
    assert torch.equal(one_, two)


def test_bad_trees_are_skipped(lla):
    B, N, D = 6, 5, 70
    x, a, s = torch.randn(B, N, D, device="cuda"), -torch.rand(B, N, D, device="cuda"), torch.randn(B, D, device="cuda")
    parent = torch.tensor([[-1, 0, 1, 2, 3], [-1, 1, 0, 0, 0], [-3, 0, 0, 0, 0], [-1, -2, 1, 0, 0], [0, 0, 0, 0, 0],
                           [-1, -1, -1, 1 << 30, 0]], dtype=torch.int32, device="cuda")
    out = torch.full((B, N, D), 7.0, device="cuda")
    lla.gated_decode_tree(x, a, s, parent, out=out)
    assert lla.device_error() == lla.LLA_ERR_DEVICE
    assert bool((out[1:] == 7).all()) and not bool((out[0] == 7).any())
    s0 = s.clone()
    count = torch.tensor([2, -1, 4, 3, 0, 3], dtype=torch.int32, device="cuda")
    path = torch.tensor([[0, 1, 9], [0, 1, 2], [0, 1, 2], [0, 5, 1], [9, 9, 9], [0, -1, 1]], dtype=torch.int32, device="cuda")
    lla.gated_decode_commit(x, a, s, count, path)
    assert lla.device_error() == lla.LLA_ERR_DEVICE
    assert torch.equal(s[1:], s0[1:]) and not bool((s[0] == s0[0]).any())
    lla.gated_decode_commit(x, a, s, torch.full((B,), N + 1, dtype=torch.int32, device="cuda"))
    assert lla.device_error() == lla.LLA_ERR_DEVICE and torch.equal(s[1:], s0[1:])


def test_graphs_and_streams(lla):
    B, T, D = 3, 1500, 132
    x = torch.randn(B, T, D, device="cuda").bfloat16()
    a, do, s0 = -torch.rand(B, T, D, device="cuda"), torch.randn_like(x), torch.randn(1, D, device="cuda")
    end = torch.empty(B, D, device="cuda")
    out = lla.gated_forward(x, a, state0=s0, state_out=end)
    grads = lla.gated_backward(a, out, do, state0=s0, dstate_out=end)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    end2 = torch.empty_like(end)
    out2 = lla.gated_forward(x, a, state0=s0, state_out=end2, stream=side)
    grads2 = lla.gated_backward(a, out2, do, state0=s0, dstate_out=end2, stream=side)
    side.synchronize()
    assert torch.equal(out, out2) and all(torch.equal(p, q) for p, q in zip(grads, grads2))
    g = torch.cuda.CUDAGraph()
    end3 = torch.zeros_like(end)
    with torch.cuda.graph(g):
        out3 = lla.gated_forward(x, a, state0=s0, state_out=end3)
        grads3 = lla.gated_backward(a, out3, do, state0=s0, dstate_out=end3)
    for _ in range(2):
        out3.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, out3) and all(torch.equal(p, q) for p, q in zip(grads, grads3))


def test_more_than_2_31_elements(lla):
    """Rows behind element 2^31: those of the last ones alone, going on from the state before them."""
    T, D = 2_100_000, 1032
    x = torch.empty(1, T, D, dtype=torch.bfloat16, device="cuda").normal_()
    a = torch.empty(1, T, D, dtype=torch.bfloat16, device="cuda").uniform_(-1, 0)
    end = torch.empty(1, D, device="cuda")
    out = lla.gated_forward(x, a, state_out=end)
    n = T - 2048 * 1024  # both walks then take the rows in the same pieces
    x1, a1 = x[:, -n:].contiguous(), a[:, -n:].contiguous()
    tail = lla.gated_forward(x1, a1, state0=out[0, -n - 1:-n].float().contiguous())
    # the state before them was rounded to bf16; gates of e^-0.5 on average forget it within some 50 rows
    assert torch.equal(out[:, -n + 200:], tail[:, 200:])
    dx, da, _ = lla.gated_backward(a, out, x)
    tx, ta, _ = lla.gated_backward(a1, tail, x1)
    assert torch.equal(dx[:, -n + 200:], tx[:, 200:]) and torch.equal(da[:, -n + 201:], ta[:, 201:])


@pytest.mark.parametrize("B,T,D,packed", [(2, 3000, 64, False), (3, 40, 64, False), (1, 3000, 65, False), (1, 3000, 32, True)])
def test_a_wait_that_runs_out_is_reported(lla, B, T, D, packed):
    """The hook lets every block wait for what never comes, for half a millisecond; the walk ends, the status is read, and
    the next call is right."""
    x, a = torch.randn(B, T, D, device="cuda"), -torch.rand(B, T, D, device="cuda")
    cu = torch.tensor([0, 1000, 3000], dtype=torch.int32, device="cuda")

    def calls():
        out = lla.gated_forward_varlen(x[0], a[0], cu) if packed else lla.gated_forward(x, a)
        return out, (lla.gated_backward_varlen(a[0], x[0], x[0], cu) if packed else lla.gated_backward(a, x, x))[0]

    want = calls()
    lla.debug_set_waits(1_000_000, hold=True)
    try:
        calls()
        status = lla.device_error()
    finally:
        lla.debug_set_waits(0, hold=False)
    assert status == lla.LLA_ERR_TIMEOUT
    for got, ref in zip(calls(), want):
        assert torch.equal(got, ref)
