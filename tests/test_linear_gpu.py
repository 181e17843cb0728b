"""GPU checks of linear attention with one decay per head against the 64-bit pair sums of tests/_linear.py."""
import numpy as np
import pytest

from tests import _linear as L

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


def slopes(H, seed=0):
    """Decays from fast (about 0.5) to slow (about 0.996), one head without decay, one that forgets at once."""
    la = -np.exp2(-8.0 * np.arange(1, H + 1) / H) * (0.9 + 0.2 * np.random.default_rng(seed).random(H))
    if H >= 3:
        la[1] = 0.0
        la[2] = -np.inf
    return la.astype(np.float32)


def problem(B, H, T, dk, dv, dtype, B0, seed=0):
    """{name: (float64 array, CUDA tensor)}"""
    r = np.random.default_rng(seed)
    p = {"q": L.make(r, (B, H, T, dk), dtype, dk ** -0.5), "k": L.make(r, (B, H, T, dk), dtype, dk ** -0.5),
         "v": L.make(r, (B, H, T, dv), dtype), "dout": L.make(r, (B, H, T, dv), dtype),
         "ds": L.make(r, (B, H, dk, dv), "f32", dk ** -0.5)}
    if B0:
        p["s0"] = L.make(r, (B0, H, dk, dv), "f32", dk ** -0.5)
    la = slopes(H, seed)
    p["la"] = la.astype(np.float64), torch.from_numpy(la)
    return {n: (a, t.cuda()) for n, (a, t) in p.items()}


def val(p, n):
    return p[n][0] if n in p else None


def dev(p, n):
    return p[n][1] if n in p else None


def sizes(*x):
    return [None if a is None else np.abs(a) for a in x]


def host(t):
    return t.double().cpu().numpy()


SHAPES = [
    # B, H, T, dk, dv, dtype, B0
    (1, 1, 1, 64, 64, "bf16", 0), (3, 4, 1, 128, 64, "bf16", 3), (2, 3, 2, 16, 8, "bf16", 1),
    (2, 3, 63, 64, 128, "bf16", 2), (1, 4, 64, 128, 128, "bf16", 1), (2, 4, 65, 8, 24, "bf16", 0),
    (1, 4, 127, 72, 80, "bf16", 1), (2, 4, 128, 128, 64, "bf16", 2), (1, 5, 129, 64, 64, "bf16", 0),
    (2, 4, 255, 96, 72, "bf16", 2), (2, 4, 256, 128, 128, "bf16", 0), (2, 8, 700, 128, 128, "bf16", 1),
    (1, 4, 1301, 80, 104, "bf16", 1), (1, 4, 300, 50, 33, "bf16", 1), (2, 3, 130, 127, 128, "bf16", 2),
    (1, 1, 1, 1, 1, "f32", 0), (2, 3, 1, 20, 30, "f32", 2), (1, 4, 64, 64, 64, "f32", 1), (2, 4, 65, 128, 128, "f32", 2),
    (2, 4, 200, 100, 36, "f32", 1), (1, 3, 1000, 17, 65, "f32", 0),
]


@pytest.mark.parametrize("B,H,T,dk,dv,dtype,B0", SHAPES)
def test_forward(lla, B, H, T, dk, dv, dtype, B0):
    p = problem(B, H, T, dk, dv, dtype, B0, seed=T)
    s1 = torch.full((B, H, dk, dv), float("nan"), device="cuda")
    out = lla.linear_forward(dev(p, "q"), dev(p, "k"), dev(p, "v"), dev(p, "la"), state0=dev(p, "s0"), state_out=s1)
    x = [val(p, n) for n in ("q", "k", "v", "la", "s0")]
    ref, ref_s = L.forward(*x)
    size, size_s = L.forward(*sizes(*x[:3]), x[3], *sizes(x[4]))
    L.check(host(out), ref, size, dtype, T + dk, "out")
    L.check(host(s1), ref_s, size_s, "f32", T, "state")
    # without a state to write, the outputs are the same
    again = lla.linear_forward(dev(p, "q"), dev(p, "k"), dev(p, "v"), dev(p, "la"), state0=dev(p, "s0"))
    assert torch.equal(out, again)


@pytest.mark.parametrize("B,H,T,dk,dv,dtype,B0", SHAPES)
def test_backward(lla, B, H, T, dk, dv, dtype, B0):
    p = problem(B, H, T, dk, dv, dtype, B0, seed=T + 1)
    got = lla.linear_backward(*(dev(p, n) for n in ("q", "k", "v", "la", "dout")), state0=dev(p, "s0"),
                              dstate_out=dev(p, "ds"))
    x = [val(p, n) for n in ("q", "k", "v", "la", "dout", "s0", "ds")]
    ref = list(L.backward(*x))
    size = list(L.backward(*sizes(*x[:3]), x[3], *sizes(*x[4:])))
    for n, i in (("dq", 0), ("dk", 1), ("dv", 2)):
        L.check(host(got[i]), ref[i], size[i], dtype, T + max(dk, dv), n)
    if not B0:
        assert got[3] is None
        return
    if B0 == 1:
        ref[3], size[3] = ref[3].sum(0, keepdims=True), size[3].sum(0, keepdims=True)
    L.check(host(got[3]), ref[3], size[3], "f32", T + B, "dstate0")


@pytest.mark.parametrize("B,H,T,dk,dv", [(1, 7, 1100, 128, 64), (2, 9, 700, 128, 128), (3, 11, 900, 64, 128),
                                         (1, 5, 800, 72, 40), (2, 8, 1300, 64, 64), (1, 16, 2000, 8, 128)])
def test_backward_where_blocks_begin_inside_chunks(lla, B, H, T, dk, dv):
    """More pieces of work than blocks, and not a multiple: every block begins and ends at another place of a chunk."""
    test_backward(lla, B, H, T, dk, dv, "bf16", 1)


@pytest.mark.parametrize("B,H,T,dk,dv", [(8, 16, 1562, 128, 64), (8, 16, 1562, 96, 104), (8, 16, 1562, 64, 64)])
def test_many_heads_whose_last_chunk_is_ragged(lla, B, H, T, dk, dv):
    """More heads than SMs, so that copies and products are apart by as much as the rings allow: every head against the
    CUDA cores' fp32 arithmetic on the same values (5e-3 of a head's norm, see tests/_linear.py: that arithmetic's own
    error is a thousandth of it), and every repetition the same to the bit."""
    g = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k = (rand(B, H, T, dk).mul_(dk ** -0.5).bfloat16() for _ in range(2))
    v, do = (rand(B, H, T, dv).bfloat16() for _ in range(2))
    la = -torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)

    def run(*x):
        return lla.linear_forward(x[0], x[1], x[2], la), *lla.linear_backward(x[0], x[1], x[2], la, x[3])[:3]

    ref = run(q.float(), k.float(), v.float(), do.float())
    first = None
    for _ in range(8):
        got = run(q, k, v, do)
        first = first or got
        for n, x, y, r in zip(("out", "dq", "dk", "dv"), got, first, ref):
            rel = (x.float() - r).norm(dim=(2, 3)) / r.norm(dim=(2, 3))
            assert float(rel.max()) <= 5e-3, (n, int(rel.argmax()), float(rel.max()))
            assert torch.equal(x, y), n


def test_calls_of_several_threads_do_not_meet(lla):
    """Prompts and gradients from threads with streams of their own give what they give alone, to the bit."""
    import threading

    def calls(seed):
        p = problem(2, 4, 700 + 100 * seed, 64, 64, "bf16", 1, seed)
        args = [dev(p, n) for n in ("q", "k", "v", "la")]
        return lambda: (lla.linear_forward(*args, state0=dev(p, "s0")),
                        *lla.linear_backward(*args, dev(p, "dout"), state0=dev(p, "s0"), dstate_out=dev(p, "ds")))

    jobs = [calls(seed) for seed in range(3)]
    alone = [job() for job in jobs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = jobs[i]()
                s.synchronize()
                if not all(torch.equal(x, y) for x, y in zip(got, alone[i])):
                    wrong.append(i)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_backward_without_state_gradient(lla):
    p = problem(2, 3, 150, 64, 64, "bf16", 0)
    got = lla.linear_backward(*(dev(p, n) for n in ("q", "k", "v", "la", "dout")))
    x = [val(p, n) for n in ("q", "k", "v", "la", "dout")]
    ref, size = L.backward(*x), L.backward(*sizes(*x[:3]), x[3], *sizes(x[4]))
    for i in range(3):
        L.check(host(got[i]), ref[i], size[i], "bf16", 214, i)


@pytest.mark.parametrize("dk,dv", [(16, 8), (128, 64), (12, 6)])
def test_backward_is_the_forward_s_difference(lla, dk, dv):
    """Along random directions: fp32 inputs, loss in 64 bits from fp32 outputs. The loss is linear in each input,
    so the difference over +-1 of a direction has no error but the forward's roundings: at most
    (T + dk + 16) 2^-23 of the terms' sizes for each side."""
    B, H, T = 2, 3, 70
    p = problem(B, H, T, dk, dv, "f32", 2, seed=5)
    args = {n: dev(p, n) for n in ("q", "k", "v", "s0")}

    def loss(a):
        s1 = torch.empty(B, H, dk, dv, device="cuda")
        o = lla.linear_forward(a["q"], a["k"], a["v"], dev(p, "la"), state0=a["s0"], state_out=s1)
        return float((o.double() * dev(p, "dout").double()).sum() + (s1.double() * dev(p, "ds").double()).sum())

    def total(a):
        o, s = L.forward(*sizes(a["q"], a["k"], a["v"]), val(p, "la"), *sizes(a["s0"]))
        return (o * np.abs(val(p, "dout"))).sum() + (s * np.abs(val(p, "ds"))).sum()

    grads = dict(zip(("q", "k", "v", "s0"), lla.linear_backward(args["q"], args["k"], args["v"], dev(p, "la"),
                                                                 dev(p, "dout"), state0=args["s0"],
                                                                 dstate_out=dev(p, "ds"))))
    r = np.random.default_rng(6)
    for n, x in args.items():
        d = torch.from_numpy(np.sign(r.standard_normal(x.shape)).astype(np.float32) * 0.25).cuda()
        up, down = {**args, n: x + d}, {**args, n: x - d}
        diff = (loss(up) - loss(down)) / 2
        want = float((grads[n].double() * d.double()).sum())
        tol = (T + dk + 16) * 2 * L.U32 * max(total({m: host(t) for m, t in a.items()}) for a in (up, down)) * 2
        assert abs(diff - want) <= tol, (n, diff, want, tol)


def pack(lengths, H, dk, dv, dtype, n0, tail, seed):
    r = np.random.default_rng(seed)
    total = sum(lengths) + tail
    p = {"q": L.make(r, (H, total, dk), dtype, dk ** -0.5), "k": L.make(r, (H, total, dk), dtype, dk ** -0.5),
         "v": L.make(r, (H, total, dv), dtype)}
    if n0:
        p["s0"] = L.make(r, (n0, H, dk, dv), "f32", dk ** -0.5)
    la = slopes(H, seed)
    p["la"] = la.astype(np.float64), torch.from_numpy(la)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    return {n: (a, t.cuda()) for n, (a, t) in p.items()}, cu


def check_packed(p, cu, out, s1, dtype, skip=()):
    n = len(cu) - 1
    for b in range(n):
        if b in skip:
            continue
        rows = slice(cu[b], cu[b + 1])
        T = cu[b + 1] - cu[b]
        s0 = val(p, "s0")
        s0 = None if s0 is None else s0[b if s0.shape[0] > 1 else 0][None]
        if T == 0:
            want = np.zeros_like(s1[b]) if s0 is None else s0[0]
            assert np.array_equal(s1[b], want)
            continue
        x = [val(p, m)[None, :, rows] for m in ("q", "k", "v")] + [val(p, "la"), s0]
        ref, ref_s = L.forward(*x)
        size, size_s = L.forward(*sizes(*x[:3]), x[3], *sizes(s0))
        L.check(out[None, :, rows], ref, size, dtype, T + x[0].shape[-1], f"out {b}")
        L.check(s1[None, b], ref_s, size_s, "f32", T, f"state {b}")


@pytest.mark.parametrize("lengths,H,dk,dv,dtype,n0,tail", [
    ([1], 3, 64, 64, "bf16", 0, 0), ([0, 0, 5, 0], 3, 64, 64, "bf16", 4, 3), ([0], 2, 64, 32, "bf16", 1, 4),
    ([1, 37, 128, 300, 129, 0, 257, 1], 4, 128, 64, "bf16", 1, 130), ([700, 3, 128, 64], 3, 64, 128, "bf16", 4, 1),
    ([100, 31, 200], 4, 24, 40, "bf16", 0, 9), ([1, 63, 64, 65, 0, 200], 3, 20, 36, "f32", 6, 70),
    ([5, 130], 3, 128, 128, "f32", 1, 0), ([90, 2], 3, 30, 50, "bf16", 1, 2),
])
def test_varlen(lla, lengths, H, dk, dv, dtype, n0, tail):
    p, cu = pack(lengths, H, dk, dv, dtype, n0, tail, seed=len(lengths))
    n, total = len(lengths), sum(lengths) + tail
    out = torch.full((H, total, dv), 7.0, device="cuda", dtype=p["q"][1].dtype)
    s1 = torch.full((n, H, dk, dv), float("nan"), device="cuda")
    got = lla.linear_forward_varlen(dev(p, "q"), dev(p, "k"), dev(p, "v"), dev(p, "la"), torch.from_numpy(cu).cuda(),
                                    max(max(lengths), 1), state0=dev(p, "s0"), state_out=s1, out=out)
    assert got is out
    o = host(out)
    check_packed(p, cu, o, host(s1), dtype)
    assert (o[:, cu[-1]:] == 7.0).all()


@pytest.mark.parametrize("dtype,dk", [("bf16", 64), ("f32", 64), ("bf16", 20)])
def test_varlen_rows_of_others_never_reach_a_sequence(lla, dtype, dk):
    """Every row outside the sequences under test holds NaN or infinities."""
    lengths, H, dv = [70, 130, 1, 200, 40], 3, 64
    p, cu = pack(lengths, H, dk, dv, dtype, 0, 60, seed=3)
    bad = [b for b in range(5) if b % 2]
    for n in ("q", "k", "v"):
        for b in bad:
            p[n][1][:, cu[b]:cu[b + 1]] = float("nan") if b == 1 else float("inf")
        p[n][1][:, cu[-1]:] = float("-inf")
    s1 = torch.zeros(5, H, dk, dv, device="cuda")
    out = torch.zeros(H, sum(lengths) + 60, dv, device="cuda", dtype=p["q"][1].dtype)
    lla.linear_forward_varlen(dev(p, "q"), dev(p, "k"), dev(p, "v"), dev(p, "la"), torch.from_numpy(cu).cuda(), 200,
                              state_out=s1, out=out)
    check_packed(p, cu, host(out), host(s1), dtype, skip=bad)
    assert (host(out)[:, cu[-1]:] == 0).all()


def test_values_that_are_not_finite_obey_causality_beyond_their_chunk(lla):
    """An infinity in v at token t leaves every row of earlier 128-token chunks as it was, and one in k or q every
    earlier row."""
    for name, t, first in (("v", 300, 256), ("k", 300, 300), ("q", 300, 300)):
        p = problem(1, 2, 500, 64, 64, "bf16", 0, seed=8)
        args = {n: dev(p, n).clone() for n in ("q", "k", "v")}
        clean = lla.linear_forward(*args.values(), dev(p, "la"))
        args[name][:, :, t] = float("nan")
        out = lla.linear_forward(*args.values(), dev(p, "la"))
        assert torch.equal(out[:, :, :first], clean[:, :, :first]), name
        if name == "q":
            assert torch.equal(out[:, :, t + 1:], clean[:, :, t + 1:])
        assert not torch.isfinite(out[:, :, t].float()).any()


@pytest.mark.parametrize("dk,dtype", [(64, "bf16"), (32, "f32")])
def test_varlen_bad_bounds_are_reported_and_skipped(dk, dtype):
    from log_linear_attention_gb300 import binding as lla
    lengths, H, dv = [50, 60, 70, 80], 2, 64
    p, good = pack(lengths, H, dk, dv, dtype, 0, 0, seed=4)
    for bad, skip in (([0, 50, 110, 40, 260], (2,)),      # falls: sequence 2 is out, 3 starts below row 110
                      ([0, 50, 110, 180, 300], (3,)),     # past the tensor
                      ([-5, 50, 110, 180, 260], (0,)),    # before it
                      ([0, 50, 230, 230, 260], (1,))):    # longer than max_T
        cu = np.array(bad, dtype=np.int32)
        out = torch.full((H, 260, dv), 3.0, device="cuda", dtype=p["q"][1].dtype)
        s1 = torch.full((4, H, dk, dv), 3.0, device="cuda")
        lla.linear_forward_varlen(dev(p, "q"), dev(p, "k"), dev(p, "v"), dev(p, "la"), torch.from_numpy(cu).cuda(),
                                  100, state_out=s1, out=out)
        assert lla.device_error() == lla.LLA_ERR_DEVICE
        assert lla.device_error() == 0
        if bad[3] == 40:
            skip = (2, 3)
        for b in skip:
            assert (host(s1)[b] == 3.0).all(), (bad, b)
        ok = [b for b in range(4) if b not in skip]
        for b in ok:
            assert not (host(s1)[b] == 3.0).all()
        check_packed(p, cu, host(out), host(s1), dtype, skip=skip)
        covered = np.zeros(260, dtype=bool)
        for b in ok:
            covered[cu[b]:cu[b + 1]] = True
        assert (host(out)[:, ~covered] == 3.0).all(), bad


@pytest.mark.parametrize("B,H,dk,dv,dtype", [
    (1, 1, 1, 1, "f32"), (3, 2, 64, 64, "bf16"), (2, 3, 128, 128, "f32"), (5, 3, 100, 36, "bf16"), (2, 2, 17, 33, "f32"),
    (2, 2, 128, 2, "bf16"), (300, 4, 16, 128, "bf16"),
])
def test_decode(lla, B, H, dk, dv, dtype):
    p = problem(B, H, 1, dk, dv, dtype, B, seed=dk)
    st = dev(p, "s0").clone()
    q, k, v = (dev(p, n)[:, :, 0].contiguous() for n in ("q", "k", "v"))
    out = lla.linear_decode_step(q, k, v, dev(p, "la"), st)
    x = [val(p, n) for n in ("q", "k", "v", "la", "s0")]
    ref, ref_s = L.forward(*x)
    size, size_s = L.forward(*sizes(*x[:3]), x[3], *sizes(x[4]))
    # the state is fp32 throughout, so a bf16 output has its own rounding alone
    err = np.abs(host(out)[:, :, None] - ref)
    assert (err <= (L.UBF if dtype == "bf16" else 0) * np.abs(ref) + (dk + 16) * 2 * L.U32 * size).all()
    L.check(host(st), ref_s, size_s, "f32", 4, "state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_tokens_is_the_whole(lla, dtype):
    """Prompts cut anywhere, the state handed on, then single tokens: each piece against the whole's sums."""
    B, H, T, dk, dv = 2, 4, 333, 64, 48
    p = problem(B, H, T, dk, dv, dtype, 1, seed=11)
    x = [val(p, n) for n in ("q", "k", "v", "la", "s0")]
    ref, ref_s = L.forward(*x)
    size, size_s = L.forward(*sizes(*x[:3]), x[3], *sizes(x[4]))
    state, outs, at = dev(p, "s0"), [], 0
    for n in (130, 1, 199):
        part = [dev(p, m)[:, :, at:at + n].contiguous() for m in ("q", "k", "v")]
        s1 = torch.empty(B, H, dk, dv, device="cuda")
        outs.append(lla.linear_forward(*part, dev(p, "la"), state0=state, state_out=s1))
        state, at = s1, at + n
    for t in range(at, T):
        part = [dev(p, m)[:, :, t].contiguous() for m in ("q", "k", "v")]
        outs.append(lla.linear_decode_step(*part, dev(p, "la"), state)[:, :, None])
    L.check(host(torch.cat(outs, 2)), ref, size, dtype, T + dk, "out")
    L.check(host(state), ref_s, size_s, "f32", T, "state")


def test_equals_the_hierarchy_with_equal_levels(lla):
    """lla_forward with lambda = 1 and one decay at every token: both are within their roundings of the sums."""
    B, H, T, dk, dv = 1, 4, 256, 64, 32
    p = problem(B, H, T, dk, dv, "f32", 0, seed=12)
    la = torch.where(torch.isinf(dev(p, "la")), torch.tensor(-2.0, device="cuda"), dev(p, "la"))
    lam = torch.ones(B, H, T, lla.num_levels(T), device="cuda")
    a = lla.linear_forward(dev(p, "q"), dev(p, "k"), dev(p, "v"), la)
    b = lla.forward(dev(p, "q"), dev(p, "k"), dev(p, "v"), la[None, :, None].expand(B, H, T).contiguous(), lam, 64)
    assert float((a - b).abs().max() / a.abs().max()) <= 1e-4  # the hierarchy's own bar for fp32


@pytest.mark.parametrize("dtype,dk", [("bf16", 64), ("f32", 30)])
def test_calls_repeat_to_the_bit(lla, dtype, dk):
    p = problem(2, 3, 400, dk, 64, dtype, 1, seed=13)
    names = ("q", "k", "v", "la")
    run = lambda: [lla.linear_forward(*(dev(p, n) for n in names), state0=dev(p, "s0"))] + list(  # noqa: E731
        lla.linear_backward(*(dev(p, n) for n in names), dev(p, "dout"), state0=dev(p, "s0"), dstate_out=dev(p, "ds")))
    first = run()
    for _ in range(3):
        for a, b in zip(first, run()):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,dk", [("bf16", 64), ("f32", 30)])
def test_graphs_and_streams(lla, dtype, dk):
    """Two captured graphs (prompt, gradients, packed prompt, token) replayed at the same time on two streams, new
    inputs copied in between replays; and a call on a stream of its own."""
    lengths = [100, 0, 260]
    work = []
    for seed in (20, 21):
        p = problem(2, 3, 300, dk, 64, dtype, 1, seed=seed)
        pk, cu = pack(lengths, 3, dk, 64, dtype, 0, 5, seed=seed)
        work.append(dict(p=p, pk=pk, cu=torch.from_numpy(cu).cuda(), s1=torch.zeros(2, 3, dk, 64, device="cuda"),
                         st=torch.zeros(2, 3, dk, 64, device="cuda")))

    def calls(w):
        p, pk = w["p"], w["pk"]
        o = lla.linear_forward(dev(p, "q"), dev(p, "k"), dev(p, "v"), dev(p, "la"), state0=dev(p, "s0"),
                               state_out=w["s1"])
        g = lla.linear_backward(dev(p, "q"), dev(p, "k"), dev(p, "v"), dev(p, "la"), dev(p, "dout"),
                                state0=dev(p, "s0"), dstate_out=dev(p, "ds"))
        out = torch.zeros(3, sum(lengths) + 5, 64, device="cuda", dtype=o.dtype)
        u = lla.linear_forward_varlen(dev(pk, "q"), dev(pk, "k"), dev(pk, "v"), dev(pk, "la"), w["cu"], 260, out=out)
        w["st"].copy_(w["s1"])
        d = lla.linear_decode_step(*(dev(p, n)[:, :, 0].contiguous() for n in ("q", "k", "v")), dev(p, "la"), w["st"])
        return [o, *g, u, d, w["s1"], w["st"]]

    want = [[x.clone() for x in calls(w)] for w in work]
    graphs, outs = [], []
    for w in work:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(calls(w))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, r in zip(outs, want):
        for a, b in zip(o, r):
            assert torch.equal(a, b)
    # new inputs in the captured buffers
    for n in ("q", "k", "v"):
        work[0]["p"][n][1].copy_(work[1]["p"][n][1])
    graphs[0].replay()
    torch.cuda.synchronize()
    again = calls(work[0])
    torch.cuda.synchronize()
    for a, b in zip(outs[0], again):
        assert torch.equal(a, b)
    # a stream of its own, given to the call
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p = work[1]["p"]
    o = lla.linear_forward(dev(p, "q"), dev(p, "k"), dev(p, "v"), dev(p, "la"), state0=dev(p, "s0"), stream=side)
    side.synchronize()
    assert torch.equal(o, want[1][0])


def test_serving_and_training_run(lla):
    """As the operators are used together: a common prefix once, packed turns that go on from its state, single
    tokens after them, then a training step of the same rows from the shared state."""
    H, dk, dv, P = 4, 64, 64, 200
    lengths = [30, 0, 150]
    pre = problem(1, H, P, dk, dv, "bf16", 0, seed=30)
    la = dev(pre, "la")
    shared = torch.empty(1, H, dk, dv, device="cuda")
    lla.linear_forward(dev(pre, "q"), dev(pre, "k"), dev(pre, "v"), la, state_out=shared)
    pk, cu = pack(lengths, H, dk, dv, "bf16", 0, 0, seed=31)
    states = torch.empty(3, H, dk, dv, device="cuda")
    out = lla.linear_forward_varlen(dev(pk, "q"), dev(pk, "k"), dev(pk, "v"), la, torch.from_numpy(cu).cuda(), 150,
                                    state0=shared, state_out=states)
    tok = problem(3, H, 1, dk, dv, "bf16", 0, seed=32)
    last = lla.linear_decode_step(*(dev(tok, n)[:, :, 0].contiguous() for n in ("q", "k", "v")), la, states)
    for b, n in enumerate(lengths):
        rows = slice(cu[b], cu[b + 1])
        x = [np.concatenate([val(pre, m)[0], val(pk, m)[:, rows], val(tok, m)[b]], 1)[None] for m in ("q", "k", "v")]
        ref, ref_s = L.forward(*x, val(pre, "la"))
        size, size_s = L.forward(*sizes(*x), val(pre, "la"))
        whole = np.concatenate([host(out)[:, rows], host(last)[b][:, None]], 1)[None]
        L.check(whole, ref[:, :, P:], size[:, :, P:], "bf16", P + n + dk, b)
        L.check(host(states)[None, b], ref_s, size_s, "f32", P + n, b)
    # the whole of it as one training sequence equals the prefix with the turn's gradient handed back
    b, n = 2, 150
    turn = {m: dev(pk, m)[None, :, cu[b]:cu[b + 1]].contiguous() for m in ("q", "k", "v")}
    do = torch.randn(1, H, n, dv, device="cuda").bfloat16()
    g2 = lla.linear_backward(*turn.values(), la, do, state0=shared)
    zero = torch.zeros(1, H, P, dv, device="cuda", dtype=torch.bfloat16)
    g1 = lla.linear_backward(dev(pre, "q"), dev(pre, "k"), dev(pre, "v"), la, zero, dstate_out=g2[3])
    x = [np.concatenate([val(pre, m)[0], val(pk, m)[:, cu[b]:cu[b + 1]]], 1)[None] for m in ("q", "k", "v")]
    d = np.concatenate([host(zero), host(do)], 2)
    ref, size = L.backward(*x, val(pre, "la"), d), L.backward(*sizes(*x), val(pre, "la"), np.abs(d))
    for i in range(3):
        L.check(host(torch.cat([g1[i], g2[i]], 2)), ref[i], size[i], "bf16", P + n + dk, i)


def test_binding_refuses(lla):
    p = problem(2, 3, 20, 16, 16, "f32", 1)
    q, k, v, la, s0 = (dev(p, n) for n in ("q", "k", "v", "la", "s0"))
    for bad in (dict(la=la[:2].contiguous()), dict(la=la.double()), dict(k=k.bfloat16()), dict(k=k[:, :, :10].contiguous()),
                dict(v=v[:, :, :10].contiguous()), dict(q=q.transpose(1, 2)), dict(s0=s0.double()),
                dict(s0=torch.cat([s0] * 3)), dict(s0=s0[..., :8].contiguous()), dict(s0=s0.cpu())):
        a = {"q": q, "k": k, "v": v, "la": la, "s0": s0, **bad}
        with pytest.raises((ValueError, TypeError)):
            lla.linear_forward(a["q"], a["k"], a["v"], a["la"], state0=a["s0"])
    state = s0.expand(2, -1, -1, -1).contiguous()
    with pytest.raises(lla.LLAError):
        lla.linear_forward(q, k, v, la, state0=state, state_out=state)
    with pytest.raises(ValueError):
        lla.linear_forward(q, k, v, la, out=torch.empty(2, 3, 20, 8, device="cuda"))
    with pytest.raises(TypeError):
        lla.linear_forward(q.half(), k.half(), v.half(), la)
    with pytest.raises(ValueError):
        lla.linear_decode_step(q[:, :, 0].contiguous(), k[:, :, 0].contiguous(), v[:, :, 0].contiguous(), la, s0)
    with pytest.raises(TypeError):
        lla.linear_forward_varlen(q[0], k[0], v[0], la, torch.zeros(2, dtype=torch.int64, device="cuda"), 20)


FIRST = """
import sys, torch
from log_linear_attention_gb300 import binding as lla
q = torch.randn(2, 3, 300, 64, device="cuda").bfloat16()
la, la2 = -torch.rand(3, device="cuda"), -torch.rand(2, 3, device="cuda")
x, f = q[:, :, 0].clone(), q.float()
cu = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
state, decay = torch.zeros(2, 3, 64, 64, device="cuda"), torch.zeros(2, 3, device="cuda")
prefix, states = torch.zeros(3, 11, 64, 64, device="cuda"), torch.zeros(2, 3, 14, 64, 64, device="cuda")
lam, t = torch.rand(2, 3, 14, device="cuda"), torch.full((2,), 1050, device="cuda")
call = {"forward": lambda: lla.linear_forward(q, q, q, la), "fp32": lambda: lla.linear_forward(f, f, f, la),
        "varlen": lambda: lla.linear_forward_varlen(q[0], q[0], q[0], la, cu, 200),
        "backward": lambda: lla.linear_backward(q, q, q, la, q)[0],
        "decode": lambda: lla.linear_decode_step(x, x, x, la, state),
        "shared": lambda: lla.decode_step_shared(x, x, x, la2, lam, prefix, 1000, decay, states, t)}[sys.argv[1]]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    o = call()
for s in (state, decay, states):
    s.zero_()
g.replay()
torch.cuda.synchronize()
for s in (state, decay, states):
    s.zero_()
assert torch.equal(o, call()) and lla.device_error() == 0
print("same")
"""


@pytest.mark.parametrize("what", ["forward", "fp32", "varlen", "backward", "decode", "shared"])
def test_first_call_of_a_process_may_be_captured(what):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST, what], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("B,H,T,dk,dv", [(4, 16, 8192, 128, 64), (10, 17, 1100, 64, 128), (1, 2, 20000, 128, 128),
                                         (200, 5, 130, 64, 64)])
def test_full_sizes_sampled(lla, B, H, T, dk, dv):
    """The headline shape, more heads than SMs, a long document of two heads, many short sequences: some heads
    against the recurrence in 64 bits. The norm bounds of tests/_linear.py; states are fp32 sums of T terms."""
    g = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k = (rand(B, H, T, dk).mul_(dk ** -0.5).bfloat16() for _ in range(2))
    v, do = (rand(B, H, T, dv).bfloat16() for _ in range(2))
    la = -torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
    s0, ds = rand(B, H, dk, dv) * 0.1, rand(B, H, dk, dv) * 0.1
    s1 = torch.empty_like(s0)
    out = lla.linear_forward(q, k, v, la, state0=s0, state_out=s1)
    got = [out, s1, *lla.linear_backward(q, k, v, la, do, state0=s0, dstate_out=ds)]
    for b, h in ((0, 0), (B - 1, H - 1), (B // 2, H // 2)):
        ref = L.tokens(q[b, h][None], k[b, h][None], v[b, h][None], la[h][None], s0[b, h][None], do[b, h][None],
                       ds[b, h][None])
        for n, x, r in zip(("out", "state", "dq", "dk", "dv", "dstate0"), got, ref):
            rel = float((x[b, h].double() - r[0]).norm() / r[0].norm())
            assert rel <= (5e-3 if x.dtype == torch.bfloat16 else 4 * (T + 16) ** 0.5 * L.U32), (n, b, h, rel)


@pytest.mark.parametrize("B,H,T,dk,dv", [(8, 20, 1024, 128, 64), (8, 20, 512, 64, 128), (2, 4, 2048, 128, 64),
                                         (2, 4, 2048, 64, 64), (1, 3, 1024, 96, 128), (3, 60, 128, 128, 128)])
def test_whole_last_chunks_wait_for_their_rows(lla, B, H, T, dk, dv):
    """Prompts of whole chunks whose state nobody takes, while another stream keeps the memory busy, so that copies are
    late: a block's last chunk adds to no state, and its product has to wait for its rows of v all the same. More heads
    than SMs, and cuts down to a chunk a block. Every head against the CUDA cores' fp32 arithmetic (5e-3 of a head's
    norm, see tests/_linear.py) and every repetition to the bit."""
    g = torch.Generator(device="cuda").manual_seed(T + dv)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    inputs = []
    for _ in range(3):
        q, k = (rand(B, H, T, dk).mul_(dk ** -0.5).bfloat16() for _ in range(2))
        inputs.append((q, k, rand(B, H, T, dv).bfloat16()))
    la = -torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
    refs = [lla.linear_forward(*(t.float() for t in x), la) for x in inputs]
    # the same rows as packed sequences of whole chunks
    rows = [[t.transpose(0, 1).reshape(H, B * T, -1).contiguous() for t in x] for x in inputs]
    cu = torch.arange(B + 1, device="cuda", dtype=torch.int32) * T
    a, b = (torch.empty(1 << 28, device="cuda") for _ in range(2))  # 1 GiB each
    busy, here = torch.cuda.Stream(), torch.cuda.current_stream()
    busy.wait_stream(here)
    first = [None, None]
    for turn in range(6):
        with torch.cuda.stream(busy):
            for _ in range(4):
                b.copy_(a)
        got = []
        for x, p in zip(inputs, rows):  # other rows lie in shared memory from call to call
            got.append((lla.linear_forward(*x, la),
                        lla.linear_forward_varlen(*p, la, cu, T).reshape(H, B, T, dv).transpose(0, 1)))
        for i, (outs, r) in enumerate(zip(got, refs)):
            for out in outs:
                rel = (out.float() - r).norm(dim=(2, 3)) / r.norm(dim=(2, 3))
                assert float(rel.max()) <= 5e-3, (turn, i, int(rel.argmax()), float(rel.max()))
        if turn:
            assert all(torch.equal(x, y) for xs, ys in zip(got, first) for x, y in zip(xs, ys)), turn
        else:
            first = got
    busy.synchronize()


@pytest.mark.parametrize("B,H,T,dk,dv", [(1, 2, 128, 64, 64), (2, 2, 384, 128, 128), (1, 2, 2048, 72, 40),
                                         (40, 2, 300, 128, 64)])
def test_states_keep_the_bits_of_fp32(lla, B, H, T, dk, dv):
    """One token of each 128 has a key and a query, so a state is a sum of few terms and shows each of its roundings:
    both states (after the last token; the gradient of the first) within them. Steps of 2^-22, of a term c chunks from
    where it is read: the weight's expf and its product 5/4, three parts' sums in fp32, truncated, 3/2, the sum with the
    state 1/4, together below 4; 5/4 for each chunk's decay on the way. The last eight bits of a term, which are a part
    of their own in the products, weigh up to 2^-15."""
    la = np.array([-2.0 ** -6, -2.0 ** -7])  # times a token count: exact
    r = np.random.default_rng(T + dk)
    t = np.arange(T)
    lit = (t % 128 == 37)[None, None, :, None]
    (k, kt), (q, qt), (v, vt), (do, dot) = (L.make(r, (B, H, T, d), "bf16") for d in (dk, dk, dv, dv))
    k, q, kt, qt = k * lit, q * lit, kt * torch.from_numpy(lit), qt * torch.from_numpy(lit)
    s0, s1 = torch.zeros(B, H, dk, dv, device="cuda"), torch.empty(B, H, dk, dv, device="cuda")
    x = [y.cuda() for y in (qt, kt, vt, torch.from_numpy(la).float())]
    lla.linear_forward(*x, state_out=s1)
    ds0 = lla.linear_backward(*x, dot.cuda(), state0=s0)[3]
    n = (T + 127) // 128
    for what, got, a, c, gap, passed in (("state", s1, k, v, T - 1 - t, n - 1 - t // 128),
                                         ("dstate0", ds0, q, do, t + 1, t // 128)):
        w = L.powers(la, gap)[..., None]
        ref = np.swapaxes(a * w, -1, -2) @ c
        bound = np.swapaxes(np.abs(a) * w * (4 + 1.25 * passed)[:, None], -1, -2) @ np.abs(c) * 2.0 ** -22
        worst = np.max(np.abs(host(got) - ref) - bound)
        assert worst <= 1e-37, (what, worst)


@pytest.mark.parametrize("B,H,T,dk,dv", [(6, 30, 640, 64, 64), (6, 30, 640, 8, 128), (6, 30, 500, 128, 64),
                                         (3, 30, 640, 128, 128)])
def test_gradients_beside_a_busy_stream(lla, B, H, T, dk, dv):
    """Gradients whose groups of pieces are of one item and of two, while another stream keeps the memory busy: every
    head against the CUDA cores' fp32 arithmetic (5e-3 of a head's norm), every repetition to the bit."""
    g = torch.Generator(device="cuda").manual_seed(T + dk)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k = (rand(B, H, T, dk).mul_(dk ** -0.5).bfloat16() for _ in range(2))
    v, do = (rand(B, H, T, dv).bfloat16() for _ in range(2))
    la = -torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
    ref = lla.linear_backward(q.float(), k.float(), v.float(), la, do.float())
    a, b = (torch.empty(1 << 28, device="cuda") for _ in range(2))  # 1 GiB each
    busy = torch.cuda.Stream()
    busy.wait_stream(torch.cuda.current_stream())
    first = None
    for _ in range(8):
        with torch.cuda.stream(busy):
            b.copy_(a)
        got = lla.linear_backward(q, k, v, la, do)
        first = first or got
        for n, x, y, r in zip(("dq", "dk", "dv"), got, first, ref):
            rel = (x.float() - r).norm(dim=(2, 3)) / r.norm(dim=(2, 3))
            assert float(rel.max()) <= 5e-3, (n, int(rel.argmax()), float(rel.max()))
            assert torch.equal(x, y), n
    busy.synchronize()


def test_a_rank_s_part_of_the_decays(lla):
    """slopes[r h : (r + 1) h] begins at any multiple of 4 bytes, and so does a part of cu_seqlens: the same bits as from
    tensors of their own."""
    B, H, T, dk, dv = 2, 3, 200, 64, 64
    for dtype in ("bf16", "f32"):
        p = problem(B, 4 * H, T, dk, dv, dtype, B, seed=40)
        cu = torch.tensor([7, 0, 60, B * T - 5], dtype=torch.int32, device="cuda")
        for r in range(4):
            heads = slice(r * H, (r + 1) * H)
            part, whole = dev(p, "la")[heads], dev(p, "la")[heads].clone()
            assert whole.data_ptr() % 16 == 0 and part.data_ptr() % 16 == (12 * r) % 16
            q, k, v, do = (dev(p, n)[:, heads].contiguous() for n in ("q", "k", "v", "dout"))
            s0 = dev(p, "s0")[:, heads].contiguous()
            rows = [x.transpose(0, 1).reshape(H, B * T, -1).contiguous() for x in (q, k, v)]
            tok = [x[:, :, 0].contiguous() for x in (q, k, v)]
            got = []
            for la, c in ((part, cu[1:]), (whole, cu[1:].clone())):
                st, s1 = s0.clone(), torch.empty_like(s0)
                got.append([lla.linear_forward(q, k, v, la, state0=s0, state_out=s1), s1,
                            lla.linear_forward_varlen(*rows, la, c, B * T, out=torch.zeros_like(rows[2])),
                            *lla.linear_backward(q, k, v, la, do, state0=s0),
                            lla.linear_decode_step(*tok, la, st), st])
            assert all(torch.equal(x, y) for x, y in zip(*got)), (dtype, r)
    store = torch.zeros(B * H * 64 + 3, device="cuda")  # decays in the last bytes of the output
    with pytest.raises(lla.LLAError):
        lla.linear_decode_step(*tok, store[-H - 2:-2], st, out=store[:B * H * 64].view(B, H, 64))


@pytest.mark.parametrize("dtype,n", [("bf16", 3), ("bf16", 80), ("f32", 70)])
def test_varlen_bounds_above_the_rows(lla, dtype, n):
    """max_T beyond every row of the tensors is the same call as max_T of all of them, to the bit: a bound of 2^31 - 1
    moved bf16 to the CUDA cores, and with 64 sequences or more was refused."""
    H, dk, dv = 3, 64, 64
    lengths = [(37 * b) % 150 for b in range(n)]
    p, cu = pack(lengths, H, dk, dv, dtype, 0, 5, seed=n)
    x = [dev(p, m) for m in ("q", "k", "v", "la")]
    total, c = sum(lengths) + 5, torch.from_numpy(cu).cuda()
    got = []
    for most in (total, total + 1, 1 << 30, 2 ** 31 - 1):
        s1 = torch.empty(n, H, dk, dv, device="cuda")
        got.append((lla.linear_forward_varlen(*x, c, most, state_out=s1, out=torch.zeros_like(x[2])), s1))
    check_packed(p, cu, host(got[0][0]), host(got[0][1]), dtype)
    for a, b in got[1:]:
        assert torch.equal(a, got[0][0]) and torch.equal(b, got[0][1])


@pytest.mark.parametrize("dtype,chunk", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_gradients_of_values_that_are_not_finite(lla, dtype, chunk, bad):
    """One element (t, column 5) of each input: what depends on it is not finite, what may share its chunk is as the
    header says, and every other element keeps its bits. dq_i = sum_{j <= i} (dO_i . v_j) k_j, dk_i = sum_{j >= i}
    (v_i . dO_j) q_j, dv_i = sum_{j >= i} (k_i . q_j) dO_j."""
    T, t, col, d = 500, 300, 5, 64
    p = problem(1, 2, T, d, d, dtype, 0, seed=41)
    clean = [lla.linear_backward(*(dev(p, n) for n in ("q", "k", "v", "la", "dout")))[i] for i in range(3)]
    lo, hi = t // chunk * chunk, t // chunk * chunk + chunk
    everywhere = slice(None)
    # input: for dq, dk, dv the rows and columns that may change
    reach = {"k": ((slice(lo, None), col), None, (slice(t, t + 1), everywhere)),
             "q": (None, (slice(0, hi), col), (slice(0, t + 1), everywhere)),
             "dout": ((slice(t, t + 1), everywhere), (slice(0, t + 1), everywhere), (slice(0, hi), col)),
             "v": ((slice(t, None), everywhere), (slice(t, t + 1), everywhere), None)}
    for name, may in reach.items():
        x = {n: dev(p, n) for n in ("q", "k", "v", "la", "dout")}
        x[name] = x[name].clone()
        x[name][:, :, t, col] = bad
        got = lla.linear_backward(*x.values())[:3]
        for n, g, c, m in zip(("dq", "dk", "dv"), got, clean, may):
            same = torch.ones(T, d, dtype=torch.bool, device="cuda")
            if m is not None:
                same[m] = False
                assert not torch.isfinite(g[:, :, t][..., m[1]].float()).all(), (name, n)
            assert torch.equal(g[:, :, same], c[:, :, same]), (name, n)


def test_without_torch_s_private_calls(lla, monkeypatch):
    """The public calls name the same device and stream: the same bits, on a stream of its own too."""
    from types import SimpleNamespace as N
    p = problem(2, 3, 200, 64, 64, "bf16", 0, seed=42)
    x = [dev(p, n) for n in ("q", "k", "v", "la")]
    want = lla.linear_forward(*x)
    device, stream = lla._cuda_calls(N(_C=N(), cuda=torch.cuda))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert device() == lla._current_device() and stream(device()) == lla._raw_stream(device()) == side.cuda_stream
    monkeypatch.setattr(lla, "_current_device", device)
    monkeypatch.setattr(lla, "_raw_stream", stream)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = lla.linear_forward(*x)
    given = lla.linear_forward(*x, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(given, want)


@pytest.mark.parametrize("B,H,T,dk,dv,dtype,B0", [(1, 64, 20001, 128, 128, "f32", 1), (5, 22, 18000, 128, 127, "bf16", 5),
                                                  (3, 40, 20001, 126, 128, "f32", 1)])
def test_long_prompts_of_many_heads_in_groups(lla, B, H, T, dk, dv, dtype, B0):
    """More chunk states than the CUDA-core path keeps at a time: each head has the bits of a call of its own, whole
    sequences to a group and parts of one."""
    g = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k = (rand(B, H, T, dk).mul_(dk ** -0.5).to(t) for _ in range(2))
    v, do = (rand(B, H, T, dv).to(t) for _ in range(2))
    la = -torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
    s0, ds, s1 = rand(B0, H, dk, dv), rand(B, H, dk, dv), torch.empty(B, H, dk, dv, device="cuda")
    out = lla.linear_forward(q, k, v, la, state0=s0, state_out=s1)
    grads = lla.linear_backward(q, k, v, la, do, state0=s0, dstate_out=ds)
    cut = lambda x, b, h: x[min(b, x.shape[0] - 1), h][None, None].clone()  # noqa: E731
    # parts of the gradient of a shared state, summed in order as the call does
    total = torch.zeros_like(s0) if B0 == 1 else None
    for b in range(B):
        for h in range(H):
            if B0 > 1 and (h, b) not in ((0, 0), (1, 1), (H - 1, 2), (H // 2, 3), (3, 4), (H - 1, 4)):
                continue
            x = [cut(y, b, h) for y in (q, k, v)]
            a = la[h:h + 1].clone()
            mine = lla.linear_backward(*x, a, cut(do, b, h), state0=cut(s0, b, h), dstate_out=cut(ds, b, h))
            if B0 == 1:
                total[0, h] += mine[3][0, 0]
            else:
                assert torch.equal(mine[3][0, 0], grads[3][b, h]), (b, h)
            for got, want in zip(grads[:3], mine[:3]):
                assert torch.equal(got[b, h], want[0, 0]), (b, h)
            if (b + h) % 7 == 0 or h in (0, H - 1):
                s = torch.empty(1, 1, dk, dv, device="cuda")
                o = lla.linear_forward(*x, a, state0=cut(s0, b, h), state_out=s)
                assert torch.equal(out[b, h], o[0, 0]) and torch.equal(s1[b, h], s[0, 0]), (b, h)
    if B0 == 1:
        assert torch.equal(total, grads[3])


def test_packed_rows_of_many_heads_in_groups(lla):
    H, dk, dv, lengths = 64, 128, 126, [9000, 0, 7001, 1, 4000]
    total, n = sum(lengths) + 3, len(lengths)
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k, v = (rand(H, total, d) for d in (dk, dk, dv))
    la = -torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)).cuda()
    for s0 in (rand(n, H, dk, dv), rand(1, H, dk, dv), None):
        s1, out = torch.empty(n, H, dk, dv, device="cuda"), torch.full((H, total, dv), 7.0, device="cuda")
        lla.linear_forward_varlen(q, k, v, la, cu, 9000, state0=s0, state_out=s1, out=out)
        for h in (0, 1, 50, 51, 52, 53, H - 1):
            s, o = torch.empty(n, 1, dk, dv, device="cuda"), torch.full((1, total, dv), 7.0, device="cuda")
            lla.linear_forward_varlen(q[h:h + 1].clone(), k[h:h + 1].clone(), v[h:h + 1].clone(), la[h:h + 1], cu, 9000,
                                      state0=None if s0 is None else s0[:, h:h + 1].contiguous(), state_out=s, out=o)
            assert torch.equal(out[h], o[0]) and torch.equal(s1[:, h], s[:, 0]), h


MEMORY = """
import torch
from log_linear_attention_gb300 import binding as lla
q, k, v, do = (torch.randn(1, 64, 40000, 128, device="cuda") for _ in range(4))
la, out = -torch.rand(64, device="cuda"), torch.empty_like(v)
outs = [torch.empty_like(q) for _ in range(3)]
del outs  # torch keeps the memory for the gradients
lla.linear_forward(q[:, :1, :64].contiguous(), q[:, :1, :64].contiguous(), q[:, :1, :64].contiguous(), la[:1])
torch.cuda.synchronize()
free = torch.cuda.mem_get_info()[0]
lla.linear_forward(q, k, v, la, out=out)
lla.linear_backward(q, k, v, la, do)
torch.cuda.synchronize()
taken = free - torch.cuda.mem_get_info()[0]
assert lla.device_error() == 0 and taken <= (1 << 30) + (64 << 20), taken
print("kept within", taken)
"""


def test_long_prompts_keep_their_workspace_within_a_bound():
    """64 heads, T = 40000, 128 x 128 in fp32: 2.6 GB of chunk states forwards and twice that backwards, 1 GiB at a time."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", MEMORY], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "kept within" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("n", [1024, 1025, 2500])
@pytest.mark.parametrize("dtype,dk", [("bf16", 64), ("f32", 20)])
def test_varlen_more_sequences_than_a_block_has_threads(dtype, dk, n):
    """The table of the sequences is made in rounds of 1024: lengths of zero and more, a few long ones, and bounds that
    break the rules on both sides of a round's end."""
    from log_linear_attention_gb300 import binding as lla
    H, dv = 2, 32
    r = np.random.default_rng(n)
    lengths = [int(x) for x in r.integers(0, 12, n)]
    for b in (5, 1022, n - 1):
        lengths[b] = 300 + b % 7
    p, cu = pack(lengths, H, dk, dv, dtype, 0, 40, seed=n)
    total = sum(lengths) + 40
    x = [dev(p, m) for m in ("q", "k", "v", "la")]
    for spoil in ((), (700, 1023) if n == 1024 else (700, 1023, 1024)):
        bounds, skip = cu.copy(), set()
        for b in spoil:  # sequence b - 1 ends past the tensors, b begins there: both are out
            bounds[b] = total + 1 + b
            skip |= {b - 1, b}
        # whatever begins below a bound that came before it is out too
        high = np.maximum.accumulate(bounds)
        skip |= {b for b in range(n) if bounds[b] < high[b] or bounds[b + 1] < bounds[b] or bounds[b + 1] > total}
        s1 = torch.full((n, H, dk, dv), 3.0, device="cuda")
        out = torch.full((H, total, dv), 7.0, device="cuda", dtype=x[2].dtype)
        lla.linear_forward_varlen(*x, torch.from_numpy(bounds).cuda(), 400, state_out=s1, out=out)
        assert lla.device_error() == (lla.LLA_ERR_DEVICE if spoil else 0)
        o, s = host(out), host(s1)
        check_packed(p, bounds, o, s, dtype, skip=skip)
        covered = np.zeros(total, dtype=bool)
        for b in range(n):
            if b in skip:
                assert (s[b] == 3.0).all(), b
            else:
                covered[bounds[b]:bounds[b + 1]] = True
        assert (o[:, ~covered] == 7.0).all()


@pytest.mark.parametrize("lengths,dk,dv,dtype,n0", [([5000, 3, 2701, 64, 0, 4097], 64, 64, "f32", 6),
                                                    ([3000, 1, 2999], 36, 100, "f32", 1),
                                                    ([4000, 129], 50, 33, "bf16", 2), ([6000, 5, 4100], 128, 64, "bf16", 3)])
def test_varlen_of_many_chunks(lla, lengths, dk, dv, dtype, n0):
    p, cu = pack(lengths, 3, dk, dv, dtype, n0, 17, seed=len(lengths))
    s1 = torch.empty(len(lengths), 3, dk, dv, device="cuda")
    out = torch.full((3, sum(lengths) + 17, dv), 7.0, device="cuda", dtype=p["q"][1].dtype)
    lla.linear_forward_varlen(*(dev(p, m) for m in ("q", "k", "v", "la")), torch.from_numpy(cu).cuda(), max(lengths),
                              state0=dev(p, "s0"), state_out=s1, out=out)
    check_packed(p, cu, host(out), host(s1), dtype)
    assert (host(out)[:, cu[-1]:] == 7.0).all()


def test_outputs_given_and_streams_given(lla):
    """Every call with its output tensor and its stream named, against the same call without, to the bit."""
    B, H, T, dk, dv = 2, 3, 300, 64, 64
    p = problem(B, H, T, dk, dv, "bf16", B, seed=50)
    q, k, v, la, do, s0, ds = (dev(p, n) for n in ("q", "k", "v", "la", "dout", "s0", "ds"))
    rows = [x.transpose(0, 1).reshape(H, B * T, -1).contiguous() for x in (q, k, v)]
    cu = torch.tensor([0, 200, B * T], dtype=torch.int32, device="cuda")
    tok = [x[:, :, 0].contiguous() for x in (q, k, v)]
    lam, pre = torch.rand(B, H, 9, device="cuda"), torch.randn(H, 8, dk, dv, device="cuda")
    t = torch.full((B,), 100, dtype=torch.int64, device="cuda")

    def calls(stream, given):
        new = lambda like: torch.zeros_like(like) if given else None  # noqa: E731
        st, own, decay = s0.clone(), torch.zeros(B, H, 9, dk, dv, device="cuda"), torch.zeros(B, H, device="cuda")
        outs = [new(v), new(rows[2]), new(tok[2]), new(tok[2])]
        s1, s2 = torch.empty_like(s0), torch.empty_like(s0)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        got = [lla.linear_forward(q, k, v, la, state0=s0, state_out=s1, out=outs[0], stream=stream),
               lla.linear_forward_varlen(*rows, la, cu, B * T, state0=s0, state_out=s2, out=outs[1], stream=stream),
               lla.linear_decode_step(*tok, la, st, out=outs[2], stream=stream),
               lla.decode_step_shared(*tok, -la[None].expand(B, H).abs().contiguous().clamp(max=2.0), lam, pre, 100, decay,
                                      own, t, out=outs[3], stream=stream)]
        grads = lla.linear_backward(q, k, v, la, do, state0=s0, dstate_out=ds, stream=stream)
        torch.cuda.synchronize()
        if given:
            assert all(a is b for a, b in zip(got, outs))
        return [*got, *grads, s1, s2, st, decay, own[:, :, 0].clone()]

    want = calls(None, False)
    for stream, given in ((None, True), (torch.cuda.Stream(), False), (torch.cuda.Stream(), True)):
        for i, (a, b) in enumerate(zip(calls(stream, given), want)):
            assert torch.equal(a, b), i


def test_offsets_past_32_bits(lla):
    """Tensors of more than 2^31 elements: the first and the last head against fp32 arithmetic on that head alone (5e-3
    of its norm, see tests/_linear.py); token steps to the bit."""
    B, H, T, d = 33, 64, 16400, 64
    assert B * H * T * d > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(7)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, k, v, do = rand(B, H, T, d).mul_(d ** -0.5), rand(B, H, T, d).mul_(d ** -0.5), rand(B, H, T, d), rand(B, H, T, d)
    la = -torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
    got = [lla.linear_forward(q, k, v, la), *lla.linear_backward(q, k, v, la, do)[:3]]
    for b, h in ((0, 0), (B - 1, H - 1)):
        x = [t[b, h][None, None].float() for t in (q, k, v)]
        a = la[h:h + 1].clone()
        ref = [lla.linear_forward(*x, a), *lla.linear_backward(*x, a, do[b, h][None, None].float())[:3]]
        for y, r in zip(got, ref):
            assert float((y[b, h].float() - r[0, 0]).norm() / r.norm()) <= 5e-3, (b, h)
    del got, do
    # the same rows packed, one tensor of [H, B T, d]: its last sequence lies past 2^31 elements
    rows = [t.view(H, B * T, d) for t in (q, k, v)]
    cu = torch.tensor([0, 1000, (B - 1) * T, B * T], dtype=torch.int32, device="cuda")
    out = lla.linear_forward_varlen(*rows, la, cu, B * T)
    x = [t[H - 1:, (B - 1) * T:].float().contiguous() for t in rows]
    ref = lla.linear_forward(*(t[None] for t in x), la[H - 1:].clone())
    assert float((out[H - 1, (B - 1) * T:].float() - ref[0, 0]).norm() / ref.norm()) <= 5e-3
    del out, rows, q, k, v
    # one token: states of more than 2^31 elements
    B, d = 2100, 128
    state = torch.randn(B, H, d, d, generator=g, device="cuda")
    assert state.numel() > 2 ** 31
    q, k, v = (torch.randn(B, H, d, generator=g, device="cuda") for _ in range(3))
    last = state[-1:].clone()
    out = lla.linear_decode_step(q, k, v, la, state)
    one = lla.linear_decode_step(q[-1:].clone(), k[-1:].clone(), v[-1:].clone(), la, last)
    assert torch.equal(out[-1:], one) and torch.equal(state[-1:], last)


def test_shared_offsets_past_32_bits(lla):
    B, H, L, d, P = 130, 64, 18, 128, 70001
    states = torch.randn(B, H, L, d, d, device="cuda")
    assert states.numel() > 2 ** 31
    q, k, v = (torch.randn(B, H, d, device="cuda") for _ in range(3))
    la, lam = -torch.rand(B, H, device="cuda"), torch.rand(B, H, L, device="cuda")
    pre, decay = torch.randn(H, L, d, d, device="cuda"), -torch.rand(B, H, device="cuda")
    t = P + torch.arange(B, device="cuda") * 7
    last, kept = states[-1:].clone(), decay[-1:].clone()
    out = lla.decode_step_shared(q, k, v, la, lam, pre, P, decay, states, t)
    one = lla.decode_step_shared(*(x[-1:].clone() for x in (q, k, v, la, lam)), pre, P, kept, last, t[-1:].clone())
    assert torch.equal(out[-1:], one) and torch.equal(states[-1:], last) and torch.equal(decay[-1:], kept)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_varlen_many_rows_under_a_loose_bound(lla, dtype):
    """4000 sequences of 37 million rows with max_T as large as all of them: a bound times the sequences counted as chunks
    that there might be, and the call was refused. Some sequences against calls of their own in fp32."""
    n, d = 4000, 16
    r = np.random.default_rng(9)
    lengths = r.integers(0, 17000, n)
    lengths[[3, 2500]] = 1 << 20, 1 << 19
    cu = np.concatenate([[0], np.cumsum(lengths)])
    total = int(cu[-1])
    assert n * (total // 64) > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(9)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, v = (torch.randn(1, total, d, generator=g, device="cuda", dtype=t) for _ in range(3))
    la = torch.full((1,), -0.01, device="cuda")
    s1 = torch.empty(n, 1, d, d, device="cuda")
    out = lla.linear_forward_varlen(q, k, v, la, torch.from_numpy(cu.astype(np.int32)).cuda(), total, state_out=s1)
    for b in (0, 3, 4, 1999, 2500, n - 1):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        s = torch.empty(1, 1, d, d, device="cuda")
        ref = lla.linear_forward(*(x[:, None, rows].float().contiguous() for x in (q, k, v)), la, state_out=s)
        # fp32: sums of some 100 terms (the decay's reach) in other orders
        assert float((out[:, rows].float() - ref[0]).norm() / ref.norm()) <= (5e-3 if dtype == "bf16" else 1e-5), b
        assert float((s1[b] - s[0]).norm() / s.norm()) <= 1e-4, b
