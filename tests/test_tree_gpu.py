"""GPU checks of trees of drafted tokens over recurrent states and of their commits: against sums over each node's branch
in 64 bits, against decode steps, and all of them together as a server runs them."""
import numpy as np
import pytest

from tests import _drafts as R
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


def np64(t):
    return t.double().cpu().numpy()


def normal(r, shape, dtype, scale=1.0):
    a, t = L.make(r, shape, dtype, scale)
    return a, t.cuda()


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def draft(r, B, H, N, dk, dv, dtype, Lmax, t, one_tree=False, chain=0.4, live=None):
    """Random tokens, states with NaN in the slots that t - 1 does not hold, and trees."""
    d = {"q": normal(r, (B, H, N, dk), dtype, dk ** -0.5), "k": normal(r, (B, H, N, dk), dtype, dk ** -0.5),
         "v": normal(r, (B, H, N, dv), dtype), "states": normal(r, (B, H, Lmax, dk, dv), "f32", dk ** -0.5)}
    for n, x in (("log_a", -np.logaddexp(0, r.standard_normal((B, H, N)) - 2)),
                 ("lam", np.logaddexp(0, r.standard_normal((B, H, N, Lmax)))), ("g", -0.7 * r.random(H))):
        x = x.astype(np.float32)
        d[n] = x.astype(np.float64), torch.from_numpy(x).cuda()
    for b in range(B):
        for m in range(Lmax):
            if m not in R.held(t[b] - 1):
                d["states"][1][b, :, m] = float("nan")
    live = [int(r.integers(1, N + 1)) if live is None else live for _ in range(B)]
    trees = [R.random_tree(r, N, live[0], chain)] * B if one_tree else [R.random_tree(r, N, n, chain) for n in live]
    d["parent"] = trees, ints(trees[0] if one_tree else trees)
    dead = ints(trees) == -2
    for n in ("q", "k", "v", "log_a", "lam"):
        d[n][1].transpose(1, 2)[dead] = float("nan")
    d["t"] = t, ints(t, torch.int64)
    return d


def gate_units(log_a, n):
    """What a branch's weight may be off by, in units of 2^-24 (see tree_check): the exponent is the difference of two sums
    of up to n log decays, each of whose additions rounds."""
    return 2 * n * (np.abs(log_a).max() * n + 1)


CASES = [  # B, H, N, dk, dv, Lmax, t
    (1, 1, 1, 16, 16, 2, [0]), (1, 1, 1, 16, 16, 2, [1]), (2, 2, 5, 64, 64, 8, [3, 64]), (2, 1, 16, 32, 16, 9, [0, 200]),
    (3, 2, 17, 128, 64, 12, [1, 1023, 1024]), (2, 2, 33, 48, 32, 11, [511, 700]), (1, 2, 64, 128, 128, 18, [65535]),
    (2, 1, 65, 100, 36, 13, [4000, 1]), (1, 1, 128, 128, 64, 18, [130900]), (2, 3, 7, 1, 1, 7, [31, 32]),
    (1, 2, 40, 9, 70, 10, [333]), (2, 2, 12, 127, 97, 6, [15, 16]), (1, 1, 20, 17, 3, 40, [(1 << 38) + 12345]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,N,dk,dv,Lmax,t", CASES)
def test_tree(lla, B, H, N, dk, dv, Lmax, t, dtype):
    r = np.random.default_rng(N * dk + dv)
    for one_tree, chain in ((False, 0.4), (True, 0.98), (False, 0.0)):
        d = draft(r, B, H, N, dk, dv, dtype, Lmax, t, one_tree, chain)
        trees = d["parent"][0]
        g = {n: x[1] for n, x in d.items()}
        out = torch.full((B, H, N, dv), 7.0, device="cuda", dtype=g["v"].dtype)
        before = g["states"].clone()
        got = lla.decode_tree(g["q"], g["k"], g["v"], g["log_a"], g["lam"], g["states"], g["t"], g["parent"], out=out)
        assert got is out and torch.equal(before.view(torch.int32), g["states"].view(torch.int32))
        twice = torch.full_like(out, 7.0)
        lla.decode_tree(g["q"], g["k"], g["v"], g["log_a"], g["lam"], g["states"], g["t"], g["parent"], out=twice)
        assert torch.equal(out, twice)
        # linear: one state without holes
        state, st = normal(r, (B, H, dk, dv), "f32", dk ** -0.5)
        lin = torch.full_like(out, 7.0)
        lla.linear_decode_tree(g["q"], g["k"], g["v"], g["g"], st, g["parent"], out=lin)
        for b in range(B):
            alive = np.array(trees[b]) != -2
            deep = max(len(R.branch(trees[b], i)) for i in range(N) if alive[i])
            for h in range(H):
                a = [d[n][0][b, h] for n in ("q", "k", "v", "log_a", "lam", "states")]
                ref, size = R.tree(*a, t[b], trees[b])
                terms = dk * (Lmax + deep)
                R.tree_check(np64(out[b, h])[alive], ref[alive], size[alive], dtype, terms, gate_units(a[3], deep + 1),
                             (b, h))
                ref, size = R.linear_tree(*a[:3], d["g"][0][h], state[b, h], trees[b])
                R.tree_check(np64(lin[b, h])[alive], ref[alive], size[alive], dtype, terms,
                             gate_units(d["g"][0], deep + 1), ("linear", b, h))
            assert bool((out[b][:, ~torch.from_numpy(alive).cuda()] == 7).all())
            assert bool((lin[b][:, ~torch.from_numpy(alive).cuda()] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,N,dk,dv,Lmax,t", CASES)
def test_commit(lla, B, H, N, dk, dv, Lmax, t, dtype):
    r = np.random.default_rng(N * dk + dv + 1)
    for most in (1, 4, N):
        d = draft(r, B, H, N, dk, dv, dtype, Lmax, t, live=N)
        g = {n: x[1] for n, x in d.items()}
        # any nodes in any order, the same one twice among them; the first sequence takes as many as it may
        paths = [[int(x) for x in r.integers(0, N, min(most, (1 << (Lmax - 1)) - t[b]) if b == 0 else
                                             int(r.integers(0, min(most, (1 << (Lmax - 1)) - t[b]) + 1)))] for b in range(B)]
        M = max(1, max(len(p) for p in paths))
        path = ints([p + [-9] * (M - len(p)) for p in paths])
        count = ints([len(p) for p in paths])
        before = g["states"].clone()
        assert lla.decode_commit(g["k"], g["v"], g["log_a"], g["states"], g["t"], count, path) is g["states"]
        state, st = normal(r, (B, H, dk, dv), "f32", dk ** -0.5)
        lla.linear_decode_commit(g["k"], g["v"], g["g"], st, count, path)
        for b in range(B):
            n = len(paths[b])
            held = R.held(t[b] + n - 1) if n else {}
            for h in range(H):
                k, v, la, s = (d[x][0][b, h] for x in ("k", "v", "log_a", "states"))
                ref, size = R.commit(k, v, la, s, t[b], paths[b])
                for m in range(Lmax):
                    if m in held:
                        R.tree_check(np64(g["states"][b, h, m]), ref[m], size[m], "f32", n + Lmax, gate_units(la, n + 1),
                                     (b, h, m))
                    else:
                        assert torch.equal(g["states"][b, h, m].view(torch.int32), before[b, h, m].view(torch.int32))
                ref, size = R.linear_commit(k, v, d["g"][0][h], state[b, h], paths[b])
                R.tree_check(np64(st[b, h]), ref, size, "f32", n + 2, gate_units(d["g"][0], n + 1), ("linear", b, h))
        # without a path: the first tokens in order
        first = ints([min(N, most, (1 << (Lmax - 1)) - x) for x in t])
        one, two = before.clone(), before.clone()
        lla.decode_commit(g["k"], g["v"], g["log_a"], one, g["t"], first)
        lla.decode_commit(g["k"], g["v"], g["log_a"], two, g["t"], first, torch.arange(N, dtype=torch.int32,
                                                                                        device="cuda").repeat(B, 1))
        assert torch.equal(one.view(torch.int32), two.view(torch.int32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_chain_is_decode_steps(lla, dtype):
    """Outputs of a chain and its commit against the steps that it stands for, carries of every size among them."""
    B, H, N, dk, dv, Lmax = 5, 2, 24, 64, 32, 12
    r = np.random.default_rng(5)
    t = [0, 1, 120, 1000, 1020]
    d = draft(r, B, H, N, dk, dv, dtype, Lmax, t, chain=1.0, live=N)
    g = {n: x[1] for n, x in d.items()}
    tree = lla.decode_tree(g["q"], g["k"], g["v"], g["log_a"], g["lam"], g["states"], g["t"], g["parent"])
    lin_state = torch.randn(B, H, dk, dv, device="cuda") * dk ** -0.5
    lin = lla.linear_decode_tree(g["q"], g["k"], g["v"], g["g"], lin_state, g["parent"])
    states, state = g["states"].clone(), lin_state.clone()
    tol = 2e-2 if dtype == "bf16" else 2e-5  # of the largest output: two roundings to bf16; fp32 sums in another order
    for i in range(N):
        tok = [g[n][:, :, i].contiguous() for n in ("q", "k", "v", "log_a", "lam")]
        o = lla.decode_step(*tok, states, g["t"] + i)
        assert (o.float() - tree[:, :, i].float()).abs().max() <= tol * o.float().abs().max()
        o = lla.linear_decode_step(*tok[:3], g["g"], state)
        assert (o.float() - lin[:, :, i].float()).abs().max() <= tol * o.float().abs().max()
        if i in (0, 1, 6, N - 1):
            mine, one = g["states"].clone(), lin_state.clone()
            n = ints([i + 1] * B)
            lla.decode_commit(g["k"], g["v"], g["log_a"], mine, g["t"], n)
            lla.linear_decode_commit(g["k"], g["v"], g["g"], one, n)
            assert (one - state).abs().max() <= 1e-5 * state.abs().max()
            for b in range(B):
                for m in R.held(t[b] + i):
                    a, c = mine[b, :, m], states[b, :, m]
                    assert (a - c).abs().max() <= 1e-5 * c.abs().max().clamp(min=1e-3), (i, b, m)


def test_bad_sequences_are_skipped(lla):
    B, H, N, dk, dv, Lmax = 9, 2, 4, 32, 16, 6
    t = [5, 31, 29, -1, 32, 5, 5, 5, 5]
    parent = [[-1, 0, 1, 1], [-1, -1, -1, -1], [-1, 0, 1, 2], [-1, 0, 0, 0], [-1, 0, 0, 0], [-1, 1, 0, 0], [-1, -2, 1, 0],
              [-4, 0, 0, 0], [-1, 0, 0, 1 << 20]]
    good = [0, 1]  # position 31 is the last that Lmax = 6 holds; 29 with four nodes in a row reaches 32
    q, k = torch.randn(2, B, H, N, dk, device="cuda").unbind()
    v, la, lam = torch.randn(B, H, N, dv, device="cuda"), -torch.rand(B, H, N, device="cuda"), torch.rand(B, H, N, Lmax,
                                                                                                         device="cuda")
    states = torch.randn(B, H, Lmax, dk, dv, device="cuda")
    out = torch.full((B, H, N, dv), 7.0, device="cuda")
    lla.decode_tree(q.contiguous(), k.contiguous(), v, la, lam, states, ints(t, torch.int64), ints(parent), out=out)
    assert lla.device_error() == lla.LLA_ERR_DEVICE
    for b in range(B):
        assert bool((out[b] == 7).any()) == (b not in good), b
    lin = torch.full_like(out, 7.0)
    lla.linear_decode_tree(q.contiguous(), k.contiguous(), v, la[0, :, 0].contiguous(), states[:, :, 0].contiguous(),
                           ints(parent), out=lin)
    assert lla.device_error() == lla.LLA_ERR_DEVICE
    for b in range(B):
        assert bool((lin[b] == 7).any()) == (b > 4), b
    count = [1, 1, 4, 1, 1, -1, 4, 2, 2]
    path = [[0, 9, 9], [3, 9, 9], [0, 1, 2], [0, 1, 2], [0, 1, 2], [0, 1, 2], [0, 1, 2], [4, 0, 0], [0, -1, 0]]
    was = states.clone()
    lla.decode_commit(k.contiguous(), v, la, states, ints(t, torch.int64), ints(count), ints(path))
    assert lla.device_error() == lla.LLA_ERR_DEVICE
    for b in range(B):
        assert torch.equal(states[b], was[b]) == (b not in good), b
    one, was = states[:, :, 0].contiguous(), states[:, :, 0].clone()
    lla.linear_decode_commit(k.contiguous(), v, la[0, :, 0].contiguous(), one, ints(count), ints(path))
    assert lla.device_error() == lla.LLA_ERR_DEVICE
    for b in range(B):
        assert torch.equal(one[b], was[b]) == (b in (2, 5, 6, 7, 8)), b


def test_positions_that_overflow_are_refused(lla):
    B, H, N, d, Lmax = 3, 1, 2, 16, 40
    q, k, v = torch.randn(3, B, H, N, d, device="cuda").unbind()
    la, lam = -torch.rand(B, H, N, device="cuda"), torch.rand(B, H, N, Lmax, device="cuda")
    states, out = torch.randn(B, H, Lmax, d, d, device="cuda"), torch.full((B, H, N, d), 7.0, device="cuda")
    t = ints([2 ** 63 - 1, -2 ** 63, 2 ** 39], torch.int64)
    lla.decode_tree(q.contiguous(), k.contiguous(), v.contiguous(), la, lam, states, t, ints([-1, 0]), out=out)
    assert lla.device_error() == lla.LLA_ERR_DEVICE and bool((out == 7).all())
    was = states.clone()
    lla.decode_commit(k.contiguous(), v.contiguous(), la, states, t, ints([2, 2, 1]))
    assert lla.device_error() == lla.LLA_ERR_DEVICE and torch.equal(states, was)
    # the last position that there is
    t = ints([2 ** 39 - 1] * B, torch.int64)
    lla.decode_commit(k.contiguous(), v.contiguous(), la, states, t, ints([2, 1, 0]))
    assert lla.device_error() == lla.LLA_ERR_DEVICE
    assert [torch.equal(states[b], was[b]) for b in range(B)] == [True, False, True]


def test_values_that_are_not_finite_stay_on_their_branch(lla):
    B, H, N, dk, dv, Lmax = 1, 2, 20, 64, 48, 9
    r = np.random.default_rng(8)
    for dtype in ("bf16", "f32"):
        d = draft(r, B, H, N, dk, dv, dtype, Lmax, [100], live=N)
        g, trees = {n: x[1] for n, x in d.items()}, d["parent"][0]
        call = lambda: lla.decode_tree(g["q"], g["k"], g["v"], g["log_a"], g["lam"], g["states"], g["t"], g["parent"])  # noqa: E731
        clean = call()
        for name, at in (("q", 3), ("k", 4), ("v", 5), ("log_a", 2)):
            keep = g[name].clone()
            g[name][0, 1, at] = float("nan")
            out = call()
            g[name].copy_(keep)
            hit = [i for i in range(N) if (i == at if name == "q" else at in R.branch(trees[0], i))]
            rest = [i for i in range(N) if i not in hit]
            assert torch.equal(out[0, 0], clean[0, 0]) and torch.equal(out[0, 1, rest], clean[0, 1, rest]), name
            if name != "log_a":  # a node's own log_a does not weigh its own key, but the states and the nodes above
                assert not torch.isfinite(out[0, 1, hit]).any(), name


def test_decays_of_zero(lla):
    """log_a = -inf: nothing before the node counts, in the tree and after its commit."""
    B, H, N, dk, dv, Lmax = 1, 1, 4, 32, 16, 6
    r = np.random.default_rng(9)
    d = draft(r, B, H, N, dk, dv, "f32", Lmax, [13], chain=1.0, live=N)
    g = {n: x[1] for n, x in d.items()}
    for la, lg in ((g["log_a"], g["g"]),):
        la[0, 0, 2] = -float("inf")
        lg[0] = -float("inf")
    out = lla.decode_tree(g["q"], g["k"], g["v"], g["log_a"], g["lam"], g["states"], g["t"], g["parent"])
    q, k, v, lam = (d[n][0][0, 0] for n in ("q", "k", "v", "lam"))
    ref = lam[2, 0] * (q[2] @ k[2]) * v[2]
    assert np.abs(np64(out[0, 0, 2]) - ref).max() <= 1e-5 * np.abs(ref).max()
    state = torch.randn(B, H, dk, dv, device="cuda")
    lin = lla.linear_decode_tree(g["q"], g["k"], g["v"], g["g"], state, g["parent"])
    ref = np.einsum("nd,nd->n", q, k)[:, None] * v
    assert np.abs(np64(lin[0, 0]) - ref).max() <= 1e-5 * np.abs(ref).max()
    lla.decode_commit(g["k"], g["v"], g["log_a"], g["states"], g["t"], ints([3]))
    for m, (lo, hi) in R.held(15).items():
        ref = sum((np.outer(k[s - 13], v[s - 13]) for s in range(max(lo, 15), hi)), np.zeros((dk, dv)))
        assert np.abs(np64(g["states"][0, 0, m]) - ref).max() <= 1e-6, m
    lla.linear_decode_commit(g["k"], g["v"], g["g"], state, ints([2]))
    assert np.abs(np64(state[0, 0]) - np.outer(k[1], v[1])).max() <= 1e-6


def test_graphs_streams_and_given_outputs(lla):
    B, H, N, dk, dv, Lmax = 4, 3, 21, 64, 64, 11
    r = np.random.default_rng(10)
    d = draft(r, B, H, N, dk, dv, "bf16", Lmax, [0, 7, 400, 1000], live=N)
    g = {n: x[1] for n, x in d.items()}
    args = [g[n] for n in ("q", "k", "v", "log_a", "lam", "states", "t", "parent")]
    ref = lla.decode_tree(*args)
    count, path = ints([2, 0, 1, 2]), ints([[0, 1], [0, 0], [3, 3], [1, 2]])
    done = lla.decode_commit(g["k"], g["v"], g["log_a"], g["states"].clone(), g["t"], count, path)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = lla.decode_tree(*args, stream=side)
    st = g["states"].clone()
    side.wait_stream(torch.cuda.current_stream())
    lla.decode_commit(g["k"], g["v"], g["log_a"], st, g["t"], count, path, stream=side)
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(st.view(torch.int32), done.view(torch.int32))
    graph = torch.cuda.CUDAGraph()
    st = g["states"].clone()
    with torch.cuda.graph(graph):
        st.copy_(g["states"])
        o = lla.decode_tree(g["q"], g["k"], g["v"], g["log_a"], g["lam"], st, g["t"], g["parent"])
        lla.decode_commit(g["k"], g["v"], g["log_a"], st, g["t"], count, path)
    for _ in range(2):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, ref) and torch.equal(st.view(torch.int32), done.view(torch.int32))
    # parts of larger arrays that start between 16 bytes
    whole = torch.zeros(5, N, dtype=torch.int32, device="cuda")
    whole[1:] = g["parent"]
    assert whole[1:].data_ptr() % 16
    cut = args[:7] + [whole[1:]]
    assert torch.equal(lla.decode_tree(*cut), ref)
    with pytest.raises(ValueError):
        lla.decode_tree(*args[:7], g["parent"][:, :-1].contiguous())
    with pytest.raises(lla.LLAError):
        lla.decode_tree(*args, out=g["v"])


def test_parameters_are_tensors(lla):
    """What a module holds (torch.nn.Parameter) is taken like any other tensor."""
    P = lambda x: torch.nn.Parameter(x, requires_grad=False)
    r = np.random.default_rng(14)
    d = draft(r, 2, 2, 5, 64, 64, "bf16", 9, [100, 3], live=5)
    g = {n: x[1] for n, x in d.items()}
    args = [g[n] for n in ("q", "k", "v", "log_a", "lam", "states", "t", "parent")]
    ref = lla.decode_tree(*args)
    assert torch.equal(lla.decode_tree(*(P(x) for x in args)), ref)
    count = ints([2, 1])
    one, two = g["states"].clone(), P(g["states"].clone())
    lla.decode_commit(g["k"], g["v"], g["log_a"], one, g["t"], count)
    lla.decode_commit(P(g["k"]), P(g["v"]), P(g["log_a"]), two, g["t"], P(count))
    assert torch.equal(one.view(torch.int32), two.detach().view(torch.int32))  # slots that hold nothing are NaN
    decay, state = torch.full((2,), -0.1, device="cuda"), g["states"][:, :, 0].contiguous()
    ref = lla.linear_decode_tree(*args[:3], decay, state, args[7])
    assert torch.equal(lla.linear_decode_tree(*args[:3], P(decay), P(state), args[7]), ref)


def test_two_streams_at_once(lla):
    B, H, N, dk, dv, Lmax = 32, 8, 30, 128, 64, 14
    r = np.random.default_rng(13)
    d = draft(r, B, H, N, dk, dv, "bf16", Lmax, [int(x) for x in r.integers(0, 8000, B)])
    g = {n: x[1] for n, x in d.items()}
    args = [g[n] for n in ("q", "k", "v", "log_a", "lam", "states", "t", "parent")]
    want = lla.decode_tree(*args, out=torch.zeros_like(g["v"]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream(priority=-1)]
    outs = [torch.zeros_like(g["v"]) for _ in range(6)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        lla.decode_tree(*args, out=o, stream=streams[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(104, 64), (100, 64), (64, 20), (128, 100), (40, 33), (8, 8), (72, 128),
                                   (128, 126), (100, 50), (24, 2), (33, 1), (17, 66)])
def test_every_way_of_copying(lla, dk, dv, dtype):
    """Rows of whole 16-byte pieces or not, of states and of tokens; a chain, whose nodes all count."""
    B, H, N, Lmax, t = 2, 2, 37, 13, [3000, 17]
    r = np.random.default_rng(dk + dv)
    d = draft(r, B, H, N, dk, dv, dtype, Lmax, t, chain=0.9, live=N)
    g = {n: x[1] for n, x in d.items()}
    out = lla.decode_tree(g["q"], g["k"], g["v"], g["log_a"], g["lam"], g["states"], g["t"], g["parent"])
    for b in range(B):
        deep = max(len(R.branch(d["parent"][0][b], i)) for i in range(N))
        for h in range(H):
            a = [d[n][0][b, h] for n in ("q", "k", "v", "log_a", "lam", "states")]
            ref, size = R.tree(*a, t[b], d["parent"][0][b])
            R.tree_check(np64(out[b, h]), ref, size, dtype, dk * (Lmax + deep), gate_units(a[3], deep + 1), (b, h))


def test_states_behind_element_2_31(lla):
    B, H, N, dk, dv, Lmax = 480, 16, 9, 128, 128, 18
    r = np.random.default_rng(11)
    states = torch.empty(B, H, Lmax, dk, dv, device="cuda").normal_()
    assert states.numel() > 2 ** 31
    d = draft(r, 1, H, N, dk, dv, "bf16", 2, [0], live=N)
    g = {n: x[1] for n, x in d.items()}
    rep = lambda x: x.expand(B, *x.shape[1:]).contiguous()  # noqa: E731
    lam = torch.rand(1, H, N, Lmax, device="cuda")
    t = ints([70000 + b for b in range(B)], torch.int64)
    big = [rep(g[n]) for n in ("q", "k", "v", "log_a")]
    out = lla.decode_tree(*big, rep(lam), states, t, g["parent"])
    # a call of enough heads to be cut into blocks as the large one is (fewer are cut more finely, their sums otherwise)
    last = [x[-8:].clone() for x in (*big, rep(lam), states, t)]
    assert torch.equal(lla.decode_tree(*last, g["parent"]), out[-8:])
    lla.decode_commit(last[1], last[2], last[3], last[5], last[6], ints([3] * 8))
    lla.decode_commit(big[1], big[2], big[3], states, t, ints([3] * B))
    assert torch.equal(last[5], states[-8:])


def test_a_server_round(lla):
    """A stack of a log-linear, a linear and a gated layer: prompt, a drafted tree through all three, the accepted branch
    committed, the next token; against decode steps on the accepted tokens alone."""
    B, H, T, N, d = 2, 2, 256, 10, 64
    D = H * d
    r = np.random.default_rng(12)
    Lmax = 11

    def layer(T):
        return {n: normal(r, (B, H, T, d), "bf16", d ** -0.5 if n != "v" else 1.0)[1] for n in ("q", "k", "v")}

    prompt, drafts, nxt = layer(T), layer(N), layer(1)
    la = {n: -torch.rand(B, H, m, device="cuda") * 0.2 for n, m in (("p", T), ("d", N), ("n", 1))}
    lam = {n: torch.rand(B, H, m, x, device="cuda") for n, m, x in (("p", T, lla.num_levels(T)), ("d", N, Lmax), ("n", 1, Lmax))}
    slopes = torch.tensor([-0.5, -0.01], device="cuda")
    gates = {n: -torch.rand(B, m, D, device="cuda") * 0.3 for n, m in (("p", T), ("d", N), ("n", 1))}
    merge = lambda o: o.transpose(1, 2).reshape(B, -1, D).contiguous()  # noqa: E731  heads side by side for the gated layer
    states, state, h = (torch.empty(B, H, Lmax, d, d, device="cuda"), torch.empty(B, H, d, d, device="cuda"),
                        torch.empty(B, D, device="cuda"))
    # prompt
    o1 = lla.forward(prompt["q"], prompt["k"], prompt["v"], la["p"], lam["p"], 64)
    lla.prefill_state(prompt["k"], prompt["v"], la["p"], states)
    o2 = lla.linear_forward(prompt["q"], prompt["k"], o1, slopes, state_out=state)
    lla.gated_forward(merge(o2), gates["p"], state_out=h)
    # draft
    parent = R.random_tree(r, N)
    t = ints([T] * B, torch.int64)
    d1 = lla.decode_tree(drafts["q"], drafts["k"], drafts["v"], la["d"], lam["d"], states, t, ints(parent))
    d2 = lla.linear_decode_tree(drafts["q"], drafts["k"], d1, slopes, state, ints(parent))
    d3 = lla.gated_decode_tree(merge(d2), gates["d"], h, ints(parent))
    # decode steps along the accepted branch
    way = R.branch(parent, N - 1)
    s1, s2, s3 = states.clone(), state.clone(), h.clone()
    pick = lambda x, i: x[:, :, i].contiguous()  # noqa: E731
    for step, j in enumerate(way):
        e1 = lla.decode_step(*(pick(drafts[n], j) for n in ("q", "k", "v")), pick(la["d"], j), pick(lam["d"], j), s1, t + step)
        e2 = lla.linear_decode_step(pick(drafts["q"], j), pick(drafts["k"], j), e1, slopes, s2)
        e3 = lla.gated_decode_step(e2.reshape(B, D), gates["d"][:, j].contiguous(), s3)
    # each layer rounds to bf16, and a rounding that falls the other way goes through the next layers: 3 x 2^-8 and growth
    assert (e3.float() - d3[:, N - 1].float()).abs().max() <= 4e-2 * e3.float().abs().max()
    # commit
    count, path = ints([len(way)] * B), ints([way] * B)
    lla.decode_commit(drafts["k"], drafts["v"], la["d"], states, t, count, path)
    lla.linear_decode_commit(drafts["k"], d1, slopes, state, count, path)
    lla.gated_decode_commit(merge(d2), gates["d"], h, count, path)
    for m in R.held(T + len(way) - 1):
        assert (states[:, :, m] - s1[:, :, m]).abs().max() <= 1e-5 * s1[:, :, m].abs().max()
    assert (state - s2).abs().max() <= 4e-2 * s2.abs().max() and (h - s3).abs().max() <= 4e-2 * s3.abs().max()
    # the next token
    a = lla.decode_step(*(pick(nxt[n], 0) for n in ("q", "k", "v")), pick(la["n"], 0), pick(lam["n"], 0), states, t + len(way))
    b = lla.decode_step(*(pick(nxt[n], 0) for n in ("q", "k", "v")), pick(la["n"], 0), pick(lam["n"], 0), s1, t + len(way))
    assert (a.float() - b.float()).abs().max() <= 2e-2 * b.float().abs().max()
