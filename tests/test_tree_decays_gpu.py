"""GPU checks of the weights that trees of drafted tokens and commits form from log decays: each weight by itself, behind
gates that forget by any amount, against 64 bits and against decode steps.

Keys and queries are ones, node j's value is the unit vector of column j and the state of slot m that of column N + m, so
every column of an output is one weight: nothing but its own roundings stands beside it."""
import numpy as np
import pytest

from tests import _drafts as R

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

U32, UBF = R.U32, R.UBF


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


def f32(x):
    x = np.asarray(x, dtype=np.float32)
    return x.astype(np.float64), torch.from_numpy(x).cuda()


def np64(t):
    return t.double().cpu().numpy()


def weights(log_a, lam, t, parent, dv):
    """(weights [N, dv], |D| of each) of one head; row i: node j's at column j, slot m's at column N + m."""
    N = len(parent)
    w, D = np.zeros((N, dv)), np.zeros((N, dv))
    for i in range(N):
        if parent[i] == -2:
            continue
        way = R.branch(parent, i)
        pos, d = t + len(way) - 1, 0.0
        for step in reversed(range(len(way))):
            w[i, way[step]], D[i, way[step]] = lam[i, R.level(pos, t + step)] * np.exp(d), abs(d)
            d += log_a[way[step]]
        for m, (lo, _) in R.held(t - 1).items():
            w[i, N + m], D[i, N + m] = lam[i, R.level(pos, lo)] * np.exp(d), abs(d)
    return w, D


def close(got, w, D, dtype, what, steps=0):
    """The exponent D is rounded twice (2 x 2^-24 |D|; what the sums' low halves leave out is far below one unit), expf is two
    units in the last place off at most (4 x 2^-24), its product with lambda rounds once, one unit to spare; bf16 outputs
    round once more. ``steps``: units that w itself, an output of decode steps, may be off by. 1e-37: weights below fp32's
    normal numbers."""
    finite = np.isfinite(D)
    bound = np.where(finite, (2 * np.where(finite, D, 0.0) + 6 + steps) * U32 * np.abs(w), 0.0)
    if dtype == "bf16":
        bound = bound + UBF * (np.abs(w) + bound) * (2 if steps else 1)
    got = np64(got) if torch.is_tensor(got) else got
    assert np.isfinite(got).all(), what
    worst = np.abs(got - w) - bound - 1e-37
    at = np.unravel_index(np.argmax(worst), worst.shape)
    assert worst[at] <= 0, (what, at, got[at], w[at])


GATES = {  # what some gates of a draft are, the others lie between 0 and -2
    "strong": [-30.0], "underflow": [-90.0, -103.0, -105.0], "1e4": [-1e4], "1e9": [-1e9], "lowest": [-3.4e38],
    "-inf": [-np.inf], "order": None, "many": [-20.0, -33.0, -60.0],
    "all": [-30.0, -200.0, -1e4, -1e6, -1e9, -3.4e38, -np.inf],
}


def gates(r, name, N):
    if name == "order":
        la = np.array([-1e9, -33, -0.5, -33, -0.5, -0.5, -20, -0.1] * (N // 8 + 1))[:N]
    else:
        la = -2 * r.random(N)
        for at in r.permutation(N)[:max(1, N // 6)]:
            la[at] = r.choice(GATES[name])
    return la.astype(np.float32)


def call(r, lla, names, N, L, dtype, t, parent, dv=64):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    B, H = len(t), len(names)
    la, lat = f32(np.stack([[gates(r, n, N) for n in names] for _ in range(B)]))
    lam, lamt = f32(0.25 + r.random((B, H, N, L)))
    one = torch.ones(B, H, N, 1, device="cuda", dtype=dt)
    v = torch.eye(N, dv, device="cuda", dtype=dt).expand(B, H, N, dv).contiguous()
    st = torch.eye(L, dv - N, device="cuda")
    states = torch.cat([torch.zeros(L, N, device="cuda"), st], 1).reshape(1, 1, L, 1, dv).expand(B, H, L, 1, dv).contiguous()
    out = torch.zeros_like(v)
    lla.decode_tree(one, one, v, lat, lamt, states, ints(t, torch.int64), ints(parent), out=out)
    return la, lam, lat, lamt, one, v, states, out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,L,chain", [(8, 9, 1.0), (24, 9, 1.0), (24, 9, 0.6), (48, 9, 0.9), (50, 12, 0.3)])
def test_tree_weights(lla, N, L, chain, dtype):
    r = np.random.default_rng(N + int(10 * chain))
    t = [0, 1, 100, (1 << (L - 1)) - N]
    names = list(GATES)
    parent = [R.random_tree(r, N, N if b % 2 else int(r.integers(1, N + 1)), chain) for b in range(len(t))]
    la, lam, _, _, _, _, _, out = call(r, lla, names, N, L, dtype, t, parent)
    for b in range(len(t)):
        for h, name in enumerate(names):
            w, D = weights(la[b, h], lam[b, h], t[b], parent[b], 64)
            close(out[b, h], w, D, dtype, (b, name))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_trees(lla, dtype):
    """As many nodes as there may be, in one column of depths and in a bush."""
    r = np.random.default_rng(3)
    for chain in (1.0, 0.2):
        N, L, dv, names = 119, 9, 128, ["1e9", "all"]
        parent = [R.random_tree(r, N, N, chain)] * 2
        la, lam, _, _, _, _, _, out = call(r, lla, names, N, L, dtype, [0, 100], parent, dv)
        for b, t in enumerate((0, 100)):
            for h, name in enumerate(names):
                w, D = weights(la[b, h], lam[b, h], t, parent[b], dv)
                close(out[b, h], w, D, dtype, (chain, b, name))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tree_weights_are_those_of_decode_steps(lla, dtype):
    r = np.random.default_rng(6)
    N, L, t, names = 24, 9, [0, 77], list(GATES)
    parent = [R.random_tree(r, N, N, 1.0), R.random_tree(r, N, N, 0.8)]
    la, lam, lat, lamt, one, v, states, out = call(r, lla, names, N, L, dtype, t, parent)
    for i in (5, 11, N - 1):
        ways = [R.branch(p, i) for p in parent]
        for b, way in enumerate(ways):
            st = states[b:b + 1].clone()
            for step, j in enumerate(way):
                pick = lambda x: x[b:b + 1, :, j].contiguous()  # noqa: E731
                o = lla.decode_step(pick(one), pick(one), pick(v), pick(lat), pick(lamt), st, ints([t[b] + step], torch.int64))
            for h, name in enumerate(names):
                _, D = weights(la[b, h], lam[b, h], t[b], parent[b], 64)
                # a step multiplies by expf of its gate: 4 + 1 units each, lambda's product one more
                close(out[b, h, i], np64(o[0, h]), D[i], dtype, (b, i, name), steps=5 * len(way) + 2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_tree_weights(lla, dtype):
    N, dv = 40, 64
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    r = np.random.default_rng(7)
    g, gt = f32([-0.01, -3.0, -30.0, -1e4, -1e9, -3.4e38, -np.inf, 0.0])
    H = len(g)
    one = torch.ones(1, H, N, 1, device="cuda", dtype=dt)
    v = torch.eye(N, dv, device="cuda", dtype=dt).expand(1, H, N, dv).contiguous()
    state = torch.zeros(1, H, 1, dv, device="cuda")
    state[..., N] = 1
    parent = R.random_tree(r, N, N, 0.8)
    out = lla.linear_decode_tree(one, one, v, gt, state, ints(parent))
    for h in range(H):
        w, D = np.zeros((N, dv)), np.zeros((N, dv))
        for i in range(N):
            way = R.branch(parent, i)
            for step, j in enumerate(way):
                n = len(way) - 1 - step
                d = g[h] * n if n else 0.0
                w[i, j], D[i, j] = np.exp(d), abs(d)
            w[i, N], D[i, N] = np.exp(g[h] * len(way)), abs(g[h] * len(way))
        close(out[0, h], w, D, dtype, float(g[h]))


@pytest.mark.parametrize("gate", [float("nan"), float("inf"), 200.0, -float("inf"), -1e9])
def test_the_first_gate_of_an_empty_state_weighs_nothing(lla, gate):
    """At t = 0 there is nothing that a root's gate could decay, whatever it is."""
    N, L, dv = 6, 5, 16
    r = np.random.default_rng(9)
    parent = [-1, 0, 1, -1, 3, 1]
    q, k = (torch.from_numpy(r.standard_normal((1, 1, N, 8)).astype(np.float32)).cuda() for _ in range(2))
    v = torch.from_numpy(r.standard_normal((1, 1, N, dv)).astype(np.float32)).cuda()
    la, lam = -torch.rand(1, 1, N, device="cuda"), torch.rand(1, 1, N, L, device="cuda")
    la[0, 0, [0, 3]] = 0.0
    states, t = torch.full((1, 1, L, 8, dv), float("nan"), device="cuda"), ints([0], torch.int64)
    want = lla.decode_tree(q, k, v, la, lam, states, t, ints(parent))
    odd = la.clone()
    odd[0, 0, [0, 3]] = gate
    assert torch.equal(lla.decode_tree(q, k, v, odd, lam, states, t, ints(parent)), want)


@pytest.mark.parametrize("t", [1, 6, 37])
@pytest.mark.parametrize("name", list(GATES))
def test_commit_weights(lla, name, t):
    """A slot's share of each token is the sum of the gates after it, added one by one from the end: an exponent of n gates is
    off by n x 2^-24 |D| at most."""
    r = np.random.default_rng(t)
    N, L, dv = 40, 9, 64
    la, lat = f32(gates(r, name, N).reshape(1, 1, N))
    one = torch.ones(1, 1, N, 1, device="cuda")
    v = torch.eye(N, dv, device="cuda").reshape(1, 1, N, dv).contiguous()
    for n in (1, 7, N):
        states = torch.zeros(1, 1, L, 1, dv, device="cuda")
        for m in range(L):
            states[0, 0, m, 0, N + m] = 1 if m in R.held(t - 1) else float("nan")
        lla.decode_commit(one, v, lat, states, ints([t], torch.int64), ints([n]))
        got = np64(states[0, 0, :, 0])
        after = [la[0, 0, s + 1:n].sum() for s in range(n)]
        whole = la[0, 0, :n].sum()
        for m, (lo, hi) in R.held(t + n - 1).items():
            w, D = np.zeros(dv), np.zeros(dv)
            for s in range(n):
                if lo <= t + s < hi:
                    w[s], D[s] = np.exp(after[s]), abs(after[s])
            for o, (x, y) in R.held(t - 1).items():
                if lo <= x and y <= hi:
                    w[N + o], D[N + o] = np.exp(whole), abs(whole)
            close(got[m], w, D * n, "f32", (name, n, m))
