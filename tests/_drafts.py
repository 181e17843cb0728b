"""Plain 64-bit forms of the gated linear recurrence and of trees of drafted tokens, and what roundings may cost.

The recurrence is written as sums over the rows that a row sees, its gradients as their transposes; the trees as the
sums over a node's own branch. Arrays are numpy float64.
"""
import numpy as np

U32 = 2.0 ** -24  # half a step of fp32, relative
UBF = 2.0 ** -8   # half a step of bf16, relative


def weights(log_a):
    """[D, T, T]: product of the gates after row s up to row t (1 at s = t), 0 above the diagonal. log_a [T, D]."""
    T, D = log_a.shape
    w = np.zeros((D, T, T))
    a = np.exp(log_a)
    for s in range(T):
        p = np.ones(D)
        w[:, s, s] = p
        for t in range(s + 1, T):
            p = p * a[t]
            w[:, t, s] = p
    return w


def gated(x, log_a, s0=None):
    """(h [T, D], last state [D]) of one sequence."""
    T, D = x.shape
    if T == 0:
        return x.copy(), np.zeros(D) if s0 is None else s0.copy()
    w = weights(log_a)
    h = np.einsum("dts,sd->td", w, x)
    if s0 is not None:
        h = h + w[:, :, 0].T * np.exp(log_a[0]) * s0
    return h, h[-1]


def gated_grads(log_a, h, dout, s0=None, ds=None):
    """(dx, dlog_a, dstate0) of one sequence for the outputs h as given."""
    T, D = h.shape
    ds = np.zeros(D) if ds is None else ds
    if T == 0:
        return h.copy(), h.copy(), ds.copy()
    w = weights(log_a)
    dx = np.einsum("dts,td->sd", w, dout) + w[:, -1].T * ds
    before = np.concatenate([(np.zeros(D) if s0 is None else s0)[None], h[:-1]])
    f = dx * np.exp(log_a)
    return dx, f * before, f[0]


def gated_check(got, ref, size, dtype, what, factors=1):
    """Every value within what its roundings may cost.

    ``size``: the values that the same sums take with absolute values, where each row's own share is counted once for
    every row that carries it on (see gated_size): a step rounds the gate (expf: one unit in the last place, 2^-23),
    the product of gates, the state, and one product in eight rows for each of the three compositions; 5 x 2^-24
    together, 2^-21 with a little to spare. ``factors``: further fp32 factors of the result."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), what
    bound = 2.0 ** -21 * size + factors * U32 * np.abs(ref)
    if dtype == "bf16":
        bound = bound + UBF * (np.abs(ref) + bound)
    worst = np.max(np.abs(got - ref) - bound - 1e-37) if got.size else 0
    assert worst <= 0, (what, worst)


def gated_size(x, log_a, s0=None):
    """sum_s (t - s + 1) w_ts |x_s|, with the entering state as one more row: [T, D], and its last row."""
    T, D = x.shape
    if T == 0:
        return np.zeros((0, D)), np.zeros(D) if s0 is None else np.abs(s0)
    x = np.abs(x)
    a = np.exp(log_a)
    h = np.zeros(D) if s0 is None else np.abs(s0)
    e = h.copy()
    out = np.zeros((T, D))
    for t in range(T):
        h = a[t] * h + x[t]
        e = a[t] * e + h
        out[t] = e
    return out, out[-1]


# ---- trees

def branch(parent, i):
    """Nodes from the root of node i's branch to i."""
    way = []
    while i >= 0:
        way.append(i)
        i = parent[i]
    return way[::-1]


def held(pos):
    """{slot: (first, last + 1)} of the Fenwick partition of 0..pos (none for pos = -1)."""
    if pos < 0:
        return {}
    got, end = {0: (pos, pos + 1)}, pos
    while end > 0:
        low = end & -end
        got[low.bit_length()] = (end - low, end)
        end -= low
    return got


def level(t, s):
    return int(t ^ s).bit_length()


def tree(q, k, v, log_a, lam, states, t, parent):
    """(outputs [N, dv], their sizes) of one head: q, k [N, dk], v [N, dv], log_a [N], lam [N, L], states [L, dk, dv].
    Rows of places without a node are 0."""
    N, dv = q.shape[0], v.shape[1]
    out, size = np.zeros((N, dv)), np.zeros((N, dv))
    for i in range(N):
        if parent[i] == -2:
            continue
        way = branch(parent, i)
        pos = t + len(way) - 1
        D = 0.0
        for step in reversed(range(len(way))):
            j = way[step]
            w = lam[i, level(pos, t + step)] * np.exp(D)
            out[i] += w * (q[i] @ k[j]) * v[j]
            size[i] += abs(w) * (np.abs(q[i]) @ np.abs(k[j])) * np.abs(v[j])
            D += log_a[j]
        for m, (lo, _) in held(t - 1).items():
            w = lam[i, level(pos, lo)] * np.exp(D)
            out[i] += w * (q[i] @ states[m])
            size[i] += abs(w) * (np.abs(q[i]) @ np.abs(states[m]))
    return out, size


def linear_tree(q, k, v, g, state, parent):
    """As tree, one state [dk, dv] and the log decay g."""
    N, dv = q.shape[0], v.shape[1]
    out, size = np.zeros((N, dv)), np.zeros((N, dv))
    for i in range(N):
        if parent[i] == -2:
            continue
        way = branch(parent, i)
        for step, j in enumerate(way):
            n = len(way) - 1 - step
            w = 1.0 if n == 0 else np.exp(g * n)
            out[i] += w * (q[i] @ k[j]) * v[j]
            size[i] += w * (np.abs(q[i]) @ np.abs(k[j])) * np.abs(v[j])
        w = np.exp(g * len(way))
        out[i] += w * (q[i] @ state)
        size[i] += w * (np.abs(q[i]) @ np.abs(state))
    return out, size


def commit(k, v, log_a, states, t, path):
    """(states after the tokens of ``path``, their sizes) of one head; slots that the last leaves empty as they were."""
    out, size = states.copy(), np.abs(states)
    n = len(path)
    if n == 0:
        return out, size
    la = np.array([log_a[j] for j in path])
    after = [np.exp(la[s + 1:].sum()) for s in range(n)]
    for m, (lo, hi) in held(t + n - 1).items():
        new, big = np.zeros_like(states[0]), np.zeros_like(states[0])
        for o, (x, y) in held(t - 1).items():
            if lo <= x and y <= hi:
                new += np.exp(la.sum()) * states[o]
                big += np.exp(la.sum()) * np.abs(states[o])
        for s, j in enumerate(path):
            if lo <= t + s < hi:
                new += after[s] * np.outer(k[j], v[j])
                big += after[s] * np.abs(np.outer(k[j], v[j]))
        out[m], size[m] = new, big
    return out, size


def linear_commit(k, v, g, state, path):
    n = len(path)
    if n == 0:
        return state.copy(), np.abs(state)
    out, size = np.exp(g * n) * state, np.exp(g * n) * np.abs(state)
    for s, j in enumerate(path):
        w = 1.0 if s == n - 1 else np.exp(g * (n - 1 - s))
        out = out + w * np.outer(k[j], v[j])
        size = size + w * np.abs(np.outer(k[j], v[j]))
    return out, size


def tree_check(got, ref, size, dtype, terms, gate, what):
    """Every value within what its roundings may cost.

    ``terms`` products are summed, each sum rounding to 2^-24 (tensor cores truncate: 2^-23). ``gate``: what the weights
    may be off by in units of 2^-24, the sum of a branch's log decays times its length (each addition rounds) and the
    exponential's unit. bf16: states in two parts leave out 2^-16 of each element, and the result is rounded once."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), what
    bound = ((terms + 16) * 2 + gate + 4) * U32 * size
    if dtype == "bf16":
        bound = bound + 2.0 ** -16 * size
        bound = bound + UBF * (np.abs(ref) + bound)
    worst = np.max(np.abs(got - ref) - bound - 1e-37) if got.size else 0
    assert worst <= 0, (what, worst)


def random_tree(r, N, live=None, chain=0.4):
    """Parents of a tree of ``live`` nodes in N places, -2 behind them."""
    live = N if live is None else live
    return [-2 if i >= live else -1 if i == 0 else i - 1 if r.random() < chain else int(r.integers(-1, i))
            for i in range(N)]
