"""CPU checks of the gated recurrence, of trees of drafted tokens and of their commits: argument errors found on the
host, and the tests' own 64-bit forms against token-by-token recurrences and against differences."""
import os

import numpy as np
import pytest

from log_linear_attention_gb300 import binding, build
from tests import _drafts as R

A = 4096        # a 16-byte-aligned fake address: only ever used in calls that fail validation
Z = 1 << 40     # far from A's tensors
BAD, UNS = binding.LLA_ERR_INVALID_ARG, binding.LLA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH) or not hasattr(binding.load(), "lla_gated_forward"):
        build.build()
    return binding.load()


@pytest.mark.parametrize("over,expect", [
    (dict(x=None), BAD), (dict(log_a=None), BAD), (dict(out=None), BAD), (dict(x=A + 8), BAD), (dict(log_a=A + 4), BAD),
    (dict(out=Z + 8), BAD), (dict(state_out=A + 8), BAD), (dict(state0=A + 4, B0=1), BAD),
    (dict(state0=A, B0=0), BAD), (dict(state0=None, B0=1), BAD), (dict(state0=A, B0=2), BAD), (dict(B0=-1), BAD),
    (dict(out=A), BAD),                                  # in place
    (dict(out=A + 16), BAD), (dict(state_out=Z), BAD),   # onto the output
    (dict(state0=2 * Z, B0=3, state_out=2 * Z), BAD),
    (dict(B=0), BAD), (dict(T=0), BAD), (dict(D=0), BAD), (dict(dtype=2), BAD), (dict(gate=2), BAD),
    (dict(dtype=1, gate=0), BAD),                        # 16-bit gates of fp32 inputs
    (dict(B=2 ** 20, T=2 ** 20, D=2), UNS), (dict(T=2 ** 31 - 1), UNS), (dict(B=2 ** 28, T=1), UNS),
    (dict(B=1, T=1, D=2 ** 30 + 1), UNS),
])
def test_gated_forward_refuses(lib, over, expect):
    a = dict(x=A, log_a=A, state0=None, out=Z, state_out=None, B=3, B0=0, T=5, D=16, dtype=0, gate=1)
    a.update(over)
    assert lib.lla_gated_forward(a["x"], a["log_a"], a["state0"], a["out"], a["state_out"], a["B"], a["B0"], a["T"],
                                 a["D"], None, a["dtype"], a["gate"]) == expect


@pytest.mark.parametrize("over,expect", [
    (dict(cu=None), BAD), (dict(cu=A + 4), BAD), (dict(n=0), BAD), (dict(total=0), BAD), (dict(state0=A, n0=2), BAD),
    (dict(out=None), BAD), (dict(cu=Z + 16), BAD), (dict(n=2 ** 29), UNS), (dict(total=2 ** 31 - 1), UNS),
])
def test_gated_varlen_refuses(lib, over, expect):
    a = dict(cu=A, n=4, n0=0, state0=None, out=Z, total=50, D=16)
    a.update(over)
    assert lib.lla_gated_forward_varlen(A, A, a["state0"], a["out"], None, a["cu"], a["n"], a["n0"], a["total"], a["D"],
                                        None, 1, 1) == expect
    assert lib.lla_gated_backward_varlen(A, A, a["state0"], A, None, a["out"], 2 * Z, None, a["cu"], a["n"], a["n0"],
                                         a["total"], a["D"], None, 1, 1) == expect


@pytest.mark.parametrize("over,expect", [
    (dict(log_a=None), BAD), (dict(out=None), BAD), (dict(dout=None), BAD), (dict(dx=None), BAD), (dict(da=None), BAD),
    (dict(da=2 * Z + 4), BAD), (dict(ds=3 * Z), BAD),   # a gradient of a state that is not there
    (dict(dstate_out=A + 4), BAD), (dict(dx=A), BAD), (dict(da=Z), BAD), (dict(da=A + 32), BAD),
    (dict(state0=A, B0=3, ds=A), BAD), (dict(dtype=1, gate=0), BAD),
])
def test_gated_backward_refuses(lib, over, expect):
    a = dict(log_a=A, out=A, state0=None, dout=A, dstate_out=None, dx=Z, da=2 * Z, ds=None, B0=0, dtype=0, gate=0)
    a.update(over)
    assert lib.lla_gated_backward(a["log_a"], a["out"], a["state0"], a["dout"], a["dstate_out"], a["dx"], a["da"],
                                  a["ds"], 3, a["B0"], 5, 16, None, a["dtype"], a["gate"]) == expect


@pytest.mark.parametrize("over,expect", [
    (dict(x=None), BAD), (dict(state=None), BAD), (dict(state=A + 4), BAD), (dict(out=None), BAD), (dict(B=0), BAD),
    (dict(D=0), BAD), (dict(out=A), BAD), (dict(state=A), BAD), (dict(state=Z), BAD), (dict(gate=0), BAD),
    (dict(B=2 ** 21, D=2 ** 20), UNS),
])
def test_gated_step_refuses(lib, over, expect):
    a = dict(x=A, state=2 * Z, out=Z, B=2, D=16, gate=1)
    a.update(over)
    assert lib.lla_gated_decode_step(a["x"], A, a["state"], a["out"], None, a["B"], a["D"], 1, a["gate"]) == expect


@pytest.mark.parametrize("over,expect", [
    (dict(parent=None), BAD), (dict(parent=A + 4), BAD), (dict(state=None), BAD), (dict(out=None), BAD), (dict(B=0), BAD),
    (dict(BP=2), BAD), (dict(BP=0), BAD), (dict(N=0), BAD), (dict(N=129), UNS), (dict(D=0), BAD), (dict(out=A), BAD),
    (dict(B=65536, BP=1), UNS), (dict(gate=3), BAD),
])
def test_gated_tree_refuses(lib, over, expect):
    a = dict(state=A, parent=A, out=Z, B=3, BP=1, N=5, D=16, gate=1)
    a.update(over)
    assert lib.lla_gated_decode_tree(A, A, a["state"], a["parent"], a["out"], None, a["B"], a["BP"], a["N"], a["D"], 0,
                                     a["gate"]) == expect


@pytest.mark.parametrize("over,expect", [
    (dict(count=None), BAD), (dict(count=A + 4), BAD), (dict(path=A + 4), BAD), (dict(M=0), BAD),
    (dict(path=None, M=3), BAD), (dict(M=129), UNS), (dict(N=129), UNS), (dict(N=0), BAD), (dict(state=A), BAD),
    (dict(state=None), BAD), (dict(B=65536), UNS),
])
def test_gated_commit_refuses(lib, over, expect):
    a = dict(state=Z, count=A, path=A, B=3, N=5, M=3, D=16)
    a.update(over)
    assert lib.lla_gated_decode_commit(A, A, a["state"], a["count"], a["path"], None, a["B"], a["N"], a["M"], a["D"], 1,
                                       1) == expect


@pytest.mark.parametrize("over,expect", [
    (dict(q=None), BAD), (dict(lam=None), BAD), (dict(states=None), BAD), (dict(t=None), BAD), (dict(parent=None), BAD),
    (dict(out=None), BAD), (dict(t=A + 8), BAD), (dict(parent=A + 4), BAD), (dict(q=A + 2), BAD), (dict(B=0), BAD),
    (dict(H=0), BAD), (dict(N=0), BAD), (dict(dk=0), BAD), (dict(dv=0), BAD), (dict(Lmax=0), BAD), (dict(Lmax=41), BAD),
    (dict(BP=2), BAD), (dict(N=129), UNS), (dict(dk=129), UNS), (dict(dv=129), UNS), (dict(B=2 ** 16, BP=1, H=2 ** 16), UNS),
    (dict(dtype=2), BAD), (dict(out=A + 64), BAD),
])
def test_tree_refuses(lib, over, expect):
    a = dict(q=A, lam=A, states=A, t=A, parent=A, out=Z, B=3, BP=1, H=2, N=5, dk=16, dv=16, Lmax=5, dtype=1)
    a.update(over)
    assert lib.lla_decode_tree(a["q"], A, A, A, a["lam"], a["states"], a["t"], a["parent"], a["out"], None, a["B"],
                               a["BP"], a["H"], a["N"], a["dk"], a["dv"], a["Lmax"], a["dtype"]) == expect
    if not {"lam", "t", "Lmax"} & set(over):
        assert lib.lla_linear_decode_tree(a["q"], A, A, A, a["states"], a["parent"], a["out"], None, a["B"], a["BP"],
                                          a["H"], a["N"], a["dk"], a["dv"], a["dtype"]) == expect


@pytest.mark.parametrize("over,expect", [
    (dict(k=None), BAD), (dict(states=None), BAD), (dict(t=None), BAD), (dict(count=None), BAD), (dict(path=A + 4), BAD),
    (dict(count=A + 8), BAD), (dict(M=0), BAD), (dict(path=None), BAD), (dict(M=129), UNS), (dict(N=129), UNS),
    (dict(dk=129), UNS), (dict(dv=129), UNS), (dict(Lmax=41), BAD), (dict(states=A), BAD), (dict(H=0), BAD),
    (dict(dtype=-1), BAD),
])
def test_commit_refuses(lib, over, expect):
    a = dict(k=A, states=Z, t=A, count=A, path=A, B=3, H=2, N=5, M=3, dk=16, dv=16, Lmax=5, dtype=1)
    a.update(over)
    assert lib.lla_decode_commit(a["k"], A, A, a["states"], a["t"], a["count"], a["path"], None, a["B"], a["H"], a["N"],
                                 a["M"], a["dk"], a["dv"], a["Lmax"], a["dtype"]) == expect
    if not {"t", "Lmax"} & set(over):
        assert lib.lla_linear_decode_commit(a["k"], A, A, a["states"], a["count"], a["path"], None, a["B"], a["H"],
                                            a["N"], a["M"], a["dk"], a["dv"], a["dtype"]) == expect


def test_tensors_are_checked_before_the_library(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 5, 8)
    i = torch.zeros(5, dtype=torch.int32)
    q = torch.zeros(1, 2, 5, 8)
    for call in (lambda: binding.gated_forward(x, x), lambda: binding.gated_backward(x, x, x),
                 lambda: binding.gated_forward_varlen(x[0], x[0], i), lambda: binding.gated_decode_step(x[0], x[0], x[0]),
                 lambda: binding.gated_decode_tree(x, x, x[0], i), lambda: binding.gated_decode_commit(x, x, x[0], i),
                 lambda: binding.decode_tree(q, q, q, q[..., 0], q, q[None], i, i),
                 lambda: binding.decode_commit(q, q, q[..., 0], q[None], i, i),
                 lambda: binding.linear_decode_tree(q, q, q, x[0, 0], q, i),
                 lambda: binding.linear_decode_commit(q, q, x[0, 0], q, i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


# ---- the tests' own forms

def rows(seed, T, D):
    r = np.random.default_rng(seed)
    return r.standard_normal((T, D)), -np.logaddexp(0, r.standard_normal((T, D)) - 1), r.standard_normal(D)


def steps(x, log_a, s0):
    h, out = s0.copy(), np.zeros_like(x)
    for t in range(len(x)):
        h = np.exp(log_a[t]) * h + x[t]
        out[t] = h
    return out


@pytest.mark.parametrize("T", [1, 2, 9, 40])
def test_gated_sums_are_the_recurrence(T):
    x, log_a, s0 = rows(T, T, 3)
    if T > 4:
        log_a[3] = -np.inf
    for s in (None, s0):
        h, end = R.gated(x, log_a, s)
        ref = steps(x, log_a, np.zeros(3) if s is None else s)
        assert np.abs(h - ref).max() < 1e-13 and np.abs(end - ref[-1]).max() < 1e-13


@pytest.mark.parametrize("T", [1, 2, 7])
def test_gated_gradients_are_differences(T):
    D = 2
    x, log_a, s0 = rows(T + 50, T, D)
    r = np.random.default_rng(T)
    do, ds = r.standard_normal((T, D)), r.standard_normal(D)

    def loss(x, log_a, s0):
        h = steps(x, log_a, s0)
        return (do * h).sum() + (ds * h[-1]).sum()

    got = R.gated_grads(log_a, steps(x, log_a, s0), do, s0, ds)
    for which, (arr, grad) in enumerate(zip((x, log_a, s0), got)):
        for at in np.ndindex(arr.shape):
            e = np.zeros_like(arr)
            e[at] = 1e-5
            lo, hi = [(x, log_a, s0)[:which] + (arr + s * e,) + (x, log_a, s0)[which + 1:] for s in (-1, 1)]
            assert abs((loss(*hi) - loss(*lo)) / 2e-5 - grad[at]) < 1e-7


def log_step(q, k, v, la, lam, st, t):
    """One decode step on the recurrence's own terms: the carry by trailing zeros."""
    st = st * np.exp(la)
    if t > 0:
        c = (t & -t).bit_length() - 1
        st[c + 1] = sum(st[m] for m in range(c + 1) if m in R.held(t - 1))
    st[0] = np.outer(k, v)
    return sum(lam[m] * (q @ st[m]) for m in R.held(t)), st


@pytest.mark.parametrize("t", [0, 1, 2, 5, 7, 8, 31, 100])
def test_tree_and_commit_are_decode_steps(t):
    r = np.random.default_rng(t)
    N, dk, dv, L = 9, 4, 3, 9
    parent = R.random_tree(r, N)
    q, k = r.standard_normal((2, N, dk))
    v, la, lam = r.standard_normal((N, dv)), -r.random(N), r.random((N, L))
    st0 = r.standard_normal((L, dk, dv))
    out, _ = R.tree(q, k, v, la, lam, st0, t, parent)
    g, s0 = -0.3, r.standard_normal((dk, dv))
    lin, _ = R.linear_tree(q, k, v, g, s0, parent)
    for i in range(N):
        st, s = st0.copy(), s0.copy()
        way = R.branch(parent, i)
        for n, j in enumerate(way):
            o, st = log_step(q[j], k[j], v[j], la[j], lam[j], st, t + n)
            s = np.exp(g) * s + np.outer(k[j], v[j])
        assert np.abs(o - out[i]).max() < 1e-12 and np.abs(q[i] @ s - lin[i]).max() < 1e-12
        new, _ = R.commit(k, v, la, st0, t, way)
        for m in range(L):
            ref = st[m] if m in R.held(t + len(way) - 1) else st0[m]
            assert np.abs(new[m] - ref).max() < 1e-12, m
        assert np.abs(R.linear_commit(k, v, g, s0, way)[0] - s).max() < 1e-12
