"""CPU checks of linear attention with one decay per head and of the shared-prefix decode step: argument
errors found on the host, and the tests' own 64-bit forms against the recurrence and against differences."""
import os

import numpy as np
import pytest

from log_linear_attention_gb300 import binding, build
from tests import _linear as L

A = 4096  # a 16-byte-aligned fake address: only ever used in calls that fail validation
BAD, UNS = binding.LLA_ERR_INVALID_ARG, binding.LLA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH) or not hasattr(binding.load(), "lla_linear_forward"):
        build.build()
    return binding.load()


@pytest.mark.parametrize("over,expect", [
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(log_a=None), BAD), (dict(out=None), BAD),
    (dict(q=A + 8), BAD), (dict(out=A + 4), BAD), (dict(log_a=A + 4), BAD),
    (dict(state0=A, B0=0), BAD), (dict(state0=None, B0=1), BAD), (dict(state0=A, B0=2), BAD),
    (dict(state0=A, B0=-1), BAD), (dict(state0=A + 4, B0=1), BAD), (dict(state_out=A + 8), BAD),
    (dict(state0=A, B0=3, state_out=A), BAD),           # in place
    (dict(state0=A, B0=3, state_out=A + 1024), BAD),    # partly in place
    (dict(B=0), BAD), (dict(H=0), BAD), (dict(T=0), BAD), (dict(dk=0), BAD), (dict(dv=-1), BAD), (dict(dtype=2), BAD),
    (dict(dk=129), UNS), (dict(dv=200), UNS), (dict(B=3, H=65535), UNS), (dict(T=2 ** 31 - 1, H=21845), UNS),
])
def test_forward_refuses(lib, over, expect):
    a = dict(q=A, k=A, v=A, log_a=A, state0=None, out=A, state_out=None, B=3, B0=0, H=2, T=5, dk=16, dv=16, dtype=1)
    a.update(over)
    assert lib.lla_linear_forward(a["q"], a["k"], a["v"], a["log_a"], a["state0"], a["out"], a["state_out"], a["B"],
                                  a["B0"], a["H"], a["T"], a["dk"], a["dv"], None, a["dtype"]) == expect


@pytest.mark.parametrize("over,expect", [
    (dict(cu=None), BAD), (dict(cu=A + 4), BAD), (dict(n=0), BAD), (dict(total=0), BAD), (dict(max_T=0), BAD),
    (dict(state0=A, n0=2), BAD), (dict(state0=A, n0=1, state_out=A + 16), BAD), (dict(out=None), BAD),
    (dict(dk=130), UNS), (dict(n=65536, H=1), UNS),
])
def test_varlen_refuses(lib, over, expect):
    a = dict(cu=A, n=4, n0=0, state0=None, state_out=None, out=A, H=2, total=50, max_T=20, dk=16, dv=16)
    a.update(over)
    assert lib.lla_linear_forward_varlen(A, A, A, A, a["state0"], a["out"], a["state_out"], a["cu"], a["n"], a["n0"],
                                         a["H"], a["total"], a["max_T"], a["dk"], a["dv"], None, 1) == expect


@pytest.mark.parametrize("over,expect", [
    (dict(dout=None), BAD), (dict(dq=None), BAD), (dict(dk=A + 4), BAD), (dict(dv=None), BAD),
    (dict(dstate0=A), BAD),                      # a gradient of a state that is not there
    (dict(dstate_out=A + 4), BAD), (dict(state0=A, B0=1, dstate0=A + 4), BAD), (dict(d1=129), UNS),
])
def test_backward_refuses(lib, over, expect):
    a = dict(dout=A, dstate_out=None, dq=A, dk=A, dv=A, dstate0=None, state0=None, B0=0, d1=16)
    a.update(over)
    assert lib.lla_linear_backward(A, A, A, A, a["state0"], a["dout"], a["dstate_out"], a["dq"], a["dk"], a["dv"],
                                   a["dstate0"], 3, a["B0"], 2, 5, a["d1"], 16, None, 1) == expect


@pytest.mark.parametrize("over,expect", [
    (dict(state=None), BAD), (dict(state=A + 4), BAD), (dict(B=0), BAD), (dict(dk=129), UNS), (dict(dv=129), UNS),
    (dict(dtype=7), BAD),
])
def test_decode_refuses(lib, over, expect):
    a = dict(state=A, B=2, dk=16, dv=16, dtype=1)
    a.update(over)
    assert lib.lla_linear_decode_step(A, A, A, A, a["state"], A, None, a["B"], 2, a["dk"], a["dv"],
                                      a["dtype"]) == expect


@pytest.mark.parametrize("over,expect", [
    (dict(prefix=None), BAD), (dict(decay=None), BAD), (dict(decay=A + 4), BAD), (dict(t=None), BAD),
    (dict(P=0), BAD), (dict(P=-3), BAD), (dict(P=16), BAD),  # no position of 16 fits Lmax = 5
    (dict(P=9, Lp=4), BAD), (dict(Lp=0), BAD), (dict(Lmax=41), BAD), (dict(Lmax=0), BAD),
    (dict(dv=48), UNS), (dict(dk=257), UNS), (dict(dtype=3), BAD),
])
def test_shared_refuses(lib, over, expect):
    a = dict(prefix=A, decay=A, t=A, P=9, Lp=5, Lmax=5, dk=16, dv=16, dtype=1)
    a.update(over)
    assert lib.lla_decode_step_shared(A, A, A, A, A, a["prefix"], a["P"], a["Lp"], a["decay"], A, a["t"], A, None, 2,
                                      2, a["dk"], a["dv"], a["Lmax"], a["dtype"]) == expect


# arguments far enough apart for the sizes below, each at its own place; `over` moves one onto another
NAMES = ("q", "k", "v", "log_a", "state0", "dout", "dstate_out", "out", "state_out", "dq", "dk", "dv", "dstate0", "cu",
         "lambda", "prefix", "decay", "states", "t")
AT = {n: A + (i << 24) for i, n in enumerate(NAMES)}


@pytest.mark.parametrize("call,written,onto", [
    ("forward", "out", "v"), ("forward", "out", "q"), ("forward", "out", "state0"), ("forward", "state_out", "k"),
    ("forward", "state_out", "state0"), ("forward", "state_out", "out"), ("forward", "out", "log_a"),
    ("varlen", "out", "v"), ("varlen", "out", "cu"), ("varlen", "state_out", "state0"), ("varlen", "state_out", "out"),
    ("backward", "dq", "q"), ("backward", "dk", "dout"), ("backward", "dv", "dq"), ("backward", "dstate0", "dstate_out"),
    ("backward", "dstate0", "state0"), ("backward", "dv", "v"),
    ("decode", "out", "v"), ("decode", "states", "out"), ("decode", "states", "q"),
    ("shared", "out", "q"), ("shared", "states", "prefix"), ("shared", "decay", "log_a"), ("shared", "decay", "states"),
    ("shared", "states", "t"), ("shared", "out", "lambda"),
])
@pytest.mark.parametrize("by", [0, 16, -16])
def test_overlaps_are_refused(lib, call, written, onto, by):
    """Also by the last 16 bytes of one and the first of the other: every argument here has at least 32."""
    a = dict(AT)
    a[written] = a[onto] + by
    x = lambda *names: [a[n] for n in names]  # noqa: E731
    if call == "forward":
        st = lib.lla_linear_forward(*x("q", "k", "v", "log_a", "state0", "out", "state_out"), 3, 3, 8, 5, 16, 16, None, 1)
    elif call == "varlen":
        st = lib.lla_linear_forward_varlen(*x("q", "k", "v", "log_a", "state0", "out", "state_out", "cu"), 8, 8, 8, 50, 20,
                                           16, 16, None, 1)
    elif call == "backward":
        st = lib.lla_linear_backward(*x("q", "k", "v", "log_a", "state0", "dout", "dstate_out", "dq", "dk", "dv",
                                        "dstate0"), 3, 3, 8, 5, 16, 16, None, 1)
    elif call == "decode":
        st = lib.lla_linear_decode_step(*x("q", "k", "v", "log_a", "states", "out"), None, 3, 8, 16, 16, 1)
    else:
        st = lib.lla_decode_step_shared(*x("q", "k", "v", "log_a", "lambda", "prefix"), 9, 5,
                                        *x("decay", "states", "t", "out"), None, 4, 8, 16, 16, 5, 1)
    assert st == BAD

def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 1, 4, 16)
    with pytest.raises(ValueError, match="CUDA"):
        binding.linear_forward(x, x, x, torch.zeros(1))
    with pytest.raises(ValueError, match="CUDA"):
        binding.linear_decode_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], torch.zeros(1), torch.zeros(1, 1, 16, 16))


def problem(seed, T, dk=3, dv=2):
    r = np.random.default_rng(seed)
    q, k, v, do = (r.standard_normal((2, 2, T, d)) for d in (dk, dk, dv, dv))
    s0, ds = r.standard_normal((2, 2, 2, dk, dv))
    return q, k, v, np.array([-0.05, -0.7]), do, s0, ds


@pytest.mark.parametrize("T", [1, 2, 7])
def test_reference_is_the_recurrence(T):
    q, k, v, la, _, s0, _ = problem(1, T)
    S, out = s0.copy(), np.zeros_like(v)
    for t in range(T):
        S = np.exp(la)[:, None, None] * S + k[:, :, t, :, None] * v[:, :, t, None, :]
        out[:, :, t] = np.einsum("bhd,bhdv->bhv", q[:, :, t], S)
    o, s = L.forward(q, k, v, la, s0)
    assert np.allclose(o, out, atol=1e-13) and np.allclose(s, S, atol=1e-13)


@pytest.mark.parametrize("T", [1, 5])
def test_reference_gradients_are_the_differences(T):
    q, k, v, la, do, s0, ds = problem(2, T)

    def loss(*x):
        o, s = L.forward(x[0], x[1], x[2], la, x[3])
        return (o * do).sum() + (s * ds).sum()

    grads = L.backward(q, k, v, la, do, s0, ds)
    args = [q, k, v, s0]
    for n, g in enumerate(grads):
        for at in np.ndindex(*g.shape):
            d = []
            for e in (1e-5, -1e-5):
                x = [a.copy() for a in args]
                x[n][at] += e
                d.append(loss(*x))
            # the loss is bilinear, so the central difference is exact but for roundings (1e-16 / 1e-5 of it)
            assert abs((d[0] - d[1]) / 2e-5 - g[at]) < 1e-8


def test_no_rule_counts_on_one_chip():
    """How many SMs there are is asked of the device: the count of one chip stands in comments only."""
    import glob
    import re
    for path in glob.glob(os.path.join(build.CSRC, "lla_linear*.cu*")) + glob.glob(os.path.join(build.CSRC, "lla_shared.cu")):
        with open(path) as f:
            code = [line.split("//")[0] for line in f]
        assert not [line for line in code if re.search(r"\b15[0-9]\b", line)], path


def test_binding_does_without_torch_s_private_calls():
    from types import SimpleNamespace as N
    cuda = N(current_device=lambda: 3, current_stream=lambda index: N(cuda_stream=100 + index))
    device, stream = binding._cuda_calls(N(_C=N(), cuda=cuda))
    assert device() == 3 and stream(2) == 102
    device, stream = binding._cuda_calls(N(_C=N(_cuda_getDevice=lambda: 1, _cuda_getCurrentRawStream=lambda i: 7 + i),
                                           cuda=cuda))
    assert device() == 1 and stream(2) == 9


def test_calls_for_another_device_or_stream_run_there(monkeypatch):
    """What a call allocates belongs to the stream that writes it: device first, then stream, and a stream of another
    device is refused."""
    from contextlib import contextmanager
    from types import SimpleNamespace as N
    now = []

    def entered(kind):
        @contextmanager
        def inside(x):
            now.append((kind, x))
            try:
                yield
            finally:
                now.pop()
        return inside

    monkeypatch.setattr(binding, "_torch", lambda: N(cuda=N(device=entered("device"), stream=entered("stream"))))
    seen = lambda *args: (tuple(now), args)  # noqa: E731
    side = N(device="cuda:1")
    assert binding._elsewhere("cuda:1", None, seen, 1, 2) == ((("device", "cuda:1"),), (1, 2))
    assert binding._elsewhere("cuda:1", side, seen, 3) == ((("device", "cuda:1"), ("stream", side)), (3,))
    with pytest.raises(ValueError, match="cuda:1"):
        binding._elsewhere("cuda:0", side, seen)
    assert not now
