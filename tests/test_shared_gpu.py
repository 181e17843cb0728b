"""GPU checks of the decode step over a shared prefix: against the pair sums of the log-linear operator in 64
bits, step by step from the end of the prefix, and against lla_decode_step on the whole states."""
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


def level(t, s):
    return int(t ^ s).bit_length()


def row(q, k, v, log_a, lam, t, absolute=False):
    """o_t [H, dv] of the pair sum over s <= t: k [H, T, dk], v [H, T, dv], log_a [H, T], q [H, dk], lam [H, Lmax]."""
    s = np.arange(t + 1)
    cum = np.cumsum(log_a, 1)
    w = np.exp(cum[:, t, None] - cum[:, :t + 1]) * lam[:, [level(t, x) for x in s]]
    if absolute:
        return np.einsum("hs,hsd,hd,hsv->hv", w, np.abs(k[:, :t + 1]), np.abs(q), np.abs(v[:, :t + 1]))
    return np.einsum("hs,hs,hsv->hv", w, np.einsum("hsd,hd->hs", k[:, :t + 1], q), v[:, :t + 1])


def softplus(x):
    return np.logaddexp(0, x)


def build(lla, P, B, H, dk, dv, dtype, steps, Lmax, seed):
    """A prefix, `steps` own tokens of every sequence, and the prefix's states."""
    r = np.random.default_rng(seed)
    d = {"pk": L.make(r, (1, H, P, dk), dtype, dk ** -0.5), "pv": L.make(r, (1, H, P, dv), dtype),
         "pa": L.make(r, (1, H, P), "f32")}
    for n, w, sc in (("q", dk, dk ** -0.5), ("k", dk, dk ** -0.5), ("v", dv, 1.0)):
        d[n] = L.make(r, (B, steps, H, w), dtype, sc)
    for n, shape in (("pa", (1, H, P)), ("a", (B, steps, H))):
        x = -softplus(r.standard_normal(shape) - 2).astype(np.float32)
        d[n] = x.astype(np.float64), torch.from_numpy(x)
    x = softplus(r.standard_normal((B, steps, H, Lmax))).astype(np.float32)
    d["lam"] = x.astype(np.float64), torch.from_numpy(x)
    d = {n: (a, t.cuda()) for n, (a, t) in d.items()}
    Lp = lla.num_levels(P) + (seed & 1)
    prefix = torch.full((1, H, Lp, dk, dv), float("nan"), device="cuda")
    lla.prefill_state(d["pk"][1], d["pv"][1], d["pa"][1], prefix)
    return d, prefix[0]


def step_args(d, i, t):
    """Inputs of every sequence's own token i."""
    return [d[n][1][:, i].clone() for n in ("q", "k", "v", "a", "lam")], t


@pytest.mark.parametrize("P,B,H,dk,dv,dtype,steps", [
    (1, 2, 2, 16, 16, "f32", 20), (2, 1, 1, 20, 32, "f32", 10), (3, 3, 2, 32, 64, "bf16", 14),
    (8, 2, 2, 64, 16, "f32", 17), (63, 2, 2, 128, 64, "bf16", 5), (64, 9, 3, 128, 64, "bf16", 5),
    (65, 2, 2, 100, 128, "f32", 70), (127, 17, 2, 64, 64, "f32", 4), (300, 2, 2, 256, 32, "f32", 30),
    (511, 2, 1, 128, 128, "bf16", 6),
])
def test_steps_from_the_prefix(lla, P, B, H, dk, dv, dtype, steps):
    Lmax = lla.num_levels(P + steps) + 1
    if dk > 128:  # the prefill takes 128: two halves of the keys, side by side
        a, pa = build(lla, P, B, H, dk // 2, dv, dtype, steps, Lmax, seed=P)
        b, pb = build(lla, P, B, H, dk // 2, dv, dtype, steps, Lmax, seed=P + 2)
        d = dict(a)
        for n in ("pk", "q", "k"):
            d[n] = np.concatenate([a[n][0], b[n][0]], -1), torch.cat([a[n][1], b[n][1]], -1)
        lla.prefill_state(b["pk"][1], a["pv"][1], a["pa"][1], pb[None])
        prefix = torch.cat([pa, pb], 2).contiguous()
    else:
        d, prefix = build(lla, P, B, H, dk, dv, dtype, steps, Lmax, seed=P)
    kept = prefix.clone()
    states = torch.full((B, H, Lmax, dk, dv), float("nan"), device="cuda")
    decay = torch.full((B, H), float("nan"), device="cuda")
    for i in range(steps):
        t = torch.full((B,), P + i, dtype=torch.int64, device="cuda")
        args, _ = step_args(d, i, t)
        out = lla.decode_step_shared(*args[:4], args[4], prefix, P, decay, states, t)
        got = out.double().cpu().numpy()
        for b in range(B):
            k = np.concatenate([d["pk"][0][0], d["k"][0][b, :i + 1].transpose(1, 0, 2)], 1)
            v = np.concatenate([d["pv"][0][0], d["v"][0][b, :i + 1].transpose(1, 0, 2)], 1)
            a = np.concatenate([d["pa"][0][0], d["a"][0][b, :i + 1].T], 1)
            q, lam = d["q"][0][b, i], d["lam"][0][b, i]
            ref, size = row(q, k, v, a, lam, P + i), row(q, k, v, a, lam, P + i, absolute=True)
            # fp32 sums of P + i + dk terms and a decay of a sum of as many logs, whose rounding of 2^-24 of up to
            # sum |log a| enters every term; prefill_state itself keeps 16 bits of bf16 values' products
            logs = np.abs(a).sum(1)[:, None]
            tol = ((P + i + dk + 16) * 2 * L.U32 + (i + 2) * L.U32 * logs) * size
            if dtype == "bf16":
                tol = tol + L.UBF * np.abs(ref) + 2.0 ** -16 * size
            assert (np.abs(got[b] - ref) <= tol).all(), (i, b, np.max(np.abs(got[b] - ref) / tol))
    assert torch.equal(prefix.nan_to_num(9.0), kept.nan_to_num(9.0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equals_decode_step_on_whole_states(lla, dtype):
    """Sequences at different positions, from the prefix's end to far behind it; a whole-state batch beside it."""
    P, B, H, dk, dv, Lmax = 1000, 6, 2, 128, 64, 14
    n = [0, 1, 23, 24, 25, 400]
    r = np.random.default_rng(5)
    d, prefix = build(lla, P, B, H, dk, dv, dtype, 1, Lmax, seed=7)
    whole = torch.zeros(B, H, Lmax, dk, dv, device="cuda")
    whole[:, :, :prefix.shape[1]] = prefix.nan_to_num(0.0)
    states = torch.full((B, H, Lmax, dk, dv), float("nan"), device="cuda")
    decay = torch.full((B, H), float("nan"), device="cuda")
    for i in range(max(n) + 1):
        live = [b for b in range(B) if n[b] >= i]
        x = torch.tensor(live, device="cuda")
        tok = [L.make(r, (len(live), H, w), dtype, w ** -0.5)[1].cuda() for w in (dk, dk, dv)]
        a = torch.from_numpy(-softplus(r.standard_normal((len(live), H)) - 2).astype(np.float32)).cuda()
        lam = torch.from_numpy(softplus(r.standard_normal((len(live), H, Lmax))).astype(np.float32)).cuda()
        t = torch.full((len(live),), P + i, dtype=torch.int64, device="cuda")
        w, s, D = whole[x], states[x], decay[x]
        ref = lla.decode_step(*tok, a, lam, w, t)
        got = lla.decode_step_shared(*tok, a, lam, prefix, P, D, s, t)
        whole[x], states[x], decay[x] = w, s, D
        # both are fp32 sums of the same terms in other orders, rounded once: one step of bf16 apart at most; fp32:
        # some 1400 roundings of 2^-24, on values of at most the sum of sizes, about 30 times the largest
        scale = ref.float().abs().max()
        tol = 2 * L.UBF if dtype == "bf16" else 1400 * 30 * L.U32
        assert float((got.float() - ref.float()).abs().max() / scale) <= tol


def test_positions_outside_are_skipped():
    from log_linear_attention_gb300 import binding as lla
    P, B, H, dk, dv, Lmax = 10, 4, 2, 32, 16, 6
    d, prefix = build(lla, P, B, H, dk, dv, "f32", 1, Lmax, seed=1)
    states = torch.randn(B, H, Lmax, dk, dv, device="cuda")
    decay = torch.zeros(B, H, device="cuda")
    kept = states.clone()
    out = torch.full((B, H, dv), 5.0, device="cuda")
    t = torch.tensor([9, 32, -1, 10], dtype=torch.int64, device="cuda")
    args, _ = step_args(d, 0, t)
    lla.decode_step_shared(*args[:4], args[4], prefix, P, decay, states, t, out=out)
    assert lla.device_error() == lla.LLA_ERR_DEVICE
    assert torch.equal(states[:3], kept[:3]) and (out[:3] == 5.0).all() and (decay[:3] == 0).all()
    assert not torch.equal(states[3], kept[3]) and not (out[3] == 5.0).any()
    # slots that hold nothing own after t = 10 are left as they were
    assert torch.equal(states[3, :, 1:], kept[3, :, 1:])


def test_own_prompt_behind_an_aligned_prefix(lla):
    """P a multiple of 64: the states of a prompt of up to 64 own tokens come from prefill_state."""
    P, B, H, dk, dv, n = 192, 2, 2, 128, 64, 50
    Lmax = lla.num_levels(P + n) + 1
    d, prefix = build(lla, P, B, H, dk, dv, "f32", n + 1, Lmax, seed=3)
    a = torch.full((B, H, Lmax, dk, dv), float("nan"), device="cuda")
    own = [d[m][1][:, :n].transpose(1, 2).contiguous() for m in ("k", "v", "a")]
    lla.prefill_state(*own, a)
    Da = own[2].sum(-1).contiguous()
    b, Db = torch.full_like(a, float("nan")), torch.full((B, H), float("nan"), device="cuda")
    for i in range(n):
        args, t = step_args(d, i, torch.full((B,), P + i, dtype=torch.int64, device="cuda"))
        lla.decode_step_shared(*args[:4], args[4], prefix, P, Db, b, t)
    args, t = step_args(d, n, torch.full((B,), P + n, dtype=torch.int64, device="cuda"))
    x = lla.decode_step_shared(*args[:4], args[4], prefix, P, Da, a, t)
    y = lla.decode_step_shared(*args[:4], args[4], prefix, P, Db, b, t)
    assert float((x - y).abs().max() / x.abs().max()) <= 1e-4  # the hand-off's own bar for fp32


def test_graph_replay(lla):
    """A captured step, replayed with t advanced on the device, equals the eager steps; two graphs at once."""
    P, B, H, dk, dv, Lmax, steps = 100, 3, 2, 64, 64, 9, 6
    sets = []
    for seed in (1, 2):
        d, prefix = build(lla, P, B, H, dk, dv, "bf16", steps, Lmax, seed=seed)
        sets.append(dict(d=d, prefix=prefix, states=torch.zeros(B, H, Lmax, dk, dv, device="cuda"),
                         decay=torch.zeros(B, H, device="cuda"), t=torch.full((B,), P, dtype=torch.int64, device="cuda"),
                         args=[d[n][1][:, 0].clone() for n in ("q", "k", "v", "a", "lam")]))

    def one(s):
        o = lla.decode_step_shared(*s["args"], s["prefix"], P, s["decay"], s["states"], s["t"])
        s["t"] += 1
        return o

    def reset(s):
        s["t"].fill_(P)
        s["states"].zero_()
        s["decay"].zero_()

    def load(s, i):
        for x, n in zip(s["args"], ("q", "k", "v", "a", "lam")):
            x.copy_(s["d"][n][1][:, i])

    want = []
    for s in sets:
        rows = []
        for i in range(steps):
            load(s, i)
            rows.append(one(s).clone())
        want.append(rows)
        reset(s)
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(one(s))
        graphs.append(g)
        reset(s)
    streams = [torch.cuda.Stream() for _ in sets]
    for i in range(steps):
        for s in sets:
            load(s, i)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w[i])


def test_prefix_s_parts_are_those_of_the_call(lla):
    """Calls over two prefixes in turn, whose parts lie in the same workspace one after the other, while another stream
    keeps the memory busy: the kernel that reads the parts starts beside the one that writes them. At t = P an output is
    lam_0 (q . k) v + exp(log_a) sum_j lam_j S_j^T q, in fp32 sums of dk (slots + 1) terms, and expf within 2^-22."""
    P, B, H, dk, dv = 30011, 70, 8, 128, 64
    Lmax = lla.num_levels(P) + 1
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    prefixes = [rand(H, Lmax, dk, dv) for _ in range(2)]
    q, k, v = rand(B, H, dk), rand(B, H, dk) * dk ** -0.5, rand(B, H, dv)
    log_a, lam = -torch.rand(B, H, generator=g, device="cuda"), torch.rand(B, H, Lmax, generator=g, device="cuda")
    t = torch.full((B,), P, dtype=torch.int64, device="cuda")
    held = [0] + [x for x in range(1, Lmax) if (P - 1) >> (x - 1) & 1]
    w = torch.stack([lam[:, :, level(P, (P - 1) >> x << x)] for x in held], 2).double() * log_a.double().exp()[..., None]

    def sums(prefix, q, k, v):
        return (lam[:, :, 0, None].double() * (q * k).sum(-1, keepdim=True) * v
                + torch.einsum("bhj,hjdv,bhd->bhv", w, prefix[:, held].double(), q))

    x = [y.double() for y in (q, k, v)]
    refs = [sums(p, *x) for p in prefixes]
    sizes_ = [sums(p.abs(), *(y.abs() for y in x)) for p in prefixes]
    states, decay = torch.empty(B, H, Lmax, dk, dv, device="cuda"), torch.empty(B, H, device="cuda")
    a, b = (torch.empty(1 << 28, device="cuda") for _ in range(2))  # 1 GiB each
    busy = torch.cuda.Stream()
    busy.wait_stream(torch.cuda.current_stream())
    first = None
    for _ in range(6):
        with torch.cuda.stream(busy):
            b.copy_(a)
        got = [lla.decode_step_shared(q, k, v, log_a, lam, p, P, decay, states, t) for p in prefixes]
        for o, r, s in zip(got, refs, sizes_):
            assert ((o.double() - r).abs() <= ((dk + len(held) + 16) * 2 * L.U32 + 2.0 ** -22) * s).all()
        first = first or got
        assert all(torch.equal(o, f) for o, f in zip(got, first))
    busy.synchronize()


def test_a_part_of_the_batch(lla):
    """Sequences 1.. of a batch whose heads are odd in number: decay, decays of the step, lambda and positions begin
    between the library's 16 bytes, and the decays are updated in place all the same."""
    P, B, H, dk, dv, Lmax = 100, 4, 3, 64, 64, 9
    d, prefix = build(lla, P, B, H, dk, dv, "f32", 3, Lmax, seed=2)
    whole, part = [(torch.zeros(B, H, Lmax, dk, dv, device="cuda"), torch.full((B, H), 5.0, device="cuda")) for _ in "ab"]
    for i in range(3):
        t = torch.full((B,), P + i, dtype=torch.int64, device="cuda")
        args, _ = step_args(d, i, t)
        want = lla.decode_step_shared(*args, prefix, P, whole[1], whole[0], t)
        q, k, v, a, lam = args
        got = lla.decode_step_shared(q[1:].clone(), k[1:].clone(), v[1:].clone(), a[1:], lam[1:], prefix, P, part[1][1:],
                                     part[0][1:], t[1:])
        assert torch.equal(got, want[1:]) and torch.equal(part[1][1:], whole[1][1:])
        assert torch.equal(part[0][1:], whole[0][1:]) and (part[1][0] == 5.0).all()
    with pytest.raises(lla.LLAError):  # decays over the step's own
        lla.decode_step_shared(q[1:].clone(), k[1:].clone(), v[1:].clone(), a[1:], lam[1:], prefix, P, a[1:],
                               part[0][1:], t[1:])
