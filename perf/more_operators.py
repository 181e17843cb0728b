"""Cases of the gated linear recurrence, and of trees of drafted tokens over recurrent states with the commit of the
accepted path: their inputs, their plain forms in torch and their values in 64 bits.

    gated           gated_forward, gated_forward_varlen      h_t = exp(log_a_t) h_{t-1} + x_t, every channel by itself
    gated_backward  gated_backward, gated_backward_varlen    gradients of x, log_a and the entering state
    tree            decode_tree, linear_decode_tree, gated_decode_tree        outputs of drafted tokens
    commit          decode_commit, linear_decode_commit, gated_decode_commit  accepted tokens into the states

A drafted tree has nodes 0..N-1, parent(i) < i or -1 (a child of the last token in the states) or -2 (no node). With
position p_i = t + depth(i), D(i, j) the sum of log_a over the nodes after j on the way to i, l the Fenwick level:

    o_i = sum_{j = i or above i} lambda_i^(l(p_i,p_j)) exp(D(i,j)) (q_i . k_j) v_j
        + exp(D_i) sum_m lambda_i^(l(p_i, block m)) (S^(m))^T q_i          (log-linear; S^(m) the states of t - 1)
    linear: one state, lambda = 1, a constant log_a per head;   gated: h_i = exp(log_a_i) h_parent(i) + x_i

A commit leaves the states as if the accepted tokens had been decoded one by one.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def _gated(name, op, B, T, D, dtype, gate, B0):
    return {"name": name, "op": op, "packed": False, "B": B, "T": T, "D": D, "dtype": dtype, "gate": gate, "B0": B0}


def _packed(name, op, n, lo, hi, D, dtype, gate, B0, tail, lens):
    return {"name": name, "op": op, "packed": True, "B": n, "lo": lo, "hi": hi, "D": D, "dtype": dtype, "gate": gate,
            "B0": B0, "tail": tail, "lens": lens}


def _tree(name, kind, B, H, N, least, dk, dv, dtype, t_max, one, nodes):
    """least: fewest nodes of a sequence; one: the same tree for the whole batch; gated: dv channels a head."""
    return {"name": name, "op": "tree", "kind": kind, "B": B, "H": H, "N": N, "least": least, "dk": dk, "dv": dv,
            "dtype": dtype, "t_max": t_max, "one": one, "nodes": nodes}


def _commit(name, kind, B, H, N, most, dk, dv, dtype, t_max, nodes):
    """most: longest accepted path."""
    return {"name": name, "op": "commit", "kind": kind, "B": B, "H": H, "N": N, "most": most, "dk": dk, "dv": dv,
            "dtype": dtype, "t_max": t_max, "nodes": nodes}


def listed():
    return [
        # prompts of the headline prefill shape (16 heads of 64 channels) that go on from one shared state
        _gated("gated headline", "gated", 4, 8192, 1024, "bf16", "f32", 1),
        # one long document, gates in 16 bits as a layer under autocast leaves them
        _gated("gated long", "gated", 1, 65536, 1024, "bf16", "bf16", 0),
        # chat turns of 0 to 200 tokens, each on its own state, fp32, an odd number of channels, rows behind the last
        _packed("gated turns", "gated", 24, 0, 200, 515, "f32", "f32", 24, 77, 5),
        # training: the headline shape
        _gated("gated backward headline", "gated_backward", 4, 8192, 1024, "bf16", "f32", 0),
        # training on packed documents in fp32 from one learned state
        _packed("gated backward packed", "gated_backward", 9, 1, 1301, 240, "f32", "f32", 1, 0, 3),
        # serving: the repository's decode batch checks up to 32 drafted tokens each, every sequence its own tree
        _tree("tree batch", "log", 64, 16, 32, 20, 128, 64, "bf16", 65536, False, 1),
        # serving: one sequence and a short draft, latency counts
        _tree("tree one", "log", 1, 8, 7, 7, 64, 64, "f32", 5000, True, 2),
        # serving: linear layers, one wide tree for the whole batch
        _tree("tree linear", "linear", 64, 16, 64, 64, 128, 64, "bf16", 1, True, 3),
        # serving: gated layers of the same batch
        _tree("tree gated", "gated", 64, 16, 32, 20, 1, 64, "bf16", 1, False, 1),
        # serving: the accepted tokens of the decode batch, up to six each
        _commit("commit batch", "log", 64, 16, 32, 6, 128, 64, "bf16", 65536, 1),
        # serving: one sequence's, latency counts
        _commit("commit linear one", "linear", 1, 8, 7, 4, 64, 64, "f32", 1, 9),
        # serving: the gated layers of the decode batch
        _commit("commit gated", "gated", 64, 16, 32, 6, 1, 64, "bf16", 1, 3),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _head_dim(rng):
    return rng.choice([64, 128, 64, 128, 16, 32, 48, 80, 96, 112, rng.randint(9, 128)])


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_backward", "gated_backward", "tree", "tree", "commit"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("gated", "gated_backward"):
        gate = rng.choice(["f32", dtype])
        D = rng.choice([_log_int(rng, 1, 4096), 8 * _log_int(rng, 1, 512)])
        B = _log_int(rng, 1, 32)
        room = max(1, (1 << 25) // (D * B))
        if rng.random() < 0.6:
            T = _log_int(rng, 1, min(65536, room))
            c = _gated("", op, B, T, D, dtype, gate, rng.choice([0, 1, B]))
        else:
            hi = _log_int(rng, 1, min(8192, room))
            c = _packed("", op, B, rng.choice([0, 1, hi // 2, hi]), hi, D, dtype, gate, rng.choice([0, 1, B]),
                        rng.choice([0, 0, rng.randint(1, 300)]), rng.randint(0, 1 << 30))
    else:
        kind = rng.choice(["log", "log", "linear", "gated"])
        B, H = _log_int(rng, 1, 64), _log_int(rng, 1, 16)
        dk, dv = (1, _head_dim(rng)) if kind == "gated" else (_head_dim(rng), _head_dim(rng))
        if kind == "log":
            dv = rng.choice([16, 32, 64, 64])
        N = _log_int(rng, 1, 64)
        t_max = _log_int(rng, 1, 65536) if kind == "log" else 1
        if op == "tree":
            c = _tree("", kind, B, H, N, rng.randint(1, N), dk, dv, dtype, t_max, rng.random() < 0.3,
                      rng.randint(0, 1 << 30))
        else:
            c = _commit("", kind, B, H, N, rng.randint(1, N), dk, dv, dtype, t_max, rng.randint(0, 1 << 30))
    del c["name"]
    return c


def _lengths(c):
    if not c["packed"]:
        return [c["T"]] * c["B"]
    r = random.Random(c["lens"])
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]


def _parents(c):
    """Parents of every tree: a draft that mostly goes on from the last token, with side branches."""
    r = random.Random(c["nodes"])
    trees = []
    for _ in range(1 if c["one"] else c["B"]):
        live = c["N"] if c["one"] else r.randint(c["least"], c["N"])
        trees.append([-2 if i >= live else -1 if i == 0 else i - 1 if r.random() < 0.3 else r.randint(-1, i - 1)
                      for i in range(c["N"])])
    return trees


def _paths(c):
    """Accepted nodes of every sequence, first to last; none for some."""
    r = random.Random(c["nodes"])
    most = min(c["most"], c["N"])
    return [sorted(r.sample(range(c["N"]), r.randint(0, most))) for _ in range(c["B"])]


def _positions(c):
    r = random.Random(c["nodes"] + 1)
    return [r.randrange(c["t_max"]) for _ in range(c["B"])]


def _slots(c):
    return (c["t_max"] + c["N"] - 1).bit_length() + 1


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    def gates(*shape):
        # channels from slow to fast (half-lives of one to a thousand tokens), each token a little off its channel's rate
        rate = torch.exp(torch.rand(shape[-1], generator=g, device="cuda") * -6.9)
        return -rate * 2.0 * torch.sigmoid(normal(*shape))

    s = {"op": c["op"], "kind": c.get("kind")}
    if c["op"] in ("gated", "gated_backward"):
        lens, D, B0 = _lengths(c), c["D"], c["B0"]
        rows = max(1, sum(lens) + c.get("tail", 0))
        shape = (rows, D) if c["packed"] else (c["B"], c["T"], D)
        log_a = gates(*shape).to(DTYPES[c["gate"]])
        # inputs scaled so that the states stay of the size of one
        x = (normal(*shape) * torch.sqrt(-torch.expm1(2.0 * log_a.float()))).to(dt)
        s.update(x=x, log_a=log_a, state0=normal(B0, D) if B0 else None, cu=None, n=c["B"])
        if c["packed"]:
            cu = [0]
            for n in lens:
                cu.append(cu[-1] + n)
            s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        if c["op"] == "gated":
            s["state_out"] = torch.empty(c["B"], D, device="cuda")
            s["out"] = torch.zeros_like(x) if c["packed"] else None
        else:
            s["out"] = _plain_gated({**s, "state_out": None, "out": torch.zeros_like(x)})["out"]
            s.update(dout=normal(*shape).to(dt), dstate_out=normal(c["B"], D))
        return s
    B, H, N, dk, dv = (c[n] for n in ("B", "H", "N", "dk", "dv"))
    if c["kind"] == "gated":
        s.update(x=normal(B, N, H * dv).to(dt), log_a=gates(B, N, H * dv), state=normal(B, H * dv))
    else:
        s.update(q=normal(B, H, N, dk, scale=dk ** -0.5).to(dt), k=normal(B, H, N, dk, scale=dk ** -0.5).to(dt),
                 v=normal(B, H, N, dv).to(dt))
        if c["kind"] == "log":
            L = _slots(c)
            sp = torch.nn.functional.softplus
            s.update(log_a=-sp(normal(B, H, N) - 2.0), lam=sp(normal(B, H, N, L)),
                     states=normal(B, H, L, dk, dv, scale=dk ** -0.5),
                     t=torch.tensor(_positions(c), dtype=torch.int64, device="cuda"))
        else:
            slope = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
            s.update(log_a=-slope * (0.9 + 0.2 * torch.rand(H, generator=g, device="cuda")),
                     state=normal(B, H, dk, dv, scale=dk ** -0.5))
    if c["op"] == "tree":
        parent = torch.tensor(_parents(c), dtype=torch.int32, device="cuda")
        s["parent"] = parent[0].contiguous() if c["one"] else parent
        s["out"] = torch.zeros_like(s["x"] if c["kind"] == "gated" else s["v"])
    else:
        paths = _paths(c)
        wide = min(c["most"], N)
        s.update(path=torch.tensor([p + [-1] * (wide - len(p)) for p in paths], dtype=torch.int32, device="cuda"),
                 count=torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda"))
    return s


# ---------------------------------------------------------------- the calls

def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "gated":
        return _plain_gated(s)
    if s["op"] == "gated_backward":
        return _plain_gated_backward(s)
    return _plain_tree(s) if s["op"] == "tree" else _plain_commit(s)


def _run_own(s):
    from log_linear_attention_gb300 import binding as lla
    op, kind = s["op"], s["kind"]
    if op == "gated":
        if s["cu"] is None:
            out = lla.gated_forward(s["x"], s["log_a"], state0=s["state0"], state_out=s["state_out"])
        else:
            out = lla.gated_forward_varlen(s["x"], s["log_a"], s["cu"], state0=s["state0"], state_out=s["state_out"],
                                           out=s["out"])
        return {"out": out, "state_out": s["state_out"]}
    if op == "gated_backward":
        if s["cu"] is None:
            dx, da, ds = lla.gated_backward(s["log_a"], s["out"], s["dout"], state0=s["state0"],
                                            dstate_out=s["dstate_out"])
        else:
            dx, da, ds = lla.gated_backward_varlen(s["log_a"], s["out"], s["dout"], s["cu"], state0=s["state0"],
                                                   dstate_out=s["dstate_out"])
        return {"dx": dx, "dlog_a": da, "dstate0": ds}
    if op == "tree":
        if kind == "gated":
            return {"out": lla.gated_decode_tree(s["x"], s["log_a"], s["state"], s["parent"], out=s["out"])}
        if kind == "linear":
            return {"out": lla.linear_decode_tree(s["q"], s["k"], s["v"], s["log_a"], s["state"], s["parent"],
                                                  out=s["out"])}
        return {"out": lla.decode_tree(s["q"], s["k"], s["v"], s["log_a"], s["lam"], s["states"], s["t"], s["parent"],
                                       out=s["out"])}
    if kind == "gated":
        return {"state": lla.gated_decode_commit(s["x"], s["log_a"], s["state"], s["count"], s["path"])}
    if kind == "linear":
        return {"state": lla.linear_decode_commit(s["k"], s["v"], s["log_a"], s["state"], s["count"], s["path"])}
    return {"states": lla.decode_commit(s["k"], s["v"], s["log_a"], s["states"], s["t"], s["count"], s["path"])}


# ---------------------------------------------------------------- plain forms

def _scan(a, x):
    """h_t = a_t h_{t-1} + x_t along the rows (h before the first: 0), in doubling steps: [rows, D] fp32."""
    step = 1
    while step < x.shape[0]:
        x = torch.cat([x[:step], x[step:] + a[step:] * x[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return x


def _bounds(s):
    """(first row, row after the last) of every sequence among the rows of all."""
    if s["cu"] is None:
        T = s["log_a"].shape[1]
        start = T * torch.arange(s["n"], device=s["log_a"].device)
        return start, start + T
    cu = s["cu"].long()
    return cu[:-1], cu[1:]


def _per_sequence(state, s):
    if state is None:
        return torch.zeros(s["n"], s["log_a"].shape[-1], device=s["log_a"].device)
    return state.expand(s["n"], -1)


def _plain_gated(s):
    D = s["x"].shape[-1]
    x, a = s["x"].float().reshape(-1, D), s["log_a"].float().exp().reshape(-1, D)
    lo, hi = _bounds(s)
    some = hi > lo
    s0 = _per_sequence(s["state0"], s)
    x = x.index_add(0, lo[some], a[lo[some]] * s0[some])
    h = _scan(a.index_fill(0, lo[some], 0.0), x)
    state = s0.clone()
    state[some] = h[hi[some] - 1]
    out = h.to(s["x"].dtype).reshape(s["x"].shape)
    if s["cu"] is not None:
        s["out"][:s["cu"][-1]] = out[:s["cu"][-1]]
        out = s["out"]
    return {"out": out, "state_out": state}


def _plain_gated_backward(s):
    shape, D = s["log_a"].shape, s["log_a"].shape[-1]
    a = s["log_a"].float().exp().reshape(-1, D)
    h, do = s["out"].float().reshape(-1, D), s["dout"].float().reshape(-1, D)
    lo, hi = _bounds(s)
    some = hi > lo
    first, last = lo[some], hi[some] - 1
    s0, ds = _per_sequence(s["state0"], s), s["dstate_out"]
    rows = torch.arange(h.shape[0], device=h.device)[:, None]
    inside = (rows < hi.max()).float()
    a, do = a * inside, do * inside
    # F_t = a_t (dout_t + F_{t+1}); a sequence's last row takes dstate_out in place of F_{t+1}
    end = torch.zeros_like(a).index_add(0, last, ds[some])
    c = a.index_fill(0, last, 0.0)
    F = _scan(c.flip(0), (a * (do + end)).flip(0)).flip(0)
    after = torch.cat([F[1:], torch.zeros_like(F[:1])]).index_fill(0, last, 0.0) + end
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]]).index_copy(0, first, s0[some])
    ds0 = None
    if s["state0"] is not None:
        ds0 = ds.clone()
        ds0[some] = F[first]
        if s["state0"].shape[0] == 1:
            ds0 = ds0.sum(0, keepdim=True)
    return {"dx": ((do + after) * inside).to(s["dout"].dtype).reshape(shape),
            "dlog_a": (F * before * inside).to(s["log_a"].dtype).reshape(shape), "dstate0": ds0}


def _bit_length(x):
    return ((x[..., None] >> torch.arange(62, device=x.device)) > 0).sum(-1)


def _above(parent, B):
    """[B, N, N]: node j is node i or above it; no row for what is no node."""
    parent = parent.long().expand(B, -1)
    N = parent.shape[1]
    got = torch.zeros(B, N, N, dtype=torch.bool, device=parent.device)
    b = torch.arange(B, device=parent.device)
    for i in range(N):
        p = parent[:, i]
        got[:, i] = got[b, p.clamp(min=0)] & (p >= 0)[:, None]
        got[:, i, i] = p >= -1
    return got


def _plain_tree(s):
    kind, out = s["kind"], s["out"]
    B = out.shape[0]
    up = _above(s["parent"], B)
    live = up.diagonal(dim1=1, dim2=2)
    if kind == "gated":
        # log decays along a path in 64 bits, their differences are not
        x, la = s["x"].float(), s["log_a"].double()
        cum = up.double() @ la
        h = (cum.exp() * s["state"].double()[:, None]).float()
        for j in range(x.shape[1]):
            w = torch.where(up[:, :, j, None], cum - cum[:, j:j + 1], -torch.inf).exp().float()
            h = h + w * x[:, j:j + 1]
        out.copy_(torch.where(live[..., None], h.to(out.dtype), out))
        return {"out": out}
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    depth = up.sum(-1) - 1
    if kind == "linear":
        la = s["log_a"].double()[None, :, None]
        cum = la * (depth[:, None] + 1)
    else:
        cum = (up.double()[:, None] @ s["log_a"].double()[..., None])[..., 0]
    w = torch.where(up[:, None], cum[..., :, None] - cum[..., None, :], -torch.inf).exp().float()
    if kind == "linear":
        far = cum.exp().float()[..., None] * (q @ s["state"])
    else:
        lam, st, t = s["lam"], s["states"], s["t"]
        pos = t[:, None] + depth
        level = torch.where(up, _bit_length(pos[:, :, None] ^ pos[:, None, :]), 0)
        w = w * lam.gather(3, level[:, None].expand(-1, lam.shape[1], -1, -1))
        # the states of t - 1: slot 0 the token t - 1, slot m its bucket of 2^(m-1) tokens from ((t-1) >> m) << m
        m = torch.arange(st.shape[2], device=t.device)
        held = (t[:, None] > 0) & ((m == 0) | (((t[:, None] - 1) >> (m - 1).clamp(min=0)) & 1 == 1))
        start = ((t[:, None] - 1) >> m) << m
        level = torch.where(held[:, None] & live[..., None], _bit_length(pos[..., None] ^ start[:, None]), 0)
        u = lam.gather(3, level[:, None].expand(-1, lam.shape[1], -1, -1)) * held[:, None, None].float()
        u = u * cum.exp().float()[..., None]
        B, H, N, dk = q.shape
        held_states = torch.where(held[:, None, :, None, None], st, 0.0)
        far = (u[..., None] * q[..., None, :]).reshape(B, H, N, -1) @ held_states.reshape(B, H, -1, v.shape[-1])
    o = ((q @ k.transpose(-1, -2)) * w) @ v + far
    out.copy_(torch.where(live[:, None, :, None], o.to(out.dtype), out))
    return {"out": out}


def _plain_commit(s):
    kind, path, count = s["kind"], s["path"].long(), s["count"].long()
    B, M = path.shape
    r = torch.arange(M, device=path.device)
    real = r < count[:, None]
    node = torch.where(real, path, 0)
    b = torch.arange(B, device=path.device)[:, None]
    if kind == "gated":
        st = s["state"]
        x = s["x"].float()[b, node]
        a = torch.where(real[..., None], s["log_a"].float()[b, node].exp(), 1.0)
        for i in range(M):
            st.copy_(a[:, i] * st + torch.where(real[:, i, None], x[:, i], 0.0))
        return {"state": st}
    take = lambda y: y.float().transpose(1, 2)[b, node].transpose(1, 2)  # noqa: E731  [B, H, M, .]
    k, v = take(s["k"]), take(s["v"])
    if kind == "linear":
        la = s["log_a"].double()[None, :, None] * real[:, None]
    else:
        la = take(s["log_a"]).double() * real[:, None]
    tail = la.flip(2).cumsum(2).flip(2)
    whole = tail[:, :, 0].exp().float()
    w = torch.where(real[:, None], (tail - la).exp(), 0.0).float()
    if kind == "linear":
        st = s["state"]
        st.copy_(whole[..., None, None] * st + (k * w[..., None]).transpose(-1, -2) @ v)
        return {"state": st}
    st, t = s["states"], s["t"]
    L = st.shape[2]
    m = torch.arange(L, device=t.device)
    low = (m - 1).clamp(min=0)
    size = torch.where(m > 0, 1 << low, 1)

    def walk(pos):
        held = (pos[:, None] >= 0) & ((m == 0) | ((pos[:, None] >> low) & 1 == 1))
        return held, (pos[:, None] >> m) << m

    end = t + count - 1
    (old, old_at), (new, new_at) = walk(t - 1), walk(end)
    new = new & (count > 0)[:, None]
    inside = ((old_at[:, None, :] >= new_at[:, :, None])
              & (old_at[:, None, :] + size <= new_at[:, :, None] + size[:, None])
              & old[:, None, :] & new[:, :, None]).float()
    grown = torch.einsum("blm,bhmkv->bhlkv", inside, torch.where(old[:, None, :, None, None], st, 0.0))
    pos = (t[:, None] + r)[:, None]
    mine = (pos >= new_at[..., None]) & (pos < (new_at + size)[..., None]) & new[..., None] & real[:, None]
    kw = (k * w[..., None])[:, :, None] * mine[:, None, ..., None].float()
    grown = grown * whole[..., None, None, None] + kw.transpose(-1, -2) @ v[:, :, None]
    st.copy_(torch.where(new[:, None, :, None, None], grown, st))
    return {"states": st}


# ---------------------------------------------------------------- work

def _held(pos):
    return 1 + bin(pos).count("1") if pos >= 0 else 0


def work(case):
    """Bytes: inputs once, outputs once, states that are held. Flops: two a row and channel for the recurrence, four for
    its gradients; for trees the read of every held state by every node and the pairs of nodes on one path; for commits
    the new tokens' outer products and the sums of states."""
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] in ("gated", "gated_backward"):
        g = 2 if c["gate"] == "bf16" else 4
        n, D = sum(_lengths(c)), c["D"]
        if c["op"] == "gated":
            return {"bytes": n * D * (2 * e + g) + 4 * D * (c["B0"] + c["B"]), "flops": 2 * n * D}
        return {"bytes": n * D * (3 * e + 2 * g) + 4 * D * (2 * c["B0"] + c["B"]), "flops": 4 * n * D}
    B, H, dk, dv, kind = (c[n] for n in ("B", "H", "dk", "dv", "kind"))
    if c["op"] == "tree":
        trees = _parents(c) * (B if c["one"] else 1)
        nodes = pairs = states = reads = 0
        for tree, t in zip(trees, _positions(c)):
            depth = []
            for p in tree:
                depth.append(0 if p < 0 else depth[p] + 1)
            live = sum(p >= -1 for p in tree)
            held = _held(t - 1) if kind == "log" else 1
            nodes += live
            states += held
            reads += held * live
            pairs += sum(d + 1 for d, p in zip(depth, tree) if p >= -1)
        if kind == "gated":
            return {"bytes": H * dv * (nodes * (2 * e + 4) + 4 * B), "flops": 2 * nodes * H * dv}
        small = 4 * (1 + _slots(c)) if kind == "log" else 0
        return {"bytes": H * (nodes * (e * (2 * dk + 2 * dv) + small) + 4 * dk * dv * states),
                "flops": 2 * H * (dk * dv * reads + (dk + dv) * pairs)}
    n = read = wrote = 0
    for path, t in zip(_paths(c), _positions(c)):
        n += len(path)
        if path:
            read += _held(t - 1) if kind == "log" else 1
            wrote += _held(t + len(path) - 1) if kind == "log" else 1
    if kind == "gated":
        return {"bytes": H * dv * (n * (e + 4) + 4 * (read + wrote)), "flops": 2 * n * H * dv}
    return {"bytes": H * (n * e * (dk + dv) + 4 * dk * dv * (read + wrote)), "flops": H * dk * dv * (2 * n + read)}


# ---------------------------------------------------------------- 64 bits

def _walk(pos):
    """{slot: (first, last + 1)} of the Fenwick partition of 0..pos."""
    if pos < 0:
        return {}
    got, end = {0: (pos, pos + 1)}, pos
    while end > 0:
        low = end & -end
        got[low.bit_length()] = (end - low, end)
        end -= low
    return got


def _slot_of(walk, s):
    return next(m for m, (lo, hi) in walk.items() if lo <= s < hi)


def exact(case, seed):
    s = prepare(case, seed)
    d = {n: x.double() for n, x in s.items() if torch.is_tensor(x) and x.is_floating_point()}
    if case["op"] == "gated":
        return _exact_gated(case, s, d)
    if case["op"] == "gated_backward":
        return _exact_gated_backward(case, s, d)
    return _exact_tree(case, s, d) if case["op"] == "tree" else _exact_commit(case, s, d)


def _pieces(case):
    """Index of every sequence's rows among those of its tensors."""
    if not case["packed"]:
        return [(b, slice(None)) for b in range(case["B"])]
    got, at = [], 0
    for n in _lengths(case):
        got.append((slice(at, at + n),))
        at += n
    return got


def _entering(case, d, b):
    return d["state0"][b if case["B0"] > 1 else 0] if case["B0"] else d["log_a"].new_zeros(case["D"])


def _exact_gated(case, s, d):
    out, ends = torch.zeros_like(d["x"]), []
    if sum(_lengths(case)) // (1 if case["packed"] else case["B"]) > 200000:
        return None
    if not case["packed"]:
        h = torch.stack([_entering(case, d, b) for b in range(case["B"])])
        for t in range(case["T"]):
            h = d["log_a"][:, t].exp() * h + d["x"][:, t]
            out[:, t] = h
        return {"out": out, "state_out": h}
    for b, at in enumerate(_pieces(case)):
        h = _entering(case, d, b)
        x, a, o = d["x"][at], d["log_a"][at].exp(), out[at]
        for t in range(x.shape[0]):
            h = a[t] * h + x[t]
            o[t] = h
        ends.append(h)
    return {"out": out, "state_out": torch.stack(ends)}


def _exact_gated_backward(case, s, d):
    if case["packed"] and sum(_lengths(case)) > 100000:
        return None
    dx, da = torch.zeros_like(d["dout"]), torch.zeros_like(d["log_a"])
    enter = torch.stack([_entering(case, d, b) for b in range(case["B"])])
    # dense: all sequences at once, [T, B, D]; packed: one after another, [T, 1, D]
    if case["packed"]:
        jobs = [([b], at) for b, at in enumerate(_pieces(case))]
    else:
        jobs = [(list(range(case["B"])), slice(None))]
    grad = torch.zeros_like(enter)
    for who, at in jobs:
        turn = (lambda x: x[at][:, None]) if case["packed"] else (lambda x: x.transpose(0, 1))
        a, h, do, gx, ga = turn(d["log_a"]).exp(), turn(d["out"]), turn(d["dout"]), turn(dx), turn(da)
        g = d["dstate_out"][who]
        for t in reversed(range(a.shape[0])):
            g = g + do[t]
            gx[t] = g
            ga[t] = g * a[t] * (h[t - 1] if t else enter[who])
            g = g * a[t]
        grad[who] = g
    if case["B0"] == 1:
        grad = grad.sum(0, keepdim=True)
    return {"dx": dx, "dlog_a": da, "dstate0": grad if case["B0"] else None}


def _exact_tree(case, s, d):
    out = torch.zeros_like(d["out"])
    trees = _parents(case) * (case["B"] if case["one"] else 1)
    for b, (tree, t) in enumerate(zip(trees, _positions(case))):
        way = []  # nodes from the root to each node
        for i, p in enumerate(tree):
            way.append(None if p == -2 else (way[p] if p >= 0 else []) + [i])
        if case["kind"] == "gated":
            h = {-1: d["state"][b]}
            for i, p in enumerate(tree):
                if p > -2:
                    out[b, i] = h[i] = d["log_a"][b, i].exp() * h[p] + d["x"][b, i]
            continue
        before = _walk(t - 1) if case["kind"] == "log" else {0: None}
        for i, nodes in enumerate(way):
            if nodes is None:
                continue
            q = d["q"][b, :, i]
            after = _walk(t + len(nodes) - 1)
            decay = torch.zeros_like(q[:, 0])  # sum of log_a after the node, on the way to i
            for step in reversed(range(len(nodes))):
                j = nodes[step]
                w = decay.exp() * (q * d["k"][b, :, j]).sum(-1)
                if case["kind"] == "log":
                    w = w * d["lam"][b, :, i, _slot_of(after, t + step)]
                out[b, :, i] += w[:, None] * d["v"][b, :, j]
                decay = decay + (d["log_a"][b, :, j] if case["kind"] == "log" else d["log_a"])
            for m, block in before.items():
                state = d["states"][b, :, m] if case["kind"] == "log" else d["state"][b]
                w = decay.exp()
                if case["kind"] == "log":
                    w = w * d["lam"][b, :, i, _slot_of(after, block[0])]
                out[b, :, i] += w[:, None] * (q[:, :, None] * state).sum(1)
    return {"out": out}


def _exact_commit(case, s, d):
    """Token by token: each one a decode step without its output. Slots that the last token leaves empty stay as they
    were."""
    kind = case["kind"]
    name = "states" if kind == "log" else "state"
    st = d[name].clone()
    for b, (path, t) in enumerate(zip(_paths(case), _positions(case))):
        first = st[b].clone()
        for step, j in enumerate(path):
            if kind == "gated":
                st[b] = d["log_a"][b, j].exp() * st[b] + d["x"][b, j]
                continue
            new = d["k"][b, :, j, :, None] * d["v"][b, :, j, None, :]
            if kind == "linear":
                st[b] = d["log_a"].exp()[:, None, None] * st[b] + new
                continue
            before, after = _walk(t + step - 1), _walk(t + step)
            a = d["log_a"][b, :, j].exp()[:, None, None]
            was = st[b].clone()
            for m, (lo, hi) in after.items():
                st[b, :, m] = new if m == 0 else a * sum(was[:, n] for n, (x, y) in before.items() if lo <= x and y <= hi)
        if kind == "log" and path:
            held = _walk(t + len(path) - 1)
            for m in range(st.shape[2]):
                if m not in held:
                    st[b, :, m] = first[:, m]
    return {name: st}
