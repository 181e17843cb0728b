"""Cases of the linear-attention operators with one decay per head, and of the decode step over a
shared prefix: their inputs, their plain forms in torch and their values in 64 bits.

    linear           lla_linear_forward         prompts, [B, H, T, .], optional entering and leaving state
    linear_varlen    lla_linear_forward_varlen  packed prompts, [H, total, .] with cu_seqlens
    linear_backward  lla_linear_backward        gradients of q, k, v and the entering state
    linear_decode    lla_linear_decode_step     one token of every sequence, states updated in place
    decode_shared    lla_decode_step_shared     one log-linear decode step over a prefix kept once per head

With gamma_h = exp(log_a_h):

    S_t = gamma_h S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t                         (linear)
    o_t = sum_{s <= t} lambda_t^(l(t,s)) exp(sum_{r=s+1..t} log_a_r) (q_t . k_s) v_s   (log-linear)

The log-linear step takes the sum over s < P from the Fenwick buckets of the prefix (one set for all
sequences), and the sum over s >= P from each sequence's own buckets.
"""
import math
import random

import torch

own = False

CHUNK = 128
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def _linear(name, B, H, T, dk, dv, dtype, B0, state_out):
    return {"name": name, "op": "linear", "B": B, "H": H, "T": T, "dk": dk, "dv": dv, "dtype": dtype, "B0": B0,
            "state_out": state_out}


def _varlen(name, n, H, lo, hi, dk, dv, dtype, n0, tail, lens):
    return {"name": name, "op": "linear_varlen", "n": n, "H": H, "lo": lo, "hi": hi, "dk": dk, "dv": dv,
            "dtype": dtype, "n0": n0, "tail": tail, "lens": lens}


def _backward(name, B, H, T, dk, dv, dtype, B0):
    return {"name": name, "op": "linear_backward", "B": B, "H": H, "T": T, "dk": dk, "dv": dv, "dtype": dtype,
            "B0": B0}


def _decode(name, B, H, dk, dv, dtype):
    return {"name": name, "op": "linear_decode", "B": B, "H": H, "dk": dk, "dv": dv, "dtype": dtype}


def _shared(name, B, H, dk, dv, dtype, P, span, Lmax, at):
    return {"name": name, "op": "decode_shared", "B": B, "H": H, "dk": dk, "dv": dv, "dtype": dtype, "P": P,
            "span": span, "Lmax": Lmax, "at": at}


def listed():
    return [
        # the repository's small prefill shape, its state kept for decoding: a short prompt, latency counts
        _linear("prompt small", 2, 4, 2048, 64, 64, "bf16", 0, True),
        # the headline prefill shape: a batch of prompts that go on from one shared state
        _linear("prompt headline", 4, 16, 8192, 128, 64, "bf16", 1, True),
        # one long document (the length of the long configuration), square heads, few of them
        _linear("prompt long", 1, 16, 65536, 128, 128, "bf16", 0, True),
        # fp32 with head sizes and a length that are no multiples of anything
        _linear("prompt f32 odd", 2, 6, 1237, 100, 36, "f32", 2, True),
        # the packed benchmark mix: 32 prompts of 256 to 8192 tokens
        _varlen("packed mix", 32, 16, 256, 8192, 128, 64, "bf16", 0, 0, 1234),
        # chat turns of 0 to 200 tokens that go on from one shared state, with rows behind the last
        _varlen("packed turns", 24, 8, 0, 200, 64, 64, "bf16", 1, 77, 5),
        # training: the headline shape
        _backward("backward headline", 4, 16, 8192, 128, 64, "bf16", 0),
        # training in fp32, an odd length and head sizes, gradients of a state that the batch shares
        _backward("backward f32 odd", 3, 5, 1301, 96, 80, "f32", 1),
        # serving: the repository's decode batch
        _decode("decode batch", 64, 16, 128, 64, "bf16"),
        # serving: a single sequence, latency counts
        _decode("decode one", 1, 8, 64, 64, "bf16"),
        # serving: a long system prompt under the decode batch, up to 4096 own tokens each
        _shared("shared batch", 64, 16, 128, 64, "bf16", 30011, 4096, 18, 1),
        # serving: a few short answers under one prompt, fp32, latency counts
        _shared("shared small", 4, 4, 64, 64, "f32", 1000, 100, 14, 2),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _head_dim(rng):
    return rng.choice([64, 128, 64, 128, 16, 32, 48, 80, 96, 112, rng.randint(9, 128)])


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_varlen", "linear_backward", "linear_backward", "linear_decode",
                     "decode_shared"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    H = _log_int(rng, 1, 32)
    dk, dv = _head_dim(rng), _head_dim(rng)
    if op in ("linear", "linear_backward"):
        B = _log_int(rng, 1, 16)
        rows = {"bf16": 1 << 19, "f32": 1 << 17}[dtype] // (1 if op == "linear" else 2)
        T = _log_int(rng, 1, max(1, min(65536, rows // (B * H))))
        B0 = rng.choice([0, 1, B])
        if op == "linear":
            c = _linear("", B, H, T, dk, dv, dtype, B0, rng.random() < 0.7)
        else:
            c = _backward("", B, H, T, dk, dv, dtype, B0)
    elif op == "linear_varlen":
        n = _log_int(rng, 1, 64)
        rows = {"bf16": 1 << 19, "f32": 1 << 17}[dtype]
        hi = _log_int(rng, 1, max(1, min(8192, rows // (n * H))))
        lo = rng.choice([0, 1, hi // 2, hi])
        c = _varlen("", n, H, lo, hi, dk, dv, dtype, rng.choice([0, 1, n]), rng.choice([0, 0, rng.randint(1, 300)]),
                    rng.randint(0, 1 << 30))
    elif op == "linear_decode":
        c = _decode("", _log_int(rng, 1, 256), H, dk, dv, dtype)
    else:
        P = _log_int(rng, 1, 60000)
        span = _log_int(rng, 1, 5000)
        Lmax = max((P + span - 1).bit_length() + 1, 2)
        c = _shared("", _log_int(rng, 1, 64), H, dk, rng.choice([16, 32, 64, 64, 128]), dtype, P, span,
                    min(18, Lmax + rng.randint(0, 2)), rng.randint(0, 1 << 30))
    del c["name"]
    return c


def _lengths(c):
    r = random.Random(c["lens"])
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["n"])]


def _positions(c):
    """Position of the new token of every sequence: from P (no own token yet) to P + span - 1."""
    r = random.Random(c["at"])
    return [c["P"] + r.randrange(c["span"]) for _ in range(c["B"])]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    dt = DTYPES[c["dtype"]]
    H, dk, dv = c["H"], c["dk"], c["dv"]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    def rows(*shape):
        return normal(*shape, scale=shape[-1] ** -0.5).to(dt)

    # slopes from fast to slow over the heads, each head a little off its slope
    slope = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
    log_a = -slope * (0.9 + 0.2 * torch.rand(H, generator=g, device="cuda"))
    s = {"op": c["op"], "log_a": log_a}
    if c["op"] in ("linear", "linear_backward"):
        B, T = c["B"], c["T"]
        s.update(q=rows(B, H, T, dk), k=rows(B, H, T, dk), v=normal(B, H, T, dv).to(dt),
                 state0=normal(c["B0"], H, dk, dv, scale=dk ** -0.5) if c["B0"] else None)
        if c["op"] == "linear":
            s["state_out"] = torch.empty(B, H, dk, dv, device="cuda") if c["state_out"] else None
        else:
            s.update(dout=normal(B, H, T, dv).to(dt), dstate_out=normal(B, H, dk, dv, scale=dk ** -0.5))
    elif c["op"] == "linear_varlen":
        lens = _lengths(c)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        total = max(1, cu[-1] + c["tail"])
        s.update(q=rows(H, total, dk), k=rows(H, total, dk), v=normal(H, total, dv).to(dt),
                 cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_T=max(1, max(lens)),
                 state0=normal(c["n0"], H, dk, dv, scale=dk ** -0.5) if c["n0"] else None,
                 state_out=torch.empty(c["n"], H, dk, dv, device="cuda"),
                 out=torch.zeros(H, total, dv, dtype=dt, device="cuda"))
    elif c["op"] == "linear_decode":
        B = c["B"]
        s.update(q=rows(B, H, dk), k=rows(B, H, dk), v=normal(B, H, dv).to(dt),
                 state=normal(B, H, dk, dv, scale=dk ** -0.5))
    else:
        B, P, L = c["B"], c["P"], c["Lmax"]
        sp = torch.nn.functional.softplus
        n_levels = (P - 1).bit_length() + 1
        s.update(q=rows(B, H, dk), k=rows(B, H, dk), v=normal(B, H, dv).to(dt), log_a=-sp(normal(B, H) - 2.0),
                 lam=sp(normal(B, H, L)), prefix=normal(H, n_levels, dk, dv, scale=dk ** -0.5), P=P,
                 decay=-3.0 * torch.rand(B, H, generator=g, device="cuda"),
                 states=normal(B, H, L, dk, dv, scale=dk ** -0.5),
                 t=torch.tensor(_positions(c), dtype=torch.int64, device="cuda"))
    return s


# ---------------------------------------------------------------- the calls

def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "linear":
        return _plain_linear(s)
    if op == "linear_varlen":
        return _plain_varlen(s)
    if op == "linear_backward":
        return _plain_backward(s)
    if op == "linear_decode":
        return _plain_decode(s)
    return _plain_shared(s)


def _run_own(s):
    from log_linear_attention_gb300 import binding as lla
    op = s["op"]
    if op == "linear":
        out = lla.linear_forward(s["q"], s["k"], s["v"], s["log_a"], state0=s["state0"], state_out=s["state_out"])
        return {"out": out, "state_out": s["state_out"]}
    if op == "linear_varlen":
        out = lla.linear_forward_varlen(s["q"], s["k"], s["v"], s["log_a"], s["cu"], s["max_T"], state0=s["state0"],
                                        state_out=s["state_out"], out=s["out"])
        return {"out": out, "state_out": s["state_out"]}
    if op == "linear_backward":
        dq, dk, dv, ds = lla.linear_backward(s["q"], s["k"], s["v"], s["log_a"], s["dout"], state0=s["state0"],
                                             dstate_out=s["dstate_out"])
        return {"dq": dq, "dk": dk, "dv": dv, "dstate0": ds}
    if op == "linear_decode":
        out = lla.linear_decode_step(s["q"], s["k"], s["v"], s["log_a"], s["state"])
        return {"out": out, "state": s["state"]}
    out = lla.decode_step_shared(s["q"], s["k"], s["v"], s["log_a"], s["lam"], s["prefix"], s["P"], s["decay"],
                                 s["states"], s["t"])
    return {"out": out, "states": s["states"], "decay": s["decay"]}


# ---------------------------------------------------------------- plain forms

def _powers(log_a, n):
    """exp(log_a_h n) for every head h and entry of n (the exponent in 64 bits): [H, *n.shape] fp32."""
    e = log_a.double().reshape(-1, *([1] * n.dim())) * n.double()
    return e.exp().float()


def _scan(q, k, v, log_a, s0):
    """o_t = S_t^T q_t by chunks of CHUNK tokens: [B, H, T, dk] x [B, H, T, dv] fp32, s0 [B or 1, H, dk, dv] or None."""
    B, H, T, dk = q.shape
    dv, C = v.shape[-1], CHUNK
    N = -(-T // C)
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, N * C - T)).reshape(B, H, N, C, -1) for x in (q, k, v))
    i = torch.arange(C, device=q.device)
    gap = i[:, None] - i[None, :]
    mask = torch.where(gap >= 0, _powers(log_a, gap.clamp(min=0)), 0.0)[:, None]
    out = ((q @ k.transpose(-1, -2)) * mask) @ v
    # the state that enters chunk n: sum over earlier chunks m of gamma^(C (n-1-m)) times chunk m's own state
    chunk = (k * _powers(log_a, C - 1 - i)[:, None, :, None]).transpose(-1, -2) @ v
    n = torch.arange(N, device=q.device)
    gap = n[:, None] - 1 - n[None, :]
    carry = torch.where(gap >= 0, _powers(log_a, C * gap.clamp(min=0)), 0.0)
    enter = (carry @ chunk.reshape(B, H, N, dk * dv)).reshape(B, H, N, dk, dv)
    if s0 is not None:
        enter = enter + _powers(log_a, C * n)[..., None, None] * s0[:, :, None]
    out = out + (q * _powers(log_a, i + 1)[:, None, :, None]) @ enter
    return out.reshape(B, H, N * C, dv)[:, :, :T]


def _leave(k, v, log_a, s0, length):
    """S after `length` [B] tokens of every sequence (rows past it count nothing)."""
    T = k.shape[2]
    gap = length[:, None] - 1 - torch.arange(T, device=k.device)[None, :]
    w = torch.where(gap >= 0, _powers(log_a, gap.clamp(min=0)), 0.0).transpose(0, 1)
    s = (k * w[..., None]).transpose(-1, -2) @ v
    if s0 is not None:
        s = s + _powers(log_a, length).transpose(0, 1)[..., None, None] * s0
    return s


def _plain_linear(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    out = _scan(q, k, v, s["log_a"], s["state0"]).to(s["q"].dtype)
    if s["state_out"] is None:
        return {"out": out, "state_out": None}
    length = torch.full((q.shape[0],), q.shape[2], device=q.device)
    return {"out": out, "state_out": _leave(k, v, s["log_a"], s["state0"], length)}


def _plain_varlen(s):
    cu = s["cu"].long()
    length = cu[1:] - cu[:-1]
    i = torch.arange(s["max_T"], device=cu.device)
    real = i[None, :] < length[:, None]
    row = torch.where(real, cu[:-1, None] + i[None, :], 0)
    pad = lambda x: (x.float()[:, row] * real[None, ..., None]).transpose(0, 1)  # noqa: E731
    q, k, v = pad(s["q"]), pad(s["k"]), pad(s["v"])
    o = _scan(q, k, v, s["log_a"], s["state0"]).transpose(0, 1)
    out = torch.zeros_like(s["out"])
    out[:, row[real]] = o[:, real].to(out.dtype)
    return {"out": out, "state_out": _leave(k, v, s["log_a"], s["state0"], length)}


def _plain_backward(s):
    q, k, v, do = (s[n].float() for n in ("q", "k", "v", "dout"))
    la, s0, dsT = s["log_a"], s["state0"], s["dstate_out"]
    dt, T = s["q"].dtype, q.shape[2]
    flip = lambda x: x.flip(2)  # noqa: E731
    # adjoint states: R_t = q_t dout_t^T + gamma R_{t+1}, so dstate_out meets the last token undecayed
    r0 = dsT * _powers(-la, torch.ones((), device=q.device))[:, None, None]
    dq = _scan(do, v, k, la, None if s0 is None else s0.transpose(-1, -2))
    dk = flip(_scan(flip(v), flip(do), flip(q), la, r0.transpose(-1, -2)))
    dv = flip(_scan(flip(k), flip(q), flip(do), la, r0))
    ds0 = None
    if s0 is not None:
        t = torch.arange(T, device=q.device)
        ds0 = (q * _powers(la, t + 1)[..., None]).transpose(-1, -2) @ do
        ds0 = ds0 + _powers(la, torch.full((), T, device=q.device))[:, None, None] * dsT
        if s0.shape[0] == 1:
            ds0 = ds0.sum(0, keepdim=True)
    return {"dq": dq.to(dt), "dk": dk.to(dt), "dv": dv.to(dt), "dstate0": ds0}


def _plain_decode(s):
    st = s["state"]
    st.mul_(s["log_a"].exp()[:, None, None]).add_(s["k"].float()[..., :, None] * s["v"].float()[..., None, :])
    out = (s["q"].float()[..., None, :] @ st)[..., 0, :]
    return {"out": out.to(s["q"].dtype), "state": st}


def _bit_length(x):
    return ((x[..., None] >> torch.arange(62, device=x.device)) > 0).sum(-1)


def _plain_shared(s):
    q, k, v, lam, st, t, P = s["q"].float(), s["k"].float(), s["v"].float(), s["lam"], s["states"], s["t"], s["P"]
    L = st.shape[2]
    l = torch.arange(L, device=t.device)
    pos = t[:, None] - 1
    # bucket of slot l at pos: 2^(l-1) tokens from (pos >> l) << l; slot 0 is the token pos itself
    size = torch.where(l > 0, 1 << (l - 1).clamp(min=0), 1)
    start = (pos >> l) << l
    held = ((l == 0) | ((pos >> (l - 1).clamp(min=0)) & 1 == 1)) & (start + size > P) & (pos >= P)
    into = _bit_length(t & -t)[:, None]  # the slot that the carry of t fills
    grown = torch.where(held[:, None, :, None, None], st, 0.0) * s["log_a"].exp()[..., None, None, None]
    low = (l < into)[:, None, :, None, None]
    merged = torch.where(low, grown, 0.0).sum(2, keepdim=True)
    new = k[..., :, None] * v[..., None, :]
    fills = ((l == into) & (pos >= P))[:, None, :, None, None]
    keeps = (held & (l > into))[:, None, :, None, None]
    first = (l == 0)[None, None, :, None, None]
    st.copy_(torch.where(first, new[:, :, None], torch.where(fills, merged, torch.where(keeps, grown, st))))
    now = torch.where(first | fills | keeps, st, 0.0) * lam[..., None, None]
    out = (q[..., None, :] @ now.sum(2))[..., 0, :]
    # prefix buckets: of the walk of P - 1, at the level of t
    s["decay"].copy_(torch.where(t[:, None] > P, s["decay"], 0.0) + s["log_a"])
    j = torch.arange(s["prefix"].shape[1], device=t.device)
    j = j[(j == 0) | (((P - 1) >> (j - 1).clamp(min=0)) & 1 == 1)]
    level = _bit_length(t[:, None] ^ (((P - 1) >> j) << j))
    w = lam.gather(2, level[:, None, :].expand(-1, lam.shape[1], -1))
    each = torch.einsum("bhk,hjkv->bhjv", q, s["prefix"][:, j])
    out = out + s["decay"].exp()[..., None] * (w[..., None] * each).sum(2)
    return {"out": out.to(s["q"].dtype), "states": st, "decay": s["decay"]}


# ---------------------------------------------------------------- work

def work(case):
    """Bytes: inputs once, outputs once. Flops: the recurrence's 4 dk dv a token (update and read), for the
    backward 10 dk dv (both states, three reads); the shared step's held buckets at their reads and updates."""
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    H, dk, dv = c["H"], c["dk"], c["dv"]
    if c["op"] == "linear":
        n = c["B"] * H * c["T"]
        b = n * e * (2 * dk + 2 * dv) + 4 * H * dk * dv * (c["B0"] + (c["B"] if c["state_out"] else 0))
        return {"bytes": b, "flops": 4 * n * dk * dv}
    if c["op"] == "linear_varlen":
        n = H * sum(_lengths(c))
        return {"bytes": n * e * (2 * dk + 2 * dv) + 4 * H * dk * dv * (c["n0"] + c["n"]), "flops": 4 * n * dk * dv}
    if c["op"] == "linear_backward":
        n = c["B"] * H * c["T"]
        return {"bytes": n * e * (4 * dk + 3 * dv) + 4 * H * dk * dv * (2 * c["B0"] + c["B"]),
                "flops": 10 * n * dk * dv}
    if c["op"] == "linear_decode":
        n = c["B"] * H
        return {"bytes": n * (e * (2 * dk + 2 * dv) + 8 * dk * dv), "flops": 4 * n * dk * dv}
    P, n = c["P"], c["B"] * H
    shared = 1 + bin(P - 1).count("1")
    read = wrote = 0
    for t in _positions(c):
        read += _own_buckets(t - 1, P)
        wrote += _own_buckets(t, P)
    b = n * (e * (2 * dk + 2 * dv) + 4 * (c["Lmax"] + 3)) + 4 * H * dk * dv * (shared + read + wrote)
    return {"bytes": b, "flops": 2 * dk * dv * (n * shared + H * (read + wrote))}


def _own_buckets(pos, P):
    if pos < P:
        return 0
    return 1 + sum((pos >> i) & 1 and ((pos >> (i + 1)) << (i + 1)) + (1 << i) > P for i in range(40))


# ---------------------------------------------------------------- 64 bits

def _tokens(q, k, v, gamma, S):
    """The recurrence token by token: outputs [.., T, dv] and the last state."""
    out = torch.empty(*q.shape[:-1], v.shape[-1], dtype=torch.float64, device=q.device)
    for t in range(q.shape[-2]):
        S = gamma * S + k[..., t, :, None] * v[..., t, None, :]
        out[..., t, :] = (q[..., t, :, None] * S).sum(-2)
    return out, S


def exact(case, seed):
    s = prepare(case, seed)
    d = {n: x.double() for n, x in s.items() if torch.is_tensor(x) and x.is_floating_point()}
    q, k, v = d["q"], d["k"], d["v"]
    H, dk, dv = case["H"], case["dk"], case["dv"]
    if case["op"] in ("linear", "linear_varlen", "linear_backward", "linear_decode"):
        gamma = torch.exp(d["log_a"])[:, None, None]
    if case["op"] == "linear":
        S = q.new_zeros(case["B"], H, dk, dv) + (d["state0"] if case["B0"] else 0.0)
        out, S = _tokens(q, k, v, gamma, S)
        return {"out": out, "state_out": S if case["state_out"] else None}
    if case["op"] == "linear_varlen":
        if sum(_lengths(case)) > 200000:
            return None
        out, ends, at = torch.zeros_like(v), [], 0
        for b, n in enumerate(_lengths(case)):
            S = d["state0"][b if case["n0"] > 1 else 0] if case["n0"] else q.new_zeros(H, dk, dv)
            out[:, at:at + n], S = _tokens(q[:, at:at + n], k[:, at:at + n], v[:, at:at + n], gamma, S)
            ends.append(S)
            at += n
        return {"out": out, "state_out": torch.stack(ends)}
    if case["op"] == "linear_decode":
        out, S = _tokens(q[..., None, :], k[..., None, :], v[..., None, :], gamma, d["state"])
        return {"out": out[..., 0, :], "state": S}
    if case["op"] == "linear_backward":
        do = d["dout"]
        S = q.new_zeros(case["B"], H, dk, dv) + (d["state0"] if case["B0"] else 0.0)
        dq, gk, gv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        for t in range(case["T"]):
            S = gamma * S + k[..., t, :, None] * v[..., t, None, :]
            dq[..., t, :] = (S * do[..., t, None, :]).sum(-1)
        R = d["dstate_out"].clone()
        for t in reversed(range(case["T"])):
            R = R + q[..., t, :, None] * do[..., t, None, :]
            gk[..., t, :] = (R * v[..., t, None, :]).sum(-1)
            gv[..., t, :] = (R * k[..., t, :, None]).sum(-2)
            R = gamma * R
        if case["B0"] == 1:
            R = R.sum(0, keepdim=True)
        return {"dq": dq, "dk": gk, "dv": gv, "dstate0": R if case["B0"] else None}
    # the shared step, sequence by sequence over its buckets as sets of positions
    P, st, decay, out = case["P"], d["states"].clone(), d["decay"].clone(), q.new_zeros(case["B"], H, dv)
    for b, t in enumerate(_positions(case)):
        before = _walk(t - 1)
        after = _walk(t)
        a = torch.exp(d["log_a"][b])[:, None, None]
        decay[b] = (decay[b] if t > P else 0.0) + d["log_a"][b]
        for l, (lo, hi) in after.items():
            if hi <= P:
                continue
            if l == 0:
                S = k[b][:, :, None] * v[b][:, None, :]
            else:
                S = sum(d["states"][b, :, m] for m, (x, y) in before.items() if lo <= x and y <= hi and y > P) * a
            st[b, :, l] = S
            out[b] += d["lam"][b, :, l, None] * (q[b][:, :, None] * S).sum(1)
        for m, (lo, hi) in _walk(P - 1).items():
            l = next(n for n, (x, y) in after.items() if x <= lo and hi <= y)
            w = d["lam"][b, :, l] * torch.exp(decay[b])
            out[b] += w[:, None] * (q[b][:, :, None] * d["prefix"][:, m]).sum(1)
    return {"out": out, "states": st, "decay": decay}


def _walk(pos):
    """{slot: [first, last + 1) positions} of the Fenwick partition of 0..pos."""
    got, end = {0: (pos, pos + 1)}, pos
    while end > 0:
        low = end & -end
        got[low.bit_length()] = (end - low, end)
        end -= low
    return got
