"""Plain 64-bit forms of linear attention with one decay per head, and what roundings may cost.

Written from the sums over pairs of tokens, not from the recurrence or from chunks. Arrays are numpy
float64, q and k [B, H, T, dk], v [B, H, T, dv], log_a [H], states [B, H, dk, dv].
"""
import numpy as np

U32 = 2.0 ** -24  # half a step of fp32, relative
UBF = 2.0 ** -8   # half a step of bf16, relative


def powers(log_a, n):
    """exp(log_a n) [H, *n.shape] for n >= 0, 1 at n = 0 for every decay (0 among them)."""
    n = np.asarray(n, dtype=np.float64)
    e = np.asarray(log_a, dtype=np.float64).reshape(-1, *([1] * n.ndim))
    with np.errstate(invalid="ignore"):
        return np.where(n == 0, 1.0, np.exp(e * n))


def decay_mask(log_a, T):
    gap = np.arange(T)[:, None] - np.arange(T)[None, :]
    return np.where(gap >= 0, powers(log_a, np.maximum(gap, 0)), 0.0)


def forward(q, k, v, log_a, s0=None):
    """(out, state after the last token)."""
    T = q.shape[2]
    t = np.arange(T)
    out = ((q @ np.swapaxes(k, -1, -2)) * decay_mask(log_a, T)) @ v
    s = np.swapaxes(k * powers(log_a, T - 1 - t)[..., None], -1, -2) @ v
    if s0 is not None:
        out = out + powers(log_a, t + 1)[..., None] * (q @ s0)
        s = s + powers(log_a, np.array(T))[:, None, None] * s0
    return out, s


def backward(q, k, v, log_a, dout, s0=None, ds=None):
    """(dq, dk, dv, dstate0 per sequence) of sum(dout out) + sum(ds state)."""
    T = q.shape[2]
    t = np.arange(T)
    m = decay_mask(log_a, T)
    g = (dout @ np.swapaxes(v, -1, -2)) * m
    p = (q @ np.swapaxes(k, -1, -2)) * m
    enter, leave = powers(log_a, t + 1)[..., None], powers(log_a, T - 1 - t)[..., None]
    dq, dk, dv = g @ k, np.swapaxes(g, -1, -2) @ q, np.swapaxes(p, -1, -2) @ dout
    ds0 = np.swapaxes(q * enter, -1, -2) @ dout
    if s0 is not None:
        dq = dq + enter * (dout @ np.swapaxes(s0, -1, -2))
    if ds is not None:
        dk = dk + leave * (v @ np.swapaxes(ds, -1, -2))
        dv = dv + leave * (k @ ds)
        ds0 = ds0 + powers(log_a, np.array(T))[:, None, None] * ds
    return dq, dk, dv, ds0


def check(got, ref, size, dtype, terms, what):
    """Every element within what its roundings may cost, and the whole within what they cost on average.

    ``size``: the reference with every input's absolute value (the sum of the terms' sizes). fp32: each of
    ``terms`` additions rounds to 2^-24 (the tensor cores' truncate, so to 2^-23). bf16: the weighted scores or
    the state are rounded once, 2^-8 of every term, and the result once. On average over an output, roundings
    are uniform (half a step over sqrt 3) and independent, so two of them give sqrt(2 / 3) 2^-8 = 3.2e-3 of
    sums without cancellation beyond that of random signs; 5e-3 is half as much again. fp32 outputs average the
    same way: sqrt(terms) of them at most."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), what
    bound = (terms + 16) * 2 * U32 * size
    if dtype == "bf16":
        bound = bound + UBF * size + UBF * np.abs(ref)
    worst = np.max(np.abs(got - ref) - bound - 1e-37)
    assert worst <= 0, (what, "element", worst)
    rel = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30)
    most = 5e-3 if dtype == "bf16" else 4 * np.sqrt(terms + 16) * U32 * max(
        1.0, np.linalg.norm(size) / max(np.linalg.norm(ref), 1e-30))
    assert rel <= most, (what, "norm", rel, most)


def make(rng, shape, dtype, scale=1.0):
    """(float64 values, tensor on the CPU holding exactly them)."""
    import torch
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32))
    if dtype == "bf16":
        t = t.bfloat16()
    return t.double().numpy(), t


def tokens(q, k, v, log_a, s0, dout, ds):
    """The recurrence and its adjoint token by token in float64 on the tensors' device, for shapes too long for pair
    sums: q, k [N, T, dk], v, dout [N, T, dv], log_a [N], s0, ds [N, dk, dv]. (out, state, dq, dk, dv, dstate0)."""
    import torch
    q, k, v, dout, S = (x.double() for x in (q, k, v, dout, s0))
    g = torch.exp(log_a.double())[:, None, None]
    out, dq, gk, gv = (torch.empty_like(x) for x in (v, q, k, v))
    for t in range(q.shape[1]):
        S = g * S + k[:, t, :, None] * v[:, t, None, :]
        out[:, t] = (q[:, t, :, None] * S).sum(1)
        dq[:, t] = (S * dout[:, t, None, :]).sum(2)
    R = ds.double()
    for t in reversed(range(q.shape[1])):
        R = R + q[:, t, :, None] * dout[:, t, None, :]
        gk[:, t] = (R * v[:, t, None, :]).sum(2)
        gv[:, t] = (R * k[:, t, :, None]).sum(1)
        R = g * R
    return out, S, dq, gk, gv, R
