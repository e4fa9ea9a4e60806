"""Linear attention with a decay for each head, token by token in 64 bits, with
bounds of what a kernel's roundings can add.

A rounding to bf16 is off by at most 2^-8 of the value, to float32 by 2^-24.
Beside every result this returns the same sum over absolute values: a rounding
of relative size e on every term of the sum is off by at most e times that.
"""
import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def wide(x, H):
    """[.., heads, d] to float64 [.., H, d], each head repeated for its states."""
    x = x.detach().cpu().double()
    return x.repeat_interleave(H // x.shape[-2], -2)


def decay(log_alpha, lead, H):
    a = torch.exp(log_alpha.detach().cpu().double())
    return a.expand(lead + (H,)) if log_alpha.dim() == 1 else a


def forward(q, k, v, a, S0):
    """One sequence: q, k [T,H,dk], v [T,H,dv], a [T,H], S0 [H,dk,dv], float64.
    Returns o, S, and both over absolute values."""
    S, M = S0.clone(), S0.abs()
    o, m = torch.zeros_like(v), torch.zeros_like(v)
    for t in range(q.shape[0]):
        at = a[t][:, None, None]
        S = S * at + k[t][:, :, None] * v[t][:, None, :]
        M = M * at + k[t].abs()[:, :, None] * v[t].abs()[:, None, :]
        o[t] = (S * q[t][:, :, None]).sum(1)
        m[t] = (M * q[t].abs()[:, :, None]).sum(1)
    return o, S, m, M


def backward(q, k, v, a, do, S0, dS):
    """One sequence, as forward; do [T,H,dv], dS [H,dk,dv].  Returns dicts of the
    gradients dq, dk, dv, dlog_alpha, dS0 by the recurrence
    R_t = a_{t+1} R_{t+1} + q_t do_t^T (R_T = dS + ..), and of the same over
    absolute values."""
    out = []
    for f in (lambda x: x, torch.abs):
        Q, K, V, O = f(q), f(k), f(v), f(do)
        S, before = f(S0), []
        dq, dk, dv, dg = (torch.zeros_like(x) for x in (q, k, v, a))
        for t in range(q.shape[0]):
            S = S * a[t][:, None, None]
            before.append(S)                      # a_t S_{t-1}
            S = S + K[t][:, :, None] * V[t][:, None, :]
            dq[t] = (S * O[t][:, None, :]).sum(2)
        R = f(dS)
        for t in range(q.shape[0] - 1, -1, -1):
            R = R + Q[t][:, :, None] * O[t][:, None, :]
            dk[t] = (R * V[t][:, None, :]).sum(2)
            dv[t] = (R * K[t][:, :, None]).sum(1)
            dg[t] = (R * before[t]).sum((1, 2))
            R = R * a[t][:, None, None]
        out.append(dict(dq=dq, dk=dk, dv=dv, dlog_alpha=dg, dS0=R))
    return out


def flow_bound(g, m, q, k, C, dtype):
    """d log_alpha: the states' roundings on what passes the token (two of
    them in <S, R>), float32 sums over the chunk's tokens, its own rounding."""
    near = (q.abs() * m["dq"]).sum(-1) + (k.abs() * m["dk"]).sum(-1)
    T = g.shape[0]
    total = torch.stack([near[t // C * C:t // C * C + C].sum(0) for t in range(T)]) if T else near
    h = HALF[dtype]
    low = 2.05 * h * m["dlog_alpha"] if dtype == torch.bfloat16 else 0.0
    return h * (g.abs() + low) + low + slack(T, 2 * C, dtype) * (m["dlog_alpha"] + total)


def slack(T, d, dtype):
    """Relative bound of float32 sums over T tokens of d channels, with the
    decays' own roundings (a power of two is off by 2^-23, one per chunk and
    token on the way)."""
    return (2 * T + d + 256) * 2.0 ** -23


def o_bound(o, m, T, d, dtype):
    """Output: its own rounding; for bf16 also the rounding of q k^T and of the
    state it is read from (each term of the sum has one of the two)."""
    h = HALF[dtype]
    low = h * m if dtype == torch.bfloat16 else 0.0
    return h * (o.abs() + low) + low + slack(T, d, dtype) * m


def S_bound(M, T, d, dtype):
    """State: bf16 operands in two parts leave 2^-16 of a term."""
    return (2.0 ** -16 * (dtype == torch.bfloat16) + slack(T, d, dtype)) * M


def close(name, got, want, bound):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{name}: not finite"
    off = (got - want).abs()
    worst = (off / (bound + 1e-30)).max().item() if off.numel() else 0.0
    print(f"    {name}: {worst:.3f} of the bound", flush=True)
    assert (off <= bound + 1e-30).all(), f"{name}: {worst:.2f} times the bound"


def tables(lengths, tokens, block, slots=None, context=None):
    """The packed batch's tables, in plain Python."""
    N = len(lengths)
    offsets, block_offsets, blocks, at = [0], [0], [], 0
    slot_map, positions = [-1] * tokens, [0] * tokens
    for n, length in enumerate(lengths):
        end = min(at + max(length, 0), tokens)
        for i, first in enumerate(range(at, end, block)):
            blocks.append((first, min(block, end - first), n, i))
        for t in range(at, end):
            slot_map[t] = n if slots is None else slots[n]
            positions[t] = t - at + (0 if context is None else context[n])
        at = end
        offsets.append(at)
        block_offsets.append(len(blocks))
    rows = min(tokens, tokens // block + N)
    assert len(blocks) <= rows
    blocks += [(0, 0, -1, 0)] * (rows - len(blocks))
    i32 = lambda x: np.asarray(x, np.int32)
    return (i32(offsets), i32(block_offsets), i32(blocks).reshape(rows, 4), i32(slot_map),
            i32(positions))
