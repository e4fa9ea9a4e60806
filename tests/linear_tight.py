"""States that a call returns are float32 in bf16 calls too: inputs of few live
tokens, at which float32 sums leave less than operands of two bf16 parts would."""
import torch

import linear_ref as ref


def case(T, live, H, dk, dv, dtype, seed):
    """One sequence of T tokens, k and q zero but for those in `live`; log-decays
    of at most 1 in all.  CPU tensors q, k, v, log_alpha, d_o, S0, dS."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)
    q, k, v, do = rnd(T, H, dk), rnd(T, H, dk), rnd(T, H, dv), rnd(T, H, dv)
    dead = torch.ones(T, dtype=torch.bool)
    dead[live] = False
    q[dead] = 0
    k[dead] = 0
    la = -torch.rand(T, H, generator=g) / T
    return [x.to(dtype) for x in (q, k, v, la, do)] + [rnd(H, dk, dv) * 2.0 ** -6 for _ in range(2)]


def wanted(q, k, v, la, do, S0, dS):
    """S and dS0, and both over absolute values."""
    a = torch.exp(la.double())
    x = [y.double() for y in (q, k, v)]
    _, S, _, M = ref.forward(*x, a, S0.double())
    g, m = ref.backward(*x, a, do.double(), S0.double(), dS.double())
    return S, M, g["dS0"], m["dS0"]


def bound(M, live, chunks, blocks):
    """Units of 2^-23 (a float32 rounding, also one towards zero): three sums for
    each live token's three parts; for each chunk the power of its decay and the
    product with it; for each block besides those its join's power, product and
    sum; one for the parts' rest and the weight's product, two for the weight's
    power, two for the rounded arguments of the powers (at most 1.5 in base 2)."""
    return (3 * live + 2 * chunks + 3 * blocks + 5) * 2.0 ** -23 * M


def in_parts(x, parts):
    """x as the sum of so many bf16 numbers, each the rest of those before."""
    total = torch.zeros_like(x)
    for _ in range(parts):
        total = total + (x - total).bfloat16().double()
    return total


def planted(q, k, v, la, do, S0, dS, parts):
    """S and dS0 in 64 bits but for the operands of their sums, in so many parts."""
    a = torch.exp(la.double())
    G = la.double().cumsum(0)
    S = S0.double() * torch.exp(G[-1])[:, None, None]
    R = dS.double() * torch.exp(G[-1])[:, None, None]
    for t in range(q.shape[0]):
        S = S + k[t].double()[:, :, None] * in_parts(
            v[t].double() * torch.exp(G[-1] - G[t])[:, None], parts)[:, None, :]
        R = R + q[t].double()[:, :, None] * in_parts(
            do[t].double() * torch.exp(G[t])[:, None], parts)[:, None, :]
    return S, R


# tokens, live ones, tokens of a block, chunks and blocks in bf16
SIZES = [(40, [3, 17, 30], 64, 1, 1), (158, [5, 70, 140], 256, 3, 1), (158, [5, 70, 140], 64, 3, 3),
         (300, [60, 299], 128, 5, 3)]


# ---------------------------------------------------------------------------
# d log_alpha beyond the rounding of its operands.
# ---------------------------------------------------------------------------
def flow_case(T, H, dk, dv, per_head, seed):
    """One sequence in bf16 whose head h lives in channels (p_h, r_h) alone: S and
    R are one number each, just short of half a bf16 step above 1, so that their
    rounding is off by almost 2^-8 the same way in every chunk.  CPU tensors q, k,
    v, log_alpha ([H] float32 or [T, H]), d_o, S0, dS."""
    g = torch.Generator().manual_seed(seed)
    p, r = torch.randint(0, dk, (H,), generator=g), torch.randint(0, dv, (H,), generator=g)
    heads = torch.arange(H)

    def put(d, at, size):
        x = torch.zeros(T, H, d)
        x[:, heads, at] = size * (0.5 + torch.rand(T, H, generator=g))
        return x.bfloat16()

    q, k, v, do = put(dk, p, 2.0 ** -4), put(dk, p, 2.0 ** -7), put(dv, r, 2.0 ** -7), put(dv, r, 2.0 ** -4)
    S0, dS = torch.zeros(H, dk, dv), torch.zeros(H, dk, dv)
    S0[heads, p, r] = 1 + 0.97 * 2.0 ** -8
    dS[heads, p, r] = 1 + 0.95 * 2.0 ** -8
    la = -2.0 ** -14 * (1 + torch.rand(*((H,) if per_head else (T, H)), generator=g))
    return q, k, v, la if per_head else la.bfloat16(), do, S0, dS


def flow_bound(g, m, q, k):
    """d log_alpha [T, H] with states of two bf16 parts on either side (2^-15 of a
    term, 2^-16 from their sums and 2^-16 from the parts), and as much again for
    float32 sums within a chunk (2^-23 for each of up to 160 roundings is 2^-15.7):
    of what passes the token, and of every x and y that the sums run over."""
    near = (q.double().abs() * m["dq"]).sum(-1) + (k.double().abs() * m["dk"]).sum(-1)
    return 2.0 ** -14 * (m["dlog_alpha"] + near.sum(0))


def flow_in_parts(q, k, v, la, do, S0, dS, parts, C=64):
    """The chunk form of d log_alpha [T, H] in 64 bits with S and R read in so many
    bf16 parts."""
    T, H = q.shape[:2]
    q, k, v, do = (x.double().transpose(0, 1) for x in (q, k, v, do))
    g = (la.expand(T, H) if la.dim() == 1 else la).double().t()
    S, starts = S0.double(), []
    spans = [slice(at, min(at + C, T)) for at in range(0, T, C)]
    for s in spans:
        starts.append(S)
        G = g[:, s].cumsum(-1)
        E = G[:, -1:]
        S = S * torch.exp(E)[..., None] + \
            (k[:, s] * torch.exp(E - G)[..., None]).transpose(1, 2) @ v[:, s]
    R, out = dS.double(), torch.zeros(H, T, dtype=torch.float64)
    for s, S in zip(reversed(spans), reversed(starts)):
        G = g[:, s].cumsum(-1)
        E = G[:, -1:]
        Sr, Rr = in_parts(S, parts), in_parts(R, parts)
        D = torch.exp(G[..., :, None] - G[..., None, :]).tril(-1)
        X = (q[:, s] @ k[:, s].transpose(1, 2)) * (do[:, s] @ v[:, s].transpose(1, 2)) * D
        x = (q[:, s] * (do[:, s] @ Sr.transpose(1, 2))).sum(-1) * torch.exp(G)
        y = (k[:, s] * (v[:, s] @ Rr.transpose(1, 2))).sum(-1) * torch.exp(E - G)
        u = X.sum(-1) - X.sum(-2) + x
        out[:, s] = u.flip(-1).cumsum(-1).flip(-1) + y.cumsum(-1) - y + \
            torch.exp(E) * (Sr * Rr).sum((-1, -2))[:, None]
        R = R * torch.exp(E)[..., None] + (q[:, s] * torch.exp(G)[..., None]).transpose(1, 2) @ do[:, s]
    return out.t()
