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
