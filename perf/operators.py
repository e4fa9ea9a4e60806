"""Measured cases of the linear-attention operators: prefill, decode and gradients
of linear attention with a decay for each head, and the tables of a packed batch.

Per head h with log-decays g_t <= 0 and a memory S (d_k x d_v):
    S_t = exp(g_t) S_{t-1} + k_t v_t^T,      o_t = S_t^T q_t.
g is one value per token and head, or one constant per head.  q, k and v may
each have fewer heads than there are memories (each head of theirs then serves
a run of consecutive memories).  A packed batch holds sequences of different
lengths one behind the other; a pool of memories is addressed by slot.

``run`` computes the plain form in elementary torch operations, or, where
``own`` is true, calls the library.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 256          # tokens per chunk of the plain form
RESET = -200.0       # log-decay whose exponential is 0 in 32 bits


# ---------------------------------------------------------------------------
# Cases.
# ---------------------------------------------------------------------------
def _prefill(name, B, T, H, Hq, Hk, Hv, dk, dv, dtype, layout, gate, state=True, resets=False):
    return dict(name=name, op="prefill", B=B, T=T, H=H, Hq=Hq, Hk=Hk, Hv=Hv, dk=dk, dv=dv,
                dtype=dtype, layout=layout, gate=gate, state=state, resets=resets)


def listed():
    return [
        # one short prompt of a chat: a few chunks of one sequence, where latency counts
        _prefill("prefill_short_prompt", 1, 190, 16, 16, 16, 16, 128, 128, "bf16", "dense", "token"),
        # a serving step: prompts of different lengths packed one behind the other,
        # memories in a pool, q and k shared by groups of heads
        _prefill("prefill_packed_ragged", 37, 600, 32, 8, 8, 32, 128, 64, "bf16", "packed", "token"),
        # the library's long-context prefill shape, constant decay per head, q, k and v
        # as slices of one projection's output
        _prefill("prefill_long_fused_qkv", 2, 16384, 16, 16, 16, 16, 128, 128, "bf16", "fused",
                 "head", state=False),
        # float32 inputs, with tokens that reset the memory (document borders)
        _prefill("prefill_f32_resets", 1, 2000, 8, 8, 8, 8, 64, 128, "f32", "dense", "token",
                 resets=True),
        # single tokens: the library's decode shape
        dict(name="decode_256x32", op="decode", N=256, live=256, pool=256, H=32, Hq=32, Hk=32,
             Hv=32, dk=128, dv=128, dtype="bf16", gate="token"),
        # one request alone
        dict(name="decode_one_request", op="decode", N=1, live=1, pool=4, H=16, Hq=16, Hk=16,
             Hv=16, dk=128, dv=128, dtype="bf16", gate="head"),
        # a batch padded to a fixed size, memories scattered over a pool, shared q and k
        dict(name="decode_padded_pool", op="decode", N=64, live=45, pool=100, H=24, Hq=2, Hk=2,
             Hv=24, dk=128, dv=64, dtype="bf16", gate="token"),
        # training: the library's gradient shape
        dict(_prefill("grad_4x4096", 4, 4096, 16, 16, 16, 16, 128, 128, "bf16", "dense", "token"),
             op="grad"),
        # training on packed documents, k and v shared by groups of heads
        dict(_prefill("grad_packed_shared", 11, 500, 16, 16, 4, 4, 64, 128, "bf16", "packed",
                      "token", state=False), op="grad"),
        # float32 gradients of a short sequence, constant decay per head
        dict(_prefill("grad_f32_short", 1, 333, 4, 4, 4, 4, 64, 64, "f32", "dense", "token"),
             op="grad"),
        # tables of one serving step: few requests with a token or a prompt each
        dict(name="tables_serving_step", op="tables", N=48, tokens=8192, block=256, mean=150,
             slots=True, context=True),
        # tables of a large batch of short requests
        dict(name="tables_many_requests", op="tables", N=8000, tokens=1 << 20, block=64, mean=120,
             slots=True, context=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "grad", "grad", "tables"])
    if op == "tables":
        N = _log(rng, 1, 8000)
        tokens = _log(rng, 64, 1 << 20)
        return dict(op=op, N=N, tokens=tokens, block=64 * rng.choice([1, 2, 4, 8, 16]),
                    mean=max(1, int(tokens / N * rng.uniform(0.3, 1.2))),
                    slots=rng.random() < 0.7, context=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dk, dv = rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
    H = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 20, 32])

    def heads():
        return rng.choice([d for d in range(1, H + 1) if H % d == 0])

    Hq, Hk, Hv = H, H, H
    share = rng.choice(["none", "none", "qk", "kv", "v"])
    if share == "qk":
        Hq = Hk = heads()
    elif share == "kv":
        Hk = Hv = heads()
    elif share == "v":
        Hv = heads()
    gate = rng.choice(["token", "token", "head"])
    if op == "decode":
        N = _log(rng, 1, 256)
        live = max(1, N - rng.choice([0, 0, 1, N // 4]))
        return dict(op=op, N=N, live=live, pool=live + rng.randrange(0, 20), H=H, Hq=Hq, Hk=Hk,
                    Hv=Hv, dk=dk, dv=dv, dtype=dtype, gate=gate)
    # token-heads of one pass, at most half the largest listed case's
    most = (131072 if op == "prefill" else 65536) if dtype == "bf16" else 32768
    layout = rng.choice(["dense", "fused", "packed"])
    B = _log(rng, 1, 40) if layout == "packed" else rng.choice([1, 1, 2, 3, 4])
    T = _log(rng, 1, max(1, min(16384, most // (B * H))))
    return dict(op=op, B=B, T=T, H=H, Hq=Hq, Hk=Hk, Hv=Hv, dk=dk, dv=dv, dtype=dtype,
                layout=layout, gate=gate, state=rng.random() < 0.6,
                resets=gate == "token" and rng.random() < 0.3)


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _lengths(c):
    """Lengths of a packed batch: c["B"] sequences of one to 2 T - 1 tokens, fixed by the
    case so that its work is; one of them empty where there are many."""
    g = torch.Generator().manual_seed(1234 + 7 * c["B"] + c["T"])
    n = torch.randint(1, 2 * c["T"], (c["B"],), generator=g)
    if c["B"] > 4:
        n[c["B"] // 2] = 0
    return n.tolist()


def _gates(gen, lead, H, gate, dtype, resets=False):
    if gate == "head":       # constant retention from 1 - 2^-4 to about 1 - 2^-9
        r = 4.0 + 5.0 * torch.arange(H, device="cuda", dtype=torch.float32) / max(1, H)
        r = r + 0.2 * torch.rand(H, generator=gen, device="cuda")
        return torch.log1p(-torch.exp2(-r))
    x = torch.randn(lead + (H,), generator=gen, device="cuda")
    g = -torch.nn.functional.softplus(x) * 0.1
    if resets:
        g = torch.where(torch.rand(lead + (H,), generator=gen, device="cuda") < 1 / 64,
                        torch.full_like(g, -math.inf), g)
    return g.to(dtype)


def _qkv(gen, c, lead, dtype):
    """q, k, v of the case; k of norm one; for "fused" as slices of one buffer."""
    q = torch.randn(lead + (c["Hq"], c["dk"]), generator=gen, device="cuda")
    k = torch.randn(lead + (c["Hk"], c["dk"]), generator=gen, device="cuda")
    k = k / k.norm(dim=-1, keepdim=True)
    v = torch.randn(lead + (c["Hv"], c["dv"]), generator=gen, device="cuda")
    if c.get("layout") != "fused":
        return q.to(dtype), k.to(dtype), v.to(dtype)
    parts = [x.flatten(-2).to(dtype) for x in (q, k, v)]
    x = torch.cat(parts, -1)
    q, k, v = x.split([p.shape[-1] for p in parts], -1)
    return (q.unflatten(-1, (c["Hq"], c["dk"])), k.unflatten(-1, (c["Hk"], c["dk"])),
            v.unflatten(-1, (c["Hv"], c["dv"])))


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = dict(case=c)
    if c["op"] == "tables":
        s["lengths"] = torch.randint(0, 2 * c["mean"] + 1, (c["N"],), generator=gen, device="cuda",
                                     dtype=torch.int32)
        s["slots"] = torch.randperm(c["N"] + 5, generator=gen, device="cuda")[:c["N"]].int() \
            if c["slots"] else None
        s["context"] = torch.randint(0, 4000, (c["N"],), generator=gen, device="cuda",
                                     dtype=torch.int32) if c["context"] else None
        return s
    dtype = TYPES[c["dtype"]]
    H, dk, dv = c["H"], c["dk"], c["dv"]
    if c["op"] == "decode":
        N, n = c["N"], c["live"]
        s["q"], s["k"], s["v"] = _qkv(gen, c, (N,), dtype)
        s["g"] = _gates(gen, (N,), H, c["gate"], dtype)
        s["S"] = 0.5 * torch.randn((c["pool"], H, dk, dv), generator=gen, device="cuda")
        s["slots"] = torch.full((N,), -1, dtype=torch.int32, device="cuda")
        s["slots"][:n] = torch.randperm(c["pool"], generator=gen, device="cuda")[:n].int()
        s["o"] = torch.zeros((N, H, dv), dtype=dtype, device="cuda")
        return s
    packed = c["layout"] == "packed"
    if packed:
        n = _lengths(c)
        # a few rows behind the last sequence, as in a buffer of fixed size
        s["total"], s["longest"] = sum(n) + 3, max(max(n), 1)
        s["lengths"] = torch.tensor(n, dtype=torch.int32, device="cuda")
        lead, P = (s["total"],), c["B"] + 2
        s["slots"] = torch.randperm(P, generator=gen, device="cuda")[:c["B"]].int()
    else:
        lead, P = (c["B"], c["T"]), c["B"]
    s["q"], s["k"], s["v"] = _qkv(gen, c, lead, dtype)
    s["g"] = _gates(gen, lead, H, c["gate"], dtype, c["resets"])
    if c["state"] or (packed and c["op"] == "prefill"):
        s["S0"] = 0.5 * torch.randn((P, H, dk, dv), generator=gen, device="cuda")
    else:
        s["S0"] = None
    if c["op"] == "prefill":
        s["o"] = torch.zeros(lead + (H, dv), dtype=dtype, device="cuda")
        # packed: the pool itself, updated in place by every pass
        s["S"] = s["S0"] if packed else torch.zeros((P, H, dk, dv), device="cuda")
    else:
        s["do"] = torch.randn(lead + (H, dv), generator=gen, device="cuda").to(dtype)
        s["dS"] = 0.1 * torch.randn((P, H, dk, dv), generator=gen, device="cuda") \
            if c["state"] else None
    return s


# ---------------------------------------------------------------------------
# Plain form.
# ---------------------------------------------------------------------------
def _lin(q, k, v, g, S0):
    """Linear attention in chunks, float32; q, k [B,H,T,a], v [B,H,T,b], g [B,H,T] float64 (no
    -inf), S0 [B,H,a,b]; T a multiple of the chunk.  Returns o, the memory at every chunk's
    start, and the last memory."""
    B, H, T, a = q.shape
    b, C = v.shape[-1], min(T, CHUNK)
    n = T // C
    q, k, v = q.view(B, H, n, C, a), k.view(B, H, n, C, a), v.view(B, H, n, C, b)
    G = g.view(B, H, n, C).cumsum(-1)                      # from each chunk's start
    E = G[..., -1:]
    below = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    D = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~below, -math.inf).float())
    U = (k * torch.exp((E - G).float())[..., None]).transpose(-1, -2) @ v   # each chunk's own part
    # memories at the chunks' starts: decays between chunks times the parts
    A = torch.cat([torch.zeros_like(E[:, :, :1, 0]), E[..., 0].cumsum(-1)], -1)  # [B,H,n+1]
    before = torch.ones(n + 1, n, dtype=torch.bool, device=q.device).tril(-1)
    W = torch.exp((A[..., :, None] - A[..., None, 1:]).masked_fill(~before, -math.inf).float())
    S = (W @ U.reshape(B, H, n, a * b) +
         torch.exp(A.float())[..., None] * S0.reshape(B, H, 1, a * b)).view(B, H, n + 1, a, b)
    o = ((q @ k.transpose(-1, -2)) * D) @ v + (q @ S[:, :, :-1]) * torch.exp(G.float())[..., None]
    return o.reshape(B, H, T, b), S[:, :, :-1], S[:, :, -1]


def _rows(x, H):
    """[B,T,h,d] to [B,H,T,d] in float32, each head repeated for the memories it serves."""
    return x.transpose(1, 2).float().repeat_interleave(H // x.shape[2], 1)


def _spread(s, longest):
    """Index that spreads a packed batch over [sequences, longest] rows, and which of them are
    tokens."""
    n = s["lengths"].long()
    t = torch.arange(longest, device=n.device)
    live = t < n[:, None]
    return ((n.cumsum(0) - n)[:, None] + t).clamp(max=s["total"] - 1), live


def _batch(s):
    """The case's tensors as a dense batch [B,T,...] of a whole number of chunks: packed
    sequences spread out, tokens past the end with k = v = 0 and no decay."""
    c = s["case"]
    packed = c["layout"] == "packed"
    T = s["longest"] if packed else c["T"]
    C = min(CHUNK, -(-T // 16) * 16)
    Tp = -(-T // C) * C
    if packed:
        at, live = _spread(s, Tp)

        def rows(x):
            return torch.where(live.view(live.shape + (1,) * (x.dim() - 1)), x[at], 0)
    else:
        def rows(x):
            return torch.nn.functional.pad(x, (0,) * (2 * (x.dim() - 2)) + (0, Tp - T))
    g = s["g"]
    if c["gate"] == "head":
        g = g.expand(s["q"].shape[:-2] + (c["H"],))
    g = rows(g.double().clamp(min=RESET)).transpose(1, 2)
    q, k, v = (_rows(rows(s[x]), c["H"]) for x in ("q", "k", "v"))
    S0 = s["S0"]
    if S0 is None:
        S0 = torch.zeros((c["B"], c["H"], c["dk"], c["dv"]), device=q.device)
    elif packed:
        S0 = S0[s["slots"].long()]
    return q, k, v, g, S0, rows, T


def _unspread(s, x, into):
    """Rows [B,T,...] of a dense batch back to the packed rows of ``into``; the rows behind the
    last sequence stay as ``into`` has them."""
    n = s["lengths"].long()
    ends = n.cumsum(0)
    t = torch.arange(s["total"], device=n.device)
    seq = torch.searchsorted(ends, t, right=True)
    used = seq < len(n)
    seq = seq.clamp(max=len(n) - 1)
    at = (t - (ends - n)[seq]).clamp(max=x.shape[1] - 1)
    return torch.where(used.view((-1,) + (1,) * (into.dim() - 1)), x[seq, at].to(into.dtype), into)


def _plain_prefill(s):
    c = s["case"]
    q, k, v, g, S0, _, T = _batch(s)
    o, _, S = _lin(q, k, v, g, S0)
    o = o.transpose(1, 2)
    if c["layout"] == "packed":
        s["S"][s["slots"].long()] = S
        return dict(o=_unspread(s, o, s["o"]), S=s["S"])
    return dict(o=o[:, :T].to(s["o"].dtype), S=S)


def _plain_grad(s):
    """With R_t = exp(g_{t+1}) R_{t+1} + q_t do_t^T from R_T = dS:  dq = S do, dk = R v,
    dv = R^T k, dg_t = exp(g_t) <R_t, S_{t-1}>."""
    c = s["case"]
    packed = c["layout"] == "packed"
    q, k, v, g, S0, rows, T = _batch(s)
    B, H, Tp = q.shape[:3]
    do = rows(s["do"]).transpose(1, 2).float()
    if s["dS"] is None:
        dS = torch.zeros_like(S0)
    else:
        dS = s["dS"][s["slots"].long()] if packed else s["dS"]
    # dq: the same operator with (do, v, k) on the transposed memory
    dq, starts, last = _lin(do, v, k, g, S0.transpose(-1, -2))
    # the reverse recurrence is the operator on flipped time, each decay one token later
    back = torch.cat([torch.zeros_like(g[..., :1]), g.flip(2)[..., :-1]], -1)
    dv, Rs, R = _lin(k.flip(2), q.flip(2), do.flip(2), back, dS)
    dk, _, _ = _lin(v.flip(2), do.flip(2), q.flip(2), back, dS.transpose(-1, -2))
    dk, dv, Rs = dk.flip(2), dv.flip(2), Rs.flip(2)
    # <S, R> at the end of every chunk, then sums back from there within the chunk
    C = Tp // starts.shape[2]
    S = torch.cat([starts[:, :, 1:], last[:, :, None]], 2).transpose(-1, -2)
    later = torch.cat([g.view(B, H, -1, C)[:, :, 1:, 0], torch.zeros_like(g[:, :, :1])], -1)
    end = (S * Rs).double().sum((-1, -2)) * torch.exp(later)
    w = ((q * dq).double().sum(-1) - (k * dk).double().sum(-1)).view(B, H, -1, C)
    dg = (w.flip(-1).cumsum(-1).flip(-1) + end[..., None]).view(B, H, Tp)
    dg = torch.where(g <= RESET, 0.0, dg).transpose(1, 2)
    dS0 = R * torch.exp(g[:, :, :1, None].float())

    def out(x, like):              # [B,H,T,d] to the input's rows and heads
        x = x.unflatten(1, (like.shape[-2], -1)).sum(2).transpose(1, 2)
        if packed:
            return _unspread(s, x, torch.zeros_like(like))
        return x[:, :T].to(like.dtype)

    if c["gate"] == "head":
        dg = dg[:, :T] if not packed else dg * _spread(s, Tp)[1][..., None]
        dg = dg.sum((0, 1)).to(s["do"].dtype)
    elif packed:
        dg = _unspread(s, dg, torch.zeros_like(s["g"]))
    else:
        dg = dg[:, :T].to(s["g"].dtype)
    r = dict(dq=out(dq, s["q"]), dk=out(dk, s["k"]), dv=out(dv, s["v"]), dlog_alpha=dg)
    if s["S0"] is not None:
        r["dS0"] = dS0
        if packed:
            r["dS0"] = torch.zeros_like(s["S0"])
            r["dS0"][s["slots"].long()] = dS0
    return r


def _plain_decode(s):
    c = s["case"]
    n, H = c["live"], c["H"]
    at = s["slots"][:n].long()

    def rows(x):
        return x[:n].float().repeat_interleave(H // x.shape[1], 1)

    q, k, v = rows(s["q"]), rows(s["k"]), rows(s["v"])
    a = torch.exp(s["g"].float())
    a = a[:n] if c["gate"] == "token" else a
    S = s["S"][at] * a[..., None, None] + k[..., :, None] * v[..., None, :]
    s["o"][:n] = (S * q[..., None]).sum(-2).to(s["o"].dtype)
    s["S"][at] = S
    return dict(o=s["o"], S=s["S"])


def _plain_tables(s):
    c = s["case"]
    N, tokens, block = c["N"], c["tokens"], c["block"]
    ends = s["lengths"].long().clamp(min=0).cumsum(0).clamp(max=tokens)
    zero = ends.new_zeros(1)
    offsets = torch.cat([zero, ends])
    counts = offsets[1:] - offsets[:-1]
    block_offsets = torch.cat([zero, ((counts + block - 1) // block).cumsum(0)])
    rows = torch.arange(min(tokens, tokens // block + N), device=ends.device)
    seq = torch.searchsorted(block_offsets[1:], rows, right=True)
    used = seq < N
    at = seq.clamp(max=N - 1)
    index = rows - block_offsets[at]
    first = offsets[at] + index * block
    blocks = torch.stack([first, torch.minimum(offsets[at + 1] - first, first.new_tensor(block)),
                          at, index], 1)
    blocks = torch.where(used[:, None], blocks, blocks.new_tensor([0, 0, -1, 0]))
    t = torch.arange(tokens, device=ends.device)
    seq = torch.searchsorted(ends, t, right=True)
    used = seq < N
    at = seq.clamp(max=N - 1)
    slot = at if s["slots"] is None else s["slots"].long()[at]
    place = t - offsets[at]
    if s["context"] is not None:
        place = place + s["context"].long()[at]
    return dict(offsets=offsets.int(), block_offsets=block_offsets.int(), blocks=blocks.int(),
                slot_map=torch.where(used, slot, -1).int(),
                positions=torch.where(used, place, 0).int())


# ---------------------------------------------------------------------------
# The library.
# ---------------------------------------------------------------------------
def _tables(kdn, s):
    c = s["case"]
    return kdn.sequence_tables(s["lengths"], s["total"],
                               kdn.linear_block(s["total"], c["B"], c["H"]), slots=s["slots"])


def _own(s):
    from linear_attention_recurrent_delta_amd import kdn
    c = s["case"]
    if c["op"] == "tables":
        t = kdn.sequence_tables(s["lengths"], c["tokens"], c["block"], slots=s["slots"],
                                context=s["context"], maps=True)
        return dict(offsets=t.offsets, block_offsets=t.block_offsets, blocks=t.blocks,
                    slot_map=t.slot_map, positions=t.positions)
    if c["op"] == "decode":
        o = kdn.linear_decode(s["q"], s["k"], s["v"], s["g"], s["S"], slots=s["slots"], o=s["o"])
        return dict(o=o, S=s["S"])
    packed = c["layout"] == "packed"
    tables = _tables(kdn, s) if packed else None
    if c["op"] == "prefill":
        o, S = kdn.linear_prefill(s["q"], s["k"], s["v"], s["g"], S0=s["S0"], tables=tables,
                                  out=(s["o"], s["S"]))
        return dict(o=o, S=S)
    d = kdn.linear_prefill_backward(s["q"], s["k"], s["v"], s["do"], s["g"], S0=s["S0"],
                                    dS_out=s["dS"], tables=tables)
    r = {x: d[x] for x in ("dq", "dk", "dv", "dlog_alpha")}
    if s["S0"] is not None:
        r["dS0"] = d["dS0"]
    return r


def run(state):
    if own:
        return _own(state)
    return {"prefill": _plain_prefill, "grad": _plain_grad, "decode": _plain_decode,
            "tables": _plain_tables}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "tables":
        rows = min(c["tokens"], c["tokens"] // c["block"] + c["N"])
        n = c["N"] * (1 + bool(c["slots"]) + bool(c["context"])) + 2 * (c["N"] + 1) + 4 * rows \
            + 2 * c["tokens"]
        return {"bytes": 4 * n, "flops": 0}
    es = 2 if c["dtype"] == "bf16" else 4
    H, dk, dv = c["H"], c["dk"], c["dv"]
    if c["op"] == "decode":
        tok, seqs, state = c["live"], c["live"], True
    elif c["layout"] == "packed":
        tok, seqs, state = sum(_lengths(c)), c["B"], c["state"] or c["op"] == "prefill"
    else:
        tok, seqs, state = c["B"] * c["T"], c["B"], c["state"]
    ins = tok * (c["Hq"] * dk + c["Hk"] * dk + c["Hv"] * dv) * es
    out = tok * H * dv * es
    gate = tok * H * es if c["gate"] == "token" else 4 * H
    S = seqs * H * dk * dv * 4
    if c["op"] == "grad":      # inputs and their gradients, do; S0, dS read and dS0 written
        return {"bytes": 2 * ins + out + 2 * gate + (3 * S if state else 0),
                "flops": tok * H * 10.0 * dk * dv}
    return {"bytes": ins + out + gate + S * (2 if state else 1), "flops": tok * H * 4.0 * dk * dv}


# ---------------------------------------------------------------------------
# The definition, token by token in 64 bits.
# ---------------------------------------------------------------------------
def _forward64(q, k, v, a, S, o):
    """Tokens [T,H,.] of one stream, memory S [H,dk,dv]; fills o and returns the last memory."""
    for t in range(q.shape[0]):
        S = S * a[t][..., None, None] + k[t][..., :, None] * v[t][..., None, :]
        o[t] = (S * q[t][..., None]).sum(-2)
    return S


def _backward64(q, k, v, a, do, S, dS, dq, dk, dv, dg):
    for t in range(q.shape[0]):
        S = S * a[t][..., None, None] + k[t][..., :, None] * v[t][..., None, :]
        dq[t] = (S * do[t][..., None, :]).sum(-1)
    R, flow = dS, (dS * S).sum((-1, -2))
    for t in range(q.shape[0] - 1, -1, -1):
        R = R + q[t][..., :, None] * do[t][..., None, :]
        dk[t] = (R * v[t][..., None, :]).sum(-1)
        dv[t] = (R * k[t][..., None]).sum(-2)
        flow = flow + (q[t] * dq[t]).sum(-1) - (k[t] * dk[t]).sum(-1)
        dg[t] = torch.where(a[t] == 0, 0.0, flow)
        R = R * a[t][..., None, None]
    return R


def exact(case, seed):
    c = case
    if c["op"] == "tables":
        return None
    s = prepare(case, seed)
    H = c["H"]

    def wide(x):
        return x.double().repeat_interleave(H // x.shape[-2], -2)

    q, k, v = wide(s["q"]), wide(s["k"]), wide(s["v"])
    a = torch.exp(s["g"].double())
    if c["op"] == "decode":
        n = c["live"]
        at = s["slots"][:n].long()
        a = a[:n, :, None, None] if c["gate"] == "token" else a[:, None, None]
        new = s["S"][at].double() * a + k[:n, :, :, None] * v[:n, :, None, :]
        o, S = s["o"].double(), s["S"].double()
        o[:n], S[at] = (new * q[:n, :, :, None]).sum(-2), new
        return dict(o=o, S=S)
    if c["gate"] == "head":
        a = a.expand(q.shape[:-1])
    packed = c["layout"] == "packed"
    if packed:
        ends = s["lengths"].cumsum(0).tolist()
        parts = [(slice(e - n, e), int(p)) for e, n, p in
                 zip(ends, s["lengths"].tolist(), s["slots"].tolist())]
        view = lambda x: x  # noqa: E731
    else:                      # all sequences at once: tokens first
        parts = [(slice(0, c["T"]), slice(None))]
        view = lambda x: x.transpose(0, 1)  # noqa: E731
    P = c["B"] + 2 if packed else c["B"]
    S0 = torch.zeros((P, H, c["dk"], c["dv"]), dtype=torch.float64, device="cuda") \
        if s["S0"] is None else s["S0"].double()
    q, k, v, a = view(q), view(k), view(v), view(a)
    if c["op"] == "prefill":
        o, S = torch.zeros_like(v), S0.clone()
        for rows, p in parts:
            S[p] = _forward64(q[rows], k[rows], v[rows], a[rows], S0[p], o[rows])
        return dict(o=view(o), S=S)
    do = view(s["do"].double())
    dS = torch.zeros_like(S0) if s["dS"] is None else s["dS"].double()
    dq, dk, dv, dg = (torch.zeros_like(x) for x in (q, k, v, a))
    dS0 = torch.zeros_like(S0)
    for rows, p in parts:
        dS0[p] = _backward64(q[rows], k[rows], v[rows], a[rows], do[rows], S0[p], dS[p],
                             dq[rows], dk[rows], dv[rows], dg[rows])

    def out(x, heads):
        return view(x).unflatten(-2, (heads, -1)).sum(-2)

    r = dict(dq=out(dq, c["Hq"]), dk=out(dk, c["Hk"]), dv=out(dv, c["Hv"]),
             dlog_alpha=view(dg).flatten(0, -2).sum(0) if c["gate"] == "head" else view(dg))
    if s["S0"] is not None:
        r["dS0"] = dS0
    return r
