"""Measured cases of the operators around a recurrence: the short causal
convolution in front of it, the selective state space scan, the gated norm of its
outputs, and the norm of the residual stream before the next block.

Convolution, per channel with W taps: s_t = b + sum_j w_j x_{t-W+1+j}, y = silu(s);
the rows before a sequence are its state, the last W-1 rows of x.
Scan, per channel c and state n, with A < 0:
    dt_t = softplus(delta_t + bias),   h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t,
    y_t = (sum_n C_t h_t + D x_t) silu(z_t);
B and C are shared by groups of channels.
Gated norm, of each head's d values, r(u) = (mean(u^2) + eps)^(-1/2):
    y = x r(x) w act(z)   or   u = x act(z), y = u r(u) w.
Residual norm: h = residual + scale x, y = h r(h) w.

``run`` computes the plain form in elementary torch operations, or, where ``own``
is true, calls the library.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64            # tokens per chunk of the plain form's scan
SLAB = 1 << 27        # (token, channel, state) values that the plain form holds at once
EPS = 1e-5


# ---------------------------------------------------------------------------
# Cases.
# ---------------------------------------------------------------------------
def _conv(name, op, B, T, C, W, dtype, layout, state, bias=True):
    return dict(name=name, op=op, B=B, T=T, C=C, W=W, dtype=dtype, layout=layout, state=state,
                bias=bias)


def _scan(name, op, B, T, C, N, G, dtype, layout, state, z=True, skip=True):
    return dict(name=name, op=op, B=B, T=T, C=C, N=N, G=G, dtype=dtype, layout=layout, state=state,
                z=z, skip=skip)


def listed():
    return [
        # a serving step: prompts of different lengths packed one behind the other, q, k and v
        # of 16 heads of 128 as slices of one projection's output, states in a pool
        _conv("conv_packed_prompts", "conv", 37, 600, 6144, 4, "bf16", "packed", True),
        # single tokens, a batch padded to a fixed size, states scattered over a pool
        dict(name="conv_decode_padded", op="conv_decode", N=64, live=45, pool=100, C=6144, W=4,
             dtype="bf16", bias=True),
        # training
        _conv("conv_grad_4x4096", "conv_grad", 4, 4096, 2048, 4, "bf16", "dense", False),
        # one short prompt of a chat, where latency counts
        _scan("scan_short_prompt", "scan", 1, 190, 2048, 16, 1, "bf16", "dense", True),
        # a serving step of packed prompts, states in a pool, x and z as slices of one
        # projection's output
        _scan("scan_packed_prompts", "scan", 37, 600, 4096, 16, 1, "bf16", "packed", True),
        # single tokens of many requests
        dict(name="scan_decode_256", op="scan_decode", N=256, live=256, pool=256, C=4096, S=16, G=1,
             dtype="bf16", z=True, skip=True),
        # training on long sequences
        _scan("scan_grad_2x4096", "scan_grad", 2, 4096, 2048, 16, 1, "bf16", "dense", False),
        # training in float32 on packed documents, channels not a multiple of anything, B and C
        # shared by two groups of them, states handed on between segments
        _scan("scan_grad_packed_f32", "scan_grad", 11, 500, 518, 32, 2, "f32", "packed", True,
              z=False),
        # one token of one request: 16 heads of 128
        dict(name="gated_norm_one_token", op="norm", rows=1, H=16, d=128, dtype="bf16",
             order="norm_gate", act="silu", per_head=False),
        # training: heads of the library's prefill shape
        dict(name="gated_norm_grad_4x4096", op="norm_grad", rows=16384, H=16, d=128, dtype="bf16",
             order="norm_gate", act="silu", per_head=False),
        # a prompt's rows of a bf16 model whose residual stream is float32
        dict(name="residual_norm_16384", op="residual", rows=16384, D=4096, dtype="bf16",
             stream="f32", scale="none"),
        # training with a scale per channel, rows not a multiple of anything
        dict(name="residual_norm_grad_odd", op="residual_grad", rows=2500, D=1543, dtype="bf16",
             stream="bf16", scale="channel"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def _channels(rng, lo, hi):
    """Mostly multiples of 64, as models have them; some odd."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.3 or n < 64 else n // 64 * 64


def draw(rng):
    op = rng.choice(["conv", "conv_grad", "conv_decode", "scan", "scan", "scan_grad", "scan_grad",
                     "scan_decode", "norm", "norm_grad", "residual", "residual_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "conv_decode":
        N = _log(rng, 1, 256)
        live = max(1, N - rng.choice([0, 0, 1, N // 4]))
        return dict(op=op, N=N, live=live, pool=live + rng.randrange(0, 20),
                    C=_channels(rng, 16, 6144), W=rng.choice([2, 3, 4, 4]), dtype=dtype,
                    bias=rng.random() < 0.7)
    if op == "scan_decode":
        N = _log(rng, 1, 256)
        live = max(1, N - rng.choice([0, 0, 1, N // 4]))
        G = rng.choice([1, 1, 2])
        return dict(op=op, N=N, live=live, pool=live + rng.randrange(0, 20),
                    C=G * _channels(rng, 16, 4096 // G), S=rng.choice([8, 16, 16]), G=G, dtype=dtype,
                    z=rng.random() < 0.7, skip=rng.random() < 0.7)
    layout = rng.choice(["dense", "fused", "packed"])
    B = _log(rng, 1, 40) if layout == "packed" else rng.choice([1, 1, 2, 3, 4])
    if op in ("conv", "conv_grad"):
        C = _channels(rng, 16, 6144)
        most = 1 << 24 if op == "conv_grad" else 1 << 26
        return dict(op=op, B=B, T=_log(rng, 1, max(1, min(16384, most // (B * C)))), C=C,
                    W=rng.choice([2, 3, 4, 4]), dtype=dtype, layout=layout,
                    state=rng.random() < 0.5, bias=rng.random() < 0.7)
    if op in ("scan", "scan_grad"):
        G, N = rng.choice([1, 1, 2]), rng.choice([8, 16, 16, 32])
        C = G * _channels(rng, 16, 4096 // G)
        most = (1 << 28) // N // (2 if op == "scan_grad" else 1)
        return dict(op=op, B=B, T=_log(rng, 1, max(1, min(16384, most // (B * C)))), C=C, N=N, G=G,
                    dtype=dtype, layout=layout, state=rng.random() < 0.5, z=rng.random() < 0.7,
                    skip=rng.random() < 0.7)
    rows = _log(rng, 1, 16384)
    if op in ("norm", "norm_grad"):
        d = rng.choice([32, 64, 96, 128, 128, 256, _log(rng, 1, 1024)])
        H = _log(rng, 1, max(1, min(32, (1 << 25) // (rows * d))))
        return dict(op=op, rows=rows, H=H, d=d, dtype=dtype,
                    order=rng.choice(["norm_gate", "gate_norm"]),
                    act=rng.choice(["silu", "sigmoid"]), per_head=rng.random() < 0.3)
    return dict(op=op, rows=rows, D=_channels(rng, 16, 4096), dtype=dtype,
                stream=rng.choice([dtype, "f32"]), scale=rng.choice(["none", "one", "channel"]))


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _lengths(c):
    """Lengths of a packed batch: c["B"] sequences of one to 2 T - 1 tokens, fixed by the
    case so that its work is; one of them empty where there are many."""
    g = torch.Generator().manual_seed(4321 + 7 * c["B"] + c["T"])
    n = torch.randint(1, 2 * c["T"], (c["B"],), generator=g)
    if c["B"] > 4:
        n[c["B"] // 2] = 0
    return n.tolist()


def _slots(gen, s, N, live, pool):
    s["slots"] = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    s["slots"][:live] = torch.randperm(pool, generator=gen, device="cuda")[:live].int()


def _slices(c, parts, wide):
    """The parts as they are, or as slices of one buffer's rows (with 32 more columns)."""
    if not wide:
        return parts
    sizes = [p.shape[-1] for p in parts]
    x = torch.cat(parts + [torch.zeros_like(parts[0][..., :1]).expand(
        parts[0].shape[:-1] + (32,))], -1)
    return list(x.split(sizes + [32], -1))[:-1]


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dtype = TYPES[c["dtype"]]
    s = dict(case=c)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def rand(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    if c["op"] in ("norm", "norm_grad"):
        lead = (c["rows"], c["H"], c["d"])
        # heads of very different sizes, as a recurrence's outputs have them
        s["x"] = (randn(*lead) * torch.exp(randn(c["rows"], c["H"], 1))).to(dtype)
        s["z"] = randn(*lead).to(dtype)
        s["w"] = 1 + 0.2 * randn(*((c["H"], c["d"]) if c["per_head"] else (c["d"],)))
        if c["op"] == "norm_grad":
            s["dy"] = randn(*lead).to(dtype)
        return s
    if c["op"] in ("residual", "residual_grad"):
        n, D = c["rows"], c["D"]
        s["x"] = randn(n, D).to(dtype)
        s["res"] = (3 * randn(n, D)).to(TYPES[c["stream"]])
        s["w"] = 1 + 0.2 * randn(D)
        s["scale"] = None if c["scale"] == "none" else \
            0.5 + 0.2 * randn(1 if c["scale"] == "one" else D)
        if c["op"] == "residual_grad":     # res stands for the stream after the addition
            s["dy"] = randn(n, D).to(dtype)
            s["dh"] = randn(n, D).to(TYPES[c["stream"]])
        return s
    conv, C = c["op"].startswith("conv"), c["C"]
    if conv:
        s["w"] = randn(C, c["W"]) / math.sqrt(c["W"])
        s["b"] = 0.1 * randn(C) if c["bias"] else None
    else:
        N = c["S"] if c["op"] == "scan_decode" else c["N"]
        s["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(0.2 * randn(C, N))
        s["D"] = 1 + 0.1 * randn(C) if c["skip"] else None
        # time steps from 0.001 to 0.1
        t = torch.exp(math.log(1e-3) + math.log(100.0) * rand(C))
        s["bias"] = t + torch.log(-torch.expm1(-t))
    if c["op"].endswith("decode"):
        R = c["N"]
        _slots(gen, s, R, c["live"], c["pool"])
        lead = (R,)
        s["y"] = torch.zeros((R, C), dtype=dtype, device="cuda")
    else:
        packed = c["layout"] == "packed"
        if packed:
            n = _lengths(c)
            # a few rows behind the last sequence, as in a buffer of fixed size
            s["total"], s["longest"] = sum(n) + 3, max(max(n), 1)
            s["lengths"] = torch.tensor(n, dtype=torch.int32, device="cuda")
            lead, pool = (s["total"],), c["B"] + 2
            _slots(gen, s, c["B"], c["B"], pool)
        else:
            lead, pool = (c["B"], c["T"]), c["B"]
        s["y"] = torch.zeros(lead + (C,), dtype=dtype, device="cuda")
    wide = c.get("layout") in ("fused", "packed")
    if conv:
        s["x"], = _slices(c, [randn(*lead, C).to(dtype)], wide)
        shape = (c["W"] - 1, C)
        if c["op"] == "conv_decode":
            s["state"] = randn(c["pool"], *shape).to(dtype)
            return s
        needs = c["state"] or (packed and c["op"] == "conv")
        s["S0"] = randn(pool, *shape).to(dtype) if needs else None
        if c["op"] == "conv":
            s["S"] = s["S0"] if packed else torch.zeros((pool,) + shape, dtype=dtype, device="cuda")
        else:
            s["dy"] = randn(*lead, C).to(dtype)
            s["dS"] = randn(pool, *shape).to(dtype) if c["state"] else None
        return s
    x, z = randn(*lead, C).to(dtype), randn(*lead, C).to(dtype)
    s["x"], s["z"] = _slices(c, [x, z], wide)
    if not c["z"]:
        s["z"] = None
    s["delta"] = (0.5 * randn(*lead, C)).to(dtype)
    B, Cm = _slices(c, [randn(*lead, c["G"] * N).to(dtype) for _ in range(2)], wide)
    s["B"], s["C"] = (m.unflatten(-1, (c["G"], N)) for m in (B, Cm))
    if c["op"] == "scan_decode":
        s["S"] = 0.5 * randn(c["pool"], C, N)
        return s
    needs = c["state"] or (packed and c["op"] == "scan")
    s["S0"] = 0.5 * randn(pool, C, N) if needs else None
    if c["op"] == "scan":
        s["S"] = s["S0"] if packed else torch.zeros((pool, C, N), device="cuda")
    else:
        s["dy"] = randn(*lead, C).to(dtype)
        s["dS"] = 0.1 * randn(pool, C, N) if c["state"] else None
    return s


# ---------------------------------------------------------------------------
# Packed batches as dense ones and back.
# ---------------------------------------------------------------------------
def _rows(s):
    """A function that spreads rows [tokens, ..] over [sequences, longest, ..] with zeros
    behind each end (dense batches: as they are), and the number of tokens of each."""
    if s["case"]["layout"] != "packed":
        x = s["x"]
        return lambda x: x, torch.full((x.shape[0],), x.shape[1], device=x.device)
    n = s["lengths"].long()
    t = torch.arange(s["longest"], device=n.device)
    live = t < n[:, None]
    at = ((n.cumsum(0) - n)[:, None] + t).clamp(max=s["total"] - 1)
    return (lambda x: torch.where(live.view(live.shape + (1,) * (x.dim() - 1)), x[at], 0)), n


def _unrows(s, x, into):
    """Rows [sequences, longest, ..] back to packed ones; those behind the last sequence stay
    as ``into`` has them."""
    if s["case"]["layout"] != "packed":
        return x.to(into.dtype)
    n = s["lengths"].long()
    ends = n.cumsum(0)
    t = torch.arange(s["total"], device=n.device)
    seq = torch.searchsorted(ends, t, right=True)
    used = seq < len(n)
    seq = seq.clamp(max=len(n) - 1)
    at = (t - (ends - n)[seq]).clamp(max=x.shape[1] - 1)
    return torch.where(used.view((-1,) + (1,) * (into.dim() - 1)), x[seq, at].to(into.dtype), into)


def _start(s, shape, dtype):
    """The sequences' states."""
    c = s["case"]
    if s["S0"] is None:
        return torch.zeros((c["B"],) + shape, dtype=dtype, device="cuda")
    return (s["S0"][s["slots"].long()] if c["layout"] == "packed" else s["S0"]).to(dtype)


def _end(s, S, like):
    """The sequences' states back into the pool, or as they are."""
    if s["case"]["layout"] == "packed":
        like[s["slots"].long()] = S.to(like.dtype)
        return like
    return S.to(like.dtype)


# ---------------------------------------------------------------------------
# Plain forms.
# ---------------------------------------------------------------------------
def _act(x, name="silu"):
    g = 1 / (1 + torch.exp(-x))
    return x * g if name == "silu" else g


def _act_grad(x, name="silu"):
    g = 1 / (1 + torch.exp(-x))
    return g * (1 + x * (1 - g)) if name == "silu" else g * (1 - g)


def _taps(x, w, b):
    """[B, T + W - 1, C] to sums over W rows [B, T, C]."""
    W = w.shape[1]
    T = x.shape[1] - W + 1
    out = sum(x[:, j:j + T] * w[:, j] for j in range(W))
    return out if b is None else out + b


def _tail(x, n, W):
    """The last W - 1 of the first n + W - 1 rows of each sequence of x [B, .., C]."""
    at = n[:, None] + torch.arange(W - 1, device=x.device)
    return x.gather(1, at[..., None].expand(-1, -1, x.shape[-1]))


def _plain_conv(s):
    c = s["case"]
    rows, n = _rows(s)
    x = torch.cat([_start(s, (c["W"] - 1, c["C"]), torch.float32), rows(s["x"]).float()], 1)
    y = _act(_taps(x, s["w"], s["b"]))
    return dict(y=_unrows(s, y, s["y"]), state=_end(s, _tail(x, n, c["W"]), s["S"]))


def _plain_conv_grad(s):
    c = s["case"]
    W, C = c["W"], c["C"]
    rows, n = _rows(s)
    x = torch.cat([_start(s, (W - 1, C), torch.float32), rows(s["x"]).float()], 1)
    ds = rows(s["dy"]).float() * _act_grad(_taps(x, s["w"], s["b"]))
    T = ds.shape[1]
    pad = torch.nn.functional.pad(ds, (0, 0, W - 1, W - 1))
    dx = sum(pad[:, W - 1 - j:W - 1 - j + T + W - 1] * s["w"][:, j] for j in range(W))
    if s["dS"] is not None:
        dS = s["dS"][s["slots"].long()] if c["layout"] == "packed" else s["dS"]
        at = n[:, None] + torch.arange(W - 1, device=n.device)
        dx = dx.scatter_add(1, at[..., None].expand(-1, -1, C), dS.float())
    r = dict(dx=_unrows(s, dx[:, W - 1:], torch.zeros_like(s["x"])),
             dw=torch.stack([(ds * x[:, j:j + T]).sum((0, 1), dtype=torch.float64)
                             for j in range(W)], 1).float())
    if s["b"] is not None:
        r["db"] = ds.sum((0, 1), dtype=torch.float64).float()
    if s["S0"] is not None:
        r["dS0"] = _end(s, dx[:, :W - 1], torch.zeros_like(s["S0"]))
    return r


def _plain_conv_decode(s):
    n, at = s["case"]["live"], s["slots"][:s["case"]["live"]].long()
    x = torch.cat([s["state"][at].float(), s["x"][:n, None].float()], 1)
    s["y"][:n] = _act(_taps(x, s["w"], s["b"]))[:, 0].to(s["y"].dtype)
    s["state"][at] = x[:, 1:].to(s["state"].dtype)
    return dict(y=s["y"], state=s["state"])


def _run_along(a, u, h):
    """h_t = a_t h_{t-1} + u_t along dim 1 of [B, T, ..] from h: all h_t.  Within chunks by
    doubling, from chunk to chunk one after the other."""
    B, T = a.shape[:2]
    Q = min(CHUNK, T)
    n = -(-T // Q)
    if n * Q != T:
        more = (B, n * Q - T) + a.shape[2:]
        a, u = torch.cat([a, a.new_ones(more)], 1), torch.cat([u, u.new_zeros(more)], 1)
    a, u = a.unflatten(1, (n, Q)), u.unflatten(1, (n, Q))
    step = 1
    while step < Q:
        u = torch.cat([u[:, :, :step], u[:, :, step:] + a[:, :, step:] * u[:, :, :-step]], 2)
        a = torch.cat([a[:, :, :step], a[:, :, step:] * a[:, :, :-step]], 2)
        step *= 2
    starts = []
    for i in range(n):
        starts.append(h)
        h = u[:, i, -1] + a[:, i, -1] * h
    return (u + a * torch.stack(starts, 1)[:, :, None]).flatten(1, 2)[:, :T]


def _step(s, delta):
    x = delta + s["bias"]
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _slabs(c, tokens, N):
    """Runs of channels that the plain form works on one after the other."""
    per = c["C"] // c["G"]
    width = max(1, min(per, SLAB // (tokens * N)))
    for g in range(c["G"]):
        for lo in range(g * per, (g + 1) * per, width):
            yield g, slice(lo, min(lo + width, (g + 1) * per))


def _scan_inputs(s, rows, n):
    """The case's tensors as [B, T, ..] float32; dt of tokens past a sequence's end is zero,
    so that they keep its state."""
    x, z, delta = ((None if s[k] is None else rows(s[k]).float()) for k in ("x", "z", "delta"))
    B, C = rows(s["B"]).float(), rows(s["C"]).float()
    dt = _step(s, delta)
    live = torch.arange(x.shape[1], device=x.device) < n[:, None]
    return x, z, delta, torch.where(live[..., None], dt, 0), B, C


def _plain_scan(s):
    c = s["case"]
    rows, n = _rows(s)
    x, z, _, dt, B, C = _scan_inputs(s, rows, n)
    S0 = _start(s, (c["C"], c["N"]), torch.float32)
    y, S = torch.zeros_like(x), torch.zeros_like(S0)
    for g, at in _slabs(c, x.shape[0] * x.shape[1], c["N"]):
        a = torch.exp(dt[..., at, None] * s["A"][at])
        h = _run_along(a, (dt * x)[..., at, None] * B[:, :, g, None], S0[:, at])
        y[..., at] = (h * C[:, :, g, None]).sum(-1)
        S[:, at] = h[:, -1]
    if s["D"] is not None:
        y = y + s["D"] * x
    if z is not None:
        y = y * _act(z)
    return dict(y=_unrows(s, y, s["y"]), S=_end(s, S, s["S"]))


def _plain_scan_grad(s):
    """g_t = dp_t C_t + a_{t+1} g_{t+1} from dS, then each input's part of it."""
    c = s["case"]
    rows, n = _rows(s)
    x, z, delta, dt, B, C = _scan_inputs(s, rows, n)
    S0 = _start(s, (c["C"], c["N"]), torch.float32)
    dy = rows(s["dy"]).float()
    dp = dy if z is None else dy * _act(z)
    dS = torch.zeros_like(S0)
    if s["dS"] is not None:
        dS = s["dS"][s["slots"].long()] if c["layout"] == "packed" else s["dS"]
    y, dx, ddt = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    dA, dB, dC, dS0 = (torch.zeros_like(k) for k in (s["A"], B, C, S0))
    for g, at in _slabs(c, 2 * x.shape[0] * x.shape[1], c["N"]):
        A, Bg, Cg = s["A"][at], B[:, :, g, None], C[:, :, g, None]
        a = torch.exp(dt[..., at, None] * A)
        h = _run_along(a, (dt * x)[..., at, None] * Bg, S0[:, at])
        y[..., at] = (h * Cg).sum(-1)
        dC[:, :, g] += (dp[..., at, None] * h).sum(2)
        before = torch.cat([S0[:, None, at], h[:, :-1]], 1)
        del h
        later = torch.cat([torch.ones_like(a[:, :1]), a.flip(1)[:, :-1]], 1)
        G = _run_along(later, (dp[..., at, None] * Cg).flip(1), dS[:, at]).flip(1)
        del later
        dB[:, :, g] += ((dt * x)[..., at, None] * G).sum(2)
        own_part = (G * Bg).sum(-1)
        dx[..., at] = dt[..., at] * own_part
        dS0[:, at] = a[:, 0] * G[:, 0]
        w = G.mul_(a).mul_(before)
        ddt[..., at] = (w * A).sum(-1) + x[..., at] * own_part
        dA[at] = (w * dt[..., at, None]).sum((0, 1), dtype=torch.float64).float()
        del a, before, G, w
    if s["D"] is not None:
        y, dx = y + s["D"] * x, dx + s["D"] * dp
    live = (torch.arange(x.shape[1], device=x.device) < n[:, None])[..., None]
    ddelta = torch.where(live, ddt / (1 + torch.exp(-(delta + s["bias"]))), 0)
    out = lambda v, like: _unrows(s, v, torch.zeros_like(like))  # noqa: E731
    r = dict(dx=out(dx, s["x"]), ddelta=out(ddelta, s["delta"]), dA=dA, dB=out(dB, s["B"]),
             dC=out(dC, s["C"]), dbias=ddelta.sum((0, 1), dtype=torch.float64).float())
    if s["D"] is not None:
        r["dD"] = (dp * x).sum((0, 1), dtype=torch.float64).float()
    if z is not None:
        r["dz"] = out(dy * y * _act_grad(z), s["z"])
    if s["S0"] is not None:
        r["dS0"] = _end(s, dS0, torch.zeros_like(s["S0"]))
    return r


def _plain_scan_decode(s):
    c = s["case"]
    n, at = c["live"], s["slots"][:c["live"]].long()
    x, dt = s["x"][:n].float(), _step(s, s["delta"][:n].float())
    B, C = (s[k][:n].float().repeat_interleave(c["C"] // c["G"], 1) for k in ("B", "C"))
    S = s["S"][at] * torch.exp(dt[..., None] * s["A"]) + (dt * x)[..., None] * B
    y = (S * C).sum(-1)
    if s["D"] is not None:
        y = y + s["D"] * x
    if s["z"] is not None:
        y = y * _act(s["z"][:n].float())
    s["y"][:n] = y.to(s["y"].dtype)
    s["S"][at] = S
    return dict(y=s["y"], S=s["S"])


def _inv_rms(u):
    return ((u * u).mean(-1, keepdim=True) + EPS) ** -0.5


def _norm(x, z, w, order, act):
    if order == "norm_gate":
        return x * _inv_rms(x) * w * _act(z, act)
    u = x * _act(z, act)
    return u * _inv_rms(u) * w


def _norm_back(u, w, dn):
    """Gradients of u r(u) w for dn: du and the rows' dw."""
    r = _inv_rms(u)
    n = u * r
    t = dn * w
    return r * (t - n * (t * n).mean(-1, keepdim=True)), dn * n


def _norm_grad(x, z, w, dy, order, act):
    if order == "norm_gate":
        gate = _act(z, act)
        dx, dw = _norm_back(x, w, dy * gate)
        return dx, dy * x * _inv_rms(x) * w * _act_grad(z, act), dw
    gate = _act(z, act)
    du, dw = _norm_back(x * gate, w, dy)
    return du * gate, du * x * _act_grad(z, act), dw


def _gated_norm(s, kind):
    """The gated norm or its gradients in the type ``kind``."""
    c = s["case"]
    x, z, w = (s[k].to(kind) for k in ("x", "z", "w"))
    if c["op"] == "norm":
        return dict(y=_norm(x, z, w, c["order"], c["act"]))
    dx, dz, dw = _norm_grad(x, z, w, s["dy"].to(kind), c["order"], c["act"])
    dw = dw.sum(0 if c["per_head"] else (0, 1), dtype=torch.float64)
    return dict(dx=dx, dz=dz, dw=dw)


def _residual_norm(s, kind):
    c = s["case"]
    x, res, w = (s[k].to(kind) for k in ("x", "res", "w"))
    scale = None if s["scale"] is None else s["scale"].to(kind)
    if c["op"] == "residual":
        h = res + (x if scale is None else scale * x)
        return dict(y=h * _inv_rms(h) * w, h=h)
    du, dw = _norm_back(res, w, s["dy"].to(kind))
    d = du + s["dh"].to(kind)
    r = dict(dx=d if scale is None else d * scale, dres=d, dw=dw.sum(0, dtype=torch.float64))
    if scale is not None:
        part = (d * x).sum(0, dtype=torch.float64)
        r["dscale"] = part.sum(0, keepdim=True) if c["scale"] == "one" else part
    return r


def _rounded(s, r):
    """Outputs of the norms in their types."""
    stream = TYPES[s["case"]["stream"]] if "stream" in s["case"] else None
    kinds = dict(dw=torch.float32, dscale=torch.float32, h=stream, dres=stream)
    return {k: v.to(kinds.get(k, s["x"].dtype)) for k, v in r.items()}


# ---------------------------------------------------------------------------
# The library.
# ---------------------------------------------------------------------------
def _own(s):
    from linear_attention_recurrent_delta_amd import kdn
    c = s["case"]
    op = c["op"]
    if op == "norm":
        return dict(y=kdn.gated_norm(s["x"], s["w"], s["z"], eps=EPS, order=c["order"],
                                     activation=c["act"]))
    if op == "norm_grad":
        d = kdn.gated_norm_backward(s["x"], s["w"], s["dy"], s["z"], eps=EPS, order=c["order"],
                                    activation=c["act"])
        return dict(dx=d["dx"], dz=d["dgate"], dw=d["dweight"])
    if op == "residual":
        y, h = kdn.residual_norm(s["x"], s["res"], s["w"], scale=s["scale"], eps=EPS)
        return dict(y=y, h=h)
    if op == "residual_grad":
        d = kdn.residual_norm_backward(s["x"], s["res"], s["w"], s["dy"], s["dh"],
                                       scale=s["scale"], eps=EPS)
        r = dict(dx=d["dx"], dres=d["dresidual"], dw=d["dweight"])
        if s["scale"] is not None:
            r["dscale"] = d["dscale"]
        return r
    if op == "conv_decode":
        y = kdn.causal_conv_decode(s["x"], s["w"], s["state"], bias=s["b"], slots=s["slots"],
                                   y=s["y"])
        return dict(y=y, state=s["state"])
    if op == "scan_decode":
        y = kdn.selective_decode(s["x"], s["delta"], s["A"], s["B"], s["C"], s["S"], D=s["D"],
                                 z=s["z"], delta_bias=s["bias"], slots=s["slots"], y=s["y"])
        return dict(y=y, S=s["S"])
    tables = None
    if c["layout"] == "packed":
        block = 256 if op.startswith("conv") else kdn.selective_block(s["total"], c["B"], c["C"],
                                                                      c["N"])
        tables = kdn.sequence_tables(s["lengths"], s["total"], block, slots=s["slots"])
    if op == "conv":
        y, S = kdn.causal_conv(s["x"], s["w"], bias=s["b"], state0=s["S0"], tables=tables,
                               out=(s["y"], s["S"]))
        return dict(y=y, state=S)
    if op == "conv_grad":
        d = kdn.causal_conv_backward(s["x"], s["w"], s["dy"], bias=s["b"], state0=s["S0"],
                                     dstate_out=s["dS"], tables=tables)
        r = dict(dx=d["dx"], dw=d["dweight"])
        if s["b"] is not None:
            r["db"] = d["dbias"]
        if s["S0"] is not None:
            r["dS0"] = d["dstate0"]
        return r
    args = (s["x"], s["delta"], s["A"], s["B"], s["C"])
    kw = dict(D=s["D"], z=s["z"], delta_bias=s["bias"], S0=s["S0"], tables=tables)
    if op == "scan":
        y, S = kdn.selective_scan(*args, out=(s["y"], s["S"]), **kw)
        return dict(y=y, S=S)
    d = kdn.selective_scan_backward(*args, s["dy"], dS_out=s["dS"], **kw)
    r = {k: d[k] for k in ("dx", "ddelta", "dA", "dB", "dC")}
    r["dbias"] = d["ddelta_bias"]
    if s["D"] is not None:
        r["dD"] = d["dD"]
    if s["z"] is not None:
        r["dz"] = d["dz"]
    if s["S0"] is not None:
        r["dS0"] = d["dS0"]
    return r


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op in ("norm", "norm_grad"):
        return _rounded(state, _gated_norm(state, torch.float32))
    if op in ("residual", "residual_grad"):
        return _rounded(state, _residual_norm(state, torch.float32))
    return {"conv": _plain_conv, "conv_grad": _plain_conv_grad, "conv_decode": _plain_conv_decode,
            "scan": _plain_scan, "scan_grad": _plain_scan_grad,
            "scan_decode": _plain_scan_decode}[op](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------
def work(case):
    c = case
    op = c["op"]
    es = 2 if c["dtype"] == "bf16" else 4
    if op in ("norm", "norm_grad"):
        n = c["rows"] * c["H"] * c["d"]
        w = 4 * c["d"] * (c["H"] if c["per_head"] else 1)
        if op == "norm":
            return {"bytes": 3 * n * es + w, "flops": 10.0 * n}
        return {"bytes": 5 * n * es + 2 * w, "flops": 24.0 * n}
    if op in ("residual", "residual_grad"):
        n, rs = c["rows"] * c["D"], 2 if c["stream"] == "bf16" else 4
        p = 4 * c["D"] * (2 if c["scale"] == "channel" else 1)
        if op == "residual":
            return {"bytes": n * (2 * es + 2 * rs) + p, "flops": 6.0 * n}
        # x is only read for the scale's gradient
        return {"bytes": n * (es * (3 if c["scale"] != "none" else 2) + 3 * rs) + 2 * p,
                "flops": 14.0 * n}
    C = c["C"]
    if op == "conv_decode":
        n, W = c["live"] * C, c["W"]
        return {"bytes": n * es * (2 + 2 * (W - 1)) + 4 * C * (W + c["bias"]),
                "flops": n * (2.0 * W + 4)}
    if op == "scan_decode":
        n, N = c["live"] * C, c["S"]
        return {"bytes": n * (8 * N + es * (3 + c["z"])) + c["live"] * 2 * c["G"] * N * es
                + 4 * C * (N + 1 + c["skip"]), "flops": n * (7.0 * N + 8)}
    seqs = c["B"]
    tok = sum(_lengths(c)) if c["layout"] == "packed" else c["B"] * c["T"]
    n = tok * C
    if op in ("conv", "conv_grad"):
        W = c["W"]
        p = 4 * C * (W + c["bias"])
        state = seqs * (W - 1) * C * es
        if op == "conv":
            reads = c["state"] or c["layout"] == "packed"
            return {"bytes": 2 * n * es + p + state * (1 + reads), "flops": n * (2.0 * W + 4)}
        return {"bytes": 3 * n * es + 2 * p + (3 * state if c["state"] else 0),
                "flops": n * (6.0 * W + 8)}
    N = c["N"]
    state = seqs * C * N * 4
    p = 4 * C * (N + 1 + c["skip"])
    bc = 2 * tok * c["G"] * N * es
    if op == "scan":
        reads = c["state"] or c["layout"] == "packed"
        return {"bytes": n * es * (3 + c["z"]) + bc + p + state * (1 + reads),
                "flops": n * (7.0 * N + 8)}
    return {"bytes": n * es * (5 + 2 * c["z"]) + 2 * bc + 2 * p + (3 * state if c["state"] else 0),
            "flops": n * (22.0 * N + 24)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, token by token.
# ---------------------------------------------------------------------------
def _silu64(x):
    return x * torch.sigmoid(x)


def _dsilu64(x):
    g = torch.sigmoid(x)
    return g + x * g * (1 - g)


def _sequences(s):
    """(rows, state) of every sequence: an index of the token rows and one of the states."""
    c = s["case"]
    if c["layout"] != "packed":
        return [((b,), b) for b in range(c["B"])]
    out, at = [], 0
    for n, slot in zip(s["lengths"].tolist(), s["slots"].tolist()):
        out.append(((slice(at, at + n),), slot))
        at += n
    return out


def _exact_conv(s):
    c = s["case"]
    W, grad = c["W"], c["op"] == "conv_grad"
    w = s["w"].double()
    b = torch.zeros(c["C"], dtype=torch.float64, device="cuda") if s["b"] is None else s["b"].double()
    y = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    dw, db, dS0 = torch.zeros_like(w), torch.zeros_like(b), None
    if s["S0"] is not None:
        dS0 = torch.zeros(s["S0"].shape, dtype=torch.float64, device="cuda")
    if not grad:
        S = s["S"].double()
    for rows, slot in _sequences(s):
        x = s["x"][rows].double()
        T = x.shape[0]
        old = x.new_zeros(W - 1, c["C"]) if s["S0"] is None else s["S0"][slot].double()
        ext = torch.cat([old, x])
        pre = b.expand(T, -1).clone()
        for j in range(W):
            pre += w[:, j] * ext[j:j + T]
        if not grad:
            y[rows] = _silu64(pre)
            S[slot] = ext[T:]
            continue
        ds = s["dy"][rows].double() * _dsilu64(pre)
        dext = torch.zeros_like(ext)
        for j in range(W):
            dext[j:j + T] += w[:, j] * ds
            dw[:, j] += (ds * ext[j:j + T]).sum(0)
        db += ds.sum(0)
        if s["dS"] is not None:
            dext[T:] += s["dS"][slot].double()
        y[rows] = dext[W - 1:]
        if dS0 is not None:
            dS0[slot] = dext[:W - 1]
    if not grad:
        return dict(y=y, state=S)
    r = dict(dx=y, dw=dw)
    if s["b"] is not None:
        r["db"] = db
    if dS0 is not None:
        r["dS0"] = dS0
    return r


def _padded(s):
    """Rows of every sequence as [T, sequences, ..] in 64 bits, and which of them are tokens."""
    c = s["case"]
    if c["layout"] != "packed":
        n = [c["T"]] * c["B"]
        take = lambda x: x.double().transpose(0, 1)  # noqa: E731
    else:
        n = s["lengths"].tolist()
        T = s["longest"]

        def take(x):
            parts = x[:sum(n)].double().split(n)
            out = torch.zeros((T, len(n)) + x.shape[1:], dtype=torch.float64, device=x.device)
            for i, p in enumerate(parts):
                out[:len(p), i] = p
            return out
    T = max(max(n), 1)
    live = torch.arange(T, device="cuda")[:, None] < torch.tensor(n, device="cuda")
    return take, live[..., None]


def _unpadded(s, x, like):
    c = s["case"]
    if c["layout"] != "packed":
        return x.transpose(0, 1)
    out = torch.zeros(like.shape, dtype=torch.float64, device="cuda")
    at = 0
    for i, n in enumerate(s["lengths"].tolist()):
        out[at:at + n] = x[:n, i]
        at += n
    return out


def _exact_scan(s):
    c = s["case"]
    grad = c["op"] == "scan_grad"
    packed = c["layout"] == "packed"
    take, live = _padded(s)
    x, A = take(s["x"]), s["A"].double()
    raw = take(s["delta"]) + s["bias"].double()
    dt = torch.where(live, torch.logaddexp(raw, torch.zeros_like(raw)), 0.0)
    per = c["C"] // c["G"]
    B, C = take(s["B"]), take(s["C"])
    D = torch.zeros(c["C"], dtype=torch.float64, device="cuda") if s["D"] is None else s["D"].double()
    z = None if s["z"] is None else take(s["z"])
    T, R = x.shape[:2]
    S = torch.zeros((R, c["C"], c["N"]), dtype=torch.float64, device="cuda")
    if s["S0"] is not None:
        S = s["S0"][s["slots"].long()].double() if packed else s["S0"].double()

    def wide(m):                       # [R, G, N] to [R, C, N]
        return m.repeat_interleave(per, 1)

    y = torch.zeros_like(x)
    before = torch.zeros((T,) + S.shape, dtype=torch.float64, device="cuda") if grad else None
    for t in range(T):
        if grad:
            before[t] = S
        S = S * torch.exp(dt[t][..., None] * A) + (dt[t] * x[t])[..., None] * wide(B[t])
        y[t] = (S * wide(C[t])).sum(-1)
    y = y + D * x
    if not grad:
        if z is not None:
            y = y * _silu64(z)
        out = s["S"].double()
        if packed:
            out[s["slots"].long()] = S
        else:
            out = S
        return dict(y=_unpadded(s, y, s["y"]), S=out)
    dy = take(s["dy"])
    dp = dy if z is None else dy * _silu64(z)
    g = torch.zeros_like(S)
    if s["dS"] is not None:
        g = s["dS"][s["slots"].long()].double() if packed else s["dS"].double()
    dx, ddt = D * dp, torch.zeros_like(x)
    dA, dB, dC = torch.zeros_like(A), torch.zeros_like(B), torch.zeros_like(C)
    for t in range(T - 1, -1, -1):
        a = torch.exp(dt[t][..., None] * A)
        Bt = wide(B[t])
        S = before[t] * a + (dt[t] * x[t])[..., None] * Bt
        dC[t] = (dp[t][..., None] * S).unflatten(1, (c["G"], per)).sum(2)
        g = g + dp[t][..., None] * wide(C[t])
        dB[t] = ((dt[t] * x[t])[..., None] * g).unflatten(1, (c["G"], per)).sum(2)
        own_part = (g * Bt).sum(-1)
        dx[t] += dt[t] * own_part
        w = g * a * before[t]
        ddt[t] = (w * A).sum(-1) + x[t] * own_part
        dA += (w * dt[t][..., None]).sum(0)
        g = g * a
    ddelta = torch.where(live, ddt * torch.sigmoid(raw), 0.0)
    r = dict(dx=_unpadded(s, dx, s["x"]), ddelta=_unpadded(s, ddelta, s["delta"]), dA=dA,
             dB=_unpadded(s, dB, s["B"]), dC=_unpadded(s, dC, s["C"]), dbias=ddelta.sum((0, 1)))
    if s["D"] is not None:
        r["dD"] = (dp * x).sum((0, 1))
    if z is not None:
        r["dz"] = _unpadded(s, dy * y * _dsilu64(z), s["x"])
    if s["S0"] is not None:
        r["dS0"] = torch.zeros(s["S0"].shape, dtype=torch.float64, device="cuda")
        r["dS0"][s["slots"].long() if packed else slice(None)] = g
    return r


def _exact_norm(s):
    """Gradients by the chain rule written out for each row's scalar m = mean(u^2) + eps."""
    c = s["case"]
    x, z, w = s["x"].double(), s["z"].double(), s["w"].double()
    gate, dgate = (torch.sigmoid(z), None)
    if c["act"] == "silu":
        gate, dgate = _silu64(z), _dsilu64(z)
    else:
        dgate = gate * (1 - gate)
    first = c["order"] == "gate_norm"
    u = x * gate if first else x
    m = u.square().sum(-1, keepdim=True) / c["d"] + EPS
    out = u * w / m.sqrt()
    if c["op"] == "norm":
        return dict(y=out if first else out * gate)
    dy = s["dy"].double()
    dn = dy if first else dy * gate
    dm = (dn * u * w).sum(-1, keepdim=True) * (-0.5) / m ** 1.5
    du = dn * w / m.sqrt() + dm * 2 * u / c["d"]
    dw = dn * u / m.sqrt()
    dw = dw.sum(0) if c["per_head"] else dw.sum((0, 1))
    if first:
        return dict(dx=du * gate, dz=du * x * dgate, dw=dw)
    return dict(dx=du, dz=dy * out * dgate, dw=dw)


def _exact_residual(s):
    c = s["case"]
    x, res, w = s["x"].double(), s["res"].double(), s["w"].double()
    scale = torch.ones(1, dtype=torch.float64, device="cuda") if s["scale"] is None \
        else s["scale"].double()
    h = res + scale * x if c["op"] == "residual" else res
    m = h.square().sum(-1, keepdim=True) / c["D"] + EPS
    if c["op"] == "residual":
        return dict(y=h * w / m.sqrt(), h=h)
    dy = s["dy"].double()
    dm = (dy * h * w).sum(-1, keepdim=True) * (-0.5) / m ** 1.5
    d = s["dh"].double() + dy * w / m.sqrt() + dm * 2 * h / c["D"]
    r = dict(dx=d * scale, dres=d, dw=(dy * h / m.sqrt()).sum(0))
    if c["scale"] == "one":
        r["dscale"] = (d * x).sum().view(1)
    elif c["scale"] == "channel":
        r["dscale"] = (d * x).sum(0)
    return r


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        return _exact_norm(s)
    if op in ("residual", "residual_grad"):
        return _exact_residual(s)
    if op in ("conv", "conv_grad"):
        return _exact_conv(s)
    if op in ("scan", "scan_grad"):
        return _exact_scan(s)
    n = case["live"]
    at = s["slots"][:n].long()
    x, y = s["x"][:n].double(), s["y"].double()
    if op == "conv_decode":
        rows = torch.cat([s["state"][at].double(), x[:, None]], 1)
        pre = (rows * s["w"].double().t()).sum(1)
        if s["b"] is not None:
            pre = pre + s["b"].double()
        y[:n] = _silu64(pre)
        state = s["state"].double()
        state[at] = rows[:, 1:]
        return dict(y=y, state=state)
    raw = s["delta"][:n].double() + s["bias"].double()
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    per = case["C"] // case["G"]
    B, C = (s[k][:n].double().repeat_interleave(per, 1) for k in ("B", "C"))
    S = s["S"].double()
    S[at] = S[at] * torch.exp(dt[..., None] * s["A"].double()) + (dt * x)[..., None] * B
    out = (S[at] * C).sum(-1)
    if s["D"] is not None:
        out = out + s["D"].double() * x
    if s["z"] is not None:
        out = out * _silu64(s["z"][:n].double())
    y[:n] = out
    return dict(y=y, S=S)
