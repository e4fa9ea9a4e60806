"""The convolution and the norms around a recurrence in 64 bits, with bounds of what
a kernel's roundings can add.

u = 2^-24 is half a float32 step relative to a value; a bf16 output is off by 2^-8 of
itself at most.  Beside every result stands the same sum over absolute values: k
roundings on every term are off by at most k u times that.
"""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24


def wide(x):
    return None if x is None else x.detach().cpu().double()


def silu(x):
    return x * torch.sigmoid(x)


def dsilu(x):
    g = torch.sigmoid(x)
    return g * (1 + x * (1 - g))


def act(x, name):
    return {None: lambda v: v, "silu": silu, "sigmoid": torch.sigmoid}[name](x)


def dact(x, name):
    g = torch.sigmoid(x)
    return {None: torch.ones_like(x), "silu": dsilu(x), "sigmoid": g * (1 - g)}[name]


def act_slack(x, dtype):
    """Relative error of sigmoid(x) in units of u: e^-x is off by two units of its
    own, by the rounding of x log2(e) and of the constant unless that is taken back
    (float32; there by 2^-24 of it), the sum, the reciprocal (two) and the product by
    one each."""
    return 8 + 2 * x.abs() * (1.45 if dtype == torch.bfloat16 else 0)


def close(name, got, want, bound):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{name}: not finite"
    off = (got - want).abs()
    worst = (off / (bound + 1e-38)).max().item() if off.numel() else 0.0
    print(f"    {name}: {worst:.3f} of the bound", flush=True)
    assert (off <= bound + 1e-38).all(), f"{name}: {worst:.2f} times the bound"


# ---------------------------------------------------------------------------
# Convolution: one sequence x [T, C], state [W - 1, C], float64.
# ---------------------------------------------------------------------------
def conv(x, w, b, state, silu_on, dtype):
    """y, the state behind the sequence, and y's bound."""
    W, T = w.shape[1], x.shape[0]
    ext = torch.cat([state, x])
    s = torch.zeros_like(x) if b is None else b.expand(T, -1).clone()
    m = s.abs()
    for j in range(W):
        s = s + w[:, j] * ext[j:j + T]
        m = m + w[:, j].abs() * ext[j:j + T].abs()
    y = silu(s) if silu_on else s
    # |silu'| < 1.1; the sum has W roundings
    bound = HALF[dtype] * y.abs() + 1.01 * (1.1 * W * U * m)
    if silu_on:
        bound = bound + 1.01 * y.abs() * act_slack(s, dtype) * U
    return y, ext[T:], bound


def conv_grad(x, w, b, state, dy, dlast, silu_on, dtype):
    """Gradients dx, dweight, dbias, dstate of one sequence and their bounds; those of
    the sums over tokens in units of u of the absolute sums."""
    W, T = w.shape[1], x.shape[0]
    H = W - 1
    ext = torch.cat([state, x])
    s = torch.zeros_like(x) if b is None else b.expand(T, -1).clone()
    m = s.abs()
    for j in range(W):
        s = s + w[:, j] * ext[j:j + T]
        m = m + w[:, j].abs() * ext[j:j + T].abs()
    ds = dy * (dsilu(s) if silu_on else 1.0)
    # ds: its own roundings, those of the derivative (|silu''| <= 1/2; its terms g and
    # s g (1 - g) are each off relatively) and of s
    off = dy.abs() * 2 * U
    if silu_on:
        g = torch.sigmoid(s)
        off = dy.abs() * U * ((g + (s * g * (1 - g)).abs()) * (2 * act_slack(s, dtype) + 4) + 0.5 * W * m)
    dext, mext, eext = torch.zeros_like(ext), torch.zeros_like(ext), torch.zeros_like(ext)
    dw, mw = torch.zeros_like(w), torch.zeros_like(w)
    for j in range(W):
        dext[j:j + T] += w[:, j] * ds
        mext[j:j + T] += w[:, j].abs() * ds.abs()
        eext[j:j + T] += w[:, j].abs() * off
        dw[:, j] = (ds * ext[j:j + T]).sum(0)
        # per part at most 16 tokens of a tile and four waves in float32, and the result
        mw[:, j] = (((20 + 2) * U * ds.abs() + off) * ext[j:j + T].abs()).sum(0)
    if dlast is not None:
        dext[T:] += dlast
        mext[T:] += dlast.abs()
    db, mb = ds.sum(0), ((20 + 2) * U * ds.abs() + off).sum(0)
    bound = 1.01 * (HALF[dtype] * dext.abs() + (W + 1) * U * mext + eext)
    return dict(dx=dext[H:], dweight=dw, dbias=db, dstate0=dext[:H]), \
        dict(dx=bound[H:], dweight=1.01 * mw, dbias=1.01 * mb, dstate0=bound[:H])


# ---------------------------------------------------------------------------
# Norms, float64.
# ---------------------------------------------------------------------------
def gated(x, w, z, eps, order, name, dtype):
    """y [.., H, d] and its bound: the root, the products and the activation."""
    a = torch.ones_like(x) if z is None else act(z, name)
    u = x * a if order == "gate_norm" else x
    r = (u.square().mean(-1, keepdim=True) + eps) ** -0.5
    y = u * r * w * (a if order == "norm_gate" else 1.0)
    slack = 8.0 if z is None else 8 + 2 * act_slack(z, dtype)
    if z is not None and order == "gate_norm":
        slack = slack + slack.amax(-1, keepdim=True)     # through the sum of squares, too
    return y, 1.01 * y.abs() * (HALF[dtype] + slack * U)


def gated_grad(x, w, z, dy, eps, order, name, dtype):
    """dx, dgate, dweight summed over all but the last dimension (per row: not summed)
    and bounds of the same."""
    first = order == "gate_norm"
    a, da = (torch.ones_like(x), torch.zeros_like(x)) if z is None else (act(z, name), dact(z, name))
    u = x * a if first else x
    r = (u.square().mean(-1, keepdim=True) + eps) ** -0.5
    n, dn = u * r, dy if first else dy * a
    t = dn * w
    mean, mag = (t * n).mean(-1, keepdim=True), (t * n).abs().mean(-1, keepdim=True)
    du = r * (t - n * mean)
    top = torch.zeros_like(x) if z is None else act_slack(z, dtype)
    k = 20 + 3 * top.amax(-1, keepdim=True)              # roundings on any term of the row
    off = k * U * r * (t.abs() + n.abs() * mag)
    h = HALF[dtype]
    slope = torch.zeros_like(x)
    if z is not None:
        g = torch.sigmoid(z)
        slope = (g + (z * g * (1 - g)).abs()) if name == "silu" else (g * (1 - g) if name else da.abs())
    dx = du * a if first else du
    bx = 1.01 * (h * dx.abs() + (off + k * U * du.abs()) * (a.abs() if first else 1.0))
    dz = du * x * da if first else dy * n * w * da
    bz = 1.01 * (h * dz.abs() + (off + k * U * du.abs()) * (x * slope).abs() if first else
                 h * dz.abs() + k * U * (dy * n * w * slope).abs())
    return dict(dx=dx, dgate=dz, dweight=dn * n), \
        dict(dx=bx, dgate=bz, dweight=1.01 * k * U * (dn * n).abs())


def residual(x, res, w, scale, eps, dtype, stream):
    s = 1.0 if scale is None else scale
    h = res + s * x
    r = (h.square().mean(-1, keepdim=True) + eps) ** -0.5
    y = h * r * w
    # h's rounding to float32 (one fma), in its own element and in the sum
    off = 2 * U * (h.abs() + (h.abs() * h.abs()).sum(-1, keepdim=True) /
                   (h.square().sum(-1, keepdim=True) + 1e-300) * h.abs())
    return y, h, 1.01 * (HALF[dtype] * y.abs() + 8 * U * y.abs() + off * (r * w).abs()), \
        1.01 * (HALF[stream] + U) * h.abs()


def residual_grad(x, h, w, scale, dy, dh, eps, dtype, stream):
    s = 1.0 if scale is None else scale
    r = (h.square().mean(-1, keepdim=True) + eps) ** -0.5
    n, t = h * r, dy * w
    mean, mag = (t * n).mean(-1, keepdim=True), (t * n).abs().mean(-1, keepdim=True)
    du = r * (t - n * mean)
    off = 20 * U * r * (t.abs() + n.abs() * mag)
    dres = du + (0.0 if dh is None else dh)
    off = off + U * dres.abs()
    dx = dres * s
    part = None if x is None else dres * x
    return dict(dresidual=dres, dx=dx, dweight=dy * n, dscale=part), \
        dict(dresidual=1.01 * (HALF[stream] * dres.abs() + off),
             dx=1.01 * (HALF[dtype] * dx.abs() + (off + U * dres.abs()) * (s if scale is None else s.abs())),
             dweight=1.01 * 12 * U * (dy * n).abs(),
             dscale=None if x is None else 1.01 * off * x.abs())


# ---------------------------------------------------------------------------
# Selective scan: one sequence, float64; x, delta, z [T, C], B, C [T, G, S].
# ---------------------------------------------------------------------------
def step(delta, bias, softplus):
    v = delta if bias is None else delta + bias
    return torch.logaddexp(v, torch.zeros_like(v)) if softplus else v


def step_slack(delta, bias, softplus, dtype):
    """Relative error of a time step in units of u: the sum with the bias (what it moves
    e^v by), the exponential, and the series with its reciprocal and its rest (2^-18 of
    it in bf16 calls)."""
    v = delta if bias is None else delta + bias
    m = delta.abs() + (0 if bias is None else bias.abs())
    if not softplus:
        return m / v.abs().clamp(min=1e-300)
    s = 2 * m + 14 + 2 * v.abs() * (1.45 if dtype == torch.bfloat16 else 0)
    return s + (64 if dtype == torch.bfloat16 else 0)


def heads(m, C):
    return m.repeat_interleave(C // m.shape[1], 1)


def scan(x, delta, A, B, Cm, D, z, bias, softplus, S0, dtype):
    """y, S and their bounds.  M is the state over absolute values, E a bound of what the
    state is off by, in units of u: every decay is off by its exponential and by what the
    time step and the argument's roundings move it by."""
    T, C = x.shape
    dt, ds = step(delta, bias, softplus), step_slack(delta, bias, softplus, dtype)
    Bh, Ch = heads(B, C), heads(Cm, C)
    S, M, E = S0.clone(), S0.abs(), torch.zeros_like(S0)
    y, by = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(T):
        arg = dt[t][:, None] * A
        a = torch.exp(arg)
        off = 3 + arg.abs() * (ds[t][:, None] + 4)            # relative, of a
        u = (dt[t] * x[t])[:, None] * Bh[t]
        E = a * (E + off * M) + u.abs() * (ds[t][:, None] + 3)
        S = a * S + u
        M = a * M + u.abs()
        E = E + 2 * M                                          # sums, and parts of the scan joined
        y[t] = (S * Ch[t]).sum(-1)
        by[t] = ((E + (S.shape[-1] + 4) * M) * Ch[t].abs()).sum(-1)
    if D is not None:
        by = by + 2 * (D * x).abs()
        y = y + D * x
    out, bound = y, U * by
    if z is not None:
        g = silu(z)
        out = y * g
        bound = bound * g.abs() + out.abs() * U * (act_slack(z, dtype) + 2)
    return out, S, 1.02 * (HALF[dtype] * out.abs() + bound), 1.02 * U * E


def scan_grad(x, delta, A, B, Cm, D, z, bias, softplus, S0, dy, dS, dtype):
    """Gradients and their bounds (parameters': of this sequence's part)."""
    T, C = x.shape
    G, per = B.shape[1], C // B.shape[1]
    dt, ds = step(delta, bias, softplus), step_slack(delta, bias, softplus, dtype)
    Bh, Ch = heads(B, C), heads(Cm, C)
    gz = torch.ones_like(x) if z is None else silu(z)
    dp = dy * gz
    ep = dp.abs() * (1.0 if z is None else act_slack(z, dtype) + 2)
    S, M, E = S0.clone(), S0.abs(), torch.zeros_like(S0)
    before, y, ey = [], torch.zeros_like(x), torch.zeros_like(x)
    dC, mC = torch.zeros(T, C, B.shape[2]).double(), torch.zeros(T, C, B.shape[2]).double()
    rel = []
    for t in range(T):
        before.append((S, M, E))
        arg = dt[t][:, None] * A
        a, off = torch.exp(arg), 3 + arg.abs() * (ds[t][:, None] + 4)
        rel.append((a, off))
        u = (dt[t] * x[t])[:, None] * Bh[t]
        E = a * (E + off * M) + u.abs() * (ds[t][:, None] + 3) + 2 * (a * M + u.abs())
        S, M = a * S + u, a * M + u.abs()
        y[t], ey[t] = (S * Ch[t]).sum(-1), ((E + (S.shape[-1] + 4) * M) * Ch[t].abs()).sum(-1)
        dC[t], mC[t] = dp[t][:, None] * S, dp[t].abs()[:, None] * (E + 2 * M) + ep[t][:, None] * M
    skip = 0 if D is None else D * x
    y = y + skip
    ey = ey + 2 * (skip if D is None else skip.abs())
    R, Mr, Er = dS.clone(), dS.abs(), torch.zeros_like(dS)
    zero = torch.zeros_like(x)
    dx, ex, dd, ed = zero.clone(), zero.clone(), zero.clone(), zero.clone()
    dB, mB = torch.zeros_like(dC), torch.zeros_like(dC)
    dA, mA = torch.zeros_like(A), torch.zeros_like(A)
    N = A.shape[1] + 6
    for t in range(T - 1, -1, -1):
        a, off = rel[t]
        g = R + dp[t][:, None] * Ch[t]
        mg = Mr + dp[t].abs()[:, None] * Ch[t].abs()
        eg = Er + ep[t][:, None] * Ch[t].abs() + 3 * mg
        v = dt[t] * x[t]
        dB[t], mB[t] = v[:, None] * g, v.abs()[:, None] * (eg + (ds[t][:, None] + 3) * mg)
        own, mown = (g * Bh[t]).sum(-1), ((eg + N * mg) * Bh[t].abs()).sum(-1)
        bown = (mg * Bh[t].abs()).sum(-1)
        R, Mr, Er = a * g, a * mg, a * (eg + (off + 1) * mg)
        Sb, Mb, Eb = before[t]
        w, ew = R * Sb, Er * Mb + Mr * Eb + 2 * Mr * Mb
        wA, ewA = (w * A).sum(-1), ((ew + N * Mr * Mb) * A.abs()).sum(-1)
        dx[t] = dt[t] * own + (0 if D is None else D * dp[t])
        ex[t] = dt[t].abs() * (mown + (ds[t] + 2) * bown) + (0 if D is None else D.abs() * (ep[t] + 2 * dp[t].abs()))
        dd[t], ed[t] = wA + x[t] * own, ewA + x[t].abs() * mown + 2 * (wA.abs() + (x[t] * own).abs())
        dA = dA + w * dt[t][:, None]
        mA = mA + (ew + (24 + ds[t][:, None]) * Mr * Mb) * dt[t].abs()[:, None]
    if softplus:
        v = delta if bias is None else delta + bias
        s = torch.sigmoid(v)
        m = delta.abs() + (0 if bias is None else bias.abs())
        ed = ed * s + dd.abs() * s * (act_slack(v, dtype) + 2 + 2 * m)
        dd = dd * s
    h = HALF[dtype]
    share = lambda m: m.unflatten(1, (G, per)).sum(2)  # noqa: E731
    grads = dict(dx=dx, ddelta=dd, dB=share(dB), dC=share(dC), dA=dA, dS0=R, dD=(dp * x).sum(0),
                 ddelta_bias=dd.sum(0))
    # sums over channels: 16 lanes, runs of a set and the sets
    many = per / 16 + 10
    bounds = dict(dx=ex, ddelta=ed, dB=share(mB + many * dB.abs()), dC=share(mC + many * dC.abs()), dA=mA, dS0=Er,
                  dD=((ep + 24 * dp.abs()) * x.abs()).sum(0), ddelta_bias=(ed + 24 * dd.abs()).sum(0))
    if z is not None:
        sg = torch.sigmoid(z)
        slope = sg + (z * sg * (1 - sg)).abs()
        grads["dz"] = dy * y * dsilu(z)
        bounds["dz"] = dy.abs() * (ey + y.abs() * (2 * act_slack(z, dtype) + 6)) * slope
    low = ("dx", "ddelta", "dB", "dC", "dz")
    return grads, {k: 1.02 * (U * b + (h if k in low else U) * grads[k].abs()) for k, b in bounds.items()}
