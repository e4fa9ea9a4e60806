"""Convolution, scan and norms on the GPU in calls as programs make them: a layer of them
with shared tables and pools, captured steps, two streams at once, far addresses."""
import math

import pytest
import torch

import around_ref as ref
import test_gpu_conv as tc
import test_gpu_norm as tn
import test_gpu_scan as ts
from linear_attention_recurrent_delta_amd import kdn
from test_gpu_conv import BF, F32, i32, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    kdn.ensure_built()


def layer(total, H, d, S, pool, dtype):
    """Parameters, states and inputs of a layer: stream, convolution over x, a scan of its
    output gated by z, the heads' norm, the stream's norm."""
    C = H * d
    p = dict(w_res=1 + randn((C,), F32, 1, size=0.2), scale=randn((C,), F32, 2), w=randn((C, 4), F32, 3, size=0.5),
             b=randn((C,), F32, 4, size=0.1), A=-torch.rand(C, S, generator=tc.gen(5)).mul(S).add(0.1).cuda(),
             D=randn((C,), F32, 6), bias=randn((C,), F32, 7) - 3, w_head=1 + randn((H, d), F32, 8, size=0.2))
    s = dict(conv=randn((pool, 3, C), dtype, 9), scan=randn((pool, C, S), F32, 10))
    x = dict(x=randn((total, C), dtype, 11), res=randn((total, C), F32, 12), zx=randn((total, 2 * C + 2 * S + 8), dtype, 13),
             delta=randn((total, C), dtype, 14))
    return p, s, x


def run_layer(p, s, x, H, d, S, tables, out, ws=None):
    """One step; every output in `out`, states in place."""
    C = H * d
    n = x["x"].shape[0]
    kdn.residual_norm(x["x"], x["res"], p["w_res"], scale=p["scale"], out=(out["y"], out["h"]))
    kdn.causal_conv(out["y"], p["w"], p["b"], state0=s["conv"], tables=tables, out=(out["conv"], s["conv"]))
    z, B, Cm = x["zx"][:, :C], x["zx"][:, C:C + S].view(n, 1, S), x["zx"][:, C + S:C + 2 * S].view(n, 1, S)
    kdn.selective_scan(out["conv"], x["delta"], p["A"], B, Cm, D=p["D"], z=z, delta_bias=p["bias"], S0=s["scan"],
                       tables=tables, out=(out["scan"], s["scan"]), **({} if ws is None else dict(workspace=ws)))
    gate = x["zx"][:, C:2 * C].unflatten(-1, (H, d))
    kdn.gated_norm(out["scan"].view(n, H, d), p["w_head"], gate, out=out["o"].view(n, H, d))
    return out


def outputs(total, C, dtype):
    new = lambda t: torch.full((total, C), 7.0, dtype=t, device="cuda")  # noqa: E731
    return dict(y=new(dtype), h=new(F32), conv=new(dtype), scan=new(dtype), o=new(dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_layer_on_a_packed_batch_and_its_next_tokens(dtype):
    """Every stage against its 64-bit form on what the stage before gave; then two decode
    steps from the same pools."""
    lengths, slots, H, d, S, behind = [30, 0, 170, 1, 64], [3, 6, 0, 5, 1], 2, 24, 16, 4
    total, C, pool, eps = sum(lengths) + behind, H * d, 8, torch.tensor(1e-5).item()
    p, s, x = layer(total, H, d, S, pool, dtype)
    before = {k: v.clone() for k, v in s.items()}
    t = kdn.sequence_tables(i32(lengths), total, 64, slots=i32(slots))
    out = run_layer(p, s, x, H, d, S, t, outputs(total, C, dtype))
    ends = torch.tensor(lengths).cumsum(0).tolist()
    spans = [slice(e - n, e) for e, n in zip(ends, lengths)]
    W = ref.wide
    wy, wh, by, bh = ref.residual(W(x["x"]), W(x["res"]), W(p["w_res"]), W(p["scale"]), eps, dtype, F32)
    ref.close("y", out["y"], wy, by)
    ref.close("h", out["h"], wh, bh)
    tc.check_forward(out["y"], p["w"], p["b"], before["conv"], "silu", out["conv"], s["conv"], spans, slots)
    z, B, Cm = x["zx"][:, :C], x["zx"][:, C:C + S].view(total, 1, S), x["zx"][:, C + S:C + 2 * S].view(total, 1, S)
    args, kw = (out["conv"], x["delta"], p["A"], B, Cm), dict(D=p["D"], z=z, delta_bias=p["bias"])
    ts.check(args, kw, before["scan"], out["scan"], s["scan"], spans, slots)
    gate = x["zx"][:, C:2 * C].unflatten(-1, (H, d))
    wo, bo = ref.gated(W(out["scan"].view(total, H, d)), W(p["w_head"]), W(gate), eps, "norm_gate", "silu", dtype)
    ref.close("o", out["o"].view(total, H, d), wo, bo)
    assert (out["conv"][ends[-1]:] == 7).all() and (out["scan"][ends[-1]:] == 7).all()
    # the sequences with tokens go on, padded to six rows
    rows = i32([3, -1, 0, 5, 1, 8])
    live = [(0, 3), (2, 0), (3, 5), (4, 1)]
    for step in range(2):
        was = {k: v.clone() for k, v in s.items()}
        tok, zz, delta = randn((6, C), dtype, 20 + step), randn((6, C), dtype, 30 + step), randn((6, C), dtype, 40 + step)
        bc = randn((6, 2, S), dtype, 50 + step)
        u = kdn.causal_conv_decode(tok, p["w"], s["conv"], p["b"], slots=rows)
        one = (u, delta, p["A"], bc[:, :1], bc[:, 1:])
        y = kdn.selective_decode(*one, s["scan"], D=p["D"], z=zz, delta_bias=p["bias"], slots=rows)
        for r, slot in live:
            tc.check_forward(tok[r:r + 1], p["w"], p["b"], was["conv"], "silu", u[r:r + 1], s["conv"], [slice(0, 1)], [slot])
            ts.check(one, dict(D=p["D"], z=zz, delta_bias=p["bias"]), was["scan"], y, s["scan"], [slice(r, r + 1)], [slot])
        assert not y[1].any() and not y[5].any()
        rest = [q for q in range(pool) if q not in [b for _, b in live]]
        assert torch.equal(s["scan"][rest], was["scan"][rest]) and torch.equal(s["conv"][rest], was["conv"][rest])


def gradients(p, s, x, c, H, d, S, tables, g, ws):
    """The layer's backward pass from d_o and d_h, into g."""
    C, n = H * d, x["x"].shape[0]
    z, B, Cm = x["zx"][:, :C], x["zx"][:, C:C + S].view(n, 1, S), x["zx"][:, C + S:C + 2 * S].view(n, 1, S)
    gate = x["zx"][:, C:2 * C].unflatten(-1, (H, d))
    kdn.gated_norm_backward(c["scan"].view(n, H, d), p["w_head"], x["d_o"].view(n, H, d), gate, out=g["norm"], workspace=ws)
    kdn.selective_scan_backward(c["conv"], x["delta"], p["A"], B, Cm, g["norm"]["dx"].view(n, C), D=p["D"], z=z,
                                delta_bias=p["bias"], S0=s["scan"], dS_out=x["dS"], tables=tables, out=g["scan"], workspace=ws)
    kdn.causal_conv_backward(c["y"], p["w"], g["scan"]["dx"], p["b"], state0=s["conv"], tables=tables, out=g["conv"], workspace=ws)
    kdn.residual_norm_backward(x["x"], c["h"], p["w_res"], g["conv"]["dx"], x["d_h"], scale=p["scale"], out=g["res"], workspace=ws)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_captured_training_steps(dtype):
    """Tables, forward and backward of a layer on a packed batch in two graphs that share one
    workspace, replayed on new lengths and inputs with eager work between."""
    N, H, d, S, cap, pool = 4, 2, 24, 16, 700, 6
    C = H * d
    p, s, x = layer(cap, H, d, S, pool, dtype)
    x.update(d_o=randn((cap, C), dtype, 60), d_h=randn((cap, C), F32, 61), dS=randn((pool, C, S), F32, 62))
    lengths, slots = i32([1, 1, 1, 1]), i32([0, 1, 2, 3])
    t = kdn.sequence_tables(lengths, cap, 128, slots=slots)
    out = outputs(cap, C, dtype)
    like, par = lambda: torch.zeros(cap, C, dtype=dtype, device="cuda"), torch.zeros_like  # noqa: E731
    g = dict(norm=dict(dx=like().view(cap, H, d), dgate=like().view(cap, H, d), dweight=par(p["w_head"])),
             scan=dict(dx=like(), ddelta=like(), dz=like(), dB=torch.zeros(cap, 1, S, dtype=dtype, device="cuda"),
                       dC=torch.zeros(cap, 1, S, dtype=dtype, device="cuda"), dA=par(p["A"]), dD=par(p["D"]),
                       ddelta_bias=par(p["bias"]), dS0=par(s["scan"])),
             conv=dict(dx=like(), dweight=par(p["w"]), dbias=par(p["b"]), dstate0=par(s["conv"])),
             res=dict(dx=like(), dresidual=torch.zeros(cap, C, device="cuda"), dweight=par(p["w_res"]), dscale=par(p["scale"])))
    flat = [v for k in g for v in g[k].values()] + list(out.values()) + list(s.values())
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def forward():
        kdn.sequence_tables(lengths, cap, 128, slots=slots, out=t)
        run_layer(p, s, x, H, d, S, t, out, ws)

    def backward():
        gradients(p, s, x, out, H, d, S, t, g, ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        forward()
        backward()
    torch.cuda.synchronize()
    graphs = []
    for f in (forward, backward):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    for i, (ln, sl) in enumerate([([5, 0, 300, 64], [5, 1, 0, 2]), ([200, 200, 200, 100], [3, 2, 1, 0]),
                                  ([1, 2, 3, 4], [0, -1, 4, 5]), ([0, 0, 0, 0], [0, 1, 2, 3])]):
        for k, v in x.items():
            v.copy_(randn(v.shape, v.dtype, 80 + i))
        lengths.copy_(i32(ln))
        slots.copy_(i32(sl))
        start = {k: v.clone() for k, v in s.items()}

        def reset():
            for v in flat:
                v.zero_()
            for k, v in start.items():
                s[k].copy_(v)

        reset()
        forward()
        backward()
        torch.cuda.synchronize()
        want = [v.clone() for v in flat]
        for again in range(2):
            reset()
            ws.fill_(255)
            for graph in graphs:
                graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(flat, want):
                assert torch.equal(a, b)


def test_captured_decode():
    """A padded batch's tokens in one graph; slots and inputs change between the replays."""
    N, C, S, pool = 5, 70, 16, 8
    (x, delta, A, B, Cm), kw = ts.case((N,), C, S, 1, BF, seed=1)
    w, b = tc.params(C, 4)
    conv, scan, slots = randn((pool, 3, C), BF, 2), randn((pool, C, S), F32, 3), i32([0, 1, 2, 3, 4])
    u, y = torch.zeros(N, C, dtype=BF, device="cuda"), torch.zeros(N, C, dtype=BF, device="cuda")

    def step():
        kdn.causal_conv_decode(x, w, conv, b, slots=slots, y=u)
        kdn.selective_decode(u, delta, A, B, Cm, scan, slots=slots, y=y, **kw)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, sl in enumerate([[7, 6, 5, -1, 0], [0, 8, 1, 2, 3], [-1] * 5, [1, 2, 3, 4, 5]]):
        x.copy_(randn(x.shape, BF, 20 + i))
        slots.copy_(i32(sl))
        keep = [v.clone() for v in (conv, scan, u, y)]
        step()
        torch.cuda.synchronize()
        want = [v.clone() for v in (conv, scan, u, y)]
        for again in range(2):
            for v, k in zip((conv, scan, u, y), keep):
                v.copy_(k)
            graph.replay()
            torch.cuda.synchronize()
            for a, c in zip((conv, scan, u, y), want):
                assert torch.equal(a, c)


def test_two_calls_at_once():
    """Forward and gradients on two streams, each with workspaces of its own."""
    C, S, T = 256, 16, 1500
    data = [ts.case((1, T), C, S, 1, BF, seed=s) for s in (1, 2)]
    w, b = tc.params(C, 4)
    dy = [randn((1, T, C), BF, s) for s in (3, 4)]

    def step(i, stream=None):
        (x, delta, A, B, Cm), kw = data[i]
        u, _ = kdn.causal_conv(x, w, b, stream=stream)
        y, S_ = kdn.selective_scan(u, delta, A, B, Cm, stream=stream, **kw)
        o = kdn.gated_norm(y.view(1, T, 4, 64), wn, stream=stream)
        g = kdn.selective_scan_backward(u, delta, A, B, Cm, dy[i], stream=stream, **kw)
        c = kdn.causal_conv_backward(x, w, g["dx"], b, stream=stream)
        n = kdn.gated_norm_backward(y.view(1, T, 4, 64), wn, dy[i].view(1, T, 4, 64), stream=stream)
        yy, h = kdn.residual_norm(u, x, wr, stream=stream)
        r = kdn.residual_norm_backward(u, h, wr, dy[i], stream=stream)
        return [u, y, S_, o, yy, h] + [v for q in (g, c, n, r) for v in q.values() if v is not None]

    wn, wr = 1 + randn((64,), F32, 8, size=0.1), 1 + randn((C,), F32, 9, size=0.1)
    want = [step(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        got = [step(i, s) for i, s in enumerate(streams)]
        for s in streams:
            s.synchronize()
        for a, c in zip(want, got):
            for y, z in zip(a, c):
                assert torch.equal(y, z)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sequences_may_share_a_state_that_is_only_read(dtype):
    lengths, slots, C, S = [70, 200, 0, 5, 130], [2, 2, 2, 0, 2], 24, 16
    total = sum(lengths)
    args, kw = ts.case((total,), C, S, 1, dtype, seed=3)
    w, b = tc.params(C, 4)
    t = kdn.sequence_tables(i32(lengths), total, 64, slots=i32(slots))
    S0, conv0 = randn((3, C, S), F32, 4), randn((3, 3, C), dtype, 5)
    keep = S0.clone(), conv0.clone()
    ends = torch.tensor(lengths).cumsum(0).tolist()
    spans = [slice(e - n, e) for e, n in zip(ends, lengths)]
    y, none = kdn.selective_scan(*args, S0=S0, tables=t, out=(torch.empty_like(args[0]), None), **kw)
    u, no = kdn.causal_conv(args[0], w, b, state0=conv0, tables=t, out=(torch.empty_like(args[0]), None))
    assert none is None and no is None and torch.equal(S0, keep[0]) and torch.equal(conv0, keep[1])
    ts.check(args, kw, S0, y, None, spans, slots)
    tc.check_forward(args[0], w, b, conv0, "silu", u, None, spans, slots)


def far_rows(n, C, stride, dtype, seed):
    """n rows of C values, `stride` elements apart, of which nothing else is touched."""
    buf = torch.empty((n - 1) * stride + C, dtype=dtype, device="cuda")
    x = buf.as_strided((n, C), (stride, 1))
    x.copy_(randn((n, C), dtype, seed))
    return x


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_far_apart(dtype):
    """Offsets past 2^32 bytes."""
    n, C = 40, 48
    x = far_rows(n, C, (1 << 26) + 1, dtype, 1)
    assert (n - 1) * x.stride(0) * x.element_size() > 1 << 32
    w, b = tc.params(C, 4)
    same = x.contiguous()
    dy = randn((n, C), dtype, 3)
    for a, c in zip(kdn.causal_conv(x[None], w, b), kdn.causal_conv(same[None], w, b)):
        assert torch.equal(a, c)
    a, c = kdn.causal_conv_backward(x[None], w, dy[None], b), kdn.causal_conv_backward(same[None], w, dy[None], b)
    assert all(torch.equal(a[k], c[k]) for k in a)
    S, S2 = randn((n, 3, C), dtype, 4), randn((n, 3, C), dtype, 4)
    assert torch.equal(kdn.causal_conv_decode(x, w, S, b), kdn.causal_conv_decode(same, w, S2, b)) and torch.equal(S, S2)
    wn = torch.ones(24, device="cuda")
    heads = lambda v: v.unflatten(-1, (2, 24))  # noqa: E731
    assert torch.equal(kdn.gated_norm(heads(x), wn, heads(same)), kdn.gated_norm(heads(same), wn, heads(x)))
    wr = torch.ones(C, device="cuda")
    for a, c in zip(kdn.residual_norm(x, same, wr), kdn.residual_norm(same, x, wr)):
        assert torch.equal(a, c)
    del x
    torch.cuda.empty_cache()
    stride = (1 << 25) - 1
    n = 70 if dtype is BF else 40
    args, kw = ts.case((1, n), C, 16, 1, dtype, seed=5)
    x = far_rows(n, C, stride, dtype, 6)[None]
    same = (x.contiguous(),) + args[1:]
    assert (n - 1) * stride * x.element_size() > 1 << 32
    dy = randn((1, n, C), dtype, 7)
    for a, c in zip(kdn.selective_scan(x, *args[1:], **kw), kdn.selective_scan(*same, **kw)):
        assert torch.equal(a, c)
    a, c = kdn.selective_scan_backward(x, *args[1:], dy, **kw), kdn.selective_scan_backward(*same, dy, **kw)
    assert all(torch.equal(a[k], c[k]) for k in a)


def test_far_states():
    """States past 2^32 bytes of a pool."""
    C, S, pool = 4096, 16, 17000
    big = torch.zeros((pool, C, S), device="cuda")
    assert big.numel() * 4 > 1 << 32
    lengths, slots = [3, 20], [16999, 5]
    args, kw = ts.case((23,), C, S, 1, BF, seed=1)
    t = kdn.sequence_tables(i32(lengths), 23, kdn.selective_block(23, 2, C, S), slots=i32(slots))
    y, _ = kdn.selective_scan(*args, S0=big, tables=t, **kw)
    small = torch.zeros((2, C, S), device="cuda")
    t2 = kdn.sequence_tables(i32(lengths), 23, kdn.selective_block(23, 2, C, S), slots=i32([1, 0]))
    y2, _ = kdn.selective_scan(*args, S0=small, tables=t2, **kw)
    assert torch.equal(y, y2) and torch.equal(big[slots], small[[1, 0]])
    assert int(big.count_nonzero()) == int(small.count_nonzero())
    one = [v if i == 2 else v[:2] for i, v in enumerate(args)]
    k2 = dict(kw, z=kw["z"][:2])
    a = kdn.selective_decode(*one, big, slots=i32(slots), **k2)
    assert torch.equal(a, kdn.selective_decode(*one, small, slots=i32([1, 0]), **k2)) and torch.equal(big[slots], small[[1, 0]])
    d = kdn.selective_scan_backward(*args, randn((23, C), BF, 2), S0=big, tables=t, **kw)
    d2 = kdn.selective_scan_backward(*args, randn((23, C), BF, 2), S0=small, tables=t2, **kw)
    assert torch.equal(d["dS0"][slots], d2["dS0"][[1, 0]])
    for k in ("dx", "dA", "dB", "dC"):
        assert torch.equal(d[k], d2[k])


@pytest.mark.parametrize("N", [65, 300])
def test_many_short_sequences(N):
    """More blocks than lanes rank, most of a token or none; rows of one class of length."""
    g = tc.gen(N)
    lengths = torch.randint(0, 4, (N,), generator=g).tolist()
    lengths[N // 2] = 90
    total, C, S = sum(lengths), 160, 8
    args, kw = ts.case((total,), C, S, 1, F32, seed=2)
    S0 = randn((N, C, S), F32, 3)
    ends = torch.tensor(lengths).cumsum(0).tolist()
    spans = [slice(e - n, e) for e, n in zip(ends, lengths)]
    for block in (64, kdn.selective_block(total, N, C, S), 1 << 20):
        t = kdn.sequence_tables(i32(lengths), total, block, slots=i32(list(range(N))))
        y, last = kdn.selective_scan(*args, S0=S0, tables=t, out=(torch.empty_like(args[0]), torch.empty_like(S0)), **kw)
        ts.check(args, kw, S0, y, last, spans, range(N))
        dy = randn((total, C), F32, 4)
        d = kdn.selective_scan_backward(*args, dy, S0=S0, tables=t, **kw)
        ts.check_grad(args, kw, S0, dy, None, d, spans, range(N))
