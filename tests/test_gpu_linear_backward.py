"""Gradients of the linear attention with a decay for each head on the GPU,
against the reverse recurrence in 64 bits within bounds that count every
rounding (tests/linear_ref.py), and against differences of the prefill."""
import math

import pytest
import torch

import linear_ref as ref
from linear_attention_recurrent_delta_amd import kdn
from test_gpu_linear import BF, F32, i32, make, state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    kdn.ensure_built()


def randn(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def check(q, k, v, la, do, S0, dS, got, spans, slots):
    """spans: rows of each sequence in tensors of one token axis; slots: their
    states (-1: skipped)."""
    dtype, H = q.dtype, do.shape[-2]
    dk, dv = q.shape[-1], v.shape[-1]
    C = 64 if dtype == BF else 32
    tokens = q.shape[0]
    want = {n: torch.zeros(tokens, H, d, dtype=torch.float64)
            for n, d in (("dq", dk), ("dk", dk), ("dv", dv))}
    mags = {n: x.clone() for n, x in want.items()}
    dg = torch.zeros(tokens, H, dtype=torch.float64)
    dgb = dg.clone()
    a = ref.decay(la, (tokens,), H)
    Q, K, V, O = ref.wide(q, H), ref.wide(k, H), ref.wide(v, H), do.cpu().double()
    longest = 0
    for rows, slot in zip(spans, slots):
        if slot < 0:
            continue
        T = rows.stop - rows.start
        longest = max(longest, T)
        zero = torch.zeros(H, dk, dv, dtype=torch.float64)
        s0 = zero if S0 is None else S0[slot].cpu().double()
        ds = zero if dS is None else dS[slot].cpu().double()
        r, m = ref.backward(Q[rows], K[rows], V[rows], a[rows], O[rows], s0, ds)
        for n in want:
            want[n][rows], mags[n][rows] = r[n], m[n]
        dg[rows] = r["dlog_alpha"]
        dgb[rows] = ref.flow_bound(r["dlog_alpha"], m, Q[rows], K[rows], C, dtype)
        if got["dS0"] is not None:
            ref.close(f"dS0[{slot}]", got["dS0"][slot], r["dS0"],
                      ref.S_bound(m["dS0"], T, dk, dtype))
    for n, x in (("dq", q), ("dk", k), ("dv", v)):
        heads = x.shape[-2]
        w = want[n].unflatten(1, (heads, -1)).sum(2)
        mg = mags[n].unflatten(1, (heads, -1)).sum(2)
        ref.close(n, got[n], w, ref.o_bound(w, mg, longest + H, dk + dv, dtype))
    if got["dlog_alpha"] is None:
        return
    if la.dim() == 1:
        w = dg.sum(0)
        h = ref.HALF[dtype]
        ref.close("dlog_alpha", got["dlog_alpha"], w, h * w.abs() + (1 + h) * dgb.sum(0))
    else:
        ref.close("dlog_alpha", got["dlog_alpha"], dg, dgb)


def check_dense(q, k, v, la, do, S0, dS, got):
    B, T = q.shape[:2]
    flat = lambda x: x.flatten(0, 1)
    fl = lambda x: x if x is None or x.dim() == 1 else flat(x)
    g = {n: (x if x is None or n == "dS0" else fl(x)) for n, x in got.items()}
    check(flat(q), flat(k), flat(v), fl(la), flat(do), S0, dS, g,
          [slice(b * T, b * T + T) for b in range(B)], list(range(B)))


@pytest.mark.parametrize("T", [1, 2, 16, 17, 32, 33, 64, 65, 100, 192, 257, 600])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_lengths(T, dtype):
    H, dk, dv = 2, 128, 128
    q, k, v, la = make((2, T), H, H, H, H, dk, dv, dtype, seed=T)
    S0, dS = state(2, H, dk, dv), state(2, H, dk, dv, seed=2)
    do = randn((2, T, H, dv), dtype, 3)
    got = kdn.linear_prefill_backward(q, k, v, do, la, S0=S0, dS_out=dS)
    check_dense(q, k, v, la, do, S0, dS, got)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gate", ["token", "head"])
@pytest.mark.parametrize("with_state", [True, False])
def test_sizes(dk, dv, dtype, gate, with_state):
    H, T = 3, 290
    q, k, v, la = make((1, T), H, H, H, H, dk, dv, dtype, gate, seed=dk + 2 * dv)
    S0 = state(1, H, dk, dv) if with_state else None
    dS = state(1, H, dk, dv, seed=2) if with_state else None
    do = randn((1, T, H, dv), dtype, 3)
    got = kdn.linear_prefill_backward(q, k, v, do, la, S0=S0, dS_out=dS)
    check_dense(q, k, v, la, do, S0, dS, got)


@pytest.mark.parametrize("Hq,Hk,Hv,H", [(1, 1, 6, 6), (6, 2, 2, 6), (2, 3, 6, 6), (6, 6, 1, 6),
                                        (1, 1, 1, 4)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gate", ["token", "head"])
def test_shared_heads_and_strides(Hq, Hk, Hv, H, dtype, gate):
    q, k, v, la = make((2, 90), Hq, Hk, Hv, H, 64, 128, dtype, gate, seed=H, fused=True)
    S0, dS = state(2, H, 64, 128), state(2, H, 64, 128, seed=2)
    do = randn((2, 90, H, 128), dtype, 3)
    got = kdn.linear_prefill_backward(q, k, v, do, la, S0=S0, dS_out=dS)
    check_dense(q, k, v, la, do, S0, dS, got)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [-math.inf, -1e30, -20.0, 0.0])
@pytest.mark.parametrize("share", [0.03, 0.5, 1.0])
def test_strong_decays_and_resets(dtype, value, share):
    q, k, v, la = make((1, 290), 2, 2, 2, 2, 64, 64, dtype, seed=7)
    g = torch.Generator(device="cuda").manual_seed(8)
    hit = torch.rand(la.shape, generator=g, device="cuda") < share
    la = torch.where(hit, torch.full_like(la, value), la)
    S0, dS = state(1, 2, 64, 64), state(1, 2, 64, 64, seed=2)
    do = randn((1, 290, 2, 64), dtype, 3)
    got = kdn.linear_prefill_backward(q, k, v, do, la, S0=S0, dS_out=dS)
    check_dense(q, k, v, la, do, S0, dS, got)
    if value < -1000:
        assert not got["dlog_alpha"][hit].any(), "nothing passes a reset"


LENGTHS = [[1], [0], [5, 0, 64, 1, 129, 0], [1] * 9, [300, 2, 500, 65], [0, 0, 700, 0]]


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block", [64, 256])
@pytest.mark.parametrize("Hk", [2, 1])
def test_packed(lengths, dtype, block, Hk):
    N, H, tail = len(lengths), 2, 3
    total = sum(lengths) + tail
    slots = [(n * 5 + 2) % (N + 6) for n in range(N)] if (N + 6) % 5 else list(range(N))
    if N > 3:
        slots[1] = -1
        slots[3] = N + 6
    q, k, v, la = make((total,), H, Hk, H, H, 64, 64, dtype, seed=N)
    do = randn((total, H, 64), dtype, 3)
    for x in (q, k, v, la, do):
        x[total - tail:] = float("nan")
    S0, dS = state(N + 6, H, 64, 64), state(N + 6, H, 64, 64, seed=2)
    t = kdn.sequence_tables(i32(lengths), total, block, slots=i32(slots))
    ends = torch.tensor(lengths).cumsum(0).tolist()
    spans = [slice(e - n, e) for e, n in zip(ends, lengths)]
    if N > 3:
        q[spans[1]] = float("nan")
        do[spans[3]] = float("nan")
    got = kdn.linear_prefill_backward(q, k, v, do, la, S0=S0, dS_out=dS, tables=t)
    live = [s if 0 <= s < N + 6 else -1 for s in slots]
    for x in (q, k, v, la, do):
        x[total - tail:] = 0
    if N > 3:
        q[spans[1]] = 0
        do[spans[3]] = 0
    check(q, k, v, la, do, S0, dS, got, spans, live)
    for p in set(range(N + 6)) - set(live):
        assert not got["dS0"][p].any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_packed_many_blocks(dtype):
    """More workgroups than run at once: the blocks are taken longest first."""
    lengths, H, tail = [(23 * n * n + 5 * n) % 211 for n in range(44)], 6, 4
    total = sum(lengths) + tail
    q, k, v, la = make((total,), 2, 3, H, H, 64, 64, dtype, seed=44)
    do = randn((total, H, 64), dtype, 3)
    S0, dS = state(44, H, 64, 64), state(44, H, 64, 64, seed=2)
    t = kdn.sequence_tables(i32(lengths), total, 64)
    assert t.blocks.shape[0] * H > 256
    got = kdn.linear_prefill_backward(q, k, v, do, la, S0=S0, dS_out=dS, tables=t)
    ends = torch.tensor(lengths).cumsum(0).tolist()
    check(q, k, v, la, do, S0, dS, got, [slice(e - n, e) for e, n in zip(ends, lengths)],
          list(range(44)))


def test_packed_many_states():
    """So many states that a workgroup joins the whole of one."""
    lengths, H = [(31 * n) % 140 if n % 7 else 0 for n in range(260)], 4
    total = sum(lengths)
    q, k, v, la = make((total,), H, H, H, H, 64, 128, BF, seed=45)
    do = randn((total, H, 128), BF, 3)
    S0, dS = state(260, H, 64, 128), state(260, H, 64, 128, seed=2)
    t = kdn.sequence_tables(i32(lengths), total, 64)
    got = kdn.linear_prefill_backward(q, k, v, do, la, S0=S0, dS_out=dS, tables=t)
    ends = torch.tensor(lengths).cumsum(0).tolist()
    check(q, k, v, la, do, S0, dS, got, [slice(e - n, e) for e, n in zip(ends, lengths)],
          list(range(260)))


def test_wanted_outputs_only():
    """Without d log_alpha and dS0, into given tensors, the same bits."""
    H, T = 2, 300
    q, k, v, la = make((2, T), H, H, H, H, 64, 64, BF, seed=1)
    do = randn((2, T, H, 64), BF, 2)
    want = kdn.linear_prefill_backward(q, k, v, do, la)
    out = {n: torch.full_like(want[n], 7.0) for n in ("dq", "dk", "dv")}
    out.update(dlog_alpha=None, dS0=None)
    got = kdn.linear_prefill_backward(q, k, v, do, la, out=out)
    assert got is out
    for n in ("dq", "dk", "dv"):
        assert torch.equal(got[n], want[n])
    again = kdn.linear_prefill_backward(q, k, v, do, la)
    for n in want:
        assert torch.equal(again[n], want[n]), n


@pytest.mark.parametrize("dtype", [BF, F32])
def test_packed_without_a_pool(dtype):
    """No state anywhere: every sequence counts, whatever its slot, in the
    gradients and in the prefill."""
    lengths, H = [70, 300, 5], 2
    total = sum(lengths)
    q, k, v, la = make((total,), H, H, H, H, 64, 64, dtype, seed=4)
    do = randn((total, H, 64), dtype, 3)
    t = kdn.sequence_tables(i32(lengths), total, 128, slots=i32([9, 3, 0]))
    got = kdn.linear_prefill_backward(q, k, v, do, la, tables=t)
    assert got["dS0"].shape == (3, H, 64, 64)
    spans = [slice(0, 70), slice(70, 370), slice(370, 375)]
    check(q, k, v, la, do, None, None, got, spans, [0, 1, 2])
    o, S = kdn.linear_prefill(q, k, v, la, tables=t, out=(torch.full_like(v, 7.0), None))
    plain = kdn.sequence_tables(i32(lengths), total, 128)
    assert S is None and torch.equal(o, kdn.linear_prefill(q, k, v, la, tables=plain)[0])


def test_no_tokens():
    z = lambda *s: torch.zeros(s, dtype=BF, device="cuda")
    dS = state(3, 2, 64, 64)
    got = kdn.linear_prefill_backward(z(3, 0, 2, 64), z(3, 0, 2, 64), z(3, 0, 2, 64), z(3, 0, 2, 64),
                                      z(3, 0, 2), dS_out=dS)
    assert torch.equal(got["dS0"], dS) and got["dq"].shape == (3, 0, 2, 64)
    got = kdn.linear_prefill_backward(z(3, 0, 2, 64), z(3, 0, 2, 64), z(3, 0, 2, 64), z(3, 0, 2, 64),
                                      torch.zeros(2, device="cuda"))
    assert not got["dlog_alpha"].any() and not got["dS0"].any()
    t = kdn.sequence_tables(i32([]), 5, 64)
    got = kdn.linear_prefill_backward(z(5, 2, 64), z(5, 2, 64), z(5, 2, 64), z(5, 2, 64), z(5, 2),
                                      tables=t)
    assert all(not got[n].any() for n in ("dq", "dk", "dv", "dlog_alpha"))


@pytest.mark.parametrize("gate", ["token", "head"])
def test_against_differences(gate):
    """L = <o, do> + <S, dS> of the float32 prefill: linear in q, k, v and S0
    each, so a central difference is exact up to rounding at any step; for the
    log-decays a small step, whose third-order rest is below 1e-4 of the
    directional derivative's terms."""
    H, T, d = 3, 200, 64
    q, k, v, la = make((1, T), H, H, H, H, d, d, F32, gate, seed=5)
    S0, dS = state(1, H, d, d), state(1, H, d, d, seed=2)
    do = randn((1, T, H, d), F32, 3)

    def loss(**kw):
        x = dict(q=q, k=k, v=v, la=la, S0=S0)
        x.update(kw)
        o, S = kdn.linear_prefill(x["q"], x["k"], x["v"], x["la"], S0=x["S0"])
        return (o.double() * do.double()).sum().item() + (S.double() * dS.double()).sum().item()

    got = kdn.linear_prefill_backward(q, k, v, do, la, S0=S0, dS_out=dS)
    size = math.sqrt(sum((x.double() ** 2).sum().item() for x in (do, dS)))
    for n, x, step, grad in (("q", q, 1.0, "dq"), ("k", k, 1.0, "dk"), ("v", v, 1.0, "dv"),
                             ("S0", S0, 1.0, "dS0"), ("la", la, 1e-2, "dlog_alpha")):
        way = randn(x.shape, F32, 11)
        if n == "la":
            way = way * x.abs()           # stays a decay
        diff = (loss(**{n: x + step * way}) - loss(**{n: x - step * way})) / (2 * step)
        formula = (got[grad].double() * way.double()).sum().item()
        scale = got[grad].double().norm().item() * way.double().norm().item()
        print(f"    {n}: difference {diff:.6g}, formula {formula:.6g}, scale {scale:.3g}, {size:.3g}")
        assert abs(diff - formula) <= 2e-4 * scale


def test_captured_training_step():
    """Prefill and gradients captured into one graph and replayed on new inputs,
    eager work between, each replay as the eager call."""
    B, T, H, d = 1, 600, 2, 64
    x = make((B, T), H, 1, H, H, d, d, BF, "head", seed=1)
    do = randn((B, T, H, d), BF, 2)

    def step():
        o, S = kdn.linear_prefill(*x)
        g = kdn.linear_prefill_backward(x[0], x[1], x[2], do, x[3])
        return [o, S] + [g[n] for n in ("dq", "dk", "dv", "dlog_alpha", "dS0")]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(3):
        for y, new in zip(x, make((B, T), H, 1, H, H, d, d, BF, "head", seed=20 + i)):
            y.copy_(new)
        do.copy_(randn(do.shape, BF, 30 + i))
        want = [y.clone() for y in step()]
        torch.cuda.synchronize()
        for y in outs:
            y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
