"""Selective state space scan on the GPU against its 64-bit recurrence: prefill (dense,
packed, slices, states), single tokens, gradients."""
import math

import pytest
import torch

import around_ref as ref
from linear_attention_recurrent_delta_amd import kdn
from test_gpu_conv import BF, F32, gen, i32, randn

pytestmark = pytest.mark.gpu
GRADS = ("dx", "ddelta", "dz", "dB", "dC", "dA", "dD", "ddelta_bias", "dS0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    kdn.ensure_built()


def case(lead, C, S, G, dtype, seed=0, z=True, skip=True, bias=True):
    """x, delta, A, B, C and the keyword arguments of a call."""
    A = -torch.rand(C, S, generator=gen(seed)).mul(2 * S).add(0.1).cuda()
    kw = dict(D=randn((C,), F32, seed + 1) if skip else None, z=randn(lead + (C,), dtype, seed + 2) if z else None,
              delta_bias=randn((C,), F32, seed + 3) - 3 if bias else None)
    return (randn(lead + (C,), dtype, seed + 4), randn(lead + (C,), dtype, seed + 5), A,
            randn(lead + (G, S), dtype, seed + 6), randn(lead + (G, S), dtype, seed + 7)), kw


def wide(args, kw, rows):
    """One sequence's rows in 64 bits."""
    x, delta, A, B, C = args
    cut = lambda v: None if v is None else ref.wide(v[rows])  # noqa: E731
    return (cut(x), cut(delta), ref.wide(A), cut(B), cut(C), ref.wide(kw["D"]), cut(kw["z"]),
            ref.wide(kw["delta_bias"]), kw.get("softplus", True))


def state(args, S0, slot):
    return torch.zeros(args[2].shape).double() if S0 is None else ref.wide(S0[slot])


def check(args, kw, S0, y, S, spans, slots):
    for rows, slot in zip(spans, slots):
        wy, wS, by, bS = ref.scan(*wide(args, kw, rows), state(args, S0, slot), args[0].dtype)
        ref.close("y", y[rows], wy, by)
        if S is not None:
            ref.close("S", S[slot], wS, bS)


def flat(args, kw):
    """A dense batch's tensors as rows."""
    n = args[0].shape[0] * args[0].shape[1]
    f = lambda v: None if v is None else v.reshape((n,) + v.shape[2:])  # noqa: E731
    return tuple(v if i == 2 else f(v) for i, v in enumerate(args)), dict(kw, z=f(kw["z"]))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("S", [8, 16, 32])
@pytest.mark.parametrize("T", [1, 3, 4, 15, 16, 17, 64, 65, 128, 129, 200])
def test_lengths(dtype, S, T):
    B, C = 2, 20
    args, kw = case((B, T), C, S, 1, dtype, seed=T)
    S0 = randn((B, C, S), F32, 9)
    y, last = kdn.selective_scan(*args, S0=S0, **kw)
    spans = [slice(n * T, n * T + T) for n in range(B)]
    a, k = flat(args, kw)
    check(a, k, S0, y.view(-1, C), last, spans, [0, 1])
    keep = S0.clone()
    y2, same = kdn.selective_scan(*args, S0=keep, out=(torch.empty_like(y), keep), **kw)
    assert same is keep and torch.equal(keep, last) and torch.equal(y, y2)
    y3, none = kdn.selective_scan(*args, S0=S0, out=(torch.empty_like(y), None), **kw)
    assert none is None and torch.equal(y, y3)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C,G", [(1, 1), (7, 1), (16, 1), (17, 1), (48, 3), (130, 2), (300, 1), (34, 34)])
@pytest.mark.parametrize("z,skip,bias", [(True, True, True), (False, False, False)])
def test_channels(dtype, C, G, z, skip, bias):
    T, S = 70, 16
    args, kw = case((1, T), C, S, G, dtype, seed=C, z=z, skip=skip, bias=bias)
    y, last = kdn.selective_scan(*args, **kw)
    a, k = flat(args, kw)
    check(a, k, None, y[0], last, [slice(0, T)], [0])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_without_softplus(dtype):
    args, kw = case((1, 90), 24, 16, 1, dtype, seed=1)
    args = (args[0], (args[1].float().abs() * 0.1).to(dtype)) + args[2:]
    kw["delta_bias"] = kw["delta_bias"].abs() * 0.01
    y, last = kdn.selective_scan(*args, softplus=False, **kw)
    a, k = flat(args, dict(kw, softplus=False))
    check(a, k, None, y[0], last, [slice(0, 90)], [0])
    S, pool = torch.zeros(1, 24, 16, device="cuda"), None
    for t in range(3):
        step = [v if i == 2 else v[:, t] for i, v in enumerate(args)]
        out = kdn.selective_decode(*step, S, softplus=False, D=kw["D"], z=kw["z"][:, t], delta_bias=kw["delta_bias"])
    _, w, _, b = ref.scan(*wide(a, k, slice(0, 3)), torch.zeros(24, 16).double(), dtype)
    ref.close("S", S[0], w, b)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("S", [8, 16, 32])
def test_cut_sequences(dtype, S):
    """A few channels and many tokens: blocks, their joins, and the same bits again."""
    B, T, C = 2, 2333, 33
    args, kw = case((B, T), C, S, 1, dtype, seed=S)
    S0 = randn((B, C, S), F32, 9)
    assert kdn.load().kdn_selective_scan_workspace_size(kdn.DTYPES[dtype], B, T, C, S, 1, None, None) > 0
    y, last = kdn.selective_scan(*args, S0=S0, **kw)
    a, k = flat(args, kw)
    check(a, k, S0, y.view(-1, C), last, [slice(0, T), slice(T, 2 * T)], [0, 1])
    keep = S0.clone()
    y2, _ = kdn.selective_scan(*args, S0=keep, out=(torch.empty_like(y), keep), **kw)
    assert torch.equal(y, y2) and torch.equal(keep, last)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C,G,S,more,odd", [(64, 1, 16, 8, 0), (50, 2, 16, 3, 1), (33, 1, 8, 5, 3), (40, 1, 32, 1, 2)])
def test_slices(dtype, C, G, S, more, odd):
    """Everything as slices of one projection's rows, at any element: the same bits."""
    B, T = 2, 75
    args, kw = case((B, T), C, S, G, dtype, seed=C)
    parts = [args[0], kw["z"], args[1], args[3].flatten(-2), args[4].flatten(-2)]
    row = sum(p.shape[-1] for p in parts) + more
    buf = torch.full((B * T * row + odd + 8,), math.nan, dtype=dtype, device="cuda")
    both, at, views = buf[odd:odd + B * T * row].view(B, T, row), 0, []
    for p in parts:
        both[..., at:at + p.shape[-1]] = p
        views.append(both[..., at:at + p.shape[-1]])
        at += p.shape[-1]
    cut = (views[0], views[2], args[2], views[3].unflatten(-1, (G, S)), views[4].unflatten(-1, (G, S)))
    kw2 = dict(kw, z=views[1])
    assert not any(v.is_contiguous() for i, v in enumerate(cut) if i != 2)
    for a, b in zip(kdn.selective_scan(*args, **kw), kdn.selective_scan(*cut, **kw2)):
        assert torch.equal(a, b)
    dy = randn((B, T, C), dtype, 8)
    a, b = kdn.selective_scan_backward(*args, dy, **kw), kdn.selective_scan_backward(*cut, dy, **kw2)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    S1, S2 = randn((B, C, S), F32, 5), randn((B, C, S), F32, 5)
    tok = lambda v: [w if i == 2 else w[:, 3] for i, w in enumerate(v)]  # noqa: E731
    a = kdn.selective_decode(*tok(args), S1, **dict(kw, z=kw["z"][:, 3]))
    b = kdn.selective_decode(*tok(cut), S2, **dict(kw2, z=views[1][:, 3]))
    assert torch.equal(a, b) and torch.equal(S1, S2)


LENGTHS = [([70, 1, 200, 0, 3, 64, 2], 5, 64), ([1, 1, 1, 1], 0, 64), ([0, 0, 5], 3, 64), ([300, 129, 2], 1, 128),
           ([513], 0, 256), ([40, 300, 90, 10], 2, 1024)]


def packed(lengths, behind, block, C, S, G, dtype, seed=1):
    N, total = len(lengths), sum(lengths) + behind
    pool = N + 3
    slots = torch.randperm(pool, generator=gen(N))[:N].tolist()
    skip = N - 1 if N > 3 else None
    given = [(-1 if n == skip else s) for n, s in enumerate(slots)]
    args, kw = case((total,), C, S, G, dtype, seed=seed)
    if behind:
        for v in (args[0], args[1], args[3], args[4], kw["z"]):
            v[-behind:] = math.nan
    t = kdn.sequence_tables(i32(lengths), total, block, slots=i32(given))
    ends = torch.tensor(lengths).cumsum(0).tolist()
    spans = [slice(e - n, e) for e, n in zip(ends, lengths)]
    live = [n for n in range(N) if n != skip]
    untouched = [s for s in range(pool) if s not in [slots[n] for n in live]]
    return args, kw, t, pool, spans, live, [slots[n] for n in live], untouched, skip


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("S,G", [(16, 1), (8, 2), (32, 1)])
@pytest.mark.parametrize("lengths,behind,block", LENGTHS)
def test_packed(dtype, S, G, lengths, behind, block):
    C = 36
    args, kw, t, pool, spans, live, slots, untouched, skip = packed(lengths, behind, block, C, S, G, dtype)
    S0 = randn((pool, C, S), F32, 2)
    y, last = torch.full((sum(lengths) + behind, C), 7.0, dtype=dtype, device="cuda"), S0.clone()
    kdn.selective_scan(*args, S0=S0, tables=t, out=(y, last), **kw)
    keep, y2 = S0.clone(), torch.full_like(y, 7.0)
    kdn.selective_scan(*args, S0=keep, tables=t, out=(y2, keep), **kw)
    assert torch.equal(last, keep) and torch.equal(y, y2)
    check(args, kw, S0, y, last, [spans[n] for n in live], slots)
    assert torch.equal(last[untouched], S0[untouched]) and (y[sum(lengths):] == 7).all()
    if skip is not None:
        assert (y[spans[skip]] == 7).all()
    new = torch.full_like(S0, 9.0)
    kdn.selective_scan(*args, tables=t, out=(y, new), **kw)
    check(args, kw, None, y, new, [spans[n] for n in live], slots)
    assert (new[untouched] == 9).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("S,G,C", [(16, 1, 80), (8, 5, 35), (32, 2, 150)])
def test_many_sequences(dtype, S, G, C):
    """More runs of channels than the GPU has waves for, fives of them and not fours: a wave a run."""
    B, T = 300, 37
    args, kw = case((B, T), C, S, G, dtype, seed=S)
    S0 = randn((B, C, S), F32, 9)
    y, last = kdn.selective_scan(*args, S0=S0, **kw)
    a, k = flat(args, kw)
    some = (0, 1, 2, 150, 298, 299)
    check(a, k, S0, y.view(-1, C), last, [slice(n * T, n * T + T) for n in some], some)
    keep = S0.clone()
    y2, _ = kdn.selective_scan(*args, S0=keep, out=(torch.empty_like(y), keep), **kw)
    assert torch.equal(y, y2) and torch.equal(keep, last)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,C,block", [(40, 430, 256), (40, 430, 64), (63, 300, 64), (300, 80, 64), (5, 330, 1024),
                                       (3, 40, 128)])
def test_uneven_packed_sequences(dtype, n, C, block):
    """Lengths from none to hundreds, few and many runs, blocks by length and not; skipped
    sequences and rows behind the last are left alone."""
    S, G = 16, 2
    lengths = [(7 * i * i) % 41 if i % 9 else 130 * (i % 5) for i in range(n)]
    total = sum(lengths) + 19
    args, kw = case((total,), C, S, G, dtype, seed=n)
    slots = [n + 3 - i for i in range(n)]
    slots[1] = -1
    tables = kdn.sequence_tables(i32(lengths), total, block, slots=i32(slots))
    S0 = randn((n + 5, C, S), F32, 9)
    y0 = randn((total, C), dtype, 10)
    y, last = kdn.selective_scan(*args, S0=S0, tables=tables, out=(y0.clone(), S0.clone()), **kw)
    first = [sum(lengths[:i]) for i in range(n + 1)]
    on = [i for i in range(n) if slots[i] >= 0]
    some = sorted(set(on[:4] + on[::max(1, n // 12)] + on[-4:]))
    check(args, kw, S0, y, last, [slice(first[i], first[i + 1]) for i in some if lengths[i]],
          [slots[i] for i in some if lengths[i]])
    assert torch.equal(y[first[1]:first[2]], y0[first[1]:first[2]]) and torch.equal(y[first[n]:], y0[first[n]:])
    left = [i for i in range(n + 5) if i not in slots] + [slots[i] for i in on if not lengths[i]]
    assert torch.equal(last[left], S0[left])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C,S,G", [(5, 8, 1), (100, 16, 2), (64, 32, 1)])
def test_decode(dtype, C, S, G):
    N, pool = 6, 9
    args, kw = case((N,), C, S, G, dtype, seed=3)
    st, slots = randn((pool, C, S), F32, 2), [5, -1, 0, 8, 9, 3]
    before, y = st.clone(), torch.full((N, C), 7.0, dtype=dtype, device="cuda")
    kdn.selective_decode(*args, st, slots=i32(slots), y=y, **kw)
    for n, s in enumerate(slots):
        if 0 <= s < pool:
            check(args, kw, before, y, st, [slice(n, n + 1)], [s])
        else:
            assert (y[n] == 7).all()
    rest = [s for s in range(pool) if s not in slots]
    assert torch.equal(st[rest], before[rest])
    new = kdn.selective_decode(*args, before.clone(), slots=i32(slots), **kw)
    assert not new[1].any() and not new[4].any() and torch.equal(new[0], y[0])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_continues_a_prompt(dtype):
    N, T, more, C, S = 3, 37, 5, 40, 16
    args, kw = case((N, T + more), C, S, 1, dtype, seed=4)
    pre = tuple(v if i == 2 else v[:, :T].contiguous() for i, v in enumerate(args))
    y, st = kdn.selective_scan(*pre, **dict(kw, z=kw["z"][:, :T].contiguous()))
    a, k = flat(args, kw)
    ys = [y] + [kdn.selective_decode(*[v if i == 2 else v[:, t] for i, v in enumerate(args)], st,
                                     **dict(kw, z=kw["z"][:, t]))[:, None] for t in range(T, T + more)]
    n = T + more
    check(a, k, None, torch.cat(ys, 1).view(-1, C), st, [slice(i * n, i * n + n) for i in range(N)], range(N))


def check_grad(args, kw, S0, dy, dS, got, spans, slots):
    C, S = args[2].shape
    total, bound = {}, {}
    for rows, slot in zip(spans, slots):
        cot = torch.zeros(C, S).double() if dS is None else ref.wide(dS[slot])
        g, m = ref.scan_grad(*wide(args, kw, rows), state(args, S0, slot), ref.wide(dy[rows]), cot, args[0].dtype)
        for k in ("dx", "ddelta", "dB", "dC") + (("dz",) if kw["z"] is not None else ()):
            ref.close(k, got[k][rows], g[k], m[k])
        if got["dS0"] is not None:
            ref.close("dS0", got["dS0"][slot], g["dS0"], m["dS0"])
        for k in ("dA", "dD", "ddelta_bias"):
            total[k], bound[k] = total.get(k, 0) + g[k], bound.get(k, 0) + m[k]
    for k, v in total.items():
        if got[k] is not None:
            ref.close(k, got[k], v, bound[k] + ref.U * v.abs())


def dense_grad(args, kw, S0, dy, dS):
    B, T, C = args[0].shape
    d = kdn.selective_scan_backward(*args, dy, S0=S0, dS_out=dS, **kw)
    rows = {k: v if v is None or k in ("dA", "dD", "ddelta_bias", "dS0") else v.flatten(0, 1) for k, v in d.items()}
    a, k = flat(args, kw)
    check_grad(a, k, S0, dy.view(-1, C), dS, rows, [slice(n * T, n * T + T) for n in range(B)], range(B))
    return d


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("S", [8, 16, 32])
@pytest.mark.parametrize("T,C,G", [(1, 16, 1), (5, 7, 1), (16, 40, 2), (33, 17, 1), (64, 130, 1), (65, 16, 1), (130, 66, 3)])
def test_gradients(dtype, S, T, C, G):
    B = 2
    args, kw = case((B, T), C, S, G, dtype, seed=T)
    S0, dS, dy = randn((B, C, S), F32, 9), randn((B, C, S), F32, 10), randn((B, T, C), dtype, 11)
    dense_grad(args, kw, S0, dy, dS)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("z,skip,bias,softplus", [(False, False, False, True), (True, False, True, True),
                                                  (False, True, False, False)])
def test_gradients_without(dtype, z, skip, bias, softplus):
    args, kw = case((1, 100), 24, 16, 1, dtype, seed=5, z=z, skip=skip, bias=bias)
    if not softplus:
        args = (args[0], (args[1].float().abs() * 0.1).to(dtype)) + args[2:]
        kw["softplus"] = False
    d = dense_grad(args, kw, None, randn((1, 100, 24), dtype, 11), None)
    assert (d["dz"] is None) == (not z) and (d["dD"] is None) == (not skip) and (d["ddelta_bias"] is None) == (not bias)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("S", [8, 16, 32])
def test_gradients_over_many_tiles(dtype, S):
    """Several blocks and sets of runs, more tiles than workgroups of a set."""
    args, kw = case((1, 1500), 300, S, 2, dtype, seed=6)
    dy = randn((1, 1500, 300), dtype, 11)
    d = dense_grad(args, kw, None, dy, None)
    again = kdn.selective_scan_backward(*args, dy, **kw)
    for k in GRADS:
        assert torch.equal(d[k], again[k]), k


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("S,G", [(16, 1), (8, 2), (32, 1)])
@pytest.mark.parametrize("lengths,behind,block", LENGTHS)
def test_packed_gradients(dtype, S, G, lengths, behind, block):
    C, total = 36, sum(lengths) + behind
    args, kw, t, pool, spans, live, slots, untouched, skip = packed(lengths, behind, block, C, S, G, dtype)
    S0, dS, dy = randn((pool, C, S), F32, 2), randn((pool, C, S), F32, 3), randn((total, C), dtype, 4)
    if behind:
        dy[-behind:] = math.nan
    seven = lambda v: torch.full_like(v, 7.0)  # noqa: E731
    out = dict(dx=seven(dy), ddelta=seven(dy), dz=seven(dy), dB=torch.full((total, G, S), 7.0, dtype=dtype, device="cuda"),
               dC=torch.full((total, G, S), 7.0, dtype=dtype, device="cuda"), dA=seven(args[2]), dD=seven(kw["D"]),
               ddelta_bias=seven(kw["D"]), dS0=seven(S0))
    d = kdn.selective_scan_backward(*args, dy, S0=S0, dS_out=dS, tables=t, out=out, **kw)
    check_grad(args, kw, S0, dy, dS, d, [spans[n] for n in live], slots)
    for k in ("dx", "ddelta", "dz", "dB", "dC"):
        assert not d[k][sum(lengths):].any(), k
        if skip is not None:
            assert not d[k][spans[skip]].any(), k
    assert (d["dS0"][untouched] == 7).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("S,G,C", [(16, 1, 80), (8, 5, 35), (32, 2, 70)])
def test_gradients_of_many_sequences(dtype, S, G, C):
    """Short sequences, dense and packed, many more than workgroups of a set of channels."""
    B, T = 300, 5
    args, kw = case((B, T), C, S, G, dtype, seed=S)
    dense_grad(args, kw, randn((B, C, S), F32, 9), randn((B, T, C), dtype, 11), randn((B, C, S), F32, 10))
    lengths = [(7 * i * i) % 23 for i in range(150)]
    args, kw, t, pool, spans, live, slots, untouched, skip = packed(lengths, 7, 64, C, S, G, dtype)
    S0, dS = randn((pool, C, S), F32, 2), randn((pool, C, S), F32, 3)
    dy = randn((sum(lengths) + 7, C), dtype, 4)
    dy[-7:] = math.nan
    d = kdn.selective_scan_backward(*args, dy, S0=S0, dS_out=dS, tables=t, **kw)
    check_grad(args, kw, S0, dy, dS, d, [spans[n] for n in live], slots)
    for k in ("dx", "ddelta", "dz", "dB", "dC"):
        assert not d[k][-7:].any() and not d[k][spans[skip]].any(), k
    assert not d["dS0"][untouched].any()


def test_gradient_against_differences():
    """The 64-bit gradient itself against central differences of the 64-bit form."""
    T, C, S, G = 5, 4, 8, 2
    args, kw = case((T,), C, S, G, F32, seed=2)
    v = list(wide(args, kw, slice(0, T)))
    S0, dS, dy = (randn(s, F32, i).cpu().double() for i, s in ((5, (C, S)), (6, (C, S)), (7, (T, C))))
    g, _ = ref.scan_grad(*v, S0, dy, dS, F32)

    def loss():
        y, S_, _, _ = ref.scan(*v, S0, F32)
        return ((y * dy).sum() + (S_ * dS).sum()).item()

    for name, p in (("dx", v[0]), ("ddelta", v[1]), ("dA", v[2]), ("dB", v[3]), ("dC", v[4]), ("dD", v[5]), ("dz", v[6]),
                    ("ddelta_bias", v[7]), ("dS0", S0)):
        for i in range(p.numel()):
            keep, h, at = p.view(-1)[i].item(), 1e-5, []
            for s in (h, -h):
                p.view(-1)[i] = keep + s
                at.append(loss())
            p.view(-1)[i] = keep
            assert abs((at[0] - at[1]) / (2 * h) - g[name].reshape(-1)[i].item()) < 1e-7, name


@pytest.mark.parametrize("dtype", [BF, F32])
def test_far_time_steps(dtype):
    """Steps so long that the state is forgotten, so short that nothing happens, and zero."""
    T, C, S = 40, 16, 16
    args, kw = case((1, T), C, S, 1, dtype, seed=8)
    delta = args[1].clone()
    delta[0, 5], delta[0, 9], delta[0, 20], delta[0, 21] = 60.0, -40.0, 300.0, -1e4
    args = (args[0], delta) + args[2:]
    S0, dy = randn((1, C, S), F32, 9), randn((1, T, C), dtype, 11)
    y, last = kdn.selective_scan(*args, S0=S0, **kw)
    a, k = flat(args, kw)
    check(a, k, S0, y[0], last, [slice(0, T)], [0])
    dense_grad(args, kw, S0, dy, None)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_non_finite_stay_in_their_channel_and_sequence(dtype):
    lengths, C, S = [40, 150, 30], 24, 16
    args, kw = case((220,), C, S, 1, dtype, seed=3)
    S0, dy = randn((3, C, S), F32, 2), randn((220, C), dtype, 4)
    t = kdn.sequence_tables(i32(lengths), 220, 64, slots=i32([0, 1, 2]))
    call = lambda: (kdn.selective_scan(*args, S0=S0, tables=t, out=(torch.empty_like(dy), torch.empty_like(S0)), **kw),  # noqa: E731
                    kdn.selective_scan_backward(*args, dy, S0=S0, tables=t, **kw))
    (y, last), g = call()
    args[0][100, 5], kw["z"][60, 6], S0[1, 7, 3], dy[70, 8] = math.nan, math.inf, math.inf, math.nan
    (y2, last2), g2 = call()
    other = [r for r in range(220) if not 40 <= r < 190]
    same = [c for c in range(C) if c not in (5, 6, 7, 8)]
    assert torch.equal(y[other], y2[other]) and torch.equal(last[[0, 2]], last2[[0, 2]])
    assert torch.equal(y[:, same], y2[:, same]) and torch.equal(y[:100, 5], y2[:100, 5])
    for k in ("dx", "ddelta", "dz"):
        assert torch.equal(g[k][other], g2[k][other]) and torch.equal(g[k][:, same], g2[k][:, same]), k
    for k in ("dB", "dC"):
        assert torch.equal(g[k][other], g2[k][other]), k
    assert torch.equal(g["dA"][same], g2["dA"][same]) and torch.equal(g["dS0"][[0, 2]], g2["dS0"][[0, 2]])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_nothing_to_do(dtype):
    S0 = randn((2, 8, 16), F32, 1)
    args, kw = case((2, 0), 8, 16, 1, dtype)
    y, last = kdn.selective_scan(*args, S0=S0, **kw)
    assert y.shape == (2, 0, 8) and torch.equal(last, S0)
    _, last = kdn.selective_scan(*args, **kw)
    assert not last.any()
    d = kdn.selective_scan_backward(*args, args[0], dS_out=S0, **kw)
    assert torch.equal(d["dS0"], S0) and not d["dA"].any() and not d["dD"].any() and not d["ddelta_bias"].any()
    args, kw = case((0, 5), 8, 16, 1, dtype)
    assert kdn.selective_scan(*args, **kw)[0].shape == (0, 5, 8)
    args, kw = case((0,), 8, 16, 1, dtype)
    assert kdn.selective_decode(*args, S0, **kw).shape == (0, 8)
