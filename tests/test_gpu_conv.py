"""Short causal convolution on the GPU against its 64-bit form: prefill (dense, packed,
slices, states), single tokens, gradients."""
import math

import pytest
import torch

import around_ref as ref
from linear_attention_recurrent_delta_amd import kdn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    kdn.ensure_built()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(shape, dtype=F32, seed=0, size=1.0):
    return (size * torch.randn(shape, generator=gen(seed))).to(dtype).cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rows(shape, dtype, seed, wide=0, odd=0):
    """Rows [.., C] as slices of rows with `wide` more columns, `odd` elements behind an
    aligned address; NaN in what is not theirs."""
    C = shape[-1]
    row = C + wide
    n = math.prod(shape[:-1]) * row
    buf = torch.full((n + odd + 8,), math.nan, dtype=dtype, device="cuda")
    x = buf[odd:odd + n].view(shape[:-1] + (row,))[..., :C]
    x.copy_(randn(shape, dtype, seed))
    return x


def params(C, W, seed=3, bias=True):
    return randn((C, W), seed=seed, size=W ** -0.5), randn((C,), seed=seed + 1, size=0.3) if bias else None


def check_forward(x, w, b, state, act, y, S, spans, slots):
    """Every sequence (rows `spans` of x [tokens, C]) with its state (None: zero)."""
    W, C = w.shape[1], w.shape[0]
    for rows_, slot in zip(spans, slots):
        s0 = torch.zeros(W - 1, C).double() if state is None else ref.wide(state[slot])
        yy, last, bound = ref.conv(ref.wide(x[rows_]), ref.wide(w), ref.wide(b), s0, act == "silu", x.dtype)
        ref.close("y", y[rows_], yy, bound)
        if S is not None:
            assert torch.equal(ref.wide(S[slot]), last)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 2, 3, 5, 16, 17, 64, 65, 131])
def test_lengths(dtype, W, T):
    B, C = 2, 40
    x, (w, b), S0 = randn((B, T, C), dtype, 1), params(C, W), randn((B, W - 1, C), dtype, 2)
    y, S = kdn.causal_conv(x, w, b, state0=S0)
    for n in range(B):
        check_forward(x[n], w, b, S0[n:n + 1], "silu", y[n], S[n:n + 1], [slice(0, T)], [0])
    keep = S0.clone()
    y2, same = kdn.causal_conv(x, w, b, state0=keep, out=(torch.empty_like(y), keep))
    assert same is keep and torch.equal(keep, S) and torch.equal(y, y2)
    y3, none = kdn.causal_conv(x, w, b, state0=S0, out=(torch.empty_like(y), None))
    assert none is None and torch.equal(y, y3)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C", [1, 3, 7, 8, 9, 63, 64, 257, 511, 512, 513, 1030])
@pytest.mark.parametrize("act", [None, "silu"])
def test_channels(dtype, C, act):
    T = 70
    x, (w, b) = randn((1, T, C), dtype, C), params(C, 4, bias=C % 2 == 0)
    y, S = kdn.causal_conv(x, w, b, activation=act)
    check_forward(x[0], w, b, None, act, y[0], S, [slice(0, T)], [0])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C,wide,odd", [(64, 8, 0), (64, 3, 0), (64, 8, 1), (77, 5, 3), (520, 16, 4)])
def test_slices(dtype, C, wide, odd):
    """Rows of a wider tensor, at any element: the same bits as contiguous ones."""
    B, T = 3, 50
    x = rows((B, T, C), dtype, 5, wide, odd)
    w, b = params(C, 4)
    want = kdn.causal_conv(x.contiguous(), w, b)
    got = kdn.causal_conv(x, w, b)
    for a, c in zip(want, got):
        assert torch.equal(a, c)
    dy = randn((B, T, C), dtype, 6)
    want = kdn.causal_conv_backward(x.contiguous(), w, dy, b)
    got = kdn.causal_conv_backward(x, w, dy, b)
    for k in want:
        assert torch.equal(want[k], got[k]), k
    S, S2 = randn((B, 3, C), dtype, 7), randn((B, 3, C), dtype, 7)
    assert torch.equal(kdn.causal_conv_decode(x[:, 4], w, S, b),
                       kdn.causal_conv_decode(x[:, 4].contiguous(), w, S2, b))
    assert torch.equal(S, S2)


LENGTHS = [([70, 1, 200, 0, 3, 64, 2], 5, 64), ([1, 1, 1, 1], 0, 64), ([0, 0, 5], 3, 64),
           ([300, 129, 2], 1, 128), ([513], 0, 256)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("lengths,behind,block", LENGTHS)
def test_packed(dtype, W, lengths, behind, block):
    """Sequences one behind the other, states scattered over a pool, one skipped, rows
    behind the last one untouched."""
    N, C, total = len(lengths), 72, sum(lengths) + behind
    pool = N + 3
    slots = torch.randperm(pool, generator=gen(N))[:N].tolist()
    skip = N - 1 if N > 3 else None
    given = [(-1 if n == skip else s) for n, s in enumerate(slots)]
    x, (w, b), S0 = randn((total, C), dtype, 1), params(C, W), randn((pool, W - 1, C), dtype, 2)
    if behind:
        x[-behind:] = math.nan
    t = kdn.sequence_tables(i32(lengths), total, block, slots=i32(given))
    y, S = torch.full((total, C), 7.0, dtype=dtype, device="cuda"), S0.clone()
    kdn.causal_conv(x, w, b, state0=S0, tables=t, out=(y, S))
    inplace, y2 = S0.clone(), torch.full_like(y, 7.0)
    kdn.causal_conv(x, w, b, state0=inplace, tables=t, out=(y2, inplace))
    assert torch.equal(S, inplace) and torch.equal(y, y2)
    ends = torch.tensor(lengths).cumsum(0).tolist()
    spans = [slice(e - n, e) for e, n in zip(ends, lengths)]
    live = [n for n in range(N) if n != skip]
    check_forward(x, w, b, S0, "silu", y, S, [spans[n] for n in live], [slots[n] for n in live])
    untouched = [s for s in range(pool) if s not in [slots[n] for n in live]]
    assert torch.equal(S[untouched], S0[untouched])
    assert (y[ends[-1]:] == 7).all()
    if skip is not None:
        assert (y[spans[skip]] == 7).all()
    # from nothing into a pool
    new = torch.full_like(S0, 9.0)
    kdn.causal_conv(x, w, b, tables=t, out=(y, new))
    check_forward(x, w, b, None, "silu", y, new, [spans[n] for n in live], [slots[n] for n in live])
    assert (new[untouched] == 9).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_continues_a_prompt(dtype):
    """A prompt, then token by token: the bits of one long prompt."""
    N, T, more, C, W = 3, 21, 6, 100, 4
    x, (w, b) = randn((N, T + more, C), dtype, 1), params(C, W)
    want, last = kdn.causal_conv(x, w, b)
    y, S = kdn.causal_conv(x[:, :T].contiguous(), w, b)
    assert torch.equal(y, want[:, :T])
    pool = torch.full((5, W - 1, C), 3.0, dtype=dtype, device="cuda")
    slots = i32([4, 0, 2])
    pool[slots.long()] = S
    for t in range(T, T + more):
        assert torch.equal(kdn.causal_conv_decode(x[:, t], w, pool, b, slots=slots), want[:, t])
    assert torch.equal(pool[slots.long()], last) and (pool[[1, 3]] == 3).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W,C,act", [(2, 8, "silu"), (3, 65, None), (4, 520, "silu"), (4, 33, "silu")])
def test_decode(dtype, W, C, act):
    """Padding rows skipped, their outputs left, other states untouched."""
    N, pool = 6, 9
    x, (w, b), S = randn((N, C), dtype, 1), params(C, W), randn((pool, W - 1, C), dtype, 2)
    slots, before = [5, -1, 0, 8, 9, 3], S.clone()
    y = torch.full((N, C), 7.0, dtype=dtype, device="cuda")
    kdn.causal_conv_decode(x, w, S, b, activation=act, slots=i32(slots), y=y)
    for n, s in enumerate(slots):
        if not 0 <= s < pool:
            assert (y[n] == 7).all()
            continue
        check_forward(x[n:n + 1], w, b, before, act, y[n:n + 1], S, [slice(0, 1)], [s])
    rest = [s for s in range(pool) if s not in slots]
    assert torch.equal(S[rest], before[rest])


def check_grad(x, w, b, S0, dy, dS, act, got, spans, slots):
    W, C = w.shape[1], w.shape[0]
    dw, db = torch.zeros(C, W).double(), torch.zeros(C).double()
    bw, bb = torch.zeros_like(dw), torch.zeros_like(db)
    for r, slot in zip(spans, slots):
        s0 = torch.zeros(W - 1, C).double() if S0 is None else ref.wide(S0[slot])
        g, m = ref.conv_grad(ref.wide(x[r]), ref.wide(w), ref.wide(b), s0, ref.wide(dy[r]),
                             None if dS is None else ref.wide(dS[slot]), act == "silu", x.dtype)
        ref.close("dx", got["dx"][r], g["dx"], m["dx"])
        if got["dstate0"] is not None:
            ref.close("dstate0", got["dstate0"][slot], g["dstate0"], m["dstate0"])
        dw, db, bw, bb = dw + g["dweight"], db + g["dbias"], bw + m["dweight"], bb + m["dbias"]
    ref.close("dweight", got["dweight"], dw, bw + ref.U * dw.abs())
    if b is not None:
        ref.close("dbias", got["dbias"], db, bb + ref.U * db.abs())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W,T,C,act", [(2, 1, 8, "silu"), (4, 1, 70, "silu"), (4, 2, 64, None), (3, 15, 300, "silu"),
                                       (4, 16, 64, "silu"), (4, 17, 1, "silu"), (4, 64, 33, "silu"), (2, 65, 256, "silu"),
                                       (4, 300, 130, "silu"), (3, 127, 64, None)])
def test_gradients(dtype, W, T, C, act):
    B = 2
    x, (w, b), S0 = randn((B, T, C), dtype, 1), params(C, W, bias=T != 16), randn((B, W - 1, C), dtype, 2)
    dy, dS = randn((B, T, C), dtype, 3), randn((B, W - 1, C), dtype, 4)
    d = kdn.causal_conv_backward(x, w, dy, b, state0=S0, dstate_out=dS, activation=act)
    flat = {k: v if k in ("dweight", "dbias", "dstate0") else v.reshape(B * T, C) for k, v in d.items()}
    spans = [slice(0, T), slice(T, 2 * T)]
    check_grad(x.view(-1, C), w, b, S0, dy.view(-1, C), dS, act, flat, spans, [0, 1])
    # without states
    d = kdn.causal_conv_backward(x, w, dy, b, activation=act)
    flat = {k: v if k in ("dweight", "dbias", "dstate0") else v.reshape(B * T, C) for k, v in d.items()}
    check_grad(x.view(-1, C), w, b, None, dy.view(-1, C), None, act, flat, spans, [0, 1])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("lengths,behind,block", LENGTHS)
def test_packed_gradients(dtype, W, lengths, behind, block):
    N, C, total = len(lengths), 72, sum(lengths) + behind
    pool = N + 3
    slots = torch.randperm(pool, generator=gen(N))[:N].tolist()
    skip = N - 1 if N > 3 else None
    given = [(-1 if n == skip else s) for n, s in enumerate(slots)]
    x, (w, b), S0 = randn((total, C), dtype, 1), params(C, W), randn((pool, W - 1, C), dtype, 2)
    dy, dS = randn((total, C), dtype, 3), randn((pool, W - 1, C), dtype, 4)
    if behind:
        x[-behind:] = math.nan
        dy[-behind:] = math.nan
    t = kdn.sequence_tables(i32(lengths), total, block, slots=i32(given))
    out = dict(dx=torch.full((total, C), 7.0, dtype=dtype, device="cuda"), dweight=torch.full_like(w, 7.0),
               dbias=torch.full_like(b, 7.0), dstate0=torch.full_like(S0, 7.0))
    d = kdn.causal_conv_backward(x, w, dy, b, state0=S0, dstate_out=dS, tables=t, out=out)
    ends = torch.tensor(lengths).cumsum(0).tolist()
    spans = [slice(e - n, e) for e, n in zip(ends, lengths)]
    live = [n for n in range(N) if n != skip]
    check_grad(x, w, b, S0, dy, dS, "silu", d, [spans[n] for n in live], [slots[n] for n in live])
    assert not d["dx"][ends[-1]:].any()
    if skip is not None:
        assert not d["dx"][spans[skip]].any()
    untouched = [s for s in range(pool) if s not in [slots[n] for n in live]]
    assert (d["dstate0"][untouched] == 7).all()


def test_gradient_against_differences():
    """The 64-bit gradient itself against central differences of the 64-bit form."""
    T, C, W = 7, 3, 4
    x, (w, b), S0 = randn((T, C), F32, 1).cpu().double(), params(C, W), randn((W - 1, C), F32, 2).cpu().double()
    w, b = ref.wide(w), ref.wide(b)
    dy, dS = randn((T, C), F32, 3).cpu().double(), randn((W - 1, C), F32, 4).cpu().double()
    g, _ = ref.conv_grad(x, w, b, S0, dy, dS, True, F32)

    def loss():
        y, S, _ = ref.conv(x, w, b, S0, True, F32)
        return ((y * dy).sum() + (S * dS).sum()).item()

    for name, v in (("dx", x), ("dweight", w), ("dbias", b), ("dstate0", S0)):
        for i in range(v.numel()):
            keep, h = v.view(-1)[i].item(), 1e-5
            v.view(-1)[i] = keep + h
            up = loss()
            v.view(-1)[i] = keep - h
            down = loss()
            v.view(-1)[i] = keep
            # the third derivative is a few units: h^2, and 1e-16 / h of the difference
            assert abs((up - down) / (2 * h) - g[name].reshape(-1)[i].item()) < 1e-8


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_tiles_per_workgroup(dtype):
    """More tiles than parts: sums over several tiles in float32 before the 64-bit sum."""
    B, T, C, W = 1, 64 * 1000, 64, 4
    x, (w, b), dy = randn((B, T, C), dtype, 1), params(C, W), randn((B, T, C), dtype, 2)
    d = kdn.causal_conv_backward(x, w, dy, b)
    d2 = kdn.causal_conv_backward(x, w, dy, b)
    for k in d:
        assert torch.equal(d[k], d2[k])
    flat = {k: v if k in ("dweight", "dbias", "dstate0") else v[0] for k, v in d.items()}
    check_grad(x[0], w, b, None, dy[0], None, "silu", flat, [slice(0, T)], [0])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_non_finite_stay_in_their_channel_and_sequence(dtype):
    lengths, C, W = [20, 30, 10], 24, 4
    x, (w, b), S0 = randn((60, C), dtype, 1), params(C, W), randn((3, W - 1, C), dtype, 2)
    dy = randn((60, C), dtype, 3)
    t = kdn.sequence_tables(i32(lengths), 60, 64, slots=i32([0, 1, 2]))
    y, S = kdn.causal_conv(x, w, b, state0=S0, tables=t, out=(torch.empty_like(x), torch.empty_like(S0)))
    g = kdn.causal_conv_backward(x, w, dy, b, state0=S0, tables=t)
    x[49, 5], x[30, 6], S0[1, 2, 7] = math.nan, math.inf, -math.inf
    y2, S2 = kdn.causal_conv(x, w, b, state0=S0, tables=t, out=(torch.empty_like(x), torch.empty_like(S0)))
    g2 = kdn.causal_conv_backward(x, w, dy, b, state0=S0, tables=t)
    bad = torch.zeros(60, C, dtype=torch.bool, device="cuda")
    bad[49:50, 5] = True
    bad[30:34, 6] = True
    bad[20:23, 7] = True
    assert torch.equal(y[~bad], y2[~bad])
    # the gradients of the rows that such a value meets a tap with
    for at, c in ((49, 5), (30, 6), (20, 7)):
        bad[max(at - 3, 20):min(at + 4, 50), c] = True
    assert torch.equal(g["dx"][~bad], g2["dx"][~bad])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_nothing_to_do(dtype):
    w, b = params(8, 4)
    S0 = randn((2, 3, 8), dtype, 1)
    y, S = kdn.causal_conv(torch.empty(2, 0, 8, dtype=dtype, device="cuda"), w, b, state0=S0)
    assert y.shape == (2, 0, 8) and torch.equal(S, S0)
    y, S = kdn.causal_conv(torch.empty(2, 0, 8, dtype=dtype, device="cuda"), w, b)
    assert not S.any()
    y, S = kdn.causal_conv(torch.empty(0, 5, 8, dtype=dtype, device="cuda"), w, b)
    assert y.shape == (0, 5, 8) and S.shape == (0, 3, 8)
    d = kdn.causal_conv_backward(torch.empty(2, 0, 8, dtype=dtype, device="cuda"), w,
                                 torch.empty(2, 0, 8, dtype=dtype, device="cuda"), b, dstate_out=S0)
    assert not d["dweight"].any() and not d["dbias"].any() and torch.equal(d["dstate0"], S0)
    assert kdn.causal_conv_decode(torch.empty(0, 8, dtype=dtype, device="cuda"), w, S0, b).shape == (0, 8)
    y, S = kdn.causal_conv(torch.empty(2, 3, 0, dtype=dtype, device="cuda"), torch.empty(0, 4, device="cuda"))
    assert y.shape == (2, 3, 0)
