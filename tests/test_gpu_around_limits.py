"""The operators around a recurrence on the GPU at the ends of their ranges: tables of any
block length, sums over many tokens, rounds of the norms' gradients, sizes of nothing."""
import math

import pytest
import torch

import around_ref as ref
import test_gpu_conv as tc
import test_gpu_norm as tn
import test_gpu_scan as ts
from linear_attention_recurrent_delta_amd import kdn
from test_gpu_conv import BF, F32, gen, i32, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    kdn.ensure_built()


def uneven(N, most, seed):
    """Lengths with none, one, a tile and its neighbours among them."""
    lengths = torch.randint(0, most, (N,), generator=gen(seed)).tolist()
    for i, n in enumerate((0, 1, 64, 63, 65, 0, 128)):
        lengths[(7 * i + 3) % N] = n
    return lengths


# sequences, longest, channels: one search step, two and three; one sequence; short ones only
TABLES = [(1, 300, 24), (40, 200, 520), (64, 130, 40), (65, 130, 40), (300, 150, 72), (4500, 4, 8)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,most,C", TABLES)
def test_conv_on_tables_of_any_block(dtype, N, most, C):
    """One batch on tables of many block lengths, a scan's among them: the same bits, the
    pool's other states, skipped sequences and rows behind the last left as they were."""
    lengths = uneven(N, most, N) if N > 1 else [most]
    behind, W = 5, 4
    total = sum(lengths) + behind
    slots = torch.randperm(N + 3, generator=gen(N)).tolist()[:N]
    given = [-1 if n % 11 == 10 else s for n, s in enumerate(slots)]
    x, (w, b), S0 = randn((total, C), dtype, 1), tc.params(C, W), randn((N + 3, W - 1, C), dtype, 2)
    dy, dS = randn((total, C), dtype, 3), randn((N + 3, W - 1, C), dtype, 4)
    x[-behind:], dy[-behind:] = math.nan, math.nan
    ends = torch.tensor(lengths).cumsum(0).tolist()
    first = None
    for block in (64, 128, 4096, kdn.selective_block(total, N, C, 16), kdn.selective_block(total, N, 8192, 16), 1 << 20,
                  (1 << 31) - 64):
        t = kdn.sequence_tables(i32(lengths), total, block, slots=i32(given))
        y, S = torch.full((total, C), 7.0, dtype=dtype, device="cuda"), S0.clone()
        kdn.causal_conv(x, w, b, state0=S0, tables=t, out=(y, S))
        keep, y2 = S0.clone(), torch.full_like(y, 7.0)
        kdn.causal_conv(x, w, b, state0=keep, tables=t, out=(y2, keep))
        d = kdn.causal_conv_backward(x, w, dy, b, state0=S0, dstate_out=dS, tables=t)
        assert torch.equal(y, y2) and torch.equal(S, keep), block
        if first is None:
            first = y, S, d
            on = [n for n in range(N) if given[n] >= 0]
            some = sorted(set(on[:12] + on[::max(1, N // 12)] + on[-4:]))
            spans = [slice(ends[n] - lengths[n], ends[n]) for n in some]
            tc.check_forward(x, w, b, S0, "silu", y, S, spans, [slots[n] for n in some])
            off = [n for n in range(N) if given[n] < 0]
            for n in off:
                assert (y[ends[n] - lengths[n]:ends[n]] == 7).all()
            assert (y[-behind:] == 7).all() and not d["dx"][-behind:].any()
            if N <= 300:
                tc.check_grad(x, w, b, S0, dy, dS, "silu", d, [slice(ends[n] - lengths[n], ends[n]) for n in on],
                              [slots[n] for n in on])
            continue
        assert torch.equal(y, first[0]) and torch.equal(S, first[1]), block
        for k in ("dx", "dstate0"):
            assert torch.equal(d[k], first[2][k]), (block, k)
        if N <= 300:
            tc.check_grad(x, w, b, S0, dy, dS, "silu", d, [slice(ends[n] - lengths[n], ends[n]) for n in on],
                          [slots[n] for n in on])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_conv_and_scan_on_one_table(dtype):
    """The table of a scan of many channels, whose block is the whole batch, for both."""
    N, C, S = 96, 4096, 16
    lengths = uneven(N, 40, 5)
    total = sum(lengths)
    block = kdn.selective_block(total, N, C, S)
    assert block >= total
    t = kdn.sequence_tables(i32(lengths), total, block, slots=i32(list(range(N))[::-1]))
    args, kw = ts.case((total,), C, S, 1, dtype, seed=1)
    w, b = tc.params(C, 4)
    conv0, S0 = randn((N, 3, C), dtype, 2), randn((N, C, S), F32, 3)
    u, last = kdn.causal_conv(args[0], w, b, state0=conv0, tables=t, out=(torch.empty_like(args[0]), torch.empty_like(conv0)))
    y, Sn = kdn.selective_scan(u, *args[1:], S0=S0, tables=t, out=(torch.empty_like(u), torch.empty_like(S0)), **kw)
    ends = torch.tensor(lengths).cumsum(0).tolist()
    some = [n for n in range(0, N, 9)]
    spans, slots = [slice(ends[n] - lengths[n], ends[n]) for n in some], [N - 1 - n for n in some]
    tc.check_forward(args[0], w, b, conv0, "silu", u, last, spans, slots)
    ts.check((u,) + args[1:], kw, S0, y, Sn, spans, slots)


@pytest.mark.parametrize("block", [64, 1 << 20])
def test_conv_of_no_sequence(block):
    """Rows and no sequence: outputs left as they were, gradients zero."""
    x, (w, b) = torch.full((700, 40), math.nan, device="cuda"), tc.params(40, 4)
    t = kdn.sequence_tables(torch.empty(0, dtype=torch.int32, device="cuda"), 700, block)
    y = torch.full_like(x, 7.0)
    kdn.causal_conv(x, w, b, tables=t, out=(y, None))
    assert (y == 7).all()
    d = kdn.causal_conv_backward(x, w, x, b, tables=t)
    assert not d["dx"].any() and not d["dweight"].any() and not d["dbias"].any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_captured_conv_on_a_long_block(dtype):
    """A captured convolution finds its tiles in tables that change between the replays."""
    N, C, cap = 70, 72, 3000
    x, (w, b), dy = randn((cap, C), dtype, 1), tc.params(C, 4), randn((cap, C), dtype, 2)
    lengths, state = i32([1] * N), randn((N, 3, C), dtype, 3)
    t = kdn.sequence_tables(lengths, cap, 1 << 20)
    y, S = torch.zeros_like(x), torch.zeros_like(state)
    d = dict(dx=torch.zeros_like(x), dweight=torch.zeros_like(w), dbias=torch.zeros_like(b), dstate0=torch.zeros_like(state))
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def step():
        kdn.sequence_tables(lengths, cap, 1 << 20, out=t)
        kdn.causal_conv(x, w, b, state0=state, tables=t, out=(y, S))
        kdn.causal_conv_backward(x, w, dy, b, state0=state, tables=t, out=d, workspace=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    flat = [y, S] + list(d.values())
    for ln in ([0] * N, [cap] + [0] * (N - 1), [(5 * i * i) % 43 for i in range(N)], [0] * (N - 1) + [129]):
        lengths.copy_(i32(ln))
        for v in flat:
            v.zero_()
        step()
        torch.cuda.synchronize()
        want = [v.clone() for v in flat]
        for _ in range(2):
            for v in flat:
                v.zero_()
            ws.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            for a, c in zip(flat, want):
                assert torch.equal(a, c)


def spike(shape, rest, dtype=F32):
    """Values that all count in a sum, behind one that hides each of them from a float32
    register: what a long chain of such sums loses is `rest` a step."""
    x = torch.full(shape, rest, dtype=dtype, device="cuda")
    x[0] = 2.0 ** 24
    return x


def column_sums(x):
    return sum(part.double().sum(0) for part in x.split(4096))


def test_conv_sums_over_many_tokens():
    """dweight and dbias over 768 tiles of a few wide parts.  A lane adds 16 tokens of each of at
    most 32 tiles in float32, then four waves' sums are added, all else is 64 bits, and the
    result is rounded: 517 roundings of the sum of absolute values at most."""
    T, C = 64 * 768, 8192
    x, dy, w, b = torch.ones(1, T, C, device="cuda"), spike((T, C), 0.9), torch.zeros(C, 2, device="cuda"), torch.zeros(C, device="cuda")
    d = kdn.causal_conv_backward(x, w, dy[None], b, activation=None)
    want = column_sums(dy)
    for got in (d["dbias"], d["dweight"][:, 1]):
        off = (got.double() - want).abs().max().item() / want.max().item() / ref.U
        print(f"    {off:.0f} roundings", flush=True)
        assert off <= 517


@pytest.mark.parametrize("per_head,tokens,H", [(True, 24576, 512), (False, 64 * 24576, 8)])
def test_gated_norm_sums_over_many_rows(per_head, tokens, H):
    """dweight over 768 rows for each place of the workgroups that run at once.  A thread adds at most 256
    rows in float32, then 16 rows' places; n is off by 8 roundings (its root, two products) and
    the result by one."""
    d = 64
    x, dy = torch.ones(tokens, H, d, device="cuda"), spike((tokens, H, d), 0.9)
    w = torch.ones((H, d) if per_head else (d,), device="cuda")
    if not per_head:
        dy[0, 1:] = 0.9
    got = kdn.gated_norm_backward(x, w, dy)["dweight"].double()
    n = (1.0 + torch.tensor(1e-5).double().item()) ** -0.5
    want = n * (column_sums(dy) if per_head else column_sums(dy.view(-1, d)))
    off = (got - want).abs().max().item() / want.max().item() / ref.U
    print(f"    {off:.0f} roundings", flush=True)
    assert off <= 256 + 16 + 8 + 1


@pytest.mark.parametrize("scale", ["one", "channel"])
def test_residual_norm_sums_over_many_rows(scale):
    """dweight and dscale over 768 rows for each of the workgroups that run at once: a thread adds at most 256 in float32.
    n is off by 8 roundings, the result by one; one scale adds four columns of a thread and
    nine steps of a workgroup, too."""
    tokens, D = 512 * 768, 2048
    h, one = torch.ones(tokens, D, device="cuda"), torch.ones(D, device="cuda")
    dy = spike((tokens, D), 0.9)
    d = kdn.residual_norm_backward(None, h, one, dy, out=dict(dx=None, dresidual=torch.empty_like(h), dweight=torch.empty(D, device="cuda"),
                                                              dscale=None))
    want = (1.0 + torch.tensor(1e-5).double().item()) ** -0.5 * column_sums(dy)
    off = (d["dweight"].double() - want).abs().max().item() / want.max().item() / ref.U
    print(f"    dweight {off:.0f} roundings", flush=True)
    assert off <= 256 + 8 + 1
    s = torch.ones(D if scale == "channel" else 1, device="cuda")
    got = kdn.residual_norm_backward(h, h, one, torch.zeros_like(h), dy, scale=s)["dscale"].double()
    want = column_sums(dy) if scale == "channel" else column_sums(dy).sum().view(1)
    off = (got - want).abs().max().item() / want.max().item() / ref.U
    print(f"    dscale {off:.0f} roundings", flush=True)
    assert off <= 256 + 1 + (0 if scale == "channel" else 4 + 9)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_gradients_beyond_one_run_of_sums(dtype):
    """More rows than one run of the float32 sums takes, rows as slices: each row's gradients are
    those of its own half, bit for bit, and the sums are the halves'."""
    d, n = 8, 512 * 256 * 256 + 12345
    draw = lambda w: torch.rand((n, w), device="cuda", generator=torch.Generator("cuda").manual_seed(w)).to(dtype)  # noqa: E731
    h, x, dy, w = draw(d + 3)[:, 1:1 + d], draw(d + 2)[:, 2:], draw(d), 0.5 + torch.rand(d, device="cuda")
    assert kdn.load().kdn_residual_norm_backward_workspace_size(n, d, d, None) == 4 * 512 * 2 * 2 * d
    assert kdn.load().kdn_gated_norm_backward_workspace_size(n, 1, d, 0, None) == 4 * 1024 * 2 * d
    for call in (lambda r: kdn.residual_norm_backward(x[r], h[r], w, dy[r], scale=w),
                 lambda r: kdn.gated_norm_backward(h[r].unsqueeze(1), w, dy[r].unsqueeze(1), x[r].unsqueeze(1))):
        full = call(slice(None))
        half = [call(slice(0, n // 2 - 77)), call(slice(n // 2 - 77, n))]
        for k in ("dx", "dresidual", "dgate"):
            if k in full:
                assert torch.equal(full[k], torch.cat([a[k] for a in half])), k
        # dy, h and w are positive and so are dweight's terms; a sum of one call is off by 256
        # rows of a thread, 256 or 512 threads of a column and the result at most
        want = sum(a["dweight"].double() for a in half)
        assert ((full["dweight"].double() - want).abs() <= 2 * (256 + 512 + 1) * ref.U * want).all()


def test_scan_sums_over_many_tokens():
    """dD over 768 tiles, which one workgroup of so many channels could take: a wave adds 8 tokens of each of at most 256
    tiles in float32 (two in a lane, four lanes), then eight waves' sums are added, and the
    result is rounded."""
    T, C, S = 64 * 768, 32768, 8
    x, dy = torch.ones(1, T, C, dtype=BF, device="cuda"), spike((T, C), 0.1, BF)
    none, A = torch.zeros(1, T, 1, S, dtype=BF, device="cuda"), -torch.ones(C, S, device="cuda")
    d = kdn.selective_scan_backward(x, x, A, none, none, dy[None], D=torch.ones(C, device="cuda"))
    want = column_sums(dy)
    off = (d["dD"].double() - want).abs().max().item() / want.max().item() / ref.U
    print(f"    {off:.0f} roundings", flush=True)
    assert off <= 256 + 4 + 8 + 1


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gated_gradients_of_no_heads(dtype):
    """A weight for all heads, and none of them: its gradient is zero, not left as it was."""
    e = torch.empty(5, 0, 16, dtype=dtype, device="cuda")
    for z in (None, e):
        out = dict(dx=e, dgate=z, dweight=torch.full((16,), 7.0, device="cuda"))
        kdn.gated_norm_backward(e.clone(), torch.ones(16, device="cuda"), e.clone(), z, out=out)
        assert not out["dweight"].any()
    d = kdn.gated_norm_backward(e, torch.ones(0, 16, device="cuda"), e)
    assert d["dweight"].shape == (0, 16)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("packed", [False, True])
def test_scan_gradients_of_no_channels(dtype, packed):
    """Tokens with B and C and no channel: their gradients are zero, not left as they were."""
    lead, S = (20,) if packed else (2, 10), 16
    t = kdn.sequence_tables(i32([12, 0, 5]), 20, 64) if packed else None
    e = torch.empty(lead + (0,), dtype=dtype, device="cuda")
    for G in (0, 1, 3):
        B = torch.full(lead + (G, S), math.nan, dtype=dtype, device="cuda")
        seven = lambda: torch.full(lead + (G, S), 7.0, dtype=dtype, device="cuda")  # noqa: E731
        none = torch.empty(0, device="cuda")
        out = dict(dx=e, ddelta=e.clone(), dz=None, dB=seven(), dC=seven(), dA=torch.empty(0, S, device="cuda"), dD=None,
                   ddelta_bias=None, dS0=None)
        kdn.selective_scan_backward(e, e, torch.empty(0, S, device="cuda"), B, B, e, D=none, tables=t, out=out)
        assert not out["dB"].any() and not out["dC"].any()


def test_scan_of_very_many_short_sequences():
    """2^23 runs of channels: each sequence's outputs and gradients are those that it has alone."""
    N, T, C, S = 1 << 15, 4, 4096, 16
    args, kw = ts.case((N, T), C, S, 1, BF, seed=1)
    dy = randn((N, T, C), BF, 11)
    y, last = kdn.selective_scan(*args, **kw)
    for n in (0, 1, 9999, N - 1):
        one = [v if i == 2 else v[n:n + 1] for i, v in enumerate(args)]
        wy, ws = kdn.selective_scan(*one, **dict(kw, z=kw["z"][n:n + 1]))
        # (few runs go to another kernel, whose sums are in another order)
        rows = tuple(v if i == 2 else v[0] for i, v in enumerate(one))
        ts.check(rows, dict(kw, z=kw["z"][n]), None, y[n], last[n:n + 1], [slice(0, T)], [0])
        ts.check(rows, dict(kw, z=kw["z"][n]), None, wy[0], ws, [slice(0, T)], [0])
    del last
    like = torch.empty_like
    out = dict(dx=like(dy), ddelta=like(dy), dz=like(dy), dB=like(args[3]), dC=like(args[4]), dA=like(args[2]), dD=like(kw["D"]),
               ddelta_bias=like(kw["D"]), dS0=None)
    d = kdn.selective_scan_backward(*args, dy, out=out, **kw)
    for n in (0, 1, 9999, N - 1):
        one = [v if i == 2 else v[n:n + 1] for i, v in enumerate(args)]
        g = kdn.selective_scan_backward(*one, dy[n:n + 1], **dict(kw, z=kw["z"][n:n + 1]))
        for k in ("dx", "ddelta", "dz"):
            assert torch.equal(d[k][n:n + 1], g[k]), k
    assert all(torch.isfinite(d[k]).all() for k in ("dB", "dC", "dA", "dD", "ddelta_bias"))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,C,S", [(2, 5, 20, 16), (1, 70, 33, 8), (2, 2333, 33, 32), (2, 2333, 33, 16), (300, 37, 80, 16)])
def test_states_that_forget_at_once(dtype, B, T, C, S):
    """A = -inf in some states: exp(dt A) is zero at every token and one at none, whatever the
    length leaves of a tile."""
    args, kw = ts.case((B, T), C, S, 1, dtype, seed=T)
    S0 = randn((B, C, S), F32, 9)
    A, far = args[2].clone(), args[2].clone()
    A[:, ::3], far[:, ::3] = -math.inf, -1e30
    A[3] = -math.inf
    far[3] = -1e30
    y, last = kdn.selective_scan(*args[:2], A, *args[3:], S0=S0, **kw)
    want, state = kdn.selective_scan(*args[:2], far, *args[3:], S0=S0, **kw)
    assert torch.isfinite(y).all() and torch.equal(y, want) and torch.equal(last, state)
    tok = lambda a: [v if i == 2 else v[:, 0] for i, v in enumerate(args[:2] + (a,) + args[3:])]  # noqa: E731
    kw["z"] = kw["z"][:, 0]
    a, b = S0.clone(), S0.clone()
    assert torch.equal(kdn.selective_decode(*tok(A), a, **kw), kdn.selective_decode(*tok(far), b, **kw)) and torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("S", [8, 16, 32])
@pytest.mark.parametrize("C,G", [(24, 1), (7, 1), (40, 2)])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_a_non_finite_state_stays_in_its_channel_and_state(dtype, S, C, G, bad):
    """The last state of a group's last channel, whose run has lanes behind its channels."""
    T, per = 100, C // G
    args, kw = ts.case((1, T), C, S, G, dtype, seed=S)
    S0, dS, dy = randn((1, C, S), F32, 9), randn((1, C, S), F32, 10), randn((1, T, C), dtype, 11)
    want = kdn.selective_scan_backward(*args, dy, S0=S0, dS_out=dS, **kw)
    S0[0, per - 1, S - 1] = dS[0, per - 1, S - 1] = bad
    got = kdn.selective_scan_backward(*args, dy, S0=S0, dS_out=dS, **kw)
    for k in ("dB", "dC"):
        assert torch.equal(got[k][:, :, 1:], want[k][:, :, 1:]) and torch.equal(got[k][..., :-1], want[k][..., :-1]), k
    rest = torch.arange(C, device="cuda") != per - 1
    for k in ("dx", "ddelta", "dz"):
        assert torch.equal(got[k][..., rest], want[k][..., rest]), k
    for k in ("dA", "dD", "ddelta_bias"):
        assert torch.equal(got[k][rest], want[k][rest]), k
    assert torch.equal(got["dA"][per - 1, :-1], want["dA"][per - 1, :-1])
    assert torch.equal(got["dS0"][0, rest], want["dS0"][0, rest])
    assert torch.equal(got["dS0"][0, per - 1, :-1], want["dS0"][0, per - 1, :-1])


@pytest.mark.parametrize("dtype,stream", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("scale", ["none", "one", "channel"])
@pytest.mark.parametrize("rows,D", [(2500, 1543), (1100, 4096), (3001, 513), (40000, 100)])
def test_rounds_of_residual_gradients(dtype, stream, scale, rows, D):
    """Several rounds of a workgroup over rows wider than a wave (and one case of rows within
    one): the row ahead, the turns of the sums' memory, the last round that is not full."""
    x, res = randn((rows, D), dtype, 1), randn((rows, D), stream, 2, size=3.0)
    w = 1 + randn((D,), F32, 3, size=0.3)
    s = None if scale == "none" else 0.5 + randn((1 if scale == "one" else D,), F32, 4, size=0.3)
    dy = randn((rows, D), dtype, 5)
    tn.check_residual(x, res, w, s, dy, randn((rows, D), stream, 6))
    tn.check_residual(x, res, w, s, dy, None)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("order,act", tn.KINDS)
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("tokens,H,d", [(1700, 3, 1000), (1100, 3, 2048), (2100, 2, 515)])
def test_rounds_of_gated_gradients(dtype, order, act, per_head, tokens, H, d):
    gate = act != "no gate"
    act = act if gate else "silu"
    x, z, w, dy = tn.case((tokens,), H, d, dtype, per_head, seed=d, gate=gate)
    g = kdn.gated_norm_backward(x, w, dy, z, eps=tn.EPS, order=order, activation=act)
    tn.check_gated(x, z, w, dy, order, act, dtype, None, g)
    again = kdn.gated_norm_backward(x, w, dy, z, eps=tn.EPS, order=order, activation=act)
    assert all(g[k] is None or torch.equal(g[k], again[k]) for k in g)
