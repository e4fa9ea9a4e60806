"""Linear attention on the GPU in calls as programs make them: states that
sequences share, slices, two streams at once, captured training steps."""
import math

import pytest
import torch

from linear_attention_recurrent_delta_amd import kdn
from test_gpu_linear import BF, F32, check_dense, check_packed, i32, make, packed_case, state
from test_gpu_linear_backward import check as check_gradients, randn

pytestmark = pytest.mark.gpu
GRADS = ("dq", "dk", "dv", "dlog_alpha", "dS0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    kdn.ensure_built()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sequences_may_share_a_state_that_is_only_read(dtype):
    """One prefix, several continuations: the same slot where no state is written."""
    lengths, slots, H, d = [70, 200, 0, 5, 130], [2, 2, 2, 0, 2], 2, 64
    q, k, v, la, t = packed_case(lengths, 0, H, d, d, dtype, 3, 64, slots)
    S0, dS, do = state(3, H, d, d), state(3, H, d, d, seed=2), randn(v.shape, dtype, 4)
    keep = S0.clone()
    o, S = kdn.linear_prefill(q, k, v, la, S0=S0, tables=t, out=(torch.full_like(v, 7.0), None))
    assert S is None and torch.equal(S0, keep)
    grads = dict(dq=torch.full_like(q, 7.0), dk=torch.full_like(k, 7.0), dv=torch.full_like(v, 7.0),
                 dlog_alpha=torch.full_like(la, 7.0), dS0=None)
    got = kdn.linear_prefill_backward(q, k, v, do, la, S0=S0, dS_out=dS, tables=t, out=grads)
    ends = torch.tensor(lengths).cumsum(0).tolist()
    spans = [slice(e - n, e) for e, n in zip(ends, lengths)]
    check_gradients(q, k, v, la, do, S0, dS, got, spans, slots)
    for n, rows in enumerate(spans):           # outputs: each sequence as a call of its own
        one = kdn.sequence_tables(i32([lengths[n]]), lengths[n], 64, slots=i32([slots[n]]))
        want, _ = kdn.linear_prefill(q[rows], k[rows], v[rows], la[rows], S0=S0, tables=one,
                                     out=(torch.empty_like(v[rows]), None))
        assert torch.equal(o[rows], want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block", [64, 256])
def test_packed_from_nothing_into_a_pool(dtype, block):
    """No S0: the states start at zero and end in their slots, empty ones as zero."""
    lengths, slots, H, d = [70, 0, 300, 1, 64], [4, 0, 6, -1, 2], 2, 64
    q, k, v, la, t = packed_case(lengths, 2, H, d, d, dtype, 5, block, slots)
    S, o = torch.full((7, H, d, d), 3.0, device="cuda"), torch.full_like(v, 7.0)
    before, o_before = S.clone(), o.clone()
    kdn.linear_prefill(q, k, v, la, tables=t, out=(o, S))
    check_packed(q, k, v, la, lengths, slots, None, o, S, before, o_before)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H", [1, 3])
def test_log_decays_at_any_element(dtype, H):
    """log_alpha and its gradient behind an odd number of elements."""
    T, d = 200, 64
    q, k, v, la = make((1, T), H, H, H, H, d, d, dtype, seed=H)
    do, S0 = randn(v.shape, dtype, 4), state(1, H, d, d)

    def odd(x):
        y = torch.full((x.numel() + 8,), math.nan, dtype=dtype, device="cuda")
        y = y[1:1 + x.numel()].view(x.shape)
        return y.copy_(x)

    moved = odd(la)
    assert moved.data_ptr() % 16 == la.element_size() and la.data_ptr() % 16 == 0
    for x, y in zip(kdn.linear_prefill(q, k, v, la, S0=S0), kdn.linear_prefill(q, k, v, moved, S0=S0)):
        assert torch.equal(x, y)
    want = kdn.linear_prefill_backward(q, k, v, do, la, S0=S0)
    out = {n: torch.full_like(x, 7.0) for n, x in want.items()}
    out["dlog_alpha"] = odd(torch.full_like(la, 7.0))
    got = kdn.linear_prefill_backward(q, k, v, do, moved, S0=S0, out=out)
    for n in GRADS:
        assert torch.equal(got[n], want[n]), n
    S, S2 = S0.repeat(T, 1, 1, 1), S0.repeat(T, 1, 1, 1)
    a = kdn.linear_decode(q[0], k[0], v[0], la[0], S)
    b = kdn.linear_decode(q[0], k[0], v[0], odd(la[0]), S2)
    assert torch.equal(a, b) and torch.equal(S, S2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_last_token_of_a_batch(dtype):
    """One token of each sequence out of a longer buffer, and q, k, v of one tensor."""
    B, T, H, d = 5, 9, 2, 64
    q, k, v, la = make((B, T), H, H, H, H, d, d, dtype, seed=3)
    S0, last = state(B, H, d, d), la[:, -1:].contiguous()
    cut = lambda x: x[:, -1:]
    assert not cut(q).is_contiguous()
    want = kdn.linear_prefill(*(cut(x).contiguous() for x in (q, k, v)), last, S0=S0)
    got = kdn.linear_prefill(cut(q), cut(k), cut(v), last, S0=S0)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check_dense(*(cut(x) for x in (q, k, v)), last, S0, *got, H)
    o, S = kdn.linear_prefill(q, q, q, la, S0=S0)
    want = kdn.linear_prefill(q, q.clone(), q.clone(), la, S0=S0)
    assert torch.equal(o, want[0]) and torch.equal(S, want[1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_constant_resets(dtype):
    """A head whose constant decay is -infinity has no memory, its neighbour has."""
    T, H, d = 300, 2, 64
    q, k, v, _ = make((1, T), H, H, H, H, d, d, dtype, seed=8)
    la = torch.tensor([-math.inf, -0.01], device="cuda")
    S0, dS, do = state(1, H, d, d), state(1, H, d, d, seed=2), randn(v.shape, dtype, 4)
    check_dense(q, k, v, la, S0, *kdn.linear_prefill(q, k, v, la, S0=S0), H)
    got = kdn.linear_prefill_backward(q, k, v, do, la, S0=S0, dS_out=dS)
    assert got["dlog_alpha"][0] == 0 and not got["dS0"][0, 0].any()
    check_gradients(q[0], k[0], v[0], la, do[0], S0, dS,
                    {n: x if n in ("dlog_alpha", "dS0") else x[0] for n, x in got.items()},
                    [slice(0, T)], [0])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_what_is_not_finite_stays_in_its_sequence(dtype):
    """Infinities and NaN of one sequence reach no other one, and no output of
    their own head in the chunks before theirs."""
    lengths, H, d = [150, 200, 90], 2, 64
    q, k, v, la, t = packed_case(lengths, 0, H, d, d, dtype, 6, 128)
    S0, dS, do = state(3, H, d, d), state(3, H, d, d, seed=2), randn(v.shape, dtype, 4)
    call = lambda: (kdn.linear_prefill(q, k, v, la, S0=S0, tables=t,
                                       out=(torch.empty_like(v), torch.empty_like(S0))),
                    kdn.linear_prefill_backward(q, k, v, do, la, S0=S0, dS_out=dS, tables=t))
    (o, S), g = call()
    for x, at, bad in ((q, 290, math.nan), (k, 291, math.inf), (v, 292, -math.inf), (do, 293, math.nan)):
        x[at, 0] = bad
    S0[1, 1], dS[1, 0] = math.inf, math.nan
    (o2, S2), g2 = call()
    others = [n for n in range(340) if not 150 <= n < 350 and n < o.shape[0]]
    assert torch.equal(o[others], o2[others]) and torch.equal(S[[0, 2]], S2[[0, 2]])
    assert torch.equal(o[150:278, 0], o2[150:278, 0])       # two chunks of 64 without them
    for n in ("dq", "dk", "dv", "dlog_alpha"):
        assert torch.equal(g[n][others], g2[n][others]), n
    assert torch.equal(g["dS0"][[0, 2]], g2["dS0"][[0, 2]])
    assert o2[300:350, 0].isnan().all() and o2[150:350, 1].isnan().all()


def test_two_calls_at_once():
    """Prefill and gradients on two streams, each with a workspace of its own."""
    H, d = 8, 128
    x = [make((1, 2000), H, H, H, H, d, d, BF, seed=s) for s in (1, 2)]
    do = [randn((1, 2000, H, d), BF, s) for s in (3, 4)]

    def step(i, stream=None):
        o, S = kdn.linear_prefill(*x[i], stream=stream)
        g = kdn.linear_prefill_backward(*x[i][:3], do[i], x[i][3], stream=stream)
        return [o, S] + [g[n] for n in GRADS]

    want = [step(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [step(i, s) for i, s in enumerate(streams)]
        for s in streams:
            s.synchronize()
        for a, b in zip(want, got):
            for y, z in zip(a, b):
                assert torch.equal(y, z)


@pytest.mark.parametrize("gate", ["token", "head"])
def test_captured_packed_training_steps(gate):
    """Tables, prefill and gradients of a packed batch in two graphs that share
    one workspace, replayed in turn on new lengths and inputs with eager work
    between, each replay as the eager call."""
    N, H, d, cap, P = 4, 2, 64, 700, 6
    buf = make((cap,), H, 1, H, H, d, d, BF, gate, seed=1)
    do, dS, S0 = randn((cap, H, d), BF, 2), state(P, H, d, d, seed=3), state(P, H, d, d)
    lengths, slots = i32([1, 1, 1, 1]), i32([0, 1, 2, 3])
    t = kdn.sequence_tables(lengths, cap, 128, slots=slots)
    pk, _ = kdn._packed(t, P, do.device)
    size = kdn.load().kdn_linear_prefill_backward_workspace_size(
        1, N, 0, H, H, 1, H, d, d, kdn.GATE_TOKEN if gate == "token" else kdn.GATE_HEAD, pk, None)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert kdn.linear_workspace(*buf, tables=t).numel() <= size
    o, S = torch.zeros(cap, H, d, dtype=BF, device="cuda"), torch.zeros_like(S0)
    g = dict(dq=torch.zeros_like(buf[0]), dk=torch.zeros_like(buf[1]), dv=torch.zeros_like(buf[2]),
             dlog_alpha=torch.zeros_like(buf[3], dtype=BF), dS0=torch.zeros_like(S0))

    def forward():
        kdn.sequence_tables(lengths, cap, 128, slots=slots, out=t)
        kdn.linear_prefill(*buf, S0=S0, tables=t, out=(o, S), workspace=ws)

    def backward():
        kdn.linear_prefill_backward(*buf[:3], do, buf[3], S0=S0, dS_out=dS, tables=t, out=g,
                                    workspace=ws)

    outs = [o, S] + [g[n] for n in GRADS]
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
        for x, y in zip(buf, make((cap,), H, 1, H, H, d, d, BF, gate, seed=80 + i)):
            x.copy_(y)
        do.copy_(randn(do.shape, BF, 30 + i))
        lengths.copy_(i32(ln))
        slots.copy_(i32(sl))
        for x in outs:
            x.fill_(0)
        forward()
        backward()
        torch.cuda.synchronize()
        want = [x.clone() for x in outs]
        for again in range(2):
            for x in outs:
                x.fill_(0)
            ws.fill_(255)
            for graph in graphs:
                graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs, want):
                assert torch.equal(a, b)
