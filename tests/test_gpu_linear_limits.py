"""Linear attention and the packed batch's tables on the GPU at the ends of their
ranges, against the recurrence in 64 bits (tests/linear_ref.py)."""
import pytest
import torch

import linear_ref as ref
import linear_tight as tight
from linear_attention_recurrent_delta_amd import kdn
from test_gpu_linear import BF, F32, check_packed, i32, make, packed_case, state
from test_gpu_linear_backward import check as check_gradients, randn

pytestmark = pytest.mark.gpu
NEVER_CUT = 2 ** 31 - 64         # the longest block there is


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    kdn.ensure_built()


# ---------------------------------------------------------------------------
# Blocks of any length.
# ---------------------------------------------------------------------------
def block_tables(lengths, tokens, block):
    """offsets, block_offsets and blocks in plain Python, for any number of tokens."""
    offsets, block_offsets, blocks = [0], [0], []
    for n, length in enumerate(lengths):
        first = offsets[-1]
        end = min(first + max(length, 0), tokens)
        for i, at in enumerate(range(first, end, block)):
            blocks.append([at, min(block, end - at), n, i])
        offsets.append(end)
        block_offsets.append(len(blocks))
    rows = min(tokens, tokens // block + len(lengths))
    return offsets, block_offsets, blocks + [[0, 0, -1, 0]] * (rows - len(blocks))


@pytest.mark.parametrize("lengths,tokens,block", [
    ([65], 65, NEVER_CUT), ([64], 64, NEVER_CUT), ([1], 1, NEVER_CUT), ([100, 0, 70, 1, 64], 300, NEVER_CUT),
    ([2 ** 31 - 1, 5], 1000, NEVER_CUT), ([300] * 4097, 300 * 4097, NEVER_CUT),
    ([2 ** 31 - 6, 5], 2 ** 31 - 1, NEVER_CUT), ([2 ** 31 - 6, 5], 2 ** 31 - 1, 2 ** 30),
    ([2 ** 30 + 1, 2 ** 30 - 3], 2 ** 31 - 1, 2 ** 30), ([2 ** 30, 2 ** 30 - 1], 2 ** 31 - 1, 2 ** 20)])
def test_tables_with_long_blocks(lengths, tokens, block):
    t = kdn.sequence_tables(i32(lengths), tokens, block)
    for name, got, want in zip(("offsets", "block_offsets", "blocks"),
                               (t.offsets, t.block_offsets, t.blocks),
                               block_tables(lengths, tokens, block)):
        same = got.tolist() == want          # no diff of long lists
        assert same, name


@pytest.mark.parametrize("dtype", [BF, F32])
def test_packed_never_cut(dtype):
    """Every sequence one block, whatever its length: outputs, states, gradients."""
    lengths, H, d = [65, 0, 300, 1, 64], 2, 64
    q, k, v, la, t = packed_case(lengths, 3, H, d, d, dtype, 17, NEVER_CUT)
    assert t.block_offsets.tolist() == [0, 1, 1, 2, 3, 4]
    S0 = state(5, H, d, d)
    S, o = torch.full_like(S0, 3.0), torch.full(v.shape, 7.0, dtype=dtype, device="cuda")
    before, o_before = S.clone(), o.clone()
    kdn.linear_prefill(q, k, v, la, S0=S0, tables=t, out=(o, S))
    check_packed(q, k, v, la, lengths, None, S0, o, S, before, o_before)
    do, dS = randn(v.shape, dtype, 3), state(5, H, d, d, seed=2)
    got = kdn.linear_prefill_backward(q, k, v, do, la, S0=S0, dS_out=dS, tables=t)
    for x in (q, k, v, la, do):
        x[-3:] = 0
    ends = torch.tensor(lengths).cumsum(0).tolist()
    check_gradients(q, k, v, la, do, S0, dS, got, [slice(e - n, e) for e, n in zip(ends, lengths)],
                    list(range(5)))


def test_gradients_of_a_long_skipped_sequence():
    """A sequence of 2^26 tokens without a slot has zero gradients (its groups of
    4 channels pass 2^31); the one behind it has its own."""
    long, n, dk, dv = 2 ** 26 + 5, 70, 128, 64
    rows = long + n
    x = make((n,), 1, 1, 1, 1, dk, dv, BF, seed=5)
    do, S0 = randn((n, 1, dv), BF, 6), state(1, 1, dk, dv)
    want = kdn.linear_prefill_backward(
        x[0], x[0], x[0][..., :dv], do, x[3], S0=S0,
        tables=kdn.sequence_tables(i32([n]), n, NEVER_CUT, slots=i32([0])))
    q, la, d = (torch.empty((rows, 1) + s, dtype=BF, device="cuda") for s in ((dk,), (), (dv,)))
    for big, small in ((q, x[0]), (la, x[3]), (d, do)):
        big[long:] = small
    out = {name: torch.full((rows, 1) + s, 7.0, dtype=BF, device="cuda")
           for name, s in (("dq", (dk,)), ("dk", (dk,)), ("dv", (dv,)), ("dlog_alpha", ()))}
    out["dS0"] = torch.full_like(S0, 7.0)
    t = kdn.sequence_tables(i32([long, n]), rows, NEVER_CUT, slots=i32([-1, 0]))
    kdn.linear_prefill_backward(q, q, q[..., :dv], d, la, S0=S0, tables=t, out=out)
    for name in ("dq", "dk", "dv", "dlog_alpha"):
        assert not out[name][:long].any(), name
        assert torch.equal(out[name][long:], want[name]), name
    assert torch.equal(out["dS0"], want["dS0"])
    del q, la, d, out, big
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------
# The largest launches.
# ---------------------------------------------------------------------------
def test_largest_launches():
    """2^24 - 16 workgroups run; of 2^24 and more the runtime would start some
    only, and they are refused."""
    H, d = 16, 64
    for N in (2 ** 20 - 1, 2 ** 20, 2 ** 20 + 64):
        q = randn((N, 1, 1, d), BF, 4)
        la = torch.zeros(N, 1, H, dtype=BF, device="cuda")
        o = torch.full((N, 1, H, d), 7.0, dtype=BF, device="cuda")
        S = torch.zeros(1, H, d, d, device="cuda")
        slots = torch.full((N,), -1, dtype=torch.int32, device="cuda")
        slots[-1] = 0
        calls = (lambda: kdn.linear_prefill(q, q, q, la, out=(o, None)),
                 lambda: kdn.linear_decode(q[:, 0], q[:, 0], q[:, 0], la[:, 0], S, slots=slots))
        if N >= 2 ** 20:
            for call in calls:
                with pytest.raises(kdn.KdnError, match="SHAPE"):
                    call()
            continue
        calls[0]()
        # one token from nothing: o = (q . k) v, with q k^T and o rounded to bf16,
        # and float32 sums of 64 channels
        want = q.double().square().sum(-1, keepdim=True) * q.double()
        near = lambda x, y: ((x.double() - y).abs() <= 2.02 * 2.0 ** -8 * y.abs()).all()
        assert near(o, want)
        assert near(calls[1]()[-1], want[-1, 0])


def test_refused_tables_keep_their_description():
    lengths, slots = i32([30, 0, 70]), i32([2, 0, 1])
    t = kdn.sequence_tables(lengths, 100, 64, slots=slots, maps=True)
    want = [x.clone() for x in (t.offsets, t.block_offsets, t.blocks, t.slot_map, t.positions)]
    for args in ((i32([1, 2]), 100, 64), (lengths, 300, 64), (lengths, 101, 64)):
        with pytest.raises(ValueError):
            kdn.sequence_tables(*args, out=t)
    assert (t.tokens, t.block) == (100, 64) and t.slots is slots
    for x, y in zip((t.offsets, t.block_offsets, t.blocks, t.slot_map, t.positions), want):
        assert torch.equal(x, y)
    assert kdn.sequence_tables(i32([0, 5, 9]), 100, 64, out=t) is t and t.slots is None
    assert t.offsets.tolist() == [0, 0, 5, 14]


# ---------------------------------------------------------------------------
# The gradient of one decay per head in float32.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cut", [False, True])
def test_float32_gate_gradient(dtype, cut):
    """The same sum rounded once to float32: its bf16 rounding is what the call's
    type gives, and the sum itself has more bits."""
    H, d = 5, 64
    q, k, v, la = make((2, 500 if cut else 90), H, H, H, H, d, d, dtype, "head", seed=6)
    do, S0 = randn(v.shape, dtype, 3), state(2, H, d, d)
    want = kdn.linear_prefill_backward(q, k, v, do, la, S0=S0)
    out = {n: torch.full_like(x, 7.0) for n, x in want.items()}
    out["dlog_alpha"] = torch.full((H,), 7.0, device="cuda")
    got = kdn.linear_prefill_backward(q, k, v, do, la, S0=S0, out=out)
    assert got["dlog_alpha"] is out["dlog_alpha"] and want["dlog_alpha"].dtype == dtype
    assert torch.equal(got["dlog_alpha"].to(dtype), want["dlog_alpha"])
    if dtype == BF:
        assert (got["dlog_alpha"] != want["dlog_alpha"].float()).any()
    for n in ("dq", "dk", "dv", "dS0"):
        assert torch.equal(got[n], want[n]), n
    B, T = q.shape[:2]
    flat = lambda x: x.flatten(0, 1)
    check_gradients(flat(q), flat(k), flat(v), la, flat(do), S0, None,
                    {n: x if n in ("dlog_alpha", "dS0") else flat(x) for n, x in got.items()},
                    [slice(b * T, b * T + T) for b in range(B)], list(range(B)))


# ---------------------------------------------------------------------------
# Returned states are float32.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("size", range(len(tight.SIZES)))
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shared", [False, True])
def test_returned_states_keep_24_bits(size, dk, dv, dtype, shared):
    T, live, block, chunks, blocks = tight.SIZES[size]
    if dtype == F32:
        chunks = sum(-(-min(block, T - at) // 32) for at in range(0, T, block))
    H = 4
    x = tight.case(T, live, H, dk, dv, dtype, seed=size)
    if shared:                         # neighbours with the same q and k
        for y in x[:2]:
            y[:] = y[:, :1]
    S, M, R, MR = tight.wanted(*x)
    q, k, v, la, do, S0, dS = (y.cuda() for y in x)
    N = 1
    if shared:                         # as many as make them share a workgroup
        q, k, N = q[:, :1], k[:, :1], 130
    q, k, v, la, do = (y.repeat(N, *[1] * (y.dim() - 1)) for y in (q, k, v, la, do))
    S0, dS = S0.repeat(N, 1, 1, 1), dS.repeat(N, 1, 1, 1)
    t = kdn.sequence_tables(i32([T] * N), N * T, block)
    assert t.block_offsets[:2].tolist() == [0, blocks]
    got = kdn.linear_prefill(q, k, v, la, S0=S0.clone(), tables=t)[1]
    ref.close("S", got[0], S, tight.bound(M, len(live), chunks, blocks))
    assert (got == got[0]).all()
    got = kdn.linear_prefill_backward(q, k, v, do, la, S0=S0, dS_out=dS, tables=t)["dS0"]
    ref.close("dS0", got[0], R, tight.bound(MR, len(live), chunks, blocks))
    assert (got == got[0]).all()


# ---------------------------------------------------------------------------
# Packed batches with one decay per head, in a workspace that holds anything.
# ---------------------------------------------------------------------------
def junk(n):
    """A workspace whose floats are all NaN."""
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("lengths", [[1], [5, 0, 64, 1, 129, 0], [300, 2, 500, 65], [0, 0, 700, 0],
                                     [(23 * n * n + 5 * n) % 211 for n in range(44)]],
                         ids=lambda x: f"{len(x)}x{sum(x)}")
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block", [64, 256])
@pytest.mark.parametrize("Hk", [2, 1])
def test_packed_constant_decays(lengths, dtype, block, Hk):
    """Empty sequences, skipped ones and rows behind the last: none adds to the
    decays' gradient, and nothing is read from the workspace that was not
    written."""
    N, H, d, tail = len(lengths), 2, 64, 3
    P, total = N + 3, sum(lengths) + tail
    slots = [P - 1 - n for n in range(N)]
    if N > 3:
        slots[1], slots[3] = -1, P
    q, k, v, la = make((total,), H, Hk, H, H, d, d, dtype, "head", seed=N)
    do = randn(v.shape, dtype, 3)
    for x in (q, k, v, do):
        x[total - tail:] = float("nan")
    ends = torch.tensor(lengths).cumsum(0).tolist()
    spans = [slice(e - n, e) for e, n in zip(ends, lengths)]
    if N > 3:
        q[spans[1]] = float("nan")
    S0, dS = state(P, H, d, d), state(P, H, d, d, seed=2)
    t = kdn.sequence_tables(i32(lengths), total, block, slots=i32(slots))
    pk, _ = kdn._packed(t, P, q.device)
    lib, kind = kdn.load(), kdn.DTYPES[dtype]

    S, o = S0.clone(), torch.full(v.shape, 7.0, dtype=dtype, device="cuda")
    o_before = o.clone()
    ws = junk(lib.kdn_linear_prefill_workspace_size(kind, N, 0, H, d, d, pk, None))
    kdn.linear_prefill(q, k, v, la, S0=S, tables=t, out=(o, S), workspace=ws)
    wide = [x.repeat_interleave(H // x.shape[1], 1) for x in (q, k)]
    check_packed(*wide, v, la.expand(total, H), lengths, slots, S0, o, S, S0, o_before)

    ws = junk(lib.kdn_linear_prefill_backward_workspace_size(kind, N, 0, H, H, Hk, H, d, d,
                                                             kdn.GATE_HEAD, pk, None))
    got = kdn.linear_prefill_backward(q, k, v, do, la, S0=S0, dS_out=dS, tables=t, workspace=ws)
    for x in (q, k, v, do):
        x[total - tail:] = 0
    if N > 3:
        q[spans[1]] = 0
    live = [s if 0 <= s < P else -1 for s in slots]
    check_gradients(q, k, v, la, do, S0, dS, got, spans, live)
    for p in set(range(P)) - set(live):
        assert not got["dS0"][p].any()


def test_tables_of_the_most_sequences():
    """2^31 - 1 sequences: the tiles of the scan end at the last one (a 32-bit
    counter of them would pass 2^31 and start again before the first)."""
    N, tokens = 2 ** 31 - 1, 1000
    live = {5: 70, 4096: 1, N - 4097: 64, N - 4095: 130, N - 2: 3}
    lengths = torch.zeros(N, dtype=torch.int32, device="cuda")
    for n, length in live.items():
        lengths[n] = length
    t = kdn.sequence_tables(lengths, tokens, 64, maps=True)
    at, blocks = 0, []
    for n, length in live.items():
        assert t.offsets[n].item() == at and t.block_offsets[n].item() == len(blocks)
        assert (t.slot_map[at:at + length] == n).all()
        assert t.positions[at:at + length].tolist() == list(range(length))
        blocks += [[at + i, min(64, length - i), n, i // 64] for i in range(0, length, 64)]
        at += length
        assert t.offsets[n + 1].item() == at and t.block_offsets[n + 1].item() == len(blocks)
    assert t.offsets[N].item() == at and t.block_offsets[N].item() == len(blocks)
    assert t.blocks[:len(blocks)].tolist() == blocks
    assert (t.blocks[len(blocks):] == i32([0, 0, -1, 0])).all() and (t.slot_map[at:] == -1).all()
    del t, lengths
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------
# d log_alpha beyond the rounding of its operands.
# ---------------------------------------------------------------------------
def flow_call(x, dk, dv, block, per_head):
    q, k, v, la, do, S0, dS = (y.cuda() for y in x)
    T, H = do.shape[:2]
    out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
               dlog_alpha=torch.full_like(la, 7.0), dS0=torch.empty_like(S0)[None])
    rows, tables = [q, k, v, do], None
    if block:
        tables = kdn.sequence_tables(i32([T]), T, block)
    else:
        rows = [y[None] for y in rows]
        for n in ("dq", "dk", "dv") if per_head else ("dq", "dk", "dv", "dlog_alpha"):
            out[n] = out[n][None]
        la = la if per_head else la[None]
    kdn.linear_prefill_backward(*rows, la, S0=S0[None], dS_out=dS[None], tables=tables, out=out)
    return out["dlog_alpha"] if per_head or block else out["dlog_alpha"][0]


def flow_wanted(x):
    q, k, v, la, do, S0, dS = x
    T, H = q.shape[:2]
    a = torch.exp(la.double()).expand(T, H)
    w, m = ref.backward(*(y.double() for y in (q, k, v)), a, do.double(), S0.double(), dS.double())
    return w["dlog_alpha"], tight.flow_bound(w["dlog_alpha"], m, q, k)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T,block", [(1, 0), (40, 0), (64, 0), (200, 0), (300, 0), (150, 64), (300, 512)])
def test_sum_over_tokens_is_not_of_rounded_states(dk, dv, T, block):
    """One decay per head, dense (one block or several) and packed."""
    x = tight.flow_case(T, 8, dk, dv, True, seed=T)
    w, bound = flow_wanted(x)
    got = flow_call(x, dk, dv, block, True)
    ref.close("dlog_alpha", got, w.sum(0), 2.0 ** -24 * w.sum(0).abs() + bound.sum(0))


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T", [1, 2, 40, 64])
def test_flows_of_one_chunk_are_not_of_rounded_states(dk, dv, T):
    """Decays per token, sequences of one chunk: the values' own rounding, 2^-8."""
    x = tight.flow_case(T, 8, dk, dv, False, seed=T)
    w, bound = flow_wanted(x)
    ref.close("dlog_alpha", flow_call(x, dk, dv, 0, False), w, 2.0 ** -8 * w.abs() + 1.01 * bound)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T,block", [(1, 0), (50, 0), (186, 0), (300, 0), (300, 128)])
def test_sum_over_tokens_of_any_inputs(dk, dv, T, block):
    """All channels live, sums that cancel: the same bound, over absolute values."""
    H = 3
    q, k, v, la = make((T,), H, H, H, H, dk, dv, BF, "head", seed=T)
    x = (q, k, v, la, randn(v.shape, BF, 3), state(1, H, dk, dv)[0], 0.2 * state(1, H, dk, dv, seed=2)[0])
    x = [y.cpu() for y in x]
    w, bound = flow_wanted(x)
    got = flow_call(x, dk, dv, block, True)
    ref.close("dlog_alpha", got, w.sum(0), 2.0 ** -24 * w.sum(0).abs() + bound.sum(0))
