"""Linear attention with a decay for each head on the GPU -- prefill (dense and
packed), decode and the packed batch's tables -- against the recurrence in 64
bits, within bounds that count every rounding (tests/linear_ref.py)."""
import math

import numpy as np
import pytest
import torch

import linear_ref as ref
from linear_attention_recurrent_delta_amd import kdn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    kdn.ensure_built()


def make(lead, Hq, Hk, Hv, H, dk, dv, dtype, gate="token", seed=0, fused=False, decay=0.1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    q, k, v = rnd(*lead, Hq, dk), rnd(*lead, Hk, dk), rnd(*lead, Hv, dv)
    k = k / k.norm(dim=-1, keepdim=True)
    if gate == "head":
        la = torch.log1p(-torch.exp2(-4.0 - torch.arange(H, device="cuda") * 5.0 / H))
    else:
        la = (-torch.nn.functional.softplus(rnd(*lead, H)) * decay).to(dtype)
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    if fused:
        parts = [x.flatten(-2) for x in (q, k, v)]
        pad = torch.full(lead + (16,), float("nan"), dtype=dtype, device="cuda")
        x = torch.cat([pad] + parts + [pad], -1)
        _, q, k, v, _ = x.split([16] + [p.shape[-1] for p in parts] + [16], -1)
        q, k, v = (y.unflatten(-1, (n, -1)) for y, n in ((q, Hq), (k, Hk), (v, Hv)))
    return q, k, v, la


def state(P, H, dk, dv, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return 0.5 * torch.randn(P, H, dk, dv, generator=g, device="cuda")


def check_dense(q, k, v, la, S0, o, S, H):
    B, T, dk, dv = q.shape[0], q.shape[1], q.shape[-1], v.shape[-1]
    a = ref.decay(la, (B, T), H)
    Q, K, V = ref.wide(q, H), ref.wide(k, H), ref.wide(v, H)
    for b in range(B):
        s0 = torch.zeros(H, dk, dv, dtype=torch.float64) if S0 is None else S0[b].cpu().double()
        ro, rS, m, M = ref.forward(Q[b], K[b], V[b], a[b], s0)
        ref.close(f"o[{b}]", o[b], ro, ref.o_bound(ro, m, T, dk, q.dtype))
        if S is not None:
            ref.close(f"S[{b}]", S[b], rS, ref.S_bound(M, T, dk, q.dtype))


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 200, 256, 257, 700])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_lengths(T, dtype):
    q, k, v, la = make((2, T), 2, 2, 2, 2, 128, 128, dtype, seed=T)
    S0 = state(2, 2, 128, 128)
    o, S = kdn.linear_prefill(q, k, v, la, S0=S0)
    check_dense(q, k, v, la, S0, o, S, 2)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gate", ["token", "head"])
def test_prefill_sizes(dk, dv, dtype, gate):
    q, k, v, la = make((1, 300), 3, 3, 3, 3, dk, dv, dtype, gate, seed=dk + dv)
    o, S = kdn.linear_prefill(q, k, v, la)
    check_dense(q, k, v, la, None, o, S, 3)


@pytest.mark.parametrize("Hq,Hk,Hv,H", [(1, 1, 6, 6), (6, 2, 2, 6), (2, 3, 6, 6), (6, 6, 1, 6),
                                        (1, 1, 1, 4), (5, 5, 5, 5)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_shared_heads_and_strides(Hq, Hk, Hv, H, dtype):
    q, k, v, la = make((2, 90), Hq, Hk, Hv, H, 64, 128, dtype, seed=H, fused=True)
    S0 = state(2, H, 64, 128)
    o, S = kdn.linear_prefill(q, k, v, la, S0=S0)
    check_dense(q, k, v, la, S0, o, S, H)


@pytest.mark.parametrize("Hq,Hk,H", [(1, 1, 2), (2, 1, 4), (3, 3, 6), (1, 2, 4), (2, 2, 6)])
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gate", ["token", "head"])
def test_prefill_neighbours_with_the_same_q_and_k(Hq, Hk, H, dk, dtype, gate):
    """Heads of 64 columns, whose neighbours have q and k in common: outputs,
    states, and the blocks of a cut sequence, each head with its own decay."""
    q, k, v, la = make((2, 330), Hq, Hk, H, H, dk, 64, dtype, gate, seed=H + dk, fused=True)
    if gate == "token":
        la[:, 100, 1::2] = -math.inf
    S0 = state(2, H, dk, 64)
    o, S = kdn.linear_prefill(q, k, v, la, S0=S0)
    check_dense(q, k, v, la, S0, o, S, H)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_neighbours_keep_their_infinities(dtype):
    """A value, a start or a decay that is not finite stays in its head."""
    q, k, v, la = make((1, 600), 2, 2, 4, 4, 128, 64, dtype, seed=21)
    S0 = state(1, 4, 128, 64)
    o, S = kdn.linear_prefill(q, k, v, la, S0=S0)
    v[:, 70, 1], la[:, 90, 2], S0[:, 3] = math.inf, math.nan, math.nan
    o2, S2 = kdn.linear_prefill(q, k, v, la, S0=S0)
    assert torch.equal(o[:, :, 0], o2[:, :, 0]) and torch.equal(S[:, 0], S2[:, 0])
    assert torch.equal(o[:, :64, 1:3], o2[:, :64, 1:3])
    assert not torch.isfinite(S2[:, 1:]).flatten(2).all(-1).any()
    assert o2[:, :, 3].isnan().all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [-math.inf, -1e30, -120.0, -7.0, 0.0])
@pytest.mark.parametrize("share", [0.03, 0.5, 1.0])
def test_prefill_strong_decays_and_resets(dtype, value, share):
    q, k, v, la = make((1, 290), 2, 2, 2, 2, 64, 64, dtype, seed=7)
    g = torch.Generator(device="cuda").manual_seed(8)
    la = torch.where(torch.rand(la.shape, generator=g, device="cuda") < share,
                     torch.full_like(la, value), la)
    S0 = state(1, 2, 64, 64)
    o, S = kdn.linear_prefill(q, k, v, la, S0=S0)
    check_dense(q, k, v, la, S0, o, S, 2)


def test_prefill_reset_drops_what_was_there():
    """Behind a reset nothing of a large state is left, not even a rounding."""
    q, k, v, la = make((1, 100), 2, 2, 2, 2, 64, 64, F32, seed=3)
    la[:, 70] = -math.inf
    big = torch.full((1, 2, 64, 64), 1e30, device="cuda")
    o, S = kdn.linear_prefill(q, k, v, la, S0=big)
    o2, S2 = kdn.linear_prefill(q[:, 70:].contiguous(), k[:, 70:].contiguous(),
                                v[:, 70:].contiguous(), la[:, 70:].contiguous())
    m = o2.abs().max()
    assert (o[:, 70:] - o2).abs().max() <= 1e-5 * m and (S - S2).abs().max() <= 1e-5 * S2.abs().max()


def test_prefill_continues():
    """A prompt in two pieces, the state in place, as one call."""
    q, k, v, la = make((2, 500), 4, 4, 4, 4, 128, 64, BF, seed=11)
    S0 = state(2, 4, 128, 64)
    S = S0.clone()
    cut = [x.contiguous() for y in (q, k, v, la) for x in (y[:, :201], y[:, 201:])]
    o1, r1 = kdn.linear_prefill(cut[0], cut[2], cut[4], cut[6], S0=S, out=(
        torch.empty(2, 201, 4, 64, dtype=BF, device="cuda"), S))
    o2, r2 = kdn.linear_prefill(cut[1], cut[3], cut[5], cut[7], S0=S, out=(
        torch.empty(2, 299, 4, 64, dtype=BF, device="cuda"), S))
    assert r1 is S and r2 is S
    check_dense(q, k, v, la, S0, torch.cat([o1, o2], 1), S, 4)


def test_prefill_without_state_output_and_empty():
    q, k, v, la = make((1, 600), 2, 2, 2, 2, 64, 64, BF, seed=5)
    o = torch.full((1, 600, 2, 64), float("nan"), dtype=BF, device="cuda")
    _, S = kdn.linear_prefill(q, k, v, la, out=(o, None))
    assert S is None
    check_dense(q, k, v, la, None, o, None, 2)
    # no tokens: the states pass through; no sequences: nothing
    S0 = state(3, 2, 64, 64)
    z = lambda n, t, *s: torch.zeros(n, t, *s, dtype=BF, device="cuda")
    o, S = kdn.linear_prefill(z(3, 0, 2, 64), z(3, 0, 2, 64), z(3, 0, 2, 64), z(3, 0, 2), S0=S0)
    assert o.shape == (3, 0, 2, 64) and torch.equal(S, S0)
    o, S = kdn.linear_prefill(z(3, 0, 2, 64), z(3, 0, 2, 64), z(3, 0, 2, 64), z(3, 0, 2))
    assert not S.any()
    o, S = kdn.linear_prefill(z(0, 5, 2, 64), z(0, 5, 2, 64), z(0, 5, 2, 64), z(0, 5, 2))
    assert o.shape == (0, 5, 2, 64) and S.shape == (0, 2, 64, 64)


def test_prefill_runs_alike():
    q, k, v, la = make((2, 900), 4, 4, 4, 4, 128, 128, BF, seed=9)
    a, b = kdn.linear_prefill(q, k, v, la), kdn.linear_prefill(q, k, v, la)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------------------
# Packed batches.
# ---------------------------------------------------------------------------
def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def packed_case(lengths, tail, H, dk, dv, dtype, seed, block, slots=None, pool=None):
    total = sum(max(n, 0) for n in lengths) + tail
    q, k, v, la = make((total,), H, H, H, H, dk, dv, dtype, seed=seed)
    for x in (q, k, v, la):
        if tail:
            x[-tail:] = float("nan")
    t = kdn.sequence_tables(i32(lengths), total, block, slots=None if slots is None else i32(slots))
    return q, k, v, la, t


def check_packed(q, k, v, la, lengths, slots, S0, o, S, before, o_before):
    H, dk, dv = q.shape[-2], q.shape[-1], v.shape[-1]
    at, P = 0, S.shape[0]
    seen = set()
    for n, length in enumerate(lengths):
        rows = slice(at, at + max(length, 0))
        at += max(length, 0)
        slot = n if slots is None else slots[n]
        if not 0 <= slot < P:
            assert torch.equal(o[rows], o_before[rows]), "a skipped sequence's rows were written"
            continue
        seen.add(slot)
        T = max(length, 0)
        a = ref.decay(la[rows], (T,), H)
        s0 = torch.zeros(H, dk, dv, dtype=torch.float64) if S0 is None else S0[slot].cpu().double()
        ro, rS, m, M = ref.forward(ref.wide(q[rows], H), ref.wide(k[rows], H),
                                   ref.wide(v[rows], H), a, s0)
        ref.close(f"o[seq {n}, {T} tokens]", o[rows], ro, ref.o_bound(ro, m, T, dk, q.dtype))
        ref.close(f"S[seq {n}]", S[slot], rS, ref.S_bound(M, T, dk, q.dtype))
    assert torch.equal(o[at:], o_before[at:]), "rows behind the last sequence were written"
    for p in range(P):
        if p not in seen:
            assert torch.equal(S[p], before[p]), f"state {p} belongs to no sequence"


LENGTHS = [[1], [0], [5, 0, 64, 1, 129, 0], [64, 64, 64], [1] * 9, [300, 2, 500, 65],
           [0, 0, 700, 0], [-3, 40, -1, 30]]


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block", [64, 256])
@pytest.mark.parametrize("inplace", [True, False])
def test_packed(lengths, dtype, block, inplace):
    N = len(lengths)
    slots = [(3 * n + 1) % (N + 4) for n in range(N)] if (N + 4) % 3 else list(range(N, 0, -1))
    assert len(set(slots)) == N
    q, k, v, la, t = packed_case(lengths, 5, 2, 64, 64, dtype, 20 + N, block, slots)
    S0 = state(N + 4, 2, 64, 64)
    keep = S0.clone()
    S = S0 if inplace else torch.full_like(S0, 3.0)
    before = S.clone()
    o = torch.full(v.shape, 7.0, dtype=dtype, device="cuda")
    ob = o.clone()
    kdn.linear_prefill(q, k, v, la, S0=S0, tables=t, out=(o, S))
    check_packed(q, k, v, la, lengths, slots, keep, o, S, before, ob)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dv", [64, 128])
def test_packed_many_blocks(dtype, dv):
    """More workgroups than run at once: the blocks are taken longest first.
    Neighbouring heads share q and k, sequences are cut, empty or skipped."""
    lengths = [(37 * n * n + 11 * n) % 331 for n in range(40)]
    lengths[7] = lengths[8] = 0
    H, total = 8, sum(lengths) + 9
    slots = [(7 * n + 3) % 41 for n in range(40)]
    slots[5] = -1
    q, k, v, la = make((total,), 2, 4, H, H, 64, dv, dtype, seed=91)
    t = kdn.sequence_tables(i32(lengths), total, 128, slots=i32(slots))
    assert t.blocks.shape[0] * H > 512
    S = state(41, H, 64, dv)
    keep = S.clone()
    o = torch.full(v.shape, 7.0, dtype=dtype, device="cuda")
    ob = o.clone()
    kdn.linear_prefill(q, k, v, la, S0=S, tables=t, out=(o, S))
    wide = [x.repeat_interleave(H // x.shape[1], 1) for x in (q, k)]
    check_packed(*wide, v, la, lengths, slots, keep, o, S, keep, ob)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_packed_many_states(dtype, dk, dv):
    """So many states that a workgroup joins the whole of one: cut sequences,
    whole ones, empty ones that pass theirs on, skipped ones."""
    lengths = [(53 * n) % 190 if n % 6 else 0 for n in range(172)]
    H, total = 6, sum(lengths) + 3
    slots = [(5 * n + 3) % 173 for n in range(172)]
    slots[9] = slots[12] = -1
    q, k, v, la = make((total,), H, H, H, H, dk, dv, dtype, seed=92)
    t = kdn.sequence_tables(i32(lengths), total, 64, slots=i32(slots))
    S0 = state(173, H, dk, dv)
    S = torch.full_like(S0, 3.0)
    before = S.clone()
    o = torch.full(v.shape, 7.0, dtype=dtype, device="cuda")
    ob = o.clone()
    kdn.linear_prefill(q, k, v, la, S0=S0, tables=t, out=(o, S))
    check_packed(q, k, v, la, lengths, slots, S0, o, S, before, ob)


def test_packed_thousands_of_blocks():
    """So many blocks that they are taken as they come, the same bits as in a
    batch of their first sequences, which are sorted."""
    lengths = [1 + n % 3 for n in range(4200)]
    total, few = sum(lengths), 300
    q, k, v, la, t = packed_case(lengths, 0, 2, 64, 64, BF, 95, 64)
    assert t.blocks.shape[0] > 4096
    o, S = kdn.linear_prefill(q, k, v, la, tables=t)
    rows = sum(lengths[:few])
    t2 = kdn.sequence_tables(i32(lengths[:few]), rows, 64)
    o2, S2 = kdn.linear_prefill(q[:rows], k[:rows], v[:rows], la[:rows], tables=t2)
    assert torch.equal(o[:rows], o2) and torch.equal(S[:few], S2)
    check_packed(q[:rows], k[:rows], v[:rows], la[:rows], lengths[:few], None, None, o2, S2, S2, o2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_packed_skips_sequences_without_a_slot(dtype):
    lengths, slots = [70, 130, 0, 400, 3], [2, -1, 7, 6, 0]       # pool of 6: -1, 7, 6 are none
    q, k, v, la, t = packed_case(lengths, 2, 2, 64, 128, dtype, 31, 128, slots)
    q[70:200] = float("nan")                                      # and are not looked at
    v[200:600] = float("inf")
    S = state(6, 2, 64, 128)
    keep = S.clone()
    o = torch.full(v.shape, 7.0, dtype=dtype, device="cuda")
    ob = o.clone()
    kdn.linear_prefill(q, k, v, la, S0=S, tables=t, out=(o, S))
    check_packed(q, k, v, la, lengths, slots, keep, o, S, keep, ob)


def test_packed_defaults():
    """No slots, no states: new ones; a given pool is updated in place."""
    lengths = [33, 200, 1]
    q, k, v, la, t = packed_case(lengths, 0, 2, 64, 64, BF, 41, 64)
    o, S = kdn.linear_prefill(q, k, v, la, tables=t)
    assert S.shape == (3, 2, 64, 64)
    check_packed(q, k, v, la, lengths, None, None, o, S, S, o)
    S0 = state(3, 2, 64, 64)
    keep = S0.clone()
    o, S = kdn.linear_prefill(q, k, v, la, S0=S0, tables=t)
    assert S is S0
    check_packed(q, k, v, la, lengths, None, keep, o, S, keep, o)


def test_packed_rows_that_do_not_fit_are_skipped():
    """Table rows that reach outside the call's sizes own no tokens."""
    lengths = [100, 100]
    q, k, v, la, t = packed_case(lengths, 0, 1, 64, 64, F32, 51, 64)
    good, _ = kdn.linear_prefill(q, k, v, la, tables=t)
    for row, bad in [(3, (190, 36, 1, 1)), (3, (164, 65, 1, 1)), (3, (-1, 36, 1, 1)),
                     (3, (164, 36, 2, 1)), (3, (164, 36, -1, 1)), (3, (164, 36, 1, 5)),
                     (3, (2147483647, 36, 1, 1))]:
        t2 = kdn.sequence_tables(i32(lengths), 200, 64)
        t2.blocks[row] = i32(bad)
        o = torch.full(v.shape, 7.0, device="cuda")
        S = torch.zeros(2, 1, 64, 64, device="cuda")
        kdn.linear_prefill(q, k, v, la, tables=t2, out=(o, S))
        torch.cuda.synchronize()
        assert torch.equal(o[:164], good[:164]) and (o[164:] == 7.0).all()


def test_packed_rows_of_any_length_are_sorted():
    """Lengths that no table has: the rows are skipped, the others computed."""
    lengths = [40] * 150
    q, k, v, la, t = packed_case(lengths, 0, 2, 64, 64, F32, 52, 64)
    good, _ = kdn.linear_prefill(q, k, v, la, tables=t)
    for n, bad in ((3, -2 ** 31), (9, 2 ** 31 - 1), (20, -1), (149, 65)):
        t.blocks[n, 1] = bad
    o = torch.full(v.shape, 7.0, device="cuda")
    S = torch.zeros(150, 2, 64, 64, device="cuda")
    kdn.linear_prefill(q, k, v, la, tables=t, out=(o, S))
    skipped = torch.zeros(150, 40, dtype=torch.bool, device="cuda")
    skipped[[3, 9, 20, 149]] = True
    skipped = skipped.flatten()
    assert torch.equal(o[~skipped], good[~skipped]) and (o[skipped] == 7.0).all()


# ---------------------------------------------------------------------------
# Tables.
# ---------------------------------------------------------------------------
TABLES = [([], 0, 64), ([], 10, 64), ([0], 0, 64), ([5], 5, 64), ([5], 9, 64), ([70, 0, 0, 1], 80, 64),
          ([64, 128, 129, 0, 63], 400, 64), ([10, -5, 20, -2 ** 31], 40, 128),
          ([100, 100, 100], 150, 64), ([2 ** 31 - 1, 2 ** 31 - 1, 5], 1000, 256),
          ([0] * 5000 + [3], 10, 64), ([1] * 4096, 4096, 64), ([1] * 4097, 4100, 64),
          ([2, 0, 3] * 4000, 20000, 64), ([200000, 1, 100000], 300007, 1024),
          ([300] * 100, 20000, 64)]


@pytest.mark.parametrize("case", range(len(TABLES)))
@pytest.mark.parametrize("extra", [False, True])
def test_tables(case, extra):
    lengths, tokens, block = TABLES[case]
    N = len(lengths)
    rng = np.random.RandomState(case)
    slots = rng.permutation(N + 3)[:N].tolist() if extra else None
    ctx = rng.randint(0, 1000, N).tolist() if extra else None
    want = ref.tables(lengths, tokens, block, slots, ctx)
    dev = lambda x: None if x is None else i32(x)
    t = kdn.sequence_tables(dev(lengths), tokens, block, slots=dev(slots), context=dev(ctx), maps=True)
    got = (t.offsets, t.block_offsets, t.blocks, t.slot_map, t.positions)
    for name, g, w in zip(("offsets", "block_offsets", "blocks", "slot_map", "positions"), got, want):
        assert np.array_equal(g.cpu().numpy(), w), name
    t2 = kdn.sequence_tables(dev(lengths), tokens, block)
    assert t2.slot_map is None and np.array_equal(t2.blocks.cpu().numpy(), want[2])


# ---------------------------------------------------------------------------
# Decode.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,H,Hq,Hk,Hv", [(1, 1, 1, 1, 1), (3, 6, 2, 1, 6), (130, 8, 8, 8, 8)])
@pytest.mark.parametrize("gate", ["token", "head"])
def test_decode(dk, dv, dtype, N, H, Hq, Hk, Hv, gate):
    q, k, v, la = make((N,), Hq, Hk, Hv, H, dk, dv, dtype, gate, seed=N, fused=N == 3)
    slots = torch.randperm(N + 5)[:N].tolist()
    if N > 1:
        slots[1] = -1
    if N > 100:
        slots[-3:] = [-1, N + 5, 2 ** 31 - 1]
    S = state(N + 5, H, dk, dv)
    before = S.clone()
    o = torch.full((N, H, dv), 7.0, dtype=dtype, device="cuda")
    kdn.linear_decode(q, k, v, la, S, slots=i32(slots), o=o)
    a = ref.decay(la, (N,), H)
    Q, K, V = ref.wide(q, H), ref.wide(k, H), ref.wide(v, H)
    live = [n for n in range(N) if 0 <= slots[n] < N + 5]
    at = [slots[n] for n in live]
    s = before[at].cpu().double() * a[live][:, :, None, None]
    kv = K[live][..., :, None] * V[live][..., None, :]
    new, mag = s + kv, s.abs() + kv.abs()
    ro = (new * Q[live][..., None]).sum(-2)
    m = (mag * Q[live].abs()[..., None]).sum(-2)
    # the decay is off by 2^-23 and its argument's rounding, the rest float32
    tiny = (dk + 64) * 2.0 ** -23
    ref.close("o", o[live], ro, ref.HALF[dtype] * ro.abs() + tiny * m)
    ref.close("S", S[at], new, 16 * 2.0 ** -23 * mag)
    dead = [n for n in range(N) if n not in live]
    assert (o[dead] == 7.0).all()
    rest = [p for p in range(N + 5) if p not in at]
    assert torch.equal(S[rest], before[rest])


def test_decode_resets_and_defaults():
    q, k, v, la = make((4,), 2, 2, 2, 2, 64, 64, F32, seed=2)
    la[1] = -math.inf
    S = state(4, 2, 64, 64)
    S[1] = 1e30
    o = kdn.linear_decode(q, k, v, la, S)
    want = k[1][:, :, None] * v[1][:, None, :]
    assert torch.equal(S[1], want)
    assert torch.isfinite(o).all()
    o = kdn.linear_decode(q, k, v, la, S, slots=i32([-1, 0, -1, 1]))
    assert not o[0].any() and not o[2].any() and o[1].any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_then_tokens(dtype):
    """Tables, a packed prefill into a pool, then single tokens from it: as one
    sequence each."""
    lengths, H, d, extra = [40, 300, 7], 4, 64, 3
    slots = [4, 0, 2]
    full = [make((1, n + extra), H, H, H, H, d, d, dtype, seed=60 + n) for n in lengths]
    pack = [torch.cat([f[i][0, :n] for f, n in zip(full, lengths)]) for i in range(4)]
    total = sum(lengths)
    t = kdn.sequence_tables(i32(lengths), total, kdn.linear_block(total, 3, H), slots=i32(slots),
                            maps=True)
    assert t.slot_map.tolist() == [4] * 40 + [0] * 300 + [2] * 7
    S = torch.zeros(5, H, d, d, device="cuda")
    o, _ = kdn.linear_prefill(*pack, S0=S, tables=t)
    outs = []
    for i in range(extra):
        tok = [torch.stack([f[j][0, n + i] for f, n in zip(full, lengths)]) for j in range(4)]
        outs.append(kdn.linear_decode(*tok, S, slots=t.slots))
    at = 0
    for n, (f, length) in enumerate(zip(full, lengths)):
        got = torch.cat([o[at:at + length], torch.stack([x[n] for x in outs])])
        at += length
        check_dense(*f, None, got[None], S[slots[n]][None], H)


# ---------------------------------------------------------------------------
# Streams, graphs, long offsets.
# ---------------------------------------------------------------------------
def test_other_stream():
    q, k, v, la = make((1, 600), 4, 4, 4, 4, 64, 64, BF, seed=13)
    want = kdn.linear_prefill(q, k, v, la)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = kdn.linear_prefill(q, k, v, la, stream=s)
    junk = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")   # may reuse freed memory
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    del junk


def test_captured_step():
    """A serving step -- tables, prefill into the pool, a decode step -- captured
    once and replayed on new lengths, slots and inputs."""
    N, H, d, cap = 4, 2, 64, 700
    buf = make((cap,), H, H, H, H, d, d, BF, seed=70)
    tok = make((N,), H, H, H, H, d, d, BF, seed=71)
    lengths, slots = i32([1, 1, 1, 1]), i32([0, 1, 2, 3])
    pool = torch.zeros(6, H, d, d, device="cuda")
    o = torch.zeros(cap, H, d, dtype=BF, device="cuda")
    o1 = torch.zeros(N, H, d, dtype=BF, device="cuda")
    t = kdn.sequence_tables(lengths, cap, 128, slots=slots, maps=True)
    ws = kdn.linear_workspace(*buf, tables=t)

    def step():
        kdn.sequence_tables(lengths, cap, 128, slots=slots, out=t)
        kdn.linear_prefill(*buf, S0=pool, tables=t, out=(o, pool), workspace=ws)
        kdn.linear_decode(*tok, pool, slots=slots, o=o1)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, (ln, sl) in enumerate([([5, 0, 300, 64], [5, 1, 0, 2]), ([200, 200, 200, 100], [3, 2, 1, 0]),
                                  ([1, 2, 3, 4], [0, -1, 4, 5]), ([0, 0, 0, 0], [0, 1, 2, 3])]):
        for x, y in zip(buf + tok, make((cap,), H, H, H, H, d, d, BF, seed=80 + i)
                        + make((N,), H, H, H, H, d, d, BF, seed=90 + i)):
            x.copy_(y)
        lengths.copy_(i32(ln))
        slots.copy_(i32(sl))
        pool.copy_(state(6, H, d, d, seed=i))
        o.fill_(0)
        o1.fill_(0)
        start = pool.clone()
        step()
        torch.cuda.synchronize()
        want = (o.clone(), o1.clone(), pool.clone(), t.slot_map.clone())
        pool.copy_(start)
        o.fill_(0)
        o1.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((o, o1, pool, t.slot_map), want):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Rows so far apart, and a pool so large, that bytes and elements pass 2^31."""
    T, H, d = 140, 1, 64
    wide = 2 ** 25 - 8                                 # elements between tokens: 140 * 2^25 > 2^32
    buf = torch.empty(T * wide, dtype=BF, device="cuda")
    q, k, v, la = make((1, T), H, H, H, H, d, d, BF, seed=3)
    parts = []
    for i, x in enumerate((q, k, v)):
        y = buf[i * 64: i * 64 + (T - 1) * wide + d].as_strided((1, T, H, d), (T * wide, wide, d, 1))
        y.copy_(x)
        parts.append(y)
    o, S = kdn.linear_prefill(*parts, la)
    want = kdn.linear_prefill(q, k, v, la)
    assert torch.equal(o, want[0]) and torch.equal(S, want[1])
    del buf, parts, y
    pool = torch.zeros(33000, 4, 128, 128, device="cuda")       # 2.16e9 elements
    q, k, v, la = make((2,), 4, 4, 4, 4, 128, 128, BF, seed=4)
    o = kdn.linear_decode(q, k, v, la, pool, slots=i32([32999, 32768]))
    small = torch.zeros(2, 4, 128, 128, device="cuda")
    assert torch.equal(o, kdn.linear_decode(q, k, v, la, small))
    assert torch.equal(pool[32999], small[0]) and torch.equal(pool[32768], small[1])
    assert not pool[0].any() and not pool[231].any()
