"""Host-side refusals of the linear-attention entry points and of the packed
batch's tables (no GPU needed): through the C ABI with fake addresses, none of
which is ever read, and through the binding with host tensors."""
import ctypes

import pytest
import torch

from linear_attention_recurrent_delta_amd import kdn

OK, ENULL, ESHAPE, EUNSUP, EALIGN, EALIAS, EHIP, EWS, ESCRATCH = range(9)
A, MB = 1 << 32, 1 << 26
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    return kdn.ensure_built()


def packed(tokens=100, block=64, max_blocks=None, pool=8, blocks=A + 20 * MB,
           block_offsets=A + 21 * MB, slots=A + 22 * MB, N=4):
    rows = kdn.load().kdn_sequence_max_blocks(N, tokens, block) if max_blocks is None else max_blocks
    return kdn.Packed(tokens, block, rows, pool, blocks, block_offsets, slots)


def prefill(lib, dtype=BF16, N=2, T=100, H=4, Hq=4, Hk=4, Hv=4, dk=64, dv=64, gate=0, qs=0, ks=0,
            vs=0, q=A, k=A + MB, v=A + 2 * MB, la=A + 3 * MB, S0=A + 4 * MB, o=A + 6 * MB,
            S=A + 8 * MB, pk=None, ws=A + 12 * MB, wsb=MB):
    return lib.kdn_linear_prefill(dtype, N, T, H, Hq, Hk, Hv, dk, dv, gate, qs, ks, vs, q, k, v, la,
                                  S0, o, S, pk, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), EUNSUP), (dict(gate=2), EUNSUP), (dict(gate=-1), EUNSUP), (dict(dk=32), EUNSUP),
    (dict(dv=256), EUNSUP), (dict(dk=0), ESHAPE), (dict(N=-1), ESHAPE), (dict(T=-1), ESHAPE),
    (dict(H=-4), ESHAPE), (dict(Hq=3), ESHAPE), (dict(Hk=0), ESHAPE), (dict(Hv=8), ESHAPE),
    (dict(N=1 << 20, T=1 << 20), ESHAPE), (dict(N=1 << 24, T=1, H=1 << 10, Hq=1, Hk=1, Hv=1), ESHAPE),
    (dict(qs=4 * 64 - 8), ESHAPE), (dict(ks=4 * 64 + 4), EALIGN), (dict(vs=1 << 31), ESHAPE), (dict(vs=1 << 25), ESHAPE), (dict(dtype=F32, qs=1 << 24), ESHAPE),
    (dict(dtype=F32, vs=4 * 64 + 2), EALIGN),
    (dict(q=None), ENULL), (dict(k=None), ENULL), (dict(v=None), ENULL), (dict(la=None), ENULL),
    (dict(o=None), ENULL), (dict(q=A + 8), EALIGN), (dict(o=A + 6 * MB + 4), EALIGN),
    (dict(S0=A + 4 * MB + 4), EALIGN), (dict(S=A + 8 * MB + 8), EALIGN), (dict(la=A + 3 * MB + 1), EALIGN),
    (dict(gate=1, la=A + 3 * MB + 2), EALIGN),
    (dict(o=A), EALIAS), (dict(o=A + 2 * MB + 16), EALIAS), (dict(S=A + 4 * MB + 16), EALIAS),
    (dict(S=A + 6 * MB), EALIAS), (dict(o=A + 4 * MB), EALIAS),
    # rows of o of 64 MiB: a chunk of them would pass 2^32 bytes
    (dict(N=1, T=1, H=1 << 19, Hv=1, dv=64), ESHAPE), (dict(N=1, T=1, H=1 << 18, Hv=1, dv=64, dtype=F32), ESHAPE),
    # o inside the wide rows that v is a slice of
    (dict(vs=4096, o=A + 2 * MB + 199 * 4096 * 2), EALIAS),
    (dict(T=1000, ws=None), EWS), (dict(T=1000, wsb=100), EWS), (dict(T=1000, ws=A + 12 * MB + 64), EALIGN),
    (dict(T=1000, ws=A + 8 * MB), EALIAS), (dict(T=1000, ws=A), EALIAS),
])
def test_prefill_refusals(lib, kw, want):
    if "T" in kw and kw["T"] == 1000:
        kw = dict(kw, wsb=kw.get("wsb", 8 * MB))
    assert prefill(lib, **kw) == want


@pytest.mark.parametrize("pk,kw,want", [
    (dict(), dict(T=5), ESHAPE), (dict(tokens=-1, max_blocks=3), dict(), ESHAPE),
    (dict(block=63, max_blocks=5), dict(), ESHAPE), (dict(block=0, max_blocks=5), dict(), ESHAPE),
    (dict(max_blocks=4), dict(), ESHAPE), (dict(max_blocks=6), dict(), ESHAPE),
    (dict(pool=-1), dict(), ESHAPE), (dict(blocks=None), dict(), ENULL),
    (dict(block_offsets=None), dict(), ENULL), (dict(blocks=A + 20 * MB + 4), dict(), EALIGN),
    (dict(block_offsets=A + 2), dict(), EALIGN), (dict(slots=A + 1), dict(), EALIGN),
    (dict(), dict(ws=None), EWS), (dict(), dict(wsb=8), EWS),
    (dict(blocks=A + 6 * MB), dict(wsb=64 * MB), EALIAS), (dict(slots=A + 8 * MB), dict(), EALIAS),
    (dict(), dict(ws=A + 21 * MB), EALIAS),
])
def test_packed_refusals(lib, pk, kw, want):
    args = dict(N=4, T=0)
    args.update(kw)
    assert prefill(lib, pk=packed(**pk), **args) == want


def test_prefill_workspace_size(lib):
    st = ctypes.c_int(0)
    size = lambda *a, pk=None: (lib.kdn_linear_prefill_workspace_size(*a, pk, ctypes.byref(st)), st.value)
    assert size(BF16, 1, 190, 16, 128, 128) == (0, OK)            # one block per sequence
    assert size(BF16, 1, 0, 16, 128, 128) == (0, OK)
    assert size(BF16, 0, 100, 16, 128, 128) == (0, OK)
    block = lib.kdn_linear_block(32768, 2, 16)
    n = 2 * -(-16384 // block) * 16
    assert size(BF16, 2, 16384, 16, 128, 128) == (n * 65536 + -(-n * 4 // 256) * 256, OK)
    rows = lib.kdn_sequence_max_blocks(4, 100, 64)
    n = rows * 2
    assert size(F32, 4, 0, 2, 64, 64, pk=packed()) == (n * 16384 + 256, OK)
    for bad in [(5, 1, 1, 1, 64, 64), (F32, -1, 1, 1, 64, 64), (F32, 1, 1, 1, 48, 64)]:
        assert size(*bad)[0] == 0 and st.value in (ESHAPE, EUNSUP)
    assert lib.kdn_linear_prefill_workspace_size(BF16, 1, 1, 1, 48, 64, None, None) == 0


def decode(lib, dtype=BF16, N=3, H=4, Hq=4, Hk=4, Hv=4, dk=64, dv=64, gate=0, qs=0, ks=0, vs=0, q=A,
           k=A + MB, v=A + 2 * MB, la=A + 3 * MB, slots=A + 4 * MB, pool=10, S=A + 5 * MB,
           o=A + 9 * MB):
    return lib.kdn_linear_decode(dtype, N, H, Hq, Hk, Hv, dk, dv, gate, qs, ks, vs, q, k, v, la, slots,
                                 pool, S, o, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=9), EUNSUP), (dict(gate=3), EUNSUP), (dict(dk=96), EUNSUP), (dict(N=-1), ESHAPE),
    (dict(Hq=8), ESHAPE), (dict(pool=-1), ESHAPE), (dict(slots=None, pool=2), ESHAPE),
    (dict(q=None), ENULL), (dict(la=None), ENULL), (dict(S=None), ENULL), (dict(o=None), ENULL),
    (dict(S=A + 5 * MB + 8), EALIGN), (dict(slots=A + 4 * MB + 2), EALIGN), (dict(qs=260), EALIGN),
    (dict(vs=128), ESHAPE), (dict(o=A + 5 * MB), EALIAS), (dict(o=A), EALIAS), (dict(S=A), EALIAS),
    (dict(slots=A + 9 * MB), EALIAS),
])
def test_decode_refusals(lib, kw, want):
    assert decode(lib, **kw) == want


def tables(lib, N=5, tokens=100, block=64, rows=None, lengths=A, slots=A + MB, context=A + 2 * MB,
           offsets=A + 3 * MB, block_offsets=A + 4 * MB, blocks=A + 5 * MB, slot_map=A + 6 * MB,
           positions=A + 7 * MB):
    rows = lib.kdn_sequence_max_blocks(N, tokens, block) if rows is None else rows
    return lib.kdn_sequence_tables(N, tokens, block, rows, lengths, slots, context, offsets,
                                   block_offsets, blocks, slot_map, positions, None)


@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), ESHAPE), (dict(tokens=-1), ESHAPE), (dict(block=0), ESHAPE), (dict(block=65), ESHAPE),
    (dict(rows=5), ESHAPE), (dict(rows=7), ESHAPE), (dict(lengths=None), ENULL), (dict(offsets=None), ENULL),
    (dict(block_offsets=None), ENULL), (dict(blocks=None), ENULL), (dict(blocks=A + 5 * MB + 8), EALIGN),
    (dict(lengths=A + 2), EALIGN), (dict(positions=A + 1), EALIGN), (dict(offsets=A), EALIAS),
    (dict(slot_map=A + MB), EALIAS), (dict(positions=A + 6 * MB + 396), EALIAS),
])
def test_tables_refusals(lib, kw, want):
    assert tables(lib, **kw) == want


def test_block_sizes(lib):
    assert lib.kdn_sequence_max_blocks(0, 100, 64) == 0
    assert lib.kdn_sequence_max_blocks(3, 0, 64) == 0
    assert lib.kdn_sequence_max_blocks(3, 2, 64) == 2
    assert lib.kdn_sequence_max_blocks(3, 128, 64) == 5
    assert lib.kdn_sequence_max_blocks(2 ** 31 - 1, 2 ** 31 - 1, 64) == 2 ** 31 - 1
    for bad in [(-1, 1, 64), (1, -1, 64), (1, 1, 0), (1, 1, 100)]:
        assert lib.kdn_sequence_max_blocks(*bad) == -1
    for n in [(0, 0, 0), (1, 1, 1), (16384, 1, 16), (2 ** 31 - 1, 1, 2 ** 31 - 1)]:
        b = lib.kdn_linear_block(*n)
        assert b >= 64 and b % 64 == 0
    assert lib.kdn_linear_block(-1, 1, 1) == -1


# ---------------------------------------------------------------------------
# The binding.
# ---------------------------------------------------------------------------
def z(*s, dt=torch.bfloat16):
    return torch.zeros(s, dtype=dt)


def test_binding_prefill_refusals():
    q, la = z(2, 8, 4, 64), z(2, 8, 4)
    call = kdn.linear_prefill
    with pytest.raises(ValueError, match="GPU memory"):
        call(q, q, q, la)
    with pytest.raises(ValueError, match="dtype"):
        call(q.half(), q.half(), q.half(), la.half())
    with pytest.raises(ValueError, match="dtype"):
        call(q, q.float(), q, la)
    with pytest.raises(ValueError, match="shape"):
        call(q, q[:, :4], q, la)
    with pytest.raises(ValueError, match="shape"):
        call(q[0], q[0], q[0], la[0])                       # packed rows without tables
    with pytest.raises(ValueError, match="divide"):
        call(q, z(2, 8, 3, 64), q, la)
    with pytest.raises(ValueError, match="contiguous heads"):
        call(z(2, 8, 64, 4).transpose(2, 3), q, q, la)
    with pytest.raises(ValueError, match="contiguous heads"):
        call(z(8, 2, 4, 64).transpose(0, 1), q, q, la)      # rows not at one distance
    with pytest.raises(ValueError, match="contiguous heads"):
        call(z(1, 8, 4, 64).expand(2, 8, 4, 64), q, q, la)
    with pytest.raises(TypeError, match="log_alpha"):
        call(q, q, q, None)
    with pytest.raises(TypeError, match="k must be"):
        call(q, None, q, la)


def test_binding_decode_and_tables_refusals():
    q, la = z(5, 4, 64), z(5, 4)
    with pytest.raises(ValueError, match="GPU memory"):
        kdn.linear_decode(q, q, q, la, torch.zeros(5, 4, 64, 64))
    with pytest.raises(ValueError, match="shape"):
        kdn.linear_decode(z(1, 5, 4, 64), q, q, la, torch.zeros(5, 4, 64, 64))
    with pytest.raises(ValueError):
        kdn.linear_decode(q, q, q, la, torch.zeros(5, 4, 64))
    with pytest.raises(ValueError, match="GPU memory"):
        kdn.sequence_tables(torch.zeros(3, dtype=torch.int32), 10, 64)
    with pytest.raises(ValueError, match="lengths"):
        kdn.sequence_tables([1, 2], 10, 64)
    for block in (0, 63, -64):
        with pytest.raises(kdn.KdnError):
            kdn.sequence_tables(torch.zeros(3, dtype=torch.int32), 10, block)
    with pytest.raises(kdn.KdnError):
        kdn.sequence_tables(torch.zeros(3, dtype=torch.int32), -1, 64)
    with pytest.raises(kdn.KdnError):
        kdn.linear_block(-1, 1, 1)


def backward(lib, dtype=BF16, N=2, T=100, H=4, Hq=4, Hk=4, Hv=4, dk=64, dv=64, gate=0, qs=0, ks=0,
             vs=0, q=A, k=A + MB, v=A + 2 * MB, la=A + 3 * MB, S0=A + 4 * MB, do=A + 6 * MB,
             dS=A + 8 * MB, dq=A + 10 * MB, dkk=A + 11 * MB, dvv=A + 12 * MB, dla=A + 13 * MB,
             dS0=A + 14 * MB, pk=None, ws=A + 16 * MB, wsb=MB):
    return lib.kdn_linear_prefill_backward(dtype, N, T, H, Hq, Hk, Hv, dk, dv, gate, qs, ks, vs, q, k,
                                           v, la, S0, do, dS, dq, dkk, dvv, dla, dS0, pk, ws, wsb,
                                           None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), EUNSUP), (dict(dk=96), EUNSUP), (dict(Hv=3), ESHAPE), (dict(T=-1), ESHAPE),
    (dict(do=None), ENULL), (dict(dq=None), ENULL), (dict(dkk=None), ENULL), (dict(dvv=None), ENULL),
    (dict(do=A + 6 * MB + 2), EALIGN), (dict(dS=A + 8 * MB + 4), EALIGN), (dict(dla=A + 13 * MB + 1), EALIGN),
    (dict(dq=A), EALIAS), (dict(dkk=A + 10 * MB), EALIAS), (dict(dvv=A + 6 * MB), EALIAS),
    (dict(dla=A + 3 * MB), EALIAS), (dict(dS0=A + 8 * MB), EALIAS), (dict(dS0=A + 4 * MB), EALIAS),
    (dict(wsb=1000), EWS), (dict(ws=None), EWS), (dict(ws=A + 16 * MB + 128), EALIGN),
    (dict(ws=A + 14 * MB), EALIAS), (dict(ws=A + 6 * MB), EALIAS),
    (dict(T=0, N=4, pk="max"), ESHAPE), (dict(T=3, N=4, pk="ok"), ESHAPE),
])
def test_backward_refusals(lib, kw, want):
    kw = dict(kw)
    if kw.get("pk"):
        kw["pk"] = packed(max_blocks=99) if kw["pk"] == "max" else packed()
    assert backward(lib, **kw) == want


def test_backward_workspace_size(lib):
    st = ctypes.c_int(0)

    def size(*a, pk=None):
        n = lib.kdn_linear_prefill_backward_workspace_size(*a, pk, ctypes.byref(st))
        return n, st.value

    chunk = lambda tokens, blocks, C, H, d, es: (tokens // C + blocks + 1) * H * d * d * es
    assert size(BF16, 1, 190, 4, 4, 4, 4, 64, 64, 0) == (chunk(190, 1, 64, 4, 64, 2), OK)
    # shared heads and one decay per head
    assert size(F32, 1, 100, 4, 2, 4, 1, 64, 64, 1) == (
        chunk(100, 1, 32, 4, 64, 4) + 2 * 100 * 4 * 64 * 4 + 256, OK)
    rows = lib.kdn_sequence_max_blocks(4, 100, 64)
    assert size(BF16, 4, 0, 2, 2, 2, 2, 64, 64, 0, pk=packed()) == (
        2 * (rows * 2 * 16384 + 256) + chunk(100, rows, 64, 2, 64, 2), OK)
    assert size(BF16, 0, 5, 4, 4, 4, 4, 64, 64, 0) == (0, OK)
    assert size(BF16, 1, 5, 4, 3, 4, 4, 64, 64, 0) == (0, ESHAPE)


def test_binding_backward_refusals():
    q, la = z(2, 8, 4, 64), z(2, 8, 4)
    call = kdn.linear_prefill_backward
    with pytest.raises(ValueError, match="GPU memory"):
        call(q, q, q, q, la)
    with pytest.raises(ValueError, match="dtype"):
        call(q.half(), q.half(), q.half(), q.half(), la.half())
    with pytest.raises(TypeError, match="q must be"):
        call(None, q, q, q, la)


def test_reference_gradients_against_differences():
    """The reference's own reverse recurrence (tests/linear_ref.py), in 64 bits."""
    import linear_ref as ref
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    T, H, dk, dv = 7, 2, 3, 4
    x = dict(q=rnd(T, H, dk), k=rnd(T, H, dk), v=rnd(T, H, dv), la=-rnd(T, H).abs(),
             S0=rnd(H, dk, dv))
    do, dS = rnd(T, H, dv), rnd(H, dk, dv)

    def loss(y):
        o, S, _, _ = ref.forward(y["q"], y["k"], y["v"], torch.exp(y["la"]), y["S0"])
        return ((o * do).sum() + (S * dS).sum()).item()

    grads, _ = ref.backward(x["q"], x["k"], x["v"], torch.exp(x["la"]), do, x["S0"], dS)
    for n, name in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("la", "dlog_alpha"), ("S0", "dS0")):
        for _ in range(5):
            way = rnd(*x[n].shape)
            up, down = (loss(dict(x, **{n: x[n] + e * way})) for e in (1e-5, -1e-5))
            want = (grads[name] * way).sum().item()
            assert abs((up - down) / 2e-5 - want) <= 1e-7 * (1 + abs(want)) * 10


def test_binding_q_must_be_a_tensor():
    x, la = z(2, 8, 4, 64), z(2, 8, 4)
    for call in (lambda: kdn.linear_prefill(None, x, x, la), lambda: kdn.linear_decode([1.0], x, x, la, x),
                 lambda: kdn.linear_prefill_backward(None, x, x, x, la)):
        with pytest.raises(TypeError, match="q must be"):
            call()
