"""Sizes at which the linear-attention entry points have to refuse a call, on the
host (no GPU needed): fake addresses, none of which is ever read."""
import pytest
import torch

import linear_ref as ref
import linear_tight as tight
from linear_attention_recurrent_delta_amd import kdn
from test_linear_host import (A, BF16, EALIAS, EALIGN, ESHAPE, EUNSUP, EWS, F32, MB, backward, decode,
                              packed, prefill)

M = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return kdn.ensure_built()


# A launch has less than 2^32 work-items, 2^24 workgroups of 256.
@pytest.mark.parametrize("kw", [
    dict(N=16 * M, T=1, H=1, Hq=1, Hk=1, Hv=1), dict(N=M, T=1, H=16, Hq=16, Hk=16, Hv=16),
    dict(N=M + 64, T=1, H=16, Hq=1, Hk=1, Hv=1), dict(N=2 * M, T=1, H=16, Hq=1, Hk=1, Hv=16),
    dict(N=M, T=0, H=16, Hq=16, Hk=16, Hv=16), dict(dtype=F32, N=16 * M, T=7, H=1, Hq=1, Hk=1, Hv=1)])
def test_prefill_past_one_launch(lib, kw):
    assert prefill(lib, **kw) == ESHAPE


def test_packed_prefill_past_one_launch(lib):
    heads = dict(H=16, Hq=16, Hk=16, Hv=16)
    assert prefill(lib, N=M, T=0, pk=packed(tokens=64 * M, N=M), **heads) == ESHAPE
    # few blocks, but a state of each sequence to pass on
    assert prefill(lib, N=M, T=0, pk=packed(tokens=100, N=M), **heads) == ESHAPE


@pytest.mark.parametrize("kw", [
    dict(N=16 * M, H=1, Hq=1, Hk=1, Hv=1), dict(N=M + 64, H=16, Hq=16, Hk=16, Hv=16)])
def test_decode_past_one_launch(lib, kw):
    assert decode(lib, **kw) == ESHAPE


@pytest.mark.parametrize("kw", [
    dict(N=16 * M, T=1, H=1, Hq=1, Hk=1, Hv=1),                              # the walk, 4 waves
    dict(N=8 * M, T=1, H=1, Hq=1, Hk=1, Hv=1, dk=128),                       # 8 waves
    dict(N=8 * M, T=0, H=1, Hq=1, Hk=1, Hv=1),                               # the joins
    dict(N=1, T=90 * M, H=2, Hq=1, Hk=1, Hv=1, dtype=BF16),                  # the shared heads' sums
])
def test_gradients_past_one_launch(lib, kw):
    assert backward(lib, **kw) == ESHAPE


def test_no_heads(lib):
    """No states: nothing to do, in every form."""
    none = dict(H=0, Hq=0, Hk=0, Hv=0)
    assert prefill(lib, **none) == 0 and backward(lib, **none) == 0 and decode(lib, **none) == 0
    assert prefill(lib, N=4, T=0, pk=packed(), **none) == 0


@pytest.mark.parametrize("N,tokens,block", [(4, 10, 64), (3, 200, 64), (3, 10, 128)])
def test_refused_tables_keep_their_description(lib, monkeypatch, N, tokens, block):
    """sequence_tables into given tables: what a refused call was to make is not
    written into them, whether a size does not fit or the call itself fails (the
    last case: its tensors are not in GPU memory)."""
    def same(name, x, shape, dtype, dev):
        if x is not None and x.shape != shape:
            raise ValueError(name)

    monkeypatch.setattr(kdn, "_same", same)      # host tensors pass, wrong sizes do not
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32)
    slots = i32(3)
    t = kdn.SequenceTables(10, 64, i32(4), i32(4), i32(3, 4), slots, i32(10), i32(10))
    with pytest.raises(ValueError):
        kdn.sequence_tables(i32(N), tokens, block, slots=i32(N), out=t)
    assert (t.tokens, t.block) == (10, 64) and t.slots is slots


# ---------------------------------------------------------------------------
# The gradient of one decay per head in float32.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kw,want", [
    (dict(gate=3), EUNSUP), (dict(gate=2, dla=A + 13 * MB + 2), EALIGN),
    (dict(gate=2, la=A + 3 * MB + 2), EALIGN),
    # 4 heads: 8 bytes in bfloat16, 16 in float32
    (dict(gate=1, dla=A + 14 * MB - 8, wsb=0), EWS), (dict(gate=2, dla=A + 14 * MB - 16, wsb=0), EWS),
    (dict(gate=2, dla=A + 14 * MB - 8, wsb=0), EALIAS)])
def test_float32_gate_gradient_refusals(lib, kw, want):
    assert backward(lib, **kw) == want


def test_float32_gate_gradient_sizes_and_forward(lib):
    size = lambda gate: lib.kdn_linear_prefill_backward_workspace_size(
        BF16, 2, 300, 4, 4, 2, 4, 64, 64, gate, None, None)
    assert size(kdn.GATE_HEAD_F32) == size(kdn.GATE_HEAD) > size(kdn.GATE_TOKEN)
    assert prefill(lib, gate=kdn.GATE_HEAD_F32) == EUNSUP and decode(lib, gate=kdn.GATE_HEAD_F32) == EUNSUP


@pytest.mark.parametrize("size", range(len(tight.SIZES)))
def test_bound_of_returned_states_tells_two_parts_from_three(size):
    """What test_gpu_linear_limits.py holds returned states to: three parts are
    inside, two are not, in either direction."""
    T, live, _, chunks, blocks = tight.SIZES[size]
    x = tight.case(T, live, 4, 64, 128, torch.bfloat16, seed=size)
    S, M, R, MR = tight.wanted(*x)
    for parts in (2, 3):
        for got, want, m in zip(tight.planted(*x, parts), (S, R), (M, MR)):
            inside = ((got - want).abs() <= tight.bound(m, len(live), chunks, blocks)).all()
            assert inside == (parts == 3)


@pytest.mark.parametrize("x", [2 ** 32 + 64, 2 ** 31, -2 ** 32 + 64])
def test_sizes_of_more_than_32_bits(lib, x):
    """The library takes 32-bit sizes: what does not fit is refused, not cut off."""
    lengths = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: kdn.sequence_tables(lengths, x, 64), lambda: kdn.sequence_tables(lengths, 64, x),
                 lambda: kdn.linear_block(x, 3, 4), lambda: kdn.linear_block(64, x, 4),
                 lambda: kdn.linear_block(64, 3, x),
                 lambda: kdn.sequence_tables(lengths[:1].expand(abs(x)), 64, 64)):
        with pytest.raises(kdn.KdnError, match="SHAPE"):
            call()


@pytest.mark.parametrize("T,per_head", [(1, True), (40, True), (300, True), (1, False), (40, False)])
def test_bound_of_flows_tells_one_part_from_two(T, per_head):
    """What test_gpu_linear_limits.py holds d log_alpha to, as a sum over tokens or
    a token's own: two bf16 parts of the states are inside, one is not."""
    x = tight.flow_case(T, 8, 64, 128, per_head, seed=T)
    q, k, v, la, do, S0, dS = x
    a = torch.exp(la.double()).expand(T, 8)
    w, m = ref.backward(*(y.double() for y in (q, k, v)), a, do.double(), S0.double(), dS.double())
    bound = tight.flow_bound(w["dlog_alpha"], m, q, k)
    assert (tight.flow_in_parts(*x, 8) - w["dlog_alpha"]).abs().max() <= 1e-12 * m["dlog_alpha"].max()
    for parts in (1, 2):
        off = tight.flow_in_parts(*x, parts) - w["dlog_alpha"]
        if per_head:
            assert (off.sum(0).abs() <= bound.sum(0)).all() == (parts == 2)
            assert (off.sum(0).abs() > bound.sum(0)).all() == (parts == 1)
        else:
            assert (off.abs() <= bound).all() == (parts == 2)
