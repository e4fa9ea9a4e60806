"""Sizes that the operators around a recurrence take and refuse, on the host: what is
counted is what a call launches.  Calls go through the C ABI with an input missing, so that
one whose sizes are taken ends at that."""
import ctypes

import pytest

from linear_attention_recurrent_delta_amd import kdn
from test_around_host import conv, decode, lib, scan, scan_back  # noqa: F401
from test_linear_host import BF16, ENULL, ESHAPE, F32, OK, packed

# sequences, tokens, channels of packed batches
BATCHES = [(256, 65536, 4096), (512, 65536, 6144), (1024, 32768, 4096), (128, 131072, 6144), (256, 131072, 6144),
           (1000, 100000, 6144), (37, 21815, 6144), (1, 1, 1), (4096, 4096, 8192)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,tokens,C", BATCHES)
def test_conv_takes_the_tables_of_a_scan(lib, dtype, N, tokens, C):
    """Tables with blocks of any length, those of selective_block among them."""
    st = ctypes.c_int(0)
    for block in (64, 256, lib.kdn_selective_block(tokens, N, C, 16), 1 << 20, (1 << 31) - 64):
        pk = packed(tokens, block, pool=N, N=N)
        size = lib.kdn_causal_conv_backward_workspace_size(dtype, N, 0, C, 4, pk, ctypes.byref(st))
        assert st.value == OK and size > 0, block
        assert conv(lib, dtype=dtype, N=N, T=0, C=C, pk=pk, x=None) == ENULL, block
        # parts of what tokens and sequences need, not of what the blocks have room for
        once, tiles = max(1, 512 // -(-C // (256 if dtype == BF16 else 128))), 1.25 * (tokens // 64 + N + tokens // block)
        assert size <= 4 * 5 * C * min(once * (1 + tiles // (32 * once)), tiles), block


def test_conv_counts_what_it_launches(lib):
    """2^24 workgroups: tiles of 64 tokens and 512 channels (float32: 256), and one for each sequence."""
    sizes = lambda want, **kw: conv(lib, x=None, **kw) == want  # noqa: E731
    assert sizes(ENULL, N=1, T=64 * (1 << 12), C=512 * 4000) and sizes(ESHAPE, N=1, T=64 * (1 << 12), C=512 * 4096)
    assert sizes(ENULL, dtype=F32, N=1, T=64 * (1 << 12), C=256 * 4000) and sizes(ESHAPE, dtype=F32, N=1, T=64 * (1 << 12), C=256 * 4096)
    assert sizes(ENULL, N=(1 << 23) - 1, T=1, C=512) and sizes(ESHAPE, N=1 << 23, T=1, C=512)
    assert sizes(ENULL, N=(1 << 23) - 1, T=64, C=512) and sizes(ESHAPE, N=(1 << 23) - 1, T=65, C=512)
    assert decode(lib, N=1 << 16, C=16384, x=None, pool=1 << 16) == ENULL
    assert decode(lib, N=1 << 20, C=512 * 64, x=None) == ESHAPE


def test_conv_sums_in_more_parts_of_many_tokens(lib):
    """32 tiles of 64 tokens a part at most, in whole rounds of the workgroups that run at once."""
    size = lambda T, C: lib.kdn_causal_conv_backward_workspace_size(BF16, 1, T, C, 4, None, None) // (4 * 5 * C)  # noqa: E731
    assert size(64 * 1024 - 1, 4096) == size(64 * 1024, 4096) == 32 and size(64 * 1024 + 1, 4096) == 64
    assert size(1 << 20, 6144) == 21 * 25 and size(1 << 20, 1 << 18) == 512 and size(1 << 20, 64) == 512


def test_an_empty_table_has_no_tiles(lib):
    """Tokens and no sequence: nothing to look for."""
    st = ctypes.c_int(0)
    for block in (64, 1 << 20):
        pk = kdn.Packed(1000, block, 0, 0, None, None, None)
        assert lib.kdn_causal_conv_backward_workspace_size(BF16, 0, 0, 64, 4, pk, ctypes.byref(st)) == 0 and st.value == OK


def test_gated_norm_sums_of_many_rows(lib):
    """256 rows of a column at most in one float32 sum."""
    size = lambda *a: lib.kdn_gated_norm_backward_workspace_size(*a, None)  # noqa: E731
    assert size(1 << 22, 1, 64, 0) == 4 * 1024 * 64 and size((1 << 22) + 1, 1, 64, 0) == 4 * 2048 * 64
    assert size(1 << 21, 512, 64, 1) == 4 * 2 * 256 * 512 * 64 and size(1 << 20, 8, 16384, 0) == 4 * 1024 * 32 * 16384


def test_norm_gradients_are_not_counted_by_rows(lib):
    """Gradients launch a workgroup a part, whatever the rows and their type; outputs a row's threads."""
    st, big = ctypes.c_int(0), 1 << 50
    for tokens, H, d, per_head in ((1 << 22, 32, 128, 0), (1 << 22, 32, 128, 1), (1 << 23, 1, 8192, 0), ((1 << 31) - 1, 1, 16, 0)):
        assert lib.kdn_gated_norm_backward_workspace_size(tokens, H, d, per_head, ctypes.byref(st)) > 0 and st.value == OK
        back = lambda dy, dt: lib.kdn_gated_norm_backward(dt, tokens, H, d, 0, 1, per_head, 1e-5, 0, 0, big, big, None, dy, big,  # noqa: E731
                                                          None, big, None, 0, None)
        assert back(None, BF16) == back(None, F32) == ENULL
    for tokens, D in ((1 << 23, 2048), (1 << 22, 16384), ((1 << 31) - 1, 32)):
        assert lib.kdn_residual_norm_backward_workspace_size(tokens, D, 1, ctypes.byref(st)) > 0 and st.value == OK
        assert lib.kdn_residual_norm_backward(BF16, BF16, tokens, D, 0, 1e-5, 0, 0, None, None, big, None, big, None, None, big, big,
                                              None, None, 0, None) == ENULL
    gated = lambda dt, tokens, d: lib.kdn_gated_norm(dt, tokens, 1, d, 0, 1, 0, 1e-5, 0, 0, None, None, None, None, None)  # noqa: E731
    assert gated(BF16, (1 << 27) - 8, 256) == ENULL and gated(BF16, (1 << 27) - 7, 256) == ESHAPE
    assert gated(F32, (1 << 26) - 4, 256) == ENULL and gated(F32, (1 << 26) - 3, 256) == ESHAPE
    # the sums of a weight's values, 16 a workgroup of 1024 threads
    size = lambda H: lib.kdn_gated_norm_backward_workspace_size(1, H, 1024, 1, ctypes.byref(st))  # noqa: E731
    assert size(65534) > 0 and st.value == OK and size(65535) > 0
    size = lambda H: lib.kdn_gated_norm_backward_workspace_size(1, H, 4096, 1, ctypes.byref(st))  # noqa: E731
    assert size((1 << 14) - 1) > 0 and size(1 << 14) == 0 and st.value == ESHAPE


def test_residual_norm_sums_of_many_rows(lib):
    """256 rows at most in one float32 sum."""
    size = lambda *a: lib.kdn_residual_norm_backward_workspace_size(*a, None)  # noqa: E731
    assert size(512 * 256, 4096, 0) == 4 * 512 * 4096 and size(512 * 256 + 1, 4096, 4096) == 4 * 1024 * 8192
    assert size(1 << 20, 64, 1) == 4 * 512 * 65 and size(1 << 22, 2048, 1) == 4 * 512 * 32 * 2049


def test_scan_sums_in_more_parts_of_many_tokens(lib):
    """256 tiles a part at most: the workspace beside the tiles' states and the sums over channels."""
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    for T, C, S, sets, parts in ((64 * 255, 32768, 8, 256, 1), (64 * 256, 32768, 8, 256, 2), (64 * 767, 32768, 8, 256, 3),
                                 (1 << 20, 4096, 16, 32, 72), (32 * 1000, 1024, 32, 32, 8)):
        tile = 32 if S == 32 else 64
        tiles = T // tile + -(-T // 256) + 1
        want = 2 * up(4 * tiles * C * S) + up(4 * tiles * C) + up(4 * sets * T * 2 * S) + up(4 * parts * C * (S + 2))
        assert lib.kdn_selective_scan_backward_workspace_size(BF16, 1, T, C, S, 1, None, None) == want, T


def test_gated_gradients_of_no_heads_need_a_place(lib):
    back = lambda dw, per_head: lib.kdn_gated_norm_backward(BF16, 5, 0, 16, 0, 1, per_head, 1e-5, 0, 0, None, None, None, None, None,  # noqa: E731
                                                            None, dw, None, 0, None)
    assert back(None, 0) == ENULL and back(None, 1) == OK


def test_scan_gradients_of_no_channels_need_places(lib):
    none = dict(C=0, z=None, dy=None, dl=None, dx=None, dd=None, da=None, dD=None, dz=None, dbias=None, ds=None, ws=None, wsb=0)
    assert scan_back(lib, db=None, **none) == scan_back(lib, dc=None, **none) == ENULL
    assert scan_back(lib, G=0, db=None, dc=None, **none) == OK
    assert scan_back(lib, N=0, db=None, dc=None, **none) == OK


def test_scan_counts_what_it_launches(lib):
    """2^24 workgroups: four runs of 16 channels of a block for the outputs, one for the tiles' own
    states, 512 states of a sequence for the joins, both ways for the gradients."""
    st = ctypes.c_int(0)
    call = lambda want, **kw: scan(lib, x=None, **kw) == want  # noqa: E731
    # a hundred thousand short prompts
    assert call(ENULL, N=1 << 15, T=4, C=4096, G=1) and call(ENULL, N=100000, T=4, C=2048, G=1)
    assert lib.kdn_selective_scan_workspace_size(BF16, 1 << 15, 4, 4096, 16, 1, None, ctypes.byref(st)) == 0 and st.value == OK
    assert scan_back(lib, N=1 << 15, T=4, C=4096, dy=None) == ENULL
    assert lib.kdn_selective_scan_backward_workspace_size(BF16, 1 << 15, 4, 4096, 16, 1, None, ctypes.byref(st)) > 0 and st.value == OK
    # outputs: blocks of 16 runs; joins: 4096 states of a sequence in 8 workgroups
    assert call(ENULL, N=(1 << 21) - 1, T=1, C=256, G=1) and call(ESHAPE, N=1 << 21, T=1, C=256, G=1)
    assert call(ENULL, N=(1 << 22) - 1024, T=1, C=16, S=8, G=1) and call(ESHAPE, N=(1 << 24) - 1, T=1, C=16, S=8, G=1)
    # sequences of several blocks: own states
    pk = packed(1 << 27, 64, pool=8, N=4)
    assert scan(lib, N=4, T=0, C=64, G=1, pk=pk, x=None) == ENULL and scan(lib, N=4, T=0, C=512, G=1, pk=pk, x=None) == ESHAPE
    assert scan_back(lib, N=1 << 20, T=1, C=256, dy=None) == ESHAPE
