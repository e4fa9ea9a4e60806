"""Host-side refusals of the convolution and of the norms (no GPU needed): through the
C ABI with fake addresses, none of which is ever read, and through the binding with
host tensors."""
import ctypes

import pytest
import torch

from linear_attention_recurrent_delta_amd import kdn
from test_linear_host import A, BF16, EALIAS, EALIGN, ENULL, ESHAPE, EUNSUP, EWS, F32, MB, OK, packed


@pytest.fixture(scope="module")
def lib():
    return kdn.ensure_built()


def conv(lib, dtype=BF16, N=2, T=100, C=64, W=4, act=1, xs=0, x=A, w=A + MB, b=A + 2 * MB, s0=A + 3 * MB,
         y=A + 4 * MB, s=A + 5 * MB, pk=None):
    return lib.kdn_causal_conv(dtype, N, T, C, W, act, xs, x, w, b, s0, y, s, pk, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), EUNSUP), (dict(act=2), EUNSUP), (dict(act=-1), EUNSUP), (dict(W=1), EUNSUP), (dict(W=5), EUNSUP),
    (dict(W=-1), ESHAPE), (dict(N=-1), ESHAPE), (dict(T=-1), ESHAPE), (dict(C=-1), ESHAPE),
    (dict(N=1 << 16, T=1 << 16), ESHAPE), (dict(C=1 << 26), ESHAPE), (dict(N=1, T=1 << 30, C=8192), ESHAPE),
    (dict(xs=63), ESHAPE), (dict(xs=-1), ESHAPE), (dict(xs=1 << 28), ESHAPE),
    (dict(x=None), ENULL), (dict(w=None), ENULL), (dict(y=None), ENULL),
    (dict(x=A + 1), EALIGN), (dict(y=A + 4 * MB + 1), EALIGN), (dict(s0=A + 3 * MB + 1), EALIGN), (dict(w=A + MB + 2), EALIGN),
    (dict(dtype=F32, x=A + 2), EALIGN), (dict(b=A + 2 * MB + 1), EALIGN), (dict(s=A + 5 * MB + 1), EALIGN),
    (dict(y=A), EALIAS), (dict(y=A + 2 * 100 * 64 * 2 - 2), EALIAS), (dict(s=A + 3 * MB + 2), EALIAS), (dict(s=A + 4 * MB), EALIAS),
    (dict(y=A + MB), EALIAS), (dict(xs=1000, y=A + 199 * 2000), EALIAS),
    (dict(C=0, x=None, w=None, b=None, s0=None, y=None, s=None), OK),
])
def test_conv_refusals(lib, kw, want):
    assert conv(lib, **kw) == want


@pytest.mark.parametrize("pk,kw,want", [
    (dict(), dict(T=5), ESHAPE), (dict(tokens=-1, max_blocks=3), dict(), ESHAPE), (dict(block=63, max_blocks=5), dict(), ESHAPE),
    (dict(max_blocks=4), dict(), ESHAPE), (dict(pool=-1), dict(), ESHAPE), (dict(blocks=None), dict(), ENULL),
    (dict(block_offsets=None), dict(), ENULL), (dict(blocks=A + 20 * MB + 8), dict(), EALIGN), (dict(slots=A + 1), dict(), EALIGN),
    (dict(slots=A + 4 * MB), dict(), EALIAS), (dict(blocks=A + 5 * MB), dict(), EALIAS),
])
def test_conv_packed_refusals(lib, pk, kw, want):
    assert conv(lib, pk=packed(**pk), **dict(dict(N=4, T=0), **kw)) == want
    size = lib.kdn_causal_conv_backward_workspace_size(BF16, 4, kw.get("T", 0), 64, 4, packed(**pk), None)
    assert (size == 0) == (want == ESHAPE)


def decode(lib, dtype=BF16, N=3, C=64, W=4, act=1, xs=0, x=A, w=A + MB, b=None, slots=A + 2 * MB, pool=10,
           s=A + 3 * MB, y=A + 4 * MB):
    return lib.kdn_causal_conv_decode(dtype, N, C, W, act, xs, x, w, b, slots, pool, s, y, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=7), EUNSUP), (dict(W=8), EUNSUP), (dict(N=-1), ESHAPE), (dict(pool=-1), ESHAPE), (dict(slots=None, pool=2), ESHAPE),
    (dict(N=1 << 30, slots=None, pool=1 << 30), ESHAPE), (dict(x=None), ENULL), (dict(s=None), ENULL), (dict(y=None), ENULL),
    (dict(slots=A + 2), EALIGN), (dict(y=A), EALIAS), (dict(s=A + 4 * MB), EALIAS), (dict(s=A + 2 * MB), EALIAS),
])
def test_conv_decode_refusals(lib, kw, want):
    assert decode(lib, **kw) == want


def conv_back(lib, dtype=BF16, N=2, T=100, C=64, W=4, act=1, xs=0, x=A, w=A + MB, b=A + 2 * MB, s0=A + 3 * MB,
              dy=A + 4 * MB, dl=A + 5 * MB, dx=A + 6 * MB, dw=A + 7 * MB, db=A + 8 * MB, ds=A + 9 * MB, ws=A + 10 * MB,
              wsb=MB):
    return lib.kdn_causal_conv_backward(dtype, N, T, C, W, act, xs, x, w, b, s0, dy, dl, dx, dw, db, ds, None, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), EUNSUP), (dict(dy=None), ENULL), (dict(dx=None), ENULL), (dict(dw=None), ENULL), (dict(dw=A + 7 * MB + 2), EALIGN),
    (dict(dx=A), EALIAS), (dict(dx=A + 4 * MB), EALIAS), (dict(ds=A + 5 * MB), EALIAS), (dict(db=A + 7 * MB + 4), EALIAS),
    (dict(ws=None), EWS), (dict(wsb=8), EWS), (dict(ws=A + 10 * MB + 64), EALIGN), (dict(ws=A), EALIAS), (dict(ws=A + 6 * MB), EALIAS),
    (dict(C=(1 << 26) - 1, N=1, T=1), EALIAS),
])
def test_conv_backward_refusals(lib, kw, want):
    assert conv_back(lib, **kw) == want


def test_conv_workspace_size(lib):
    st = ctypes.c_int(0)
    size = lambda *a: (lib.kdn_causal_conv_backward_workspace_size(*a, None, ctypes.byref(st)), st.value)
    assert size(BF16, 2, 100, 64, 4) == (4 * 4 * 5 * 64, OK)         # a part for each of 2 x 2 tiles
    assert size(BF16, 2, 0, 64, 4) == (0, OK)
    assert size(BF16, 4, 4096, 2048, 4) == (4 * (512 // 8) * 5 * 2048, OK)
    assert size(BF16, 4, 4096, 2048, 9)[1] == EUNSUP and size(BF16, -4, 4096, 2048, 4)[1] == ESHAPE


def scan(lib, dtype=BF16, N=2, T=100, C=64, S=16, G=2, sp=1, xs=0, ds=0, zs=0, bs=0, cs=0, x=A, dl=A + MB, a=A + 2 * MB,
         b=A + 3 * MB, c=A + 4 * MB, d=A + 5 * MB, z=A + 6 * MB, bias=A + 7 * MB, s0=A + 8 * MB, y=A + 9 * MB, s=A + 10 * MB,
         pk=None, ws=A + 32 * MB, wsb=64 * MB):
    return lib.kdn_selective_scan(dtype, N, T, C, S, G, sp, xs, ds, zs, bs, cs, x, dl, a, b, c, d, z, bias, s0, y, s, pk, ws,
                                  wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), EUNSUP), (dict(S=4), EUNSUP), (dict(S=64), EUNSUP), (dict(S=-8), ESHAPE), (dict(G=3), ESHAPE), (dict(G=0), ESHAPE),
    (dict(G=-1), ESHAPE), (dict(C=-64), ESHAPE), (dict(C=1 << 24), ESHAPE), (dict(N=-1), ESHAPE), (dict(T=-1), ESHAPE),
    (dict(N=1 << 16, T=1 << 16), ESHAPE), (dict(N=1 << 21, T=1, C=256, G=1), ESHAPE), (dict(xs=63), ESHAPE), (dict(ds=1), ESHAPE),
    (dict(zs=1 << 28), ESHAPE), (dict(bs=31), ESHAPE), (dict(cs=31), ESHAPE), (dict(x=None), ENULL), (dict(dl=None), ENULL),
    (dict(a=None), ENULL), (dict(b=None), ENULL), (dict(c=None), ENULL), (dict(y=None), ENULL), (dict(x=A + 1), EALIGN),
    (dict(b=A + 3 * MB + 1), EALIGN), (dict(a=A + 2 * MB + 4), EALIGN), (dict(s0=A + 8 * MB + 8), EALIGN), (dict(s=A + 10 * MB + 4), EALIGN),
    (dict(d=A + 5 * MB + 2), EALIGN), (dict(bias=A + 7 * MB + 1), EALIGN), (dict(dtype=F32, z=A + 6 * MB + 2), EALIGN),
    (dict(y=A), EALIAS), (dict(y=A + MB + 2), EALIAS), (dict(y=A + 6 * MB), EALIAS), (dict(s=A + 8 * MB + 16), EALIAS),
    (dict(s=A + 9 * MB), EALIAS), (dict(y=A + 2 * MB), EALIAS),
    # cut sequences need a workspace
    (dict(T=4000, ws=None), EWS), (dict(T=4000, wsb=1000), EWS), (dict(T=4000, ws=A + 32 * MB + 64), EALIGN), (dict(T=4000, ws=A + 10 * MB), EALIAS),
    (dict(T=4000, ws=A + 8 * MB), EALIAS),
])
def test_scan_refusals(lib, kw, want):
    assert scan(lib, **kw) == want


@pytest.mark.parametrize("pk,kw,want", [
    (dict(), dict(T=5), ESHAPE), (dict(tokens=-1, max_blocks=3), dict(), ESHAPE), (dict(block=63, max_blocks=5), dict(), ESHAPE),
    (dict(max_blocks=4), dict(), ESHAPE), (dict(pool=-1), dict(), ESHAPE), (dict(blocks=None), dict(), ENULL),
    (dict(block_offsets=None), dict(), ENULL), (dict(blocks=A + 20 * MB + 8), dict(), EALIGN), (dict(slots=A + 1), dict(), EALIGN),
    (dict(slots=A + 9 * MB), dict(), EALIAS), (dict(), dict(ws=None), EWS), (dict(), dict(ws=A + 20 * MB), EALIAS),
])
def test_scan_packed_refusals(lib, pk, kw, want):
    assert scan(lib, pk=packed(**pk), **dict(dict(N=4, T=0), **kw)) == want


def scan_decode(lib, dtype=BF16, N=3, C=64, S=16, G=1, xs=0, x=A, dl=A + MB, a=A + 2 * MB, b=A + 3 * MB, c=A + 4 * MB,
                slots=A + 5 * MB, pool=10, s=A + 6 * MB, y=A + 7 * MB):
    return lib.kdn_selective_decode(dtype, N, C, S, G, 1, xs, 0, 0, 0, 0, x, dl, a, b, c, None, None, None, slots, pool, s, y, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=5), EUNSUP), (dict(S=12), EUNSUP), (dict(N=-1), ESHAPE), (dict(G=5), ESHAPE), (dict(pool=-1), ESHAPE),
    (dict(slots=None, pool=2), ESHAPE), (dict(N=1 << 24, C=128, pool=1 << 24), ESHAPE), (dict(x=None), ENULL), (dict(s=None), ENULL),
    (dict(s=A + 6 * MB + 8), EALIGN), (dict(a=A + 2 * MB + 8), EALIGN), (dict(slots=A + 2), EALIGN), (dict(y=A), EALIAS), (dict(s=A + 7 * MB), EALIAS),
    (dict(slots=A + 6 * MB), EALIAS),
])
def test_scan_decode_refusals(lib, kw, want):
    assert scan_decode(lib, **kw) == want


def scan_back(lib, N=2, T=100, C=64, S=16, G=1, z=A + 6 * MB, dy=A + 9 * MB, dl=A + 10 * MB, dx=A + 11 * MB, dd=A + 12 * MB,
              da=A + 13 * MB, db=A + 14 * MB, dc=A + 15 * MB, dD=A + 16 * MB, dz=A + 17 * MB, dbias=A + 18 * MB, ds=A + 19 * MB,
              pk=None, ws=A + 32 * MB, wsb=64 * MB):
    return lib.kdn_selective_scan_backward(BF16, N, T, C, S, G, 1, 0, 0, 0, 0, 0, A, A + MB, A + 2 * MB, A + 3 * MB, A + 4 * MB,
                                           A + 5 * MB, z, A + 7 * MB, A + 8 * MB, dy, dl, dx, dd, da, db, dc, dD, dz, dbias, ds,
                                           pk, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(S=24), EUNSUP), (dict(dy=None), ENULL), (dict(dx=None), ENULL), (dict(dd=None), ENULL), (dict(da=None), ENULL), (dict(db=None), ENULL),
    (dict(dc=None), ENULL), (dict(dz=None), ENULL), (dict(z=None), ENULL), (dict(da=A + 13 * MB + 2), EALIGN), (dict(ds=A + 19 * MB + 4), EALIGN),
    (dict(dl=A + 10 * MB + 8), EALIGN), (dict(dx=A), EALIAS), (dict(dz=A + 11 * MB), EALIAS), (dict(db=A + 15 * MB), EALIAS),
    (dict(ds=A + 8 * MB), EALIAS), (dict(dbias=A + 16 * MB + 4), EALIAS), (dict(da=A + 2 * MB), EALIAS), (dict(ws=None), EWS),
    (dict(wsb=100), EWS), (dict(ws=A + 32 * MB + 16), EALIGN), (dict(ws=A + 9 * MB), EALIAS), (dict(ws=A + 19 * MB), EALIAS),
    (dict(N=1, T=1 << 30), ESHAPE),
])
def test_scan_backward_refusals(lib, kw, want):
    assert scan_back(lib, **kw) == want


def test_scan_sizes(lib):
    st = ctypes.c_int(0)
    size = lambda *a, pk=None: (lib.kdn_selective_scan_workspace_size(*a, pk, ctypes.byref(st)), st.value)  # noqa: E731
    assert size(BF16, 1, 190, 2048, 16, 1) == (0, OK) and size(BF16, 2, 0, 64, 16, 1) == (0, OK)
    n, s = size(BF16, 1, 100000, 64, 16, 1)
    assert s == OK and n >= 100000 // 64 * 64 * 17 * 4
    assert size(BF16, 1, 100, 64, 5, 1)[1] == EUNSUP and size(BF16, 1, 100, 64, 16, 7)[1] == ESHAPE
    for tokens, N, C, S in ((0, 0, 0, 0), (1, 1, 1, 8), (2 ** 31 - 1, 1, 1, 16), (22000, 37, 4096, 16), (8192, 8192, 64, 32)):
        b = lib.kdn_selective_block(tokens, N, C, S)
        assert b > 0 and b % 64 == 0
    assert lib.kdn_selective_block(-1, 1, 1, 8) == lib.kdn_selective_block(1, -1, 1, 8) == -1
    with pytest.raises(kdn.KdnError):
        kdn.selective_block(-1, 1, 1, 8)
    back = lambda *a: (lib.kdn_selective_scan_backward_workspace_size(*a, None, ctypes.byref(st)), st.value)  # noqa: E731
    assert back(BF16, 0, 5, 64, 16, 1) == (0, OK) and back(BF16, 1, 5, 64, 16, 1)[0] > 0 and back(F32, 1, 5, 64, 9, 1)[1] == EUNSUP


def gated(lib, dtype=BF16, tokens=10, H=4, d=64, order=0, act=1, per_head=0, eps=1e-5, xs=0, zs=0, x=A, w=A + MB,
          z=A + 2 * MB, y=A + 3 * MB):
    return lib.kdn_gated_norm(dtype, tokens, H, d, order, act, per_head, eps, xs, zs, x, w, z, y, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), EUNSUP), (dict(order=2), EUNSUP), (dict(act=3), EUNSUP), (dict(act=-1), EUNSUP), (dict(eps=0.0), EUNSUP),
    (dict(eps=-1.0), EUNSUP), (dict(eps=float("nan")), EUNSUP), (dict(eps=float("inf")), EUNSUP), (dict(d=0), EUNSUP),
    (dict(d=16385), EUNSUP), (dict(d=-1), ESHAPE), (dict(tokens=-1), ESHAPE), (dict(H=-1), ESHAPE), (dict(H=1 << 16), ESHAPE),
    (dict(tokens=1 << 20, H=1 << 12), ESHAPE), (dict(tokens=(1 << 31) - 1, H=1, d=8192), ESHAPE), (dict(xs=255), ESHAPE),
    (dict(zs=1 << 28), ESHAPE), (dict(x=None), ENULL), (dict(w=None), ENULL), (dict(y=None), ENULL), (dict(x=A + 1), EALIGN),
    (dict(z=A + 2 * MB + 1), EALIGN), (dict(w=A + MB + 2), EALIGN), (dict(y=A + 10 * 256 * 2 - 2), EALIAS), (dict(y=A + 2 * MB), EALIAS),
    (dict(y=A + MB), EALIAS),
])
def test_gated_refusals(lib, kw, want):
    assert gated(lib, **kw) == want


def gated_back(lib, tokens=10, H=4, d=64, z=A + 2 * MB, dy=A + 3 * MB, dx=A + 4 * MB, dz=A + 5 * MB, dw=A + 6 * MB,
               ws=A + 7 * MB, wsb=MB, per_head=0):
    return lib.kdn_gated_norm_backward(BF16, tokens, H, d, 0, 1, per_head, 1e-5, 0, 0, A, A + MB, z, dy, dx, dz, dw, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), ENULL), (dict(dx=None), ENULL), (dict(dz=None), ENULL), (dict(z=None), ENULL), (dict(dw=None), ENULL),
    (dict(dw=A + 6 * MB + 2), EALIGN), (dict(dx=A), EALIAS), (dict(dz=A + 4 * MB), EALIAS), (dict(dw=A + MB), EALIAS),
    (dict(ws=None), EWS), (dict(wsb=100), EWS), (dict(ws=A + 7 * MB + 128), EALIGN), (dict(ws=A + 3 * MB), EALIAS),
    (dict(d=16385), EUNSUP),
])
def test_gated_backward_refusals(lib, kw, want):
    assert gated_back(lib, **kw) == want


def residual(lib, dtype=BF16, sd=F32, n=10, D=64, sn=64, eps=1e-5, xs=0, rs=0, x=A, r=A + MB, w=A + 2 * MB, s=A + 3 * MB,
             y=A + 4 * MB, h=A + 5 * MB):
    return lib.kdn_residual_norm(dtype, sd, n, D, sn, eps, xs, rs, x, r, w, s, y, h, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=F32, sd=BF16), EUNSUP), (dict(sd=3), EUNSUP), (dict(D=0, sn=0), EUNSUP), (dict(D=20000, sn=0), EUNSUP),
    (dict(eps=0.0), EUNSUP), (dict(n=-1), ESHAPE), (dict(sn=2), ESHAPE), (dict(sn=-1), ESHAPE), (dict(xs=10), ESHAPE),
    (dict(rs=1 << 30), ESHAPE), (dict(sn=0), ENULL), (dict(s=None), ENULL), (dict(x=None), ENULL), (dict(r=None), ENULL),
    (dict(h=None), ENULL), (dict(r=A + MB + 2), EALIGN), (dict(h=A + 5 * MB + 2), EALIGN), (dict(y=A), EALIAS),
    (dict(h=A + MB + 4), EALIAS), (dict(h=A + MB, rs=65), EALIAS), (dict(h=A + 4 * MB), EALIAS), (dict(y=A + 3 * MB), EALIAS),
])
def test_residual_refusals(lib, kw, want):
    assert residual(lib, **kw) == want


def residual_back(lib, n=10, D=64, sn=64, x=A, h=A + MB, w=A + 2 * MB, s=A + 3 * MB, dy=A + 4 * MB, dh=A + 5 * MB,
                  dx=A + 6 * MB, dr=A + 7 * MB, dw=A + 8 * MB, ds=A + 9 * MB, ws=A + 10 * MB, wsb=MB):
    return lib.kdn_residual_norm_backward(BF16, F32, n, D, sn, 1e-5, 0, 0, x, h, w, s, dy, dh, dx, dr, dw, ds, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(h=None), ENULL), (dict(dr=None), ENULL), (dict(dw=None), ENULL), (dict(x=None), ENULL), (dict(s=None), ENULL),
    (dict(sn=0, s=None), ENULL), (dict(sn=3), ESHAPE), (dict(dr=A + 7 * MB + 2), EALIGN), (dict(dx=A + 4 * MB), EALIAS),
    (dict(dr=A + MB), EALIAS), (dict(ds=A + 8 * MB), EALIAS), (dict(ws=None), EWS), (dict(wsb=10), EWS),
    (dict(ws=A + 5 * MB), EALIAS),
])
def test_residual_backward_refusals(lib, kw, want):
    assert residual_back(lib, **kw) == want


def test_norm_workspace_sizes(lib):
    st = ctypes.c_int(0)
    g = lambda *a: (lib.kdn_gated_norm_backward_workspace_size(*a, ctypes.byref(st)), st.value)
    assert g(10, 4, 64, 0) == (4 * 40 * 64, OK) and g(10, 4, 64, 1) == (4 * 10 * 256, OK)
    assert g(1 << 20, 4, 64, 0) == (4 * 1024 * 64, OK) and g(1 << 20, 4, 64, 1) == (4 * 256 * 256, OK)
    assert g(0, 4, 64, 0) == (0, OK) and g(-1, 4, 64, 0)[1] == ESHAPE and g(1, 1, 20000, 0)[1] == EUNSUP
    r = lambda *a: (lib.kdn_residual_norm_backward_workspace_size(*a, ctypes.byref(st)), st.value)
    assert r(10, 64, 0) == (4 * 640, OK) and r(5000, 64, 64) == (4 * 512 * 128, OK) and r(10, 64, 7)[1] == ESHAPE


# ---------------------------------------------------------------------------
# The binding: host tensors, wrong shapes and types, before the library is called.
# ---------------------------------------------------------------------------
x, w4, b8 = torch.zeros(2, 5, 8), torch.zeros(8, 4), torch.zeros(8)
x16, bc = torch.zeros(8, 16), torch.zeros(2, 5, 1, 16)


@pytest.mark.parametrize("call,error", [
    (lambda: kdn.causal_conv(x, w4), ValueError),                                  # not in GPU memory
    (lambda: kdn.causal_conv(None, w4), TypeError), (lambda: kdn.causal_conv(x.half(), w4), ValueError),
    (lambda: kdn.causal_conv(x[0], w4), ValueError), (lambda: kdn.causal_conv(x, w4[0]), ValueError),
    (lambda: kdn.causal_conv(x, w4, activation="relu"), ValueError), (lambda: kdn.causal_conv(x, w4, activation="sigmoid"), ValueError),
    (lambda: kdn.causal_conv_decode(x, w4, x), ValueError), (lambda: kdn.causal_conv_decode(x[0], w4, None), ValueError),
    (lambda: kdn.causal_conv_backward(x, w4, x), ValueError),
    (lambda: kdn.selective_scan(x, x, w4, x, x), ValueError), (lambda: kdn.selective_scan(x, x, b8, x, x), ValueError),
    (lambda: kdn.selective_scan(x, x, x16, bc, bc), ValueError), (lambda: kdn.selective_scan(None, x, x16, bc, bc), TypeError),
    (lambda: kdn.selective_scan(x, None, x16, bc, bc), (TypeError, ValueError)), (lambda: kdn.selective_scan(x, x[:1], x16, bc, bc), ValueError),
    (lambda: kdn.selective_scan(x, x, x16, bc, bc.double()), ValueError), (lambda: kdn.selective_scan(x, x, x16, bc, bc, D=0.5), (TypeError, ValueError)),
    (lambda: kdn.selective_decode(x, x, x16, bc, bc, x), ValueError), (lambda: kdn.selective_decode(x[0], x[0], x16, bc[0], bc[0], None), ValueError),
    (lambda: kdn.selective_scan_backward(x, x, x16, bc, bc, x), ValueError),
    (lambda: kdn.gated_norm(x, b8), ValueError), (lambda: kdn.gated_norm(x[0, 0], b8), ValueError),
    (lambda: kdn.gated_norm(x, b8, order="both"), ValueError), (lambda: kdn.gated_norm(x, None), ValueError),
    (lambda: kdn.gated_norm(x, b8, activation="tanh"), ValueError), (lambda: kdn.gated_norm_backward(x, b8, x), ValueError),
    (lambda: kdn.residual_norm(x, x, b8), ValueError), (lambda: kdn.residual_norm(None, x, b8), (TypeError, ValueError)),
    (lambda: kdn.residual_norm(x, None, b8), TypeError), (lambda: kdn.residual_norm(x, x, b8, scale=0.5), (TypeError, ValueError)),
    (lambda: kdn.residual_norm_backward(x, x, b8, x), ValueError), (lambda: kdn.residual_norm_backward(x, x, b8, None), (TypeError, ValueError)),
])
def test_binding_refusals(call, error):
    with pytest.raises(error):
        call()


def test_strides():
    lead, dev = (2, 5), torch.device("cpu")
    wide = torch.zeros(2, 5, 12)
    s = lambda t, tail: kdn._strided("x", t, lead, tail, torch.float32, dev)
    assert s(torch.zeros(2, 5, 8), (8,)) == 0 and s(wide[..., :8], (8,)) == 12 and s(wide[..., 4:], (8,)) == 12
    assert s(wide[..., :8].unflatten(-1, (2, 4)), (2, 4)) == 12
    for bad in (torch.zeros(2, 8, 5).transpose(1, 2), torch.zeros(5, 2, 8).transpose(0, 1),
                torch.zeros(2, 1, 8).expand(2, 5, 8), torch.zeros(2, 9, 8)[:, :5], torch.zeros(2, 5, 16)[..., ::2]):
        with pytest.raises(ValueError):
            s(bad, (8,))
    one = torch.zeros(3, 7, 8)[:, 2:3]
    assert kdn._strided("x", one, (3, 1), (8,), torch.float32, dev) == 56
    assert kdn._strided("x", torch.zeros(4, 1, 8)[:1], (1, 1), (8,), torch.float32, dev) == 0
