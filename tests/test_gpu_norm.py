"""Gated norm and residual norm on the GPU against their 64-bit forms, and gradients."""
import math

import pytest
import torch

import around_ref as ref
from linear_attention_recurrent_delta_amd import kdn
from test_gpu_conv import BF, F32, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    kdn.ensure_built()


EPS = 1e-5
KINDS = [("norm_gate", "silu"), ("norm_gate", "sigmoid"), ("gate_norm", "silu"), ("gate_norm", None),
         ("norm_gate", "no gate")]


def case(lead, H, d, dtype, per_head, seed=0, gate=True):
    x = randn(lead + (H, d), F32, seed) * torch.exp(randn(lead + (H, 1), F32, seed + 1))
    z = randn(lead + (H, d), dtype, seed + 2, size=2.0) if gate else None
    w = 1 + randn((H, d) if per_head else (d,), F32, seed + 3, size=0.3)
    return x.to(dtype), z, w, randn(lead + (H, d), dtype, seed + 4)


def check_gated(x, z, w, dy, order, act, dtype, y=None, d=None):
    x, z, w, dy = (ref.wide(v) for v in (x, z, w, dy))
    if y is not None:
        ref.close("y", y, *ref.gated(x, w, z, EPS32, order, act, dtype))
    if d is None:
        return
    g, m = ref.gated_grad(x, w, z, dy, EPS32, order, act, dtype)
    ref.close("dx", d["dx"], g["dx"], m["dx"])
    if z is not None:
        ref.close("dgate", d["dgate"], g["dgate"], m["dgate"])
    over = tuple(range(x.dim() - w.dim()))
    want, bound = g["dweight"].sum(over), m["dweight"].sum(over)
    # rows of a workgroup in float32: its rounds and the rows that it holds at once
    rows = x[..., 0].numel() // (w.shape[0] if w.dim() == 2 else 1)
    mag = g["dweight"].abs().sum(over)
    ref.close("dweight", d["dweight"], want, bound + (rows / 1024 + 258) * ref.U * mag)


EPS32 = torch.tensor(EPS, dtype=torch.float32).item()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("order,act", KINDS)
@pytest.mark.parametrize("rows,H,d,per_head", [(1, 1, 1, False), (3, 2, 7, True), (5, 4, 64, False), (9, 3, 128, True),
                                               (2, 2, 130, False), (130, 5, 96, False), (3, 1, 1000, False),
                                               (2, 2, 513, True), (7, 1, 2048, False)])
def test_gated(dtype, order, act, rows, H, d, per_head):
    gate = act != "no gate"
    act = act if gate else "silu"
    x, z, w, dy = case((rows,), H, d, dtype, per_head, seed=d, gate=gate)
    y = kdn.gated_norm(x, w, z, eps=EPS, order=order, activation=act)
    g = kdn.gated_norm_backward(x, w, dy, z, eps=EPS, order=order, activation=act)
    check_gated(x, z, w, dy, order, act, dtype, y, g)
    assert gate or g["dgate"] is None


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [4096, 8192, 8199, 16384])
def test_long_rows(dtype, d):
    x, z, w, dy = case((3,), 1, d, dtype, False, seed=d)
    y = kdn.gated_norm(x, w, z, eps=EPS)
    g = kdn.gated_norm_backward(x, w, dy, z, eps=EPS)
    check_gated(x, z, w, dy, "norm_gate", "silu", dtype, y, g)
    h, s = x.view(3, d), randn((d,), F32, 5)
    check_residual(h, z.view(3, d), w, s, dy.view(3, d), None)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("order", ["norm_gate", "gate_norm"])
def test_slices(dtype, order):
    """x and the gate as slices of one projection's rows, behind an odd element."""
    B, T, H, d = 2, 9, 3, 50
    buf = torch.full((B * T * (2 * H * d + 7) + 3,), math.nan, dtype=dtype, device="cuda")
    both = buf[3:].view(B, T, 2 * H * d + 7)
    x, z, w, dy = case((B, T), H, d, dtype, True)
    both[..., :H * d], both[..., H * d + 2:2 * H * d + 2] = x.flatten(-2), z.flatten(-2)
    xs = both[..., :H * d].unflatten(-1, (H, d))
    zs = both[..., H * d + 2:2 * H * d + 2].unflatten(-1, (H, d))
    assert not xs.is_contiguous()
    kw = dict(eps=EPS, order=order)
    assert torch.equal(kdn.gated_norm(xs, w, zs, **kw), kdn.gated_norm(x, w, z, **kw))
    a, b = kdn.gated_norm_backward(xs, w, dy, zs, **kw), kdn.gated_norm_backward(x, w, dy, z, **kw)
    for k in a:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("dtype", [BF, F32])
def test_more_rows_than_workgroups(dtype):
    x, z, w, dy = case((3000,), 7, 64, dtype, False)
    g = kdn.gated_norm_backward(x, w, dy, z, eps=EPS)
    check_gated(x, z, w, dy, "norm_gate", "silu", dtype, None, g)
    again = kdn.gated_norm_backward(x, w, dy, z, eps=EPS)
    assert all(torch.equal(g[k], again[k]) for k in g)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_far_sizes(dtype):
    """Rows of zeros, and rows whose squares pass or fall below float32."""
    sizes = torch.tensor([0.0, 1e-30, 1e-12, 1.0, 1e12, 1e25, 1e36])
    x = (randn((7, 1, 64), F32, 1).clamp(-3, 3) * sizes[:, None, None].cuda()).to(dtype)
    w, z = torch.ones(64, device="cuda"), randn((7, 1, 64), dtype, 2)
    check_gated(x, z, w, None, "norm_gate", "silu", dtype, kdn.gated_norm(x, w, z, eps=EPS))
    y, h = kdn.residual_norm(x[:, 0], torch.zeros_like(x[:, 0]), w, eps=EPS)
    wy, wh, by, bh = ref.residual(ref.wide(x[:, 0]), torch.zeros(7, 64).double(), ref.wide(w), None, EPS32, dtype, dtype)
    ref.close("y", y, wy, by)
    ref.close("h", h, wh, bh)


def test_gates_at_the_ends():
    """Gates far from zero: silu and its derivative have no NaN there."""
    z = torch.tensor([-3e38, -200.0, -104.0, -88.0, -87.0, 0.0, 87.0, 104.0, 3e38], device="cuda").view(1, 1, 9)
    x, w = torch.linspace(-2, 3, 9, device="cuda").view(1, 1, 9), torch.ones(9, device="cuda")
    for act in ("silu", "sigmoid"):
        y = kdn.gated_norm(x, w, z, eps=EPS, activation=act)
        g = kdn.gated_norm_backward(x, w, torch.ones_like(x), z, eps=EPS, activation=act)
        want = torch.sigmoid(z.double()) * (z.double() if act == "silu" else 1)
        r = (x.double().square().mean() + EPS32) ** -0.5
        want = x.double() * r * want
        # 3 x 0.59 x 3e38 passes the largest float32
        assert torch.equal(want.float().isinf(), y.isinf())
        # below the smallest normal number a result may be flushed to zero
        off = (y.double() - want).abs()[..., :8]
        assert (off <= 1e-6 * want[..., :8].abs() + 1e-33).all()
        for k in ("dx", "dgate"):
            assert torch.isfinite(g[k][..., 1:-1]).all(), k
    bad = torch.tensor([math.nan, math.inf, -math.inf, 1.0], device="cuda").view(4, 1, 1).expand(4, 1, 8).contiguous()
    y = kdn.gated_norm(torch.ones(4, 1, 8, device="cuda"), torch.ones(8, device="cuda"), bad, eps=EPS, activation="sigmoid")
    assert y[0].isnan().all() and torch.isfinite(y[1:]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_do_not_mix(dtype):
    x, z, w, dy = case((40,), 2, 24, dtype, False)
    y, g = kdn.gated_norm(x, w, z), kdn.gated_norm_backward(x, w, dy, z)
    x[7, 1, 3], z[9, 0, 0] = math.nan, math.inf
    y2, g2 = kdn.gated_norm(x, w, z), kdn.gated_norm_backward(x, w, dy, z)
    keep = torch.ones(40, 2, dtype=torch.bool, device="cuda")
    keep[7, 1] = keep[9, 0] = False
    assert torch.equal(y[keep], y2[keep])
    for k in ("dx", "dgate"):
        assert torch.equal(g[k][keep], g2[k][keep])


def check_residual(x, res, w, scale, dy, dh):
    dtype, stream = x.dtype, res.dtype
    y, h = kdn.residual_norm(x, res, w, scale=scale, eps=EPS)
    W = [ref.wide(v) for v in (x, res, w, scale)]
    wy, wh, by, bh = ref.residual(W[0], W[1], W[2], W[3], EPS32, dtype, stream)
    ref.close("y", y, wy, by)
    ref.close("h", h, wh, bh)
    d = kdn.residual_norm_backward(x, h, w, dy, dh, scale=scale, eps=EPS)
    g, m = ref.residual_grad(W[0], ref.wide(h), W[2], W[3], ref.wide(dy), ref.wide(dh), EPS32, dtype, stream)
    ref.close("dresidual", d["dresidual"], g["dresidual"], m["dresidual"])
    ref.close("dx", d["dx"], g["dx"], m["dx"])
    rows = x.reshape(-1, x.shape[-1]).shape[0]
    k = (rows / 1024 + 258) * ref.U
    over = tuple(range(x.dim() - 1))
    ref.close("dweight", d["dweight"], g["dweight"].sum(over), m["dweight"].sum(over) + k * g["dweight"].abs().sum(over))
    if scale is None:
        assert d["dscale"] is None
        return
    one = scale.shape == (1,)
    add = lambda v: v.sum().view(1) if one and x.shape[-1] != 1 else v.sum(over)  # noqa: E731
    k = (rows / 1024 + 258 + (40 if one else 0)) * ref.U
    ref.close("dscale", d["dscale"], add(g["dscale"]), add(m["dscale"]) + k * add(g["dscale"].abs()))


@pytest.mark.parametrize("dtype,stream", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("scale", ["none", "one", "channel"])
@pytest.mark.parametrize("lead,D", [((1,), 1), ((3,), 9), ((2, 5), 64), ((65,), 130), ((3,), 1543), ((2,), 4096)])
def test_residual(dtype, stream, scale, lead, D):
    x, res = randn(lead + (D,), dtype, 1), randn(lead + (D,), stream, 2, size=3.0)
    w = 1 + randn((D,), F32, 3, size=0.3)
    s = None if scale == "none" else 0.5 + randn((1 if scale == "one" else D,), F32, 4, size=0.3)
    check_residual(x, res, w, s, randn(lead + (D,), dtype, 5), randn(lead + (D,), stream, 6))


@pytest.mark.parametrize("dtype,stream", [(BF, BF), (BF, F32), (F32, F32)])
def test_residual_calls(dtype, stream):
    """In place, as slices, without the cotangent of h, without dx, without dscale."""
    n, D = 37, 72
    buf = randn((n, D + 9), dtype, 1)
    x, res, w = buf[:, 5:5 + D], randn((n, D), stream, 2), 1 + randn((D,), F32, 3, size=0.3)
    s, dy = randn((D,), F32, 4), randn((n, D), dtype, 5)
    y, h = kdn.residual_norm(x.contiguous(), res, w, scale=s, eps=EPS)
    y2, h2 = kdn.residual_norm(x, res, w, scale=s, eps=EPS)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    kept = res.clone()
    y3, h3 = kdn.residual_norm(x, kept, w, scale=s, eps=EPS, out=(torch.empty_like(y), kept))
    assert h3 is kept and torch.equal(kept, h) and torch.equal(y3, y)
    full = kdn.residual_norm_backward(x, h, w, dy, torch.zeros_like(h), scale=s, eps=EPS)
    wide = torch.full((n, D + 3), math.nan, dtype=stream, device="cuda")
    wide[:, 2:2 + D] = h
    part = kdn.residual_norm_backward(x, wide[:, 2:2 + D], w, dy, scale=s, eps=EPS)
    for k in full:
        assert torch.equal(full[k], part[k]), k
    less = kdn.residual_norm_backward(None, h, w, dy, scale=s, eps=EPS,
                                      out=dict(dx=None, dresidual=torch.empty_like(h),
                                               dweight=torch.empty_like(w), dscale=None))
    assert torch.equal(less["dresidual"], full["dresidual"]) and torch.equal(less["dweight"], full["dweight"])


def test_nothing_to_do():
    w = torch.ones(16, device="cuda")
    e = torch.empty(0, 2, 16, device="cuda")
    assert kdn.gated_norm(e, w, e).shape == (0, 2, 16)
    d = kdn.gated_norm_backward(e, w, e, e)
    assert not d["dweight"].any()
    e = torch.empty(0, 16, device="cuda")
    y, h = kdn.residual_norm(e, e, w)
    assert y.shape == h.shape == (0, 16)
    d = kdn.residual_norm_backward(e, e, w, e, scale=torch.ones(16, device="cuda"))
    assert not d["dweight"].any() and not d["dscale"].any()


def test_gradients_against_differences():
    """The 64-bit gradients themselves against central differences."""
    x, z, w = (randn(s, F32, i).cpu().double() for i, s in enumerate(((2, 2, 5), (2, 2, 5), (5,))))
    dy, h = randn((2, 2, 5), F32, 4).cpu().double(), 1e-5

    def against(values, grads, loss):
        for v, g in zip(values, grads):
            for i in range(v.numel()):
                keep, at = v.view(-1)[i].item(), []
                for step in (h, -h):
                    v.view(-1)[i] = keep + step
                    at.append(loss())
                v.view(-1)[i] = keep
                # h^2 of third derivatives of a hundred units at most
                assert abs((at[0] - at[1]) / (2 * h) - g.reshape(-1)[i].item()) < 1e-7

    for order, act in (("norm_gate", "silu"), ("gate_norm", "silu"), ("norm_gate", "sigmoid"), ("gate_norm", "sigmoid")):
        g, _ = ref.gated_grad(x, w, z, dy, 0.1, order, act, F32)
        against((x, z, w), (g["dx"], g["dgate"], g["dweight"].sum((0, 1))),
                lambda: (ref.gated(x, w, z, 0.1, order, act, F32)[0] * dy).sum().item())
    res, s, dh = randn((2, 2, 5), F32, 5).cpu().double(), randn((5,), F32, 6).cpu().double(), z
    g, _ = ref.residual_grad(x, res + s * x, w, s, dy, dh, 0.1, F32, F32)

    def loss():
        y, hh, _, _ = ref.residual(x, res, w, s, 0.1, F32, F32)
        return ((y * dy).sum() + (hh * dh).sum()).item()

    against((x, res, w, s), (g["dx"], g["dresidual"], g["dweight"].sum((0, 1)), g["dscale"].sum((0, 1))), loss)
