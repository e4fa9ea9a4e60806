"""ctypes binding of libkdn.so (the C ABI declared in include/kdn.h).

Argument marshalling only: tensors become device pointers, the current HIP
stream is passed through, and a non-OK status raises.  Every step of the
recurrence runs in the library's gfx950 kernels; PyTorch provides device
memory and streams.  If the library is not built this module raises -- there
is no fallback path.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkdn.so")

# kdn_variant / kdn_dtype / kdn_status values of include/kdn.h
VARIANTS = {"deltanet": 0, "gated_deltanet": 1, "kda": 2, "diag_kdn": 3, "iso_kdn": 4}


def _p_shape(vid, N, H, dk):
    """Shape of the variance tensor p: [N,H,dk] (diagonal KDN), [N,H]
    (isotropic KDN), or None (no variance)."""
    return (N, H, dk) if vid == 3 else ((N, H) if vid == 4 else None)


def _new_p(vid, N, H, dk, device):
    shp = _p_shape(vid, N, H, dk)
    return None if shp is None else torch.empty(shp, dtype=torch.float32, device=device)
DTYPES = {torch.float32: 0, torch.bfloat16: 1}
STATUS = {0: "KDN_OK", 1: "KDN_ERR_NULL", 2: "KDN_ERR_SHAPE",
          3: "KDN_ERR_UNSUPPORTED", 4: "KDN_ERR_ALIGN", 5: "KDN_ERR_ALIAS",
          6: "KDN_ERR_HIP", 7: "KDN_ERR_WORKSPACE", 8: "KDN_ERR_SCRATCH"}

# kdn_gate values
GATE_TOKEN, GATE_HEAD, GATE_HEAD_F32 = 0, 1, 2


class Packed(ctypes.Structure):
    """kdn_packed of include/kdn.h."""
    _fields_ = [("tokens", ctypes.c_int), ("block", ctypes.c_int), ("max_blocks", ctypes.c_int),
                ("pool", ctypes.c_int), ("blocks", ctypes.c_void_p),
                ("block_offsets", ctypes.c_void_p), ("slots", ctypes.c_void_p)]


_lib = None


class KdnError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


def load(path: str = LIB_PATH):
    """Load libkdn.so and declare its signatures.  Raises if it is missing."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is not built: run `python -m linear_attention_recurrent_delta_amd.build`")
    lib = ctypes.CDLL(path)
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.kdn_chunk_prefill.restype = i
    u64 = ctypes.c_ulonglong
    lib.kdn_chunk_prefill.argtypes = [i, i, i, i, i, i, i, i, f] + [vp] * 12 + [vp, u64, vp]
    lib.kdn_chunk_prefill_noalloc.restype = i
    lib.kdn_chunk_prefill_noalloc.argtypes = [i, i, i, i, i, i, i, i, f] + [vp] * 12 + [vp]
    lib.kdn_noalloc_scratch_bytes.restype = u64
    lib.kdn_noalloc_scratch_bytes.argtypes = []
    lib.kdn_chunk_prefill_workspace_size.restype = u64
    lib.kdn_chunk_prefill_workspace_size.argtypes = [i] * 8 + [ctypes.POINTER(i)]
    lib.kdn_recurrent_decode.restype = i
    lib.kdn_recurrent_decode.argtypes = [i, i, i, i, i, i, f] + [vp] * 11
    lib.kdn_recurrent_decode_multi.restype = i
    lib.kdn_recurrent_decode_multi.argtypes = [i, i, i, i, i, i, i, f] + [vp] * 13
    lib.kdn_chunk_prefill_backward.restype = i
    lib.kdn_chunk_prefill_backward.argtypes = [i] * 8 + [f] + [vp] * 21 + [vp, u64, vp]
    lib.kdn_chunk_prefill_backward_workspace_size.restype = u64
    lib.kdn_chunk_prefill_backward_workspace_size.argtypes = [i] * 8 + [ctypes.POINTER(i)]
    ll, pk = ctypes.c_longlong, ctypes.POINTER(Packed)
    lib.kdn_sequence_tables.restype = i
    lib.kdn_sequence_tables.argtypes = [i] * 4 + [vp] * 9
    lib.kdn_sequence_max_blocks.restype = i
    lib.kdn_sequence_max_blocks.argtypes = [i] * 3
    lib.kdn_linear_block.restype = i
    lib.kdn_linear_block.argtypes = [i] * 3
    lib.kdn_linear_prefill.restype = i
    lib.kdn_linear_prefill.argtypes = [i] * 10 + [ll] * 3 + [vp] * 7 + [pk, vp, u64, vp]
    lib.kdn_linear_prefill_workspace_size.restype = u64
    lib.kdn_linear_prefill_workspace_size.argtypes = [i] * 6 + [pk, ctypes.POINTER(i)]
    lib.kdn_linear_prefill_backward.restype = i
    lib.kdn_linear_prefill_backward.argtypes = [i] * 10 + [ll] * 3 + [vp] * 12 + [pk, vp, u64, vp]
    lib.kdn_linear_prefill_backward_workspace_size.restype = u64
    lib.kdn_linear_prefill_backward_workspace_size.argtypes = [i] * 10 + [pk, ctypes.POINTER(i)]
    lib.kdn_linear_decode.restype = i
    lib.kdn_linear_decode.argtypes = [i] * 9 + [ll] * 3 + [vp] * 5 + [i] + [vp] * 3
    lib.kdn_status_string.restype = ctypes.c_char_p
    lib.kdn_status_string.argtypes = [i]
    lib.kdn_chunk_prefill_chunk_size.restype = i
    lib.kdn_chunk_prefill_chunk_size.argtypes = [i, i, i, i]
    lib.kdn_abi_version.restype = i
    lib.kdn_abi_version.argtypes = []
    if path == LIB_PATH:
        _lib = lib
    return lib


def ensure_built():
    """Build the library if no build is present, then load it."""
    if not os.path.exists(LIB_PATH):
        from . import build
        build.build()
    return load()


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_contiguous():
        raise ValueError("kdn: tensor arguments must be contiguous")
    if x.device.type != "cuda":
        raise ValueError(f"kdn: tensor arguments must be in GPU memory, not on {x.device}")
    return x.data_ptr()


def _expect(args, device):
    """Check (name, tensor or None, shape, dtype) tuples before a call: the
    shape, then the dtype, then contiguity, then that every tensor lives on
    ``device`` (a GPU).  The C library checks sizes and pointers only; a host
    tensor, a tensor on another GPU or a wrongly shaped one would otherwise
    reach the kernels."""
    for name, x, shape, dtype in args:
        if x is None:
            continue
        if not isinstance(x, torch.Tensor):
            raise TypeError(f"kdn: {name} must be a tensor or None")
        if tuple(x.shape) != tuple(shape):
            raise ValueError(f"kdn: {name} has shape {tuple(x.shape)}, expected {tuple(shape)}")
        if x.dtype != dtype:
            raise ValueError(f"kdn: {name} has dtype {x.dtype}, expected {dtype}")
        if not x.is_contiguous():
            raise ValueError(f"kdn: {name} must be contiguous")
    if device.type != "cuda":
        raise ValueError(f"kdn: tensors must be in GPU memory, not on {device}")
    for name, x, _, _ in args:
        if x is not None and x.device != device:
            raise ValueError(f"kdn: {name} is on {x.device}, the other tensors on {device}")


def _gate_specs(vid, lead, dk, dt, alpha, beta, proc_noise, obs_noise):
    """Expected (name, tensor, shape, dtype) of the gates for leading dims
    ``lead`` ([B,T,H] or [N,H])."""
    lead = tuple(lead)
    a_shape = lead if vid == 1 else lead + (dk,)
    return [("alpha", alpha, a_shape, dt), ("beta", beta, lead, dt),
            ("proc_noise", proc_noise, lead + (dk,), dt), ("obs_noise", obs_noise, lead, dt)]


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(lib, st):
    if st != 0:
        raise KdnError(st, lib.kdn_status_string(st).decode())


def kdn_status_string(status: int) -> str:
    return load().kdn_status_string(int(status)).decode()


def kdn_abi_version() -> int:
    return int(load().kdn_abi_version())


def kdn_chunk_prefill_chunk_size(dtype: int, d_k: int, d_v: int, chunk: int) -> int:
    return int(load().kdn_chunk_prefill_chunk_size(int(dtype), d_k, d_v, chunk))


def kdn_chunk_prefill(variant, dtype, B, T, H, d_k, d_v, chunk, mu, q, k, v,
                      alpha, beta, proc_noise, obs_noise, S0, p0, o, S_out,
                      p_out, workspace=None, workspace_bytes=0, stream=None):
    """Raw entry point: same arguments as the C function (tensors or ints
    for pointers, None for NULL).  A tensor workspace passes its byte size
    when ``workspace_bytes`` is 0."""
    lib = load()
    if workspace is not None and not isinstance(workspace, int) and not workspace_bytes:
        workspace_bytes = workspace.numel() * workspace.element_size()
    st = lib.kdn_chunk_prefill(
        int(variant), int(dtype), int(B), int(T), int(H), int(d_k), int(d_v),
        int(chunk), float(mu), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
        _ptr(beta), _ptr(proc_noise), _ptr(obs_noise), _ptr(S0), _ptr(p0),
        _ptr(o), _ptr(S_out), _ptr(p_out), _ptr(workspace), int(workspace_bytes),
        _stream(stream))
    _check(lib, st)


def kdn_chunk_prefill_noalloc(variant, dtype, B, T, H, d_k, d_v, chunk, mu, q, k, v,
                              alpha, beta, proc_noise, obs_noise, S0, p0, o, S_out,
                              p_out, stream=None):
    """Raw entry point: same arguments as the C function (the two-pass
    prefill on the library's static scratch; allocates nothing)."""
    lib = load()
    st = lib.kdn_chunk_prefill_noalloc(
        int(variant), int(dtype), int(B), int(T), int(H), int(d_k), int(d_v),
        int(chunk), float(mu), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
        _ptr(beta), _ptr(proc_noise), _ptr(obs_noise), _ptr(S0), _ptr(p0),
        _ptr(o), _ptr(S_out), _ptr(p_out), _stream(stream))
    _check(lib, st)


def kdn_noalloc_scratch_bytes() -> int:
    return int(load().kdn_noalloc_scratch_bytes())


def kdn_chunk_prefill_workspace_size(variant, dtype, B, T, H, d_k, d_v, chunk):
    """Bytes of workspace for the two-pass schedule; raises on invalid sizes."""
    lib = load()
    st = ctypes.c_int(0)
    n = lib.kdn_chunk_prefill_workspace_size(int(variant), int(dtype), int(B), int(T),
                                             int(H), int(d_k), int(d_v), int(chunk),
                                             ctypes.byref(st))
    _check(lib, st.value)
    return int(n)


def kdn_chunk_prefill_backward(variant, dtype, B, T, H, d_k, d_v, chunk, mu, q, k, v,
                               alpha, beta, proc_noise, obs_noise, S0, p0, d_o, dS_out,
                               dp_out, dq, dk, dv, dlog_alpha, dbeta, dproc_noise,
                               dobs_noise, dS0, dp0, workspace=None, workspace_bytes=0,
                               stream=None):
    """Raw entry point: same arguments as the C function."""
    lib = load()
    if workspace is not None and not isinstance(workspace, int) and not workspace_bytes:
        workspace_bytes = workspace.numel() * workspace.element_size()
    st = lib.kdn_chunk_prefill_backward(
        int(variant), int(dtype), int(B), int(T), int(H), int(d_k), int(d_v), int(chunk),
        float(mu), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(proc_noise),
        _ptr(obs_noise), _ptr(S0), _ptr(p0), _ptr(d_o), _ptr(dS_out), _ptr(dp_out),
        _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlog_alpha), _ptr(dbeta), _ptr(dproc_noise),
        _ptr(dobs_noise), _ptr(dS0), _ptr(dp0), _ptr(workspace), int(workspace_bytes),
        _stream(stream))
    _check(lib, st)


def kdn_chunk_prefill_backward_workspace_size(variant, dtype, B, T, H, d_k, d_v, chunk):
    """Bytes of workspace the gradient call needs; raises on invalid sizes."""
    lib = load()
    st = ctypes.c_int(0)
    n = lib.kdn_chunk_prefill_backward_workspace_size(
        int(variant), int(dtype), int(B), int(T), int(H), int(d_k), int(d_v), int(chunk),
        ctypes.byref(st))
    _check(lib, st.value)
    return int(n)


def kdn_recurrent_decode(variant, dtype, N, H, d_k, d_v, mu, q, k, v, alpha,
                         beta, proc_noise, obs_noise, S, p, o, stream=None):
    """Raw entry point: same arguments as the C function."""
    lib = load()
    st = lib.kdn_recurrent_decode(
        int(variant), int(dtype), int(N), int(H), int(d_k), int(d_v),
        float(mu), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
        _ptr(proc_noise), _ptr(obs_noise), _ptr(S), _ptr(p), _ptr(o),
        _stream(stream))
    _check(lib, st)


def kdn_recurrent_decode_multi(variant, dtype, N, T, H, d_k, d_v, mu, q, k, v,
                               alpha, beta, proc_noise, obs_noise, S0, p0, o,
                               S_out, p_out, stream=None):
    """Raw entry point: same arguments as the C function."""
    lib = load()
    st = lib.kdn_recurrent_decode_multi(
        int(variant), int(dtype), int(N), int(T), int(H), int(d_k), int(d_v),
        float(mu), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
        _ptr(proc_noise), _ptr(obs_noise), _ptr(S0), _ptr(p0), _ptr(o),
        _ptr(S_out), _ptr(p_out), _stream(stream))
    _check(lib, st)


# ---------------------------------------------------------------------------
# Tensor-shaped conveniences (allocate outputs, infer sizes, then call the
# entry points above).
# ---------------------------------------------------------------------------
def workspace(variant, q, v, chunk=0):
    """A workspace tensor (uint8, on q's device) for the two-pass prefill of
    inputs shaped like q [B,T,H,dk] and v [B,T,H,dv]; None if none is needed."""
    vid = VARIANTS[variant] if isinstance(variant, str) else int(variant)
    B, T, H, dk = q.shape
    n = kdn_chunk_prefill_workspace_size(vid, DTYPES[q.dtype], B, T, H, dk,
                                         v.shape[-1], chunk)
    if n == 0:
        return None
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def prefill(variant, q, k, v, alpha=None, beta=None, proc_noise=None,
            obs_noise=None, S0=None, p0=None, mu=1.0, chunk=0, out=None,
            workspace="auto", stream=None):
    """Chunkwise prefill.  q, k [B,T,H,dk], v [B,T,H,dv] (float32 or bf16).
    Returns (o, S, p); p is None unless the variant is a KDN ([B,H,dk] for
    diag_kdn, [B,H] for iso_kdn).  ``out`` may pass
    preallocated (o, S_out, p_out).  ``workspace``: "auto" allocates one for
    the two-pass schedule, None selects the single-pass kernel, a uint8
    tensor from :func:`workspace` is used as given."""
    vid = VARIANTS[variant] if isinstance(variant, str) else int(variant)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = DTYPES[q.dtype]
    if out is None:
        o = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
        S = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
        p = _new_p(vid, B, H, dk, q.device)
    else:
        o, S, p = out
    f32, pshape = torch.float32, _p_shape(vid, B, H, dk)
    _expect([("q", q, (B, T, H, dk), q.dtype), ("k", k, (B, T, H, dk), q.dtype),
             ("v", v, (B, T, H, dv), q.dtype)]
            + _gate_specs(vid, (B, T, H), dk, q.dtype, alpha, beta, proc_noise, obs_noise)
            + [("S0", S0, (B, H, dk, dv), f32), ("p0", p0, pshape, f32),
               ("o", o, (B, T, H, dv), q.dtype), ("S_out", S, (B, H, dk, dv), f32),
               ("p_out", p, pshape, f32)], q.device)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"kdn: workspace must be 'auto', None or a tensor, not {workspace!r}")
        workspace = globals()["workspace"](vid, q, v, chunk)
    kdn_chunk_prefill(vid, dt, B, T, H, dk, dv, chunk, mu, q, k, v, alpha, beta,
                      proc_noise, obs_noise, S0, p0, o, S, p, workspace, 0, stream)
    return o, S, p


def decode(variant, q, k, v, S, p=None, alpha=None, beta=None, proc_noise=None,
           obs_noise=None, mu=1.0, o=None, stream=None):
    """One decode step; S [N,H,dk,dv] (and p: [N,H,dk] for diag_kdn, [N,H]
    for iso_kdn) are updated in place.  Returns o [N,H,dv]."""
    vid = VARIANTS[variant] if isinstance(variant, str) else int(variant)
    N, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty((N, H, dv), dtype=q.dtype, device=q.device)
    f32 = torch.float32
    _expect([("q", q, (N, H, dk), q.dtype), ("k", k, (N, H, dk), q.dtype),
             ("v", v, (N, H, dv), q.dtype)]
            + _gate_specs(vid, (N, H), dk, q.dtype, alpha, beta, proc_noise, obs_noise)
            + [("S", S, (N, H, dk, dv), f32), ("p", p, _p_shape(vid, N, H, dk), f32),
               ("o", o, (N, H, dv), q.dtype)], q.device)
    kdn_recurrent_decode(vid, DTYPES[q.dtype], N, H, dk, dv, mu, q, k, v, alpha,
                         beta, proc_noise, obs_noise, S, p, o, stream)
    return o


def decode_multi(variant, q, k, v, alpha=None, beta=None, proc_noise=None,
                 obs_noise=None, S0=None, p0=None, mu=1.0, out=None, stream=None):
    """T decode steps in one pass over the state (speculative verify).
    q, k [N,T,H,dk], v [N,T,H,dv]; S0 [N,H,dk,dv] (None: zeros) and p0
    ([N,H,dk] diag_kdn, [N,H] iso_kdn) are read, not modified, unless ``out``
    passes them as S_out / p_out (in place).  Returns (o [N,T,H,dv], S_out,
    p_out); p_out is None unless the variant is a KDN."""
    vid = VARIANTS[variant] if isinstance(variant, str) else int(variant)
    N, T, H, dk = q.shape
    dv = v.shape[-1]
    if out is None:
        o = torch.empty((N, T, H, dv), dtype=q.dtype, device=q.device)
        S = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
        p = _new_p(vid, N, H, dk, q.device)
    else:
        o, S, p = out
    f32, pshape = torch.float32, _p_shape(vid, N, H, dk)
    _expect([("q", q, (N, T, H, dk), q.dtype), ("k", k, (N, T, H, dk), q.dtype),
             ("v", v, (N, T, H, dv), q.dtype)]
            + _gate_specs(vid, (N, T, H), dk, q.dtype, alpha, beta, proc_noise, obs_noise)
            + [("S0", S0, (N, H, dk, dv), f32), ("p0", p0, pshape, f32),
               ("o", o, (N, T, H, dv), q.dtype), ("S_out", S, (N, H, dk, dv), f32),
               ("p_out", p, pshape, f32)], q.device)
    kdn_recurrent_decode_multi(vid, DTYPES[q.dtype], N, T, H, dk, dv, mu, q, k, v,
                               alpha, beta, proc_noise, obs_noise, S0, p0, o, S, p,
                               stream)
    return o, S, p


def prefill_backward(variant, q, k, v, d_o, alpha=None, beta=None, proc_noise=None,
                     obs_noise=None, S0=None, p0=None, dS_out=None, dp_out=None, mu=1.0,
                     chunk=0, out=None, workspace=None, stream=None):
    """Gradients of :func:`prefill` (every variant) for the cotangents
    d_o [B,T,H,dv], dS_out [B,H,dk,dv] and (KDN) dp_out shaped as p0 (None:
    zero).  Returns a dict of float32 tensors: dq, dk, dv, dlog_alpha
    (alpha dL/dalpha: [B,T,H] for gated_deltanet, [B,T,H,dk] for kda and the
    KDNs, None for deltanet), dbeta (None for the KDNs), dS0, and for the KDNs
    dproc_noise, dobs_noise, dp0.  ``workspace``: a uint8 tensor of at least
    the queried size, or None to allocate one."""
    vid = VARIANTS[variant] if isinstance(variant, str) else int(variant)
    iso = vid in (3, 4)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = DTYPES[q.dtype]
    dev = q.device
    if out is None:
        f = torch.float32
        new = lambda *shape: torch.empty(shape, dtype=f, device=dev)
        out = dict(dq=new(B, T, H, dk), dk=new(B, T, H, dk), dv=new(B, T, H, dv),
                   dlog_alpha=None if vid == 0 else (new(B, T, H) if vid == 1
                                                     else new(B, T, H, dk)),
                   dbeta=None if iso else new(B, T, H), dS0=new(B, H, dk, dv),
                   dproc_noise=new(B, T, H, dk) if iso else None,
                   dobs_noise=new(B, T, H) if iso else None,
                   dp0=(new(B, H, dk) if vid == 3 else new(B, H)) if iso else None)
    f32, pshape = torch.float32, _p_shape(vid, B, H, dk)
    la_shape = (B, T, H) if vid == 1 else (B, T, H, dk)
    _expect([("q", q, (B, T, H, dk), q.dtype), ("k", k, (B, T, H, dk), q.dtype),
             ("v", v, (B, T, H, dv), q.dtype), ("d_o", d_o, (B, T, H, dv), q.dtype)]
            + _gate_specs(vid, (B, T, H), dk, q.dtype, alpha, beta, proc_noise, obs_noise)
            + [("S0", S0, (B, H, dk, dv), f32), ("p0", p0, pshape, f32),
               ("dS_out", dS_out, (B, H, dk, dv), f32), ("dp_out", dp_out, pshape, f32),
               ("dq", out["dq"], (B, T, H, dk), f32), ("dk", out["dk"], (B, T, H, dk), f32),
               ("dv", out["dv"], (B, T, H, dv), f32),
               ("dlog_alpha", out["dlog_alpha"], la_shape, f32),
               ("dbeta", out["dbeta"], (B, T, H), f32),
               ("dproc_noise", out["dproc_noise"], (B, T, H, dk), f32),
               ("dobs_noise", out["dobs_noise"], (B, T, H), f32),
               ("dS0", out["dS0"], (B, H, dk, dv), f32), ("dp0", out["dp0"], pshape, f32)],
            q.device)
    if workspace is None:
        n = kdn_chunk_prefill_backward_workspace_size(vid, dt, B, T, H, dk, dv, chunk)
        workspace = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    kdn_chunk_prefill_backward(vid, dt, B, T, H, dk, dv, chunk, mu, q, k, v, alpha, beta,
                               proc_noise, obs_noise, S0, p0, d_o, dS_out, dp_out,
                               out["dq"], out["dk"], out["dv"], out["dlog_alpha"],
                               out["dbeta"], out["dproc_noise"], out["dobs_noise"],
                               out["dS0"], out["dp0"], workspace, 0, stream)
    return out


# ---------------------------------------------------------------------------
# Linear attention with a decay for each head, and the tables of a packed batch.
# ---------------------------------------------------------------------------
@dataclasses.dataclass
class SequenceTables:
    """Tables of a packed batch (:func:`sequence_tables`), int32 on the GPU."""
    tokens: int                          # rows of the packed batch
    block: int                           # tokens of a block
    offsets: torch.Tensor                # [N + 1] first row of each sequence
    block_offsets: torch.Tensor          # [N + 1] first block of each sequence
    blocks: torch.Tensor                 # [max_blocks, 4]
    slots: torch.Tensor | None           # [N] state of each sequence (None: n)
    slot_map: torch.Tensor | None        # [tokens] state of each token
    positions: torch.Tensor | None       # [tokens] position of each token


# the current stream's handle without a Stream object around it, where torch
# has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, dev, stream, *args):
    """Call fn(*args, stream) with the tensors' device current.  These calls
    are short on the GPU too, so their checks take the quickest way that says
    yes and leave the words to the slow one."""
    if dev.type != "cuda":
        raise ValueError(f"kdn: tensors must be in GPU memory, not on {dev}")
    if stream is None:
        stream = _raw_stream(dev.index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if dev.index == torch.cuda.current_device():
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st != 0:
        _check(_lib, st)


def _same(name, x, shape, dtype, dev):
    """x is None or a contiguous GPU tensor of this shape, dtype and device."""
    if x is None or (isinstance(x, torch.Tensor) and x.shape == shape and x.dtype is dtype
                     and x.is_cuda and x.device == dev and x.is_contiguous()):
        return
    _expect([(name, x, shape, dtype)], dev)


def _new(shape, dtype, dev, stream, zero=False):
    """New memory for a call on ``stream``, allocated (and cleared) as under
    ``torch.cuda.stream(stream)``: memory of the current stream's pool could
    still be in use there."""
    if dev.type != "cuda":
        raise ValueError(f"kdn: tensors must be in GPU memory, not on {dev}")
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=dev)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev) if stream \
            else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=dev)


def _p(x):
    return None if x is None else x.data_ptr()


def _rows(name, x, lead, dtype, dev):
    """Checks of a per-token tensor [*lead, heads, d] whose rows may be slices
    of wider ones; returns the elements between tokens."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"kdn: {name} must be a tensor")
    n, shape = len(lead), x.shape
    if len(shape) == n + 2 and shape[:n] == lead and x.dtype is dtype and x.device == dev \
            and x.is_contiguous():
        return shape[n] * shape[n + 1]
    if x.dim() != n + 2 or tuple(x.shape[:n]) != lead:
        raise ValueError(f"kdn: {name} has shape {tuple(x.shape)}, expected "
                         f"{lead + ('heads', 'd')}")
    if x.dtype != dtype:
        raise ValueError(f"kdn: {name} has dtype {x.dtype}, expected {dtype}")
    if x.device != dev:
        raise ValueError(f"kdn: {name} is on {x.device}, the other tensors on {dev}")
    heads, d = x.shape[n:]
    st = x.stride()
    row = st[n - 1]
    if st[-1] != 1 or (heads > 1 and st[-2] != d) or row < heads * d or \
            (n == 2 and lead[0] > 1 and st[0] != lead[1] * row):
        if n == 2 and lead[1] == 1 and st[-1] == 1 and (heads == 1 or st[-2] == d) \
                and st[0] >= heads * d:
            return st[0]                 # one token per sequence: any distance between them
        raise ValueError(f"kdn: {name} must have contiguous heads and rows at one distance")
    return row


def _gate(log_alpha, lead, H, dtype, dev):
    if log_alpha.dim() == 1:
        want, dt, gate = (H,), torch.float32, GATE_HEAD
    else:
        want, dt, gate = lead + (H,), dtype, GATE_TOKEN
    _same("log_alpha", log_alpha, want, dt, dev)
    return gate


def _linear_heads(q, k, v, log_alpha):
    """States per token: the largest head count of q, k, v and log_alpha."""
    if not isinstance(log_alpha, torch.Tensor) or log_alpha.dim() == 0:
        raise TypeError("kdn: log_alpha must be a tensor [.., H]")
    a, b, c, H = q.shape[-2], k.shape[-2], v.shape[-2], log_alpha.shape[-1]
    if a == b == c == H:
        return H
    H = max(a, b, c, H)
    for name, n in (("q", a), ("k", b), ("v", c)):
        if n == 0 or H % n:
            raise ValueError(f"kdn: the {n} heads of {name} do not divide {H}")
    return H


def _int32(name, x):
    """x as an int the library can take (ctypes would pass its low 32 bits)."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise KdnError(2, f"{name} {x} does not fit 32 bits")
    return x


def linear_block(tokens, N, H):
    """Tokens of a block for :func:`sequence_tables` of N sequences with
    ``tokens`` rows in all and H states each."""
    n = int(load().kdn_linear_block(_int32("tokens", tokens), _int32("N", N), _int32("H", H)))
    if n < 0:
        raise KdnError(2, kdn_status_string(2))
    return n


def sequence_tables(lengths, tokens, block, slots=None, context=None, maps=False, out=None,
                    stream=None):
    """Tables of a packed batch of ``tokens`` rows, built on the GPU from the
    sequences' lengths [N] int32 (on the GPU; nothing is copied to the host).
    ``block``: tokens of a block, a multiple of 64 (:func:`linear_block`).
    ``slots`` [N] int32: state of each sequence in a pool; ``context`` [N]
    int32: tokens each sequence had before.  ``maps``: also the slot and the
    position of every token.  ``out``: a SequenceTables of the same sizes to
    fill (for a captured graph).  Returns a :class:`SequenceTables`."""
    lib = load()
    if not isinstance(lengths, torch.Tensor) or lengths.dim() != 1:
        raise ValueError("kdn: lengths must be a tensor [N]")
    N, dev, i32 = _int32("N", lengths.shape[0]), lengths.device, torch.int32
    tokens, block = _int32("tokens", tokens), _int32("block", block)
    rows = lib.kdn_sequence_max_blocks(N, tokens, block)
    if rows < 0:
        raise KdnError(2, f"tokens {tokens} must not be negative, block {block} a positive "
                          "multiple of 64")
    _same("lengths", lengths, (N,), i32, dev)
    _same("slots", slots, (N,), i32, dev)
    _same("context", context, (N,), i32, dev)
    if out is None:
        # one piece of memory, the blocks (16-byte rows) first
        n = tokens if maps else 0
        parts = _new((4 * rows + 2 * (N + 1) + 2 * n,), i32, dev, stream).split_with_sizes(
            [4 * rows, N + 1, N + 1, n, n])
        out = SequenceTables(tokens, block, parts[1], parts[2], parts[0].view(rows, 4), slots,
                             parts[3] if maps else None, parts[4] if maps else None)
    else:
        for name, x, shape in (("offsets", out.offsets, (N + 1,)),
                               ("block_offsets", out.block_offsets, (N + 1,)),
                               ("blocks", out.blocks, (rows, 4)),
                               ("slot_map", out.slot_map, (tokens,)),
                               ("positions", out.positions, (tokens,))):
            _same(name, x, shape, i32, dev)
    _call(lib.kdn_sequence_tables, dev, stream, N, tokens, block, rows, _p(lengths), _p(slots),
          _p(context), _p(out.offsets), _p(out.block_offsets), _p(out.blocks), _p(out.slot_map),
          _p(out.positions))
    # a refused call leaves `out` describing the tables it holds
    out.tokens, out.block, out.slots = tokens, block, slots
    return out


def _packed(tables, pool, dev):
    """The kdn_packed of the tables, and the number of sequences.  Without a
    pool (None) the states are by sequence and the slots are not looked at."""
    N, i32 = tables.offsets.shape[0] - 1, torch.int32
    rows = load().kdn_sequence_max_blocks(N, tables.tokens, tables.block)
    _same("offsets", tables.offsets, (N + 1,), i32, dev)
    _same("block_offsets", tables.block_offsets, (N + 1,), i32, dev)
    _same("blocks", tables.blocks, (rows, 4), i32, dev)
    _same("slots", tables.slots, (N,), i32, dev)
    return Packed(tables.tokens, tables.block, rows, N if pool is None else pool,
                  _p(tables.blocks), _p(tables.block_offsets),
                  None if pool is None else _p(tables.slots)), N


def _linear_sizes(q, tables, S0, S):
    """(lead, sequences or None, tokens per sequence, states in S0 / S_out or
    None for a packed batch without a pool)."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("kdn: q must be a tensor")
    if tables is None:
        if q.dim() != 4:
            raise ValueError(f"kdn: q has shape {tuple(q.shape)}, expected [B, T, heads, d_k]")
        return tuple(q.shape[:2]), q.shape[0], q.shape[1], q.shape[0]
    if q.dim() != 3:
        raise ValueError(f"kdn: q has shape {tuple(q.shape)}, expected [tokens, heads, d_k]")
    if q.shape[0] != tables.tokens:
        raise ValueError(f"kdn: q has {q.shape[0]} rows, the tables {tables.tokens}")
    for x in (S0, S):
        if x is not None:
            return (q.shape[0],), None, 0, x.shape[0]
    return (q.shape[0],), None, 0, None


def linear_prefill(q, k, v, log_alpha, S0=None, tables=None, out=None, workspace="auto",
                   stream=None):
    """Chunkwise prefill of linear attention with a decay for each head:
    S_t = exp(log_alpha_t) S_{t-1} + k_t v_t^T, o_t = S_t^T q_t.

    Dense: q [B,T,Hq,dk], k [B,T,Hk,dk], v [B,T,Hv,dv] (float32 or bf16; rows
    may be slices of one wider tensor), log_alpha [B,T,H] in q's dtype or [H]
    float32 (one constant per head), S0 [B,H,dk,dv] float32 or None (zeros).
    H is the largest of the head counts; the others divide it.
    Packed (``tables`` from :func:`sequence_tables`): the same without B, rows
    [tokens, ..]; S0 and S_out are pools [P,H,dk,dv] of states by slot.
    Where neither is given, states are by sequence and slots are not looked at.
    ``out`` may pass (o, S_out); S_out may be S0 (in place) or None (not
    wanted).  Without it S_out is new, and for a packed batch with S0 the pool
    S0 itself, updated in place.  Rows of o behind the last sequence are left
    as they were.  Returns (o, S_out)."""
    lib = load()
    if not isinstance(q, torch.Tensor):
        raise TypeError("kdn: q must be a tensor")
    dt, dev = q.dtype, q.device
    if dt not in DTYPES:
        raise ValueError(f"kdn: q has dtype {dt}, expected float32 or bfloat16")
    lead, N, T, pool = _linear_sizes(q, tables, S0, out[1] if out is not None else None)
    qs, ks = _rows("q", q, lead, dt, dev), _rows("k", k, lead, dt, dev)
    vs = _rows("v", v, lead, dt, dev)
    H = _linear_heads(q, k, v, log_alpha)
    dk, dv, f32 = q.shape[-1], v.shape[-1], torch.float32
    gate = _gate(log_alpha, lead, H, dt, dev)
    pk = None
    if tables is not None:
        pk, N = _packed(tables, pool, dev)
        pool = N if pool is None else pool
    if out is None:
        o = _new(lead + (H, dv), dt, dev, stream)
        if tables is None:
            S = _new((pool, H, dk, dv), f32, dev, stream)
        elif S0 is not None:
            S = S0
        else:
            if tables.slots is not None:
                raise ValueError("kdn: a pool for the tables' slots must be given (S0 or out)")
            S = _new((pool, H, dk, dv), f32, dev, stream)
    else:
        o, S = out
    if k.shape[-1] != dk:
        _same("k", k, lead + (k.shape[-2], dk), dt, dev)
    s_shape = (pool, H, dk, dv)
    _same("S0", S0, s_shape, f32, dev)
    _same("o", o, lead + (H, dv), dt, dev)
    _same("S_out", S, s_shape, f32, dev)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"kdn: workspace must be 'auto', None or a tensor, not {workspace!r}")
        workspace = _linear_workspace(DTYPES[dt], N, T, H, dk, dv, pk, dev, stream)
    nws = 0
    if workspace is not None:
        nws = workspace.numel()
        _same("workspace", workspace, (nws,), torch.uint8, dev)
    _call(lib.kdn_linear_prefill, dev, stream, DTYPES[dt], N, T, H, q.shape[-2], k.shape[-2],
          v.shape[-2], dk, dv, gate, qs, ks, vs, _p(q), _p(k), _p(v), _p(log_alpha), _p(S0),
          _p(o), _p(S), pk, _p(workspace), nws)
    return o, S


def _linear_workspace(dtype, N, T, H, dk, dv, pk, dev, stream):
    st = ctypes.c_int(0)
    n = load().kdn_linear_prefill_workspace_size(dtype, N, T, H, dk, dv, pk, ctypes.byref(st))
    _check(_lib, st.value)
    return _new((n,), torch.uint8, dev, stream) if n else None


def linear_workspace(q, k, v, log_alpha, tables=None, stream=None):
    """A workspace tensor (uint8) for :func:`linear_prefill` of these inputs,
    None if none is needed.  Calls that share one must not overlap in time."""
    H = _linear_heads(q, k, v, log_alpha)
    pk = None
    if tables is None:
        N, T = q.shape[:2]
    else:
        T = 0
        pk, N = _packed(tables, 0, q.device)
    return _linear_workspace(DTYPES[q.dtype], N, T, H, q.shape[-1], v.shape[-1], pk, q.device,
                             stream)


def linear_decode(q, k, v, log_alpha, S, slots=None, o=None, stream=None):
    """One token of linear attention for N rows: q [N,Hq,dk], k [N,Hk,dk],
    v [N,Hv,dv], log_alpha [N,H] in q's dtype or [H] float32.  S [P,H,dk,dv]
    float32 is a pool of states, updated in place; ``slots`` [N] int32 is each
    row's state (None: row n).  A row whose slot is not in the pool is skipped,
    its o left as it was (zero in a new o).  Returns o [N,H,dv]."""
    lib = load()
    if not isinstance(q, torch.Tensor):
        raise TypeError("kdn: q must be a tensor")
    dt, dev = q.dtype, q.device
    if dt not in DTYPES:
        raise ValueError(f"kdn: q has dtype {dt}, expected float32 or bfloat16")
    if q.dim() != 3:
        raise ValueError(f"kdn: q has shape {tuple(q.shape)}, expected [N, heads, d_k]")
    N, lead = q.shape[0], (q.shape[0],)
    qs, ks = _rows("q", q, lead, dt, dev), _rows("k", k, lead, dt, dev)
    vs = _rows("v", v, lead, dt, dev)
    H = _linear_heads(q, k, v, log_alpha)
    dk, dv = q.shape[-1], v.shape[-1]
    gate = _gate(log_alpha, lead, H, dt, dev)
    if not isinstance(S, torch.Tensor) or S.dim() != 4:
        raise ValueError("kdn: S must be a tensor [P, H, dk, dv]")
    pool = S.shape[0]
    if o is None:
        o = _new((N, H, dv), dt, dev, stream, zero=slots is not None)
    if k.shape[-1] != dk:
        _same("k", k, (N, k.shape[-2], dk), dt, dev)
    _same("S", S, (pool, H, dk, dv), torch.float32, dev)
    _same("o", o, (N, H, dv), dt, dev)
    _same("slots", slots, (N,), torch.int32, dev)
    _call(lib.kdn_linear_decode, dev, stream, DTYPES[dt], N, H, q.shape[-2], k.shape[-2],
          v.shape[-2], dk, dv, gate, qs, ks, vs, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          log_alpha.data_ptr(), _p(slots), pool, S.data_ptr(), o.data_ptr())
    return o


def linear_prefill_backward(q, k, v, d_o, log_alpha, S0=None, dS_out=None, tables=None, out=None,
                            workspace=None, stream=None):
    """Gradients of :func:`linear_prefill` for the cotangents d_o (shaped as o)
    and dS_out (shaped as S_out; None: zero).  Returns a dict of dq, dk, dv
    (shaped as q, k, v, contiguous) and dlog_alpha ([..,H], or [H] for one
    decay per head) in q's dtype, and dS0 float32.  A head that several states
    share gets the sum of their gradients; rows behind the last sequence of a
    packed batch get zero, and so do states of dS0 without a sequence.  ``out``
    may pass such a dict (dlog_alpha and dS0 may be None: not wanted; a given
    dlog_alpha [H] may be float32 as log_alpha [H] is, which keeps all bits of
    the sum in a bf16 call; in a given dS0 states without a sequence are left
    as they were).
    ``workspace``: a uint8 tensor of at least the queried size, or None to
    allocate one.  A packed batch without any of S0, dS_out and out["dS0"] has
    no pool: dS0 is by sequence and slots are not looked at."""
    lib = load()
    if not isinstance(q, torch.Tensor):
        raise TypeError("kdn: q must be a tensor")
    dt, dev = q.dtype, q.device
    if dt not in DTYPES:
        raise ValueError(f"kdn: q has dtype {dt}, expected float32 or bfloat16")
    lead, N, T, pool = _linear_sizes(q, tables, S0, dS_out if dS_out is not None else
                                     (out or {}).get("dS0"))
    qs, ks, vs = (_rows(n, x, lead, dt, dev) for n, x in (("q", q), ("k", k), ("v", v)))
    H = _linear_heads(q, k, v, log_alpha)
    Hq, Hk, Hv = q.shape[-2], k.shape[-2], v.shape[-2]
    dk, dv, f32 = q.shape[-1], v.shape[-1], torch.float32
    gate = _gate(log_alpha, lead, H, dt, dev)
    pk = None
    if tables is not None:
        pk, N = _packed(tables, pool, dev)
        pool = N if pool is None else pool
    la_shape, la_dt = (H,) if gate == GATE_HEAD else lead + (H,), dt
    s_shape = (pool, H, dk, dv)
    if out is None:
        new = lambda *shape: _new(shape, dt, dev, stream)
        out = dict(dq=new(*lead, Hq, dk), dk=new(*lead, Hk, dk), dv=new(*lead, Hv, dv),
                   dlog_alpha=new(*la_shape),
                   dS0=_new(s_shape, f32, dev, stream, zero=tables is not None))
    elif gate == GATE_HEAD and isinstance(out["dlog_alpha"], torch.Tensor) \
            and out["dlog_alpha"].dtype is f32:
        gate, la_dt = GATE_HEAD_F32, f32
    if k.shape[-1] != dk:
        _same("k", k, lead + (Hk, dk), dt, dev)
    for name, x, shape, t in (("d_o", d_o, lead + (H, dv), dt), ("S0", S0, s_shape, f32),
                              ("dS_out", dS_out, s_shape, f32), ("dq", out["dq"], lead + (Hq, dk), dt),
                              ("dk", out["dk"], lead + (Hk, dk), dt),
                              ("dv", out["dv"], lead + (Hv, dv), dt),
                              ("dlog_alpha", out["dlog_alpha"], la_shape, la_dt),
                              ("dS0", out["dS0"], s_shape, f32)):
        _same(name, x, shape, t, dev)
    if workspace is None:
        st = ctypes.c_int(0)
        n = lib.kdn_linear_prefill_backward_workspace_size(
            DTYPES[dt], N, T, H, Hq, Hk, Hv, dk, dv, gate, pk, ctypes.byref(st))
        _check(lib, st.value)
        workspace = _new((n,), torch.uint8, dev, stream) if n else None
    nws = 0
    if workspace is not None:
        nws = workspace.numel()
        _same("workspace", workspace, (nws,), torch.uint8, dev)
    _call(lib.kdn_linear_prefill_backward, dev, stream, DTYPES[dt], N, T, H, Hq, Hk, Hv, dk, dv,
          gate, qs, ks, vs, _p(q), _p(k), _p(v), _p(log_alpha), _p(S0), _p(d_o), _p(dS_out),
          _p(out["dq"]), _p(out["dk"]), _p(out["dv"]), _p(out["dlog_alpha"]), _p(out["dS0"]), pk,
          _p(workspace), nws)
    return out
