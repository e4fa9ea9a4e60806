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
import math
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

# kdn_activation and kdn_norm_order values
ACTIVATIONS = {None: 0, "silu": 1, "sigmoid": 2}
NORM_ORDERS = {"norm_gate": 0, "gate_norm": 1}
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
    ip = ctypes.POINTER(i)
    lib.kdn_causal_conv.restype = i
    lib.kdn_causal_conv.argtypes = [i] * 6 + [ll] + [vp] * 6 + [pk, vp]
    lib.kdn_causal_conv_decode.restype = i
    lib.kdn_causal_conv_decode.argtypes = [i] * 5 + [ll] + [vp] * 4 + [i] + [vp] * 3
    lib.kdn_causal_conv_backward.restype = i
    lib.kdn_causal_conv_backward.argtypes = [i] * 6 + [ll] + [vp] * 10 + [pk, vp, u64, vp]
    lib.kdn_causal_conv_backward_workspace_size.restype = u64
    lib.kdn_causal_conv_backward_workspace_size.argtypes = [i] * 5 + [pk, ip]
    lib.kdn_selective_block.restype = i
    lib.kdn_selective_block.argtypes = [i] * 4
    lib.kdn_selective_scan.restype = i
    lib.kdn_selective_scan.argtypes = [i] * 7 + [ll] * 5 + [vp] * 11 + [pk, vp, u64, vp]
    lib.kdn_selective_scan_workspace_size.restype = u64
    lib.kdn_selective_scan_workspace_size.argtypes = [i] * 6 + [pk, ip]
    lib.kdn_selective_decode.restype = i
    lib.kdn_selective_decode.argtypes = [i] * 5 + [i] + [ll] * 5 + [vp] * 9 + [i] + [vp] * 3
    lib.kdn_selective_scan_backward.restype = i
    lib.kdn_selective_scan_backward.argtypes = [i] * 7 + [ll] * 5 + [vp] * 20 + [pk, vp, u64, vp]
    lib.kdn_selective_scan_backward_workspace_size.restype = u64
    lib.kdn_selective_scan_backward_workspace_size.argtypes = [i] * 6 + [pk, ip]
    lib.kdn_gated_norm.restype = i
    lib.kdn_gated_norm.argtypes = [i] * 7 + [f, ll, ll] + [vp] * 5
    lib.kdn_gated_norm_backward.restype = i
    lib.kdn_gated_norm_backward.argtypes = [i] * 7 + [f, ll, ll] + [vp] * 8 + [u64, vp]
    lib.kdn_gated_norm_backward_workspace_size.restype = u64
    lib.kdn_gated_norm_backward_workspace_size.argtypes = [i] * 4 + [ip]
    lib.kdn_residual_norm.restype = i
    lib.kdn_residual_norm.argtypes = [i] * 5 + [f, ll, ll] + [vp] * 7
    lib.kdn_residual_norm_backward.restype = i
    lib.kdn_residual_norm_backward.argtypes = [i] * 5 + [f, ll, ll] + [vp] * 11 + [u64, vp]
    lib.kdn_residual_norm_backward_workspace_size.restype = u64
    lib.kdn_residual_norm_backward_workspace_size.argtypes = [i] * 3 + [ip]
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


# the current device's index; tensors in GPU memory are there, so it is initialised
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


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
    if dev.index == _current_device():
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st != 0:
        _check(_lib, st)


def _same(name, x, shape, dtype, dev):
    """x is None or a contiguous GPU tensor of this shape, dtype and device."""
    if x is None or (isinstance(x, torch.Tensor) and x.shape == shape and x.dtype is dtype
                     and x.get_device() == dev.index and x.is_contiguous()):
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


# ---------------------------------------------------------------------------
# Around a recurrence: the short causal convolution in front of it, the norms
# behind and before it.
# ---------------------------------------------------------------------------
_f32 = torch.float32


def _dtype(name, x):
    """dtype and device of a call's first per-token tensor."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"kdn: {name} must be a tensor")
    if x.dtype not in DTYPES:
        raise ValueError(f"kdn: {name} has dtype {x.dtype}, expected float32 or bfloat16")
    return x.dtype, x.device


def _strided(name, x, lead, tail, dtype, dev):
    """Checks of a per-token tensor [*lead, *tail] whose rows may be slices of
    wider ones; returns the elements between tokens (0: contiguous)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"kdn: {name} must be a tensor")
    if x.shape == lead + tail and x.dtype is dtype and x.device == dev and x.is_contiguous():
        return 0
    if x.shape != lead + tail:
        raise ValueError(f"kdn: {name} has shape {tuple(x.shape)}, expected {lead + tail}")
    if x.dtype is not dtype:
        raise ValueError(f"kdn: {name} has dtype {x.dtype}, expected {dtype}")
    if x.device != dev:
        raise ValueError(f"kdn: {name} is on {x.device}, the other tensors on {dev}")
    if x.numel() == 0:
        return 0
    n, st, row = len(lead), x.stride(), 1
    for size, step in zip(reversed(tail), reversed(st[n:])):
        if size > 1 and step != row:
            raise ValueError(f"kdn: {name} must have contiguous rows")
        row *= size
    # one distance between all tokens; dimensions of one element have none
    dist, tokens = None, 1
    for size, step in zip(reversed(lead), reversed(st[:n])):
        if size > 1:
            if dist is None:
                if step % tokens:
                    raise ValueError(f"kdn: {name} must have rows at one distance")
                dist = step // tokens
            elif step != dist * tokens:
                raise ValueError(f"kdn: {name} must have rows at one distance")
        tokens *= size
    if dist is None:
        return 0
    if dist < row:
        raise ValueError(f"kdn: {name} must have rows that do not overlap")
    return dist


def _activation(activation, among):
    if activation not in among:
        raise ValueError(f"kdn: activation must be one of {among}, not {activation!r}")
    return ACTIVATIONS[activation]


def _batch(x, tables, states, ndim, what):
    """(lead, N, T, kdn_packed or None, pool) of a dense or packed batch whose
    per-token tensors have ``ndim`` dimensions behind the tokens; the pool is that of
    the first of ``states`` which is given."""
    if tables is None:
        if x.dim() != 2 + ndim:
            raise ValueError(f"kdn: {what} has shape {tuple(x.shape)}, expected [B, T, ..]")
        B, T = x.shape[:2]
        return (B, T), _int32("B", B), _int32("T", T), None, B
    if x.dim() != 1 + ndim:
        raise ValueError(f"kdn: {what} has shape {tuple(x.shape)}, expected [tokens, ..]")
    if x.shape[0] != tables.tokens:
        raise ValueError(f"kdn: {what} has {x.shape[0]} rows, the tables {tables.tokens}")
    pool = next((_int32("pool", s.shape[0]) for s in states
                 if isinstance(s, torch.Tensor) and s.dim() > 0), None)
    pk, N = _packed(tables, pool, x.device)
    return (x.shape[0],), N, 0, pk, N if pool is None else pool


def _workspace(n, workspace, dev, stream):
    """A workspace of n bytes if none is given, and its size."""
    if workspace is None:
        workspace = _new((n,), torch.uint8, dev, stream) if n else None
    if workspace is None:
        return None, 0
    _same("workspace", workspace, (workspace.numel(),), torch.uint8, dev)
    return workspace, workspace.numel()


def _like(x, dtype, dev, stream):
    """New memory for a contiguous tensor of x's shape, the quickest way."""
    if stream is None and x.dtype is dtype and dev.type == "cuda" and x.is_contiguous():
        return torch.empty_like(x)
    return _new(x.shape, dtype, dev, stream)


def _outputs(out, specs, dev, stream):
    """A call's outputs (name, shape of or tensor like it, dtype, whether wanted or "zero"):
    those of ``out``, checked, or new ones."""
    if out is None:
        return {name: None if not want else _like(shape, kind, dev, stream)
                if isinstance(shape, torch.Tensor)
                else _new(shape, kind, dev, stream, zero=want == "zero")
                for name, shape, kind, want in specs}
    for name, shape, kind, want in specs:
        if out[name] is not None:
            _same(name, out[name], shape.shape if isinstance(shape, torch.Tensor) else shape,
                  kind, dev)
    return out


def _taps(weight, C):
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("kdn: weight must be a tensor [C, W]")
    return _int32("W", weight.shape[1])


def causal_conv(x, weight, bias=None, state0=None, tables=None, activation="silu", out=None,
                stream=None):
    """Short causal convolution of each channel and its activation ("silu" or
    None): s_t = bias + sum_j weight[:, j] x_{t-W+1+j}, y = s sigmoid(s).

    Dense: x [B,T,C] (float32 or bf16, rows may be slices of one wider tensor);
    packed (``tables`` from :func:`sequence_tables`): x [tokens,C].  weight [C,W]
    float32, W 2 to 4, bias [C] float32 or None.  ``state0`` [B or pool,W-1,C] in
    x's dtype holds the rows before each sequence (None: zeros).  ``out`` may pass
    (y, state_out); state_out may be state0 (in place) or None (not wanted).
    Without it state_out is new, and for a packed batch with state0 the pool state0
    itself, updated in place.  Rows of y behind the last sequence are left as they
    were.  Returns (y, state_out)."""
    lib = load()
    dt, dev = _dtype("x", x)
    act = _activation(activation, (None, "silu"))
    lead, N, T, pk, pool = _batch(x, tables, (state0, out[1] if out is not None else None), 1, "x")
    C = _int32("C", x.shape[-1])
    W = _taps(weight, C)
    xs = _strided("x", x, lead, (C,), dt, dev)
    s_shape = (pool, W - 1, C)
    if out is None:
        y = _like(x, dt, dev, stream)
        if tables is not None and state0 is not None:
            S = state0
        elif tables is not None and tables.slots is not None:
            raise ValueError("kdn: a pool for the tables' slots must be given (state0 or out)")
        else:
            S = _new((pool, max(W - 1, 0), C), dt, dev, stream)
    else:
        y, S = out
    _same("weight", weight, (C, W), _f32, dev)
    _same("bias", bias, (C,), _f32, dev)
    _same("state0", state0, s_shape, dt, dev)
    _same("y", y, lead + (C,), dt, dev)
    _same("state_out", S, s_shape, dt, dev)
    _call(lib.kdn_causal_conv, dev, stream, DTYPES[dt], N, T, C, W, act, xs, _p(x), _p(weight),
          _p(bias), _p(state0), _p(y), _p(S), pk)
    return y, S


def causal_conv_decode(x, weight, state, bias=None, activation="silu", slots=None, y=None,
                       stream=None):
    """One token of :func:`causal_conv` for N rows x [N,C].  ``state`` [P,W-1,C] in
    x's dtype is a pool of states, updated in place; ``slots`` [N] int32 is each
    row's state (None: row n).  A row whose slot is not in the pool is skipped, its y
    left as it was (zero in a new y).  Returns y [N,C]."""
    lib = load()
    dt, dev = _dtype("x", x)
    act = _activation(activation, (None, "silu"))
    if x.dim() != 2:
        raise ValueError(f"kdn: x has shape {tuple(x.shape)}, expected [N, C]")
    N, C = _int32("N", x.shape[0]), _int32("C", x.shape[1])
    W = _taps(weight, C)
    xs = _strided("x", x, (N,), (C,), dt, dev)
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError("kdn: state must be a tensor [P, W - 1, C]")
    pool = _int32("pool", state.shape[0])
    if y is None:
        y = _new((N, C), dt, dev, stream, zero=slots is not None)
    _same("weight", weight, (C, W), _f32, dev)
    _same("bias", bias, (C,), _f32, dev)
    _same("state", state, (pool, W - 1, C), dt, dev)
    _same("y", y, (N, C), dt, dev)
    _same("slots", slots, (N,), torch.int32, dev)
    _call(lib.kdn_causal_conv_decode, dev, stream, DTYPES[dt], N, C, W, act, xs, _p(x), _p(weight),
          _p(bias), _p(slots), pool, _p(state), _p(y))
    return y


def causal_conv_backward(x, weight, d_y, bias=None, state0=None, dstate_out=None, tables=None,
                         activation="silu", out=None, workspace=None, stream=None):
    """Gradients of :func:`causal_conv` for the cotangents d_y (shaped as y) and
    dstate_out (shaped as state_out; None: zero).  Returns a dict of dx and dstate0
    in x's dtype, dweight and dbias float32.  Rows behind the last sequence of a
    packed batch get zero, and so do states of dstate0 without a sequence.  ``out``
    may pass such a dict (dbias and dstate0 may be None: not wanted; in a given
    dstate0 states without a sequence are left as they were).  A packed batch
    without any of state0, dstate_out and out["dstate0"] has no pool: dstate0 is by
    sequence and slots are not looked at."""
    lib = load()
    dt, dev = _dtype("x", x)
    act = _activation(activation, (None, "silu"))
    lead, N, T, pk, pool = _batch(x, tables, (state0, dstate_out, (out or {}).get("dstate0")), 1, "x")
    C = _int32("C", x.shape[-1])
    W = _taps(weight, C)
    xs = _strided("x", x, lead, (C,), dt, dev)
    s_shape = (pool, W - 1, C)
    _same("weight", weight, (C, W), _f32, dev)
    _same("bias", bias, (C,), _f32, dev)
    out = _outputs(out, (("dx", x, dt, True), ("dweight", weight, _f32, True),
                         ("dbias", (C,), _f32, bias is not None),
                         ("dstate0", (pool, max(W - 1, 0), C), dt,
                          True if tables is None else "zero")), dev, stream)
    _same("d_y", d_y, lead + (C,), dt, dev)
    _same("state0", state0, s_shape, dt, dev)
    _same("dstate_out", dstate_out, s_shape, dt, dev)
    st = ctypes.c_int(0)
    n = lib.kdn_causal_conv_backward_workspace_size(DTYPES[dt], N, T, C, W, pk, ctypes.byref(st))
    _check(lib, st.value)
    workspace, n = _workspace(n, workspace, dev, stream)
    _call(lib.kdn_causal_conv_backward, dev, stream, DTYPES[dt], N, T, C, W, act, xs, _p(x),
          _p(weight), _p(bias), _p(state0), _p(d_y), _p(dstate_out), _p(out["dx"]),
          _p(out["dweight"]), _p(out["dbias"]), _p(out["dstate0"]), pk, _p(workspace), n)
    return out


def selective_block(tokens, N, C, S):
    """Tokens of a block for :func:`sequence_tables` of N sequences with ``tokens``
    rows in all and C channels of S states."""
    n = int(load().kdn_selective_block(_int32("tokens", tokens), _int32("N", N), _int32("C", C),
                                       _int32("S", S)))
    if n < 0:
        raise KdnError(2, kdn_status_string(2))
    return n


def _scan_inputs(x, delta, A, B, C, D, z, delta_bias, lead):
    """Checks of a scan's inputs: (channels, states, groups, strides)."""
    dt, dev = x.dtype, x.device
    n = len(lead)
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("kdn: A must be a tensor [C, S]")
    if not isinstance(B, torch.Tensor) or B.dim() != n + 2:
        raise ValueError("kdn: B must be a tensor [.., G, S]")
    c, s, g = _int32("C", x.shape[-1]), _int32("S", A.shape[1]), _int32("G", B.shape[-2])
    strides = (_strided("x", x, lead, (c,), dt, dev), _strided("delta", delta, lead, (c,), dt, dev),
               0 if z is None else _strided("z", z, lead, (c,), dt, dev),
               _strided("B", B, lead, (g, s), dt, dev), _strided("C", C, lead, (g, s), dt, dev))
    _same("A", A, (c, s), _f32, dev)
    _same("D", D, (c,), _f32, dev)
    _same("delta_bias", delta_bias, (c,), _f32, dev)
    return c, s, g, strides


def selective_scan(x, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True, S0=None,
                   tables=None, out=None, workspace="auto", stream=None):
    """Selective state space scan of each channel with S states:
    dt = softplus(delta + delta_bias) (or without softplus), h_t = exp(dt_t A) h_{t-1} +
    dt_t x_t B_t, y_t = (C_t . h_t + D x_t) silu(z_t).

    Dense: x, delta, z [B,T,C], B and C [B,T,G,S] (float32 or bf16, rows may be slices
    of wider ones; G groups of channels share B and C), A [C,S], D and delta_bias [C]
    float32 (None: zero), z None: no gate, S0 [B,C,S] float32 or None (zeros).
    Packed (``tables`` from :func:`sequence_tables`, blocks of :func:`selective_block`):
    the same without the batch, rows [tokens, ..]; S0 and S_out are pools [P,C,S] of
    states by slot.  ``out`` may pass (y, S_out); S_out may be S0 (in place) or None
    (not wanted).  Without it S_out is new, and for a packed batch with S0 the pool S0
    itself, updated in place.  Rows of y behind the last sequence are left as they
    were.  Returns (y, S_out)."""
    lib = load()
    dt, dev = _dtype("x", x)
    lead, N, T, pk, pool = _batch(x, tables, (S0, out[1] if out is not None else None), 1, "x")
    c, s, g, strides = _scan_inputs(x, delta, A, B, C, D, z, delta_bias, lead)
    if out is None:
        y = _like(x, dt, dev, stream)
        if tables is not None and S0 is not None:
            S = S0
        elif tables is not None and tables.slots is not None:
            raise ValueError("kdn: a pool for the tables' slots must be given (S0 or out)")
        else:
            S = _new((pool, c, s), _f32, dev, stream)
    else:
        y, S = out
    _same("S0", S0, (pool, c, s), _f32, dev)
    _same("y", y, lead + (c,), dt, dev)
    _same("S_out", S, (pool, c, s), _f32, dev)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"kdn: workspace must be 'auto', None or a tensor, not {workspace!r}")
        workspace = _scan_workspace(DTYPES[dt], N, T, c, s, g, pk, dev, stream)
    nws = 0
    if workspace is not None:
        nws = workspace.numel()
        _same("workspace", workspace, (nws,), torch.uint8, dev)
    _call(lib.kdn_selective_scan, dev, stream, DTYPES[dt], N, T, c, s, g, int(bool(softplus)),
          *strides, _p(x), _p(delta), _p(A), _p(B), _p(C), _p(D), _p(z), _p(delta_bias), _p(S0),
          _p(y), _p(S), pk, _p(workspace), nws)
    return y, S


def _scan_workspace(dtype, N, T, C, S, G, pk, dev, stream):
    st = ctypes.c_int(0)
    n = load().kdn_selective_scan_workspace_size(dtype, N, T, C, S, G, pk, ctypes.byref(st))
    _check(_lib, st.value)
    return _new((n,), torch.uint8, dev, stream) if n else None


def selective_decode(x, delta, A, B, C, S, D=None, z=None, delta_bias=None, softplus=True,
                     slots=None, y=None, stream=None):
    """One token of :func:`selective_scan` for N rows: x, delta, z [N,C], B, C [N,G,S].
    S [P,C,S] float32 is a pool of states, updated in place; ``slots`` [N] int32 is each
    row's state (None: row n).  A row whose slot is not in the pool is skipped, its y
    left as it was (zero in a new y).  Returns y [N,C]."""
    lib = load()
    dt, dev = _dtype("x", x)
    if x.dim() != 2:
        raise ValueError(f"kdn: x has shape {tuple(x.shape)}, expected [N, C]")
    N = _int32("N", x.shape[0])
    c, s, g, strides = _scan_inputs(x, delta, A, B, C, D, z, delta_bias, (N,))
    if not isinstance(S, torch.Tensor) or S.dim() != 3:
        raise ValueError("kdn: S must be a tensor [P, C, S]")
    pool = _int32("pool", S.shape[0])
    if y is None:
        y = _new((N, c), dt, dev, stream, zero=slots is not None)
    _same("S", S, (pool, c, s), _f32, dev)
    _same("y", y, (N, c), dt, dev)
    _same("slots", slots, (N,), torch.int32, dev)
    _call(lib.kdn_selective_decode, dev, stream, DTYPES[dt], N, c, s, g, int(bool(softplus)),
          *strides, _p(x), _p(delta), _p(A), _p(B), _p(C), _p(D), _p(z), _p(delta_bias), _p(slots),
          pool, _p(S), _p(y))
    return y


def selective_scan_backward(x, delta, A, B, C, d_y, D=None, z=None, delta_bias=None, softplus=True,
                            S0=None, dS_out=None, tables=None, out=None, workspace=None,
                            stream=None):
    """Gradients of :func:`selective_scan` for the cotangents d_y (shaped as y) and dS_out
    (shaped as S_out; None: zero).  Returns a dict of dx, ddelta, dz (None without z), dB,
    dC in x's dtype and dA, dD, ddelta_bias (None where their parameter is), dS0 float32.
    Rows behind the last sequence of a packed batch get zero, and so do states of dS0
    without a sequence.  ``out`` may pass such a dict (dD, ddelta_bias and dS0 may be None:
    not wanted; in a given dS0 states without a sequence are left as they were).  A packed
    batch without any of S0, dS_out and out["dS0"] has no pool: dS0 is by sequence and
    slots are not looked at."""
    lib = load()
    dt, dev = _dtype("x", x)
    lead, N, T, pk, pool = _batch(x, tables, (S0, dS_out, (out or {}).get("dS0")), 1, "x")
    c, s, g, strides = _scan_inputs(x, delta, A, B, C, D, z, delta_bias, lead)
    out = _outputs(out, (("dx", x, dt, True), ("ddelta", x, dt, True),
                         ("dz", x, dt, z is not None), ("dB", B, dt, True), ("dC", B, dt, True),
                         ("dA", A, _f32, True),
                         ("dD", (c,), _f32, D is not None),
                         ("ddelta_bias", (c,), _f32, delta_bias is not None),
                         ("dS0", (pool, c, s), _f32, True if tables is None else "zero")),
                   dev, stream)
    _same("d_y", d_y, lead + (c,), dt, dev)
    _same("S0", S0, (pool, c, s), _f32, dev)
    _same("dS_out", dS_out, (pool, c, s), _f32, dev)
    st = ctypes.c_int(0)
    n = lib.kdn_selective_scan_backward_workspace_size(DTYPES[dt], N, T, c, s, g, pk, ctypes.byref(st))
    _check(lib, st.value)
    workspace, n = _workspace(n, workspace, dev, stream)
    _call(lib.kdn_selective_scan_backward, dev, stream, DTYPES[dt], N, T, c, s, g,
          int(bool(softplus)), *strides, _p(x), _p(delta), _p(A), _p(B), _p(C), _p(D), _p(z),
          _p(delta_bias), _p(S0), _p(d_y), _p(dS_out), _p(out["dx"]), _p(out["ddelta"]),
          _p(out["dA"]), _p(out["dB"]), _p(out["dC"]), _p(out["dD"]), _p(out["dz"]),
          _p(out["ddelta_bias"]), _p(out["dS0"]), pk, _p(workspace), n)
    return out


def _heads(x, weight, gate, order, activation):
    """Sizes and codes of a gated norm."""
    dt, dev = _dtype("x", x)
    if x.dim() < 2:
        raise ValueError(f"kdn: x has shape {tuple(x.shape)}, expected [.., H, d]")
    if order not in NORM_ORDERS:
        raise ValueError(f"kdn: order must be one of {tuple(NORM_ORDERS)}, not {order!r}")
    act = _activation(activation, (None, "silu", "sigmoid"))
    shape = x.shape
    lead, H, d = shape[:-2], shape[-2], shape[-1]
    if not isinstance(weight, torch.Tensor) or weight.dim() not in (1, 2):
        raise ValueError("kdn: weight must be a tensor [d] or [H, d]")
    per_head = weight.dim() == 2
    _same("weight", weight, (H, d) if per_head else (d,), _f32, dev)
    tokens = math.prod(lead)
    xs = 0 if x.is_contiguous() else _strided("x", x, lead, (H, d), dt, dev)
    zs = 0
    if gate is not None and not (isinstance(gate, torch.Tensor) and gate.shape == shape and
                                 gate.dtype is dt and gate.get_device() == dev.index and
                                 gate.is_contiguous()):
        zs = _strided("gate", gate, lead, (H, d), dt, dev)
    return (dt, dev, _int32("tokens", tokens), _int32("H", H), _int32("d", d), NORM_ORDERS[order],
            act, int(per_head), xs, zs)


def gated_norm(x, weight, gate=None, eps=1e-5, order="norm_gate", activation="silu", out=None,
               stream=None):
    """RMS norm of each head's d values with its gate, r(u) = (mean(u^2) + eps)^-1/2:
    order "norm_gate": y = x r(x) weight act(gate); "gate_norm": u = x act(gate),
    y = u r(u) weight.  x and gate [..,H,d] (float32 or bf16; rows [H,d] may be
    slices of wider ones), weight [d] float32 for all heads or [H,d]; activation
    "silu", "sigmoid" or None; gate None: no gate.  Returns y [..,H,d] (``out`` if
    given)."""
    lib = load()
    dt, dev, tokens, H, d, order, act, per_head, xs, zs = _heads(x, weight, gate, order, activation)
    if out is None:
        out = _like(x, dt, dev, stream)
    else:
        _same("out", out, x.shape, dt, dev)
    _call(lib.kdn_gated_norm, dev, stream, DTYPES[dt], tokens, H, d, order, act, per_head,
          float(eps), xs, zs, _p(x), _p(weight), _p(gate), _p(out))
    return out


def gated_norm_backward(x, weight, d_y, gate=None, eps=1e-5, order="norm_gate", activation="silu",
                        out=None, workspace=None, stream=None):
    """Gradients of :func:`gated_norm` for d_y [..,H,d]: a dict of dx and dgate (None
    without a gate) in x's dtype and dweight float32, or ``out``, such a dict."""
    lib = load()
    dt, dev, tokens, H, d, order, act, per_head, xs, zs = _heads(x, weight, gate, order, activation)
    out = _outputs(out, (("dx", x, dt, True), ("dgate", x, dt, gate is not None),
                         ("dweight", weight, _f32, True)), dev, stream)
    _same("d_y", d_y, x.shape, dt, dev)
    st = ctypes.c_int(0)
    n = lib.kdn_gated_norm_backward_workspace_size(tokens, H, d, per_head, ctypes.byref(st))
    _check(lib, st.value)
    workspace, n = _workspace(n, workspace, dev, stream)
    _call(lib.kdn_gated_norm_backward, dev, stream, DTYPES[dt], tokens, H, d, order, act, per_head,
          float(eps), xs, zs, _p(x), _p(weight), _p(gate), _p(d_y), _p(out["dx"]),
          _p(out["dgate"]), _p(out["dweight"]), _p(workspace), n)
    return out


def _residual(x, residual, weight, scale):
    """Sizes and checks common to the residual norm and its gradients; x may be None
    (the stream's type then stands for it)."""
    sdt, dev = _dtype("residual", residual)
    dt = sdt if x is None else _dtype("x", x)[0]
    if residual.dim() < 1:
        raise ValueError("kdn: residual must be a tensor [.., D]")
    lead, D = residual.shape[:-1], residual.shape[-1]
    tokens = math.prod(lead)
    rs = 0 if residual.is_contiguous() else _strided("residual", residual, lead, (D,), sdt, dev)
    xs = 0
    if x is not None and not (x.shape == residual.shape and x.get_device() == dev.index and
                              x.is_contiguous()):
        xs = _strided("x", x, lead, (D,), dt, dev)
    _same("weight", weight, (D,), _f32, dev)
    if weight is None:
        raise TypeError("kdn: weight must be a tensor [D]")
    scale_n = 0
    if scale is not None:
        if not isinstance(scale, torch.Tensor):
            raise TypeError("kdn: scale must be a tensor [1] or [D] or None")
        scale_n = 1 if scale.shape == (1,) else D
        _same("scale", scale, (scale_n,), _f32, dev)
    return dt, sdt, dev, _int32("tokens", tokens), _int32("D", D), scale_n, xs, rs


def residual_norm(x, residual, weight, scale=None, eps=1e-5, out=None, stream=None):
    """The residual stream and the RMS norm before the next block:
    h = residual + scale x, y = h (mean(h^2) + eps)^-1/2 weight.  x [..,D] (float32
    or bf16), residual [..,D] in x's dtype or float32, weight [D] float32, scale [1]
    or [D] float32 (None: one); rows of x and residual may be slices of wider ones.
    ``out`` may pass (y, h); h may be a contiguous residual itself (in place).
    Returns (y, h): y in x's dtype, h in the residual's."""
    lib = load()
    dt, sdt, dev, tokens, D, scale_n, xs, rs = _residual(x, residual, weight, scale)
    if x is None:
        raise TypeError("kdn: x must be a tensor")
    if out is None:
        y, h = _like(x, dt, dev, stream), _like(residual, sdt, dev, stream)
    else:
        y, h = out
        for name, t, kind in (("y", y, dt), ("h", h, sdt)):
            if t is None:
                raise TypeError(f"kdn: {name} must be a tensor")
            _same(name, t, x.shape, kind, dev)
    _call(lib.kdn_residual_norm, dev, stream, DTYPES[dt], DTYPES[sdt], tokens, D, scale_n,
          float(eps), xs, rs, _p(x), _p(residual), _p(weight), _p(scale), _p(y), _p(h))
    return y, h


def residual_norm_backward(x, h, weight, d_y, d_h=None, scale=None, eps=1e-5, out=None,
                           workspace=None, stream=None):
    """Gradients of :func:`residual_norm` from h, its second output, for d_y (x's
    dtype) and d_h (h's dtype; None: zero): a dict of dx (x's dtype), dresidual (h's),
    dweight and dscale (float32; None without a scale), or ``out``, such a dict (dx
    and dscale may be None: not wanted).  x may be None where dscale is not wanted."""
    lib = load()
    dt, sdt, dev, tokens, D, scale_n, xs, rs = _residual(x, h, weight, scale)
    if not isinstance(d_y, torch.Tensor):
        raise TypeError("kdn: d_y must be a tensor")
    if x is None:
        dt, _ = _dtype("d_y", d_y)
    _same("d_y", d_y, h.shape, dt, dev)
    out = _outputs(out, (("dx", h if dt is sdt else d_y, dt, True), ("dresidual", h, sdt, True),
                         ("dweight", weight, _f32, True),
                         ("dscale", (scale_n,), _f32, scale is not None and x is not None)),
                   dev, stream)
    _same("d_h", d_h, h.shape, sdt, dev)
    st = ctypes.c_int(0)
    n = lib.kdn_residual_norm_backward_workspace_size(tokens, D, scale_n, ctypes.byref(st))
    _check(lib, st.value)
    workspace, n = _workspace(n, workspace, dev, stream)
    _call(lib.kdn_residual_norm_backward, dev, stream, DTYPES[dt], DTYPES[sdt], tokens, D, scale_n,
          float(eps), xs, rs, _p(x), _p(h), _p(weight), _p(scale), _p(d_y), _p(d_h),
          _p(out["dx"]), _p(out["dresidual"]), _p(out["dweight"]), _p(out["dscale"]),
          _p(workspace), n)
    return out
