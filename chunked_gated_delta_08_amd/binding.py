"""Thin ctypes binding of libgdr.so (include/gdr.h) over torch tensors.

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity (ValueError / TypeError before anything reaches the library),
output tensors and the workspace are allocated with torch, and the pointers and
the current HIP stream are handed to the C ABI.  Every step of the
computation runs in the library's gfx950 kernels; if the library is missing the
import fails (there is no fallback).

Layouts (token axis flattened over the batch, as in include/gdr.h):
  q, k [B*T, HK, K]   v, dO [B*T, HV, V]   beta [B*T, HV]   g_cum [B*T, HV] fp32
  h0, dht, dh0 [N, HV, K, V] fp32
"""
import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdr.so")

GDR_F32, GDR_F16, GDR_BF16 = 0, 1, 2
_DT = {torch.float32: GDR_F32, torch.float16: GDR_F16, torch.bfloat16: GDR_BF16}
STATUS = {0: "GDR_OK", -1: "GDR_ERR_INVALID", -2: "GDR_ERR_UNSUPPORTED", -3: "GDR_ERR_WORKSPACE", -4: "GDR_ERR_LAUNCH",
          -5: "GDR_ERR_SCRATCH"}
NOALLOC_SCRATCH_BYTES = 128 << 20   # GDR_NOALLOC_SCRATCH_BYTES


class GdrError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


class Problem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("HK", ctypes.c_int), ("HV", ctypes.c_int),
                ("K", ctypes.c_int), ("V", ctypes.c_int), ("BT", ctypes.c_int), ("N", ctypes.c_int),
                ("cu_seqlens", ctypes.c_void_p), ("cu_seqlens_host", ctypes.c_void_p),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int), ("seg_chunks", ctypes.c_int)]


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run chunked_gated_delta_08_amd/build.py (hipcc, gfx950)")
lib = ctypes.CDLL(LIB_PATH)
_vp, _sz = ctypes.c_void_p, ctypes.c_size_t
lib.gdr_strerror.restype = ctypes.c_char_p
lib.gdr_strerror.argtypes = [ctypes.c_int]
lib.gdr_num_chunks.restype = ctypes.c_int64
lib.gdr_num_chunks.argtypes = [ctypes.POINTER(Problem)]
lib.gdr_workspace_size.restype = _sz
lib.gdr_workspace_size.argtypes = [ctypes.POINTER(Problem)]
lib.gdr_fwd_states.restype = ctypes.c_int
lib.gdr_fwd_states.argtypes = [ctypes.POINTER(Problem)] + [_vp] * 8 + [_vp, _sz, _vp]
lib.gdr_chunk_bwd.restype = ctypes.c_int
lib.gdr_chunk_bwd.argtypes = [ctypes.POINTER(Problem)] + [_vp] * 14 + [_vp, _sz, _vp]
lib.gdr_chunk_bwd_events.restype = ctypes.c_int
lib.gdr_chunk_bwd_events.argtypes = [ctypes.POINTER(Problem)] + [_vp] * 14 + [_vp, _sz, _vp, _vp]
lib.gdr_gate_cumsum.restype = ctypes.c_int
lib.gdr_gate_cumsum.argtypes = [ctypes.POINTER(Problem), _vp, _vp, _vp]
lib.gdr_chunk_fwd.restype = ctypes.c_int
lib.gdr_chunk_fwd.argtypes = [ctypes.POINTER(Problem)] + [_vp] * 8 + [_vp, _sz, _vp]
lib.gdr_chunk_fwd_events.restype = ctypes.c_int
lib.gdr_chunk_fwd_events.argtypes = [ctypes.POINTER(Problem)] + [_vp] * 8 + [_vp, _sz, _vp, _vp]
lib.kda_workspace_size.restype = _sz
lib.kda_workspace_size.argtypes = [ctypes.POINTER(Problem)]
lib.kda_chunk_bwd_full.restype = ctypes.c_int
lib.kda_chunk_bwd_full.argtypes = [ctypes.POINTER(Problem)] + [_vp] * 14 + [_vp, _sz, _vp]
lib.kda_chunk_bwd_full_events.restype = ctypes.c_int
lib.kda_chunk_bwd_full_events.argtypes = [ctypes.POINTER(Problem)] + [_vp] * 14 + [_vp, _sz, _vp, _vp]
lib.kda_chunk_bwd.restype = ctypes.c_int
lib.kda_chunk_bwd.argtypes = [ctypes.POINTER(Problem)] + [_vp] * 17 + [_vp]
lib.gdr_noalloc_init.restype = ctypes.c_int
lib.gdr_noalloc_init.argtypes = []
lib.gdr_chunk_bwd_noalloc.restype = ctypes.c_int
lib.gdr_chunk_bwd_noalloc.argtypes = [ctypes.POINTER(Problem)] + [_vp] * 14 + [_vp]




class BigdnProblem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("F", ctypes.c_int), ("S", ctypes.c_int), ("H", ctypes.c_int),
                ("D", ctypes.c_int), ("k_scale", ctypes.c_float), ("norm_eps", ctypes.c_float),
                ("eps", ctypes.c_float)]


lib.bigdn_workspace_size.restype = _sz
lib.bigdn_workspace_size.argtypes = [ctypes.POINTER(BigdnProblem), ctypes.c_int]
lib.bigdn_fwd.restype = ctypes.c_int
lib.bigdn_fwd.argtypes = [ctypes.POINTER(BigdnProblem)] + [_vp] * 8 + [_vp, _sz, _vp]
lib.bigdn_fwd_events.restype = ctypes.c_int
lib.bigdn_fwd_events.argtypes = [ctypes.POINTER(BigdnProblem)] + [_vp] * 8 + [_vp, _sz, _vp, _vp]
lib.bigdn_bwd.restype = ctypes.c_int
lib.bigdn_bwd.argtypes = [ctypes.POINTER(BigdnProblem)] + [_vp] * 13 + [_vp, _sz, _vp]
lib.bigdn_bwd_events.restype = ctypes.c_int
lib.bigdn_bwd_events.argtypes = [ctypes.POINTER(BigdnProblem)] + [_vp] * 13 + [_vp, _sz, _vp, _vp]

EXPORTED = ["gdr_strerror", "gdr_num_chunks", "gdr_workspace_size", "gdr_fwd_states", "gdr_gate_cumsum",
            "gdr_chunk_fwd", "gdr_chunk_fwd_events", "gdr_chunk_bwd", "gdr_chunk_bwd_events", "kda_chunk_bwd",
            "kda_workspace_size", "kda_chunk_bwd_full", "kda_chunk_bwd_full_events", "bigdn_workspace_size",
            "bigdn_fwd", "bigdn_fwd_events", "bigdn_bwd", "bigdn_bwd_events", "gdr_noalloc_init",
            "gdr_chunk_bwd_noalloc"]


# ---------------------------------------------------------------- validation
_FLOATS = (torch.float32, torch.float16, torch.bfloat16)


def _need(t, name, dtype=None, shape=None, cuda=True, optional=False):
    """Raises unless `t` is a contiguous tensor of the given dtype and shape
    (on the GPU when `cuda`).  None passes only when `optional`."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _nseq(cu_seqlens, B, cuda):
    if cu_seqlens is None:
        return B
    _need(cu_seqlens, "cu_seqlens", torch.int32, cuda=cuda)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be 1-D with at least two entries")
    return cu_seqlens.numel() - 1


def check_gdr_args(q, k, v, g_cum, beta, dO=None, dht=None, h0=None, cu_seqlens=None, B=1, need_q=True,
                   need_dO=False, cuda=True):
    """Shapes and dtypes of the GDN entry points (include/gdr.h): q, k [B*T,HK,K];
    v, dO [B*T,HV,V]; beta [B*T,HV] (all one dtype); g_cum [B*T,HV] fp32;
    h0, dht [N,HV,K,V] fp32.  Returns (N, HK, HV, K, V)."""
    _need(k, "k", cuda=cuda)
    _need(v, "v", cuda=cuda)
    if k.dim() != 3 or v.dim() != 3:
        raise ValueError("k must be [B*T, HK, K] and v [B*T, HV, V]")
    if v.dtype not in _FLOATS:
        raise TypeError(f"v has dtype {v.dtype}; expected one of {_FLOATS}")
    ntok, HK, K = k.shape
    _, HV, V = v.shape
    dt = v.dtype
    _need(k, "k", dt, cuda=cuda)
    _need(v, "v", dt, (ntok, HV, V), cuda=cuda)
    if need_q:
        _need(q, "q", dt, (ntok, HK, K), cuda=cuda)
    _need(beta, "beta", dt, (ntok, HV), cuda=cuda)
    _need(g_cum, "g_cum", torch.float32, (ntok, HV), cuda=cuda)
    if need_dO:
        _need(dO, "dO", dt, (ntok, HV, V), cuda=cuda)
    if HK < 1 or HV % HK != 0:
        raise ValueError(f"HV ({HV}) must be a multiple of HK ({HK})")
    if cu_seqlens is None and ntok % B != 0:
        raise ValueError(f"the token count {ntok} is not a multiple of B = {B}")
    N = _nseq(cu_seqlens, B, cuda)
    _need(h0, "h0", torch.float32, (N, HV, K, V), cuda=cuda, optional=True)
    _need(dht, "dht", torch.float32, (N, HV, K, V), cuda=cuda, optional=True)
    return N, HK, HV, K, V


def check_kda_stage_args(q, k, v, v_new, g, beta, A, h, dO, dh, dv, BT=64, NT=None, cuda=True):
    """Shapes and dtypes of kda_chunk_bwd: q, k [ntok,H,K]; v, v_new, dO, dv
    [ntok,H,V]; beta [ntok,H]; A [ntok,H,BT] (one dtype); g [ntok,H,K] fp32;
    h, dh [NT,H,K,V] fp32 (NT given, or taken from h)."""
    _need(k, "k", cuda=cuda)
    _need(v, "v", cuda=cuda)
    if k.dim() != 3 or v.dim() != 3:
        raise ValueError("k must be [ntok, H, K] and v [ntok, H, V]")
    ntok, H, K = k.shape
    V = v.shape[-1]
    dt = k.dtype
    if dt not in _FLOATS:
        raise TypeError(f"k has dtype {dt}")
    for t, n in ((q, "q"), (k, "k")):
        _need(t, n, dt, (ntok, H, K), cuda=cuda)
    for t, n in ((v, "v"), (v_new, "v_new"), (dO, "dO"), (dv, "dv")):
        _need(t, n, dt, (ntok, H, V), cuda=cuda)
    _need(beta, "beta", dt, (ntok, H), cuda=cuda)
    _need(A, "A", dt, (ntok, H, BT), cuda=cuda)
    _need(g, "g", torch.float32, (ntok, H, K), cuda=cuda)
    _need(h, "h", torch.float32, cuda=cuda)
    nt = h.shape[0] if NT is None else NT
    _need(h, "h", torch.float32, (nt, H, K, V), cuda=cuda)
    _need(dh, "dh", torch.float32, (nt, H, K, V), cuda=cuda)


def check_kda_full_args(q, k, v, g_cum, beta, dO, dht=None, h0=None, cu_seqlens=None, B=1, cuda=True):
    """Shapes and dtypes of kda_chunk_bwd_full: q, k [ntok,H,K]; v, dO [ntok,H,V];
    beta [ntok,H] (one dtype); g_cum [ntok,H,K] fp32; h0, dht [N,H,K,V] fp32."""
    _need(k, "k", cuda=cuda)
    _need(v, "v", cuda=cuda)
    if k.dim() != 3 or v.dim() != 3:
        raise ValueError("k must be [ntok, H, K] and v [ntok, H, V]")
    ntok, H, K = k.shape
    V = v.shape[-1]
    dt = k.dtype
    if dt not in _FLOATS:
        raise TypeError(f"k has dtype {dt}")
    _need(q, "q", dt, (ntok, H, K), cuda=cuda)
    _need(v, "v", dt, (ntok, H, V), cuda=cuda)
    _need(dO, "dO", dt, (ntok, H, V), cuda=cuda)
    _need(beta, "beta", dt, (ntok, H), cuda=cuda)
    _need(g_cum, "g_cum", torch.float32, (ntok, H, K), cuda=cuda)
    if cu_seqlens is None and ntok % B != 0:
        raise ValueError(f"the token count {ntok} is not a multiple of B = {B}")
    N = _nseq(cu_seqlens, B, cuda)
    _need(h0, "h0", torch.float32, (N, H, K, V), cuda=cuda, optional=True)
    _need(dht, "dht", torch.float32, (N, H, K, V), cuda=cuda, optional=True)
    return N


def _check(code):
    if code != 0:
        raise GdrError(code, lib.gdr_strerror(code).decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_problem(B, T, HK, HV, K, V, dtype, BT=64, cu_seqlens=None, scale=None, seg_chunks=0):
    """Builds the gdr_problem struct.  cu_seqlens: int32 CUDA tensor [N+1] or None.
    seg_chunks: chunks per scan segment (0 = automatic, < 0 = no segments).
    Returns (problem, keepalive) -- keep `keepalive` referenced while the struct is used."""
    p = Problem(B, T, HK, HV, K, V, BT, 0, None, None, float(scale or 0.0), _DT[dtype], int(seg_chunks))
    keep = []
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32)
        host = cu_seqlens.detach().to("cpu").contiguous()
        keep += [cu_seqlens, host]
        p.N = host.numel() - 1
        p.cu_seqlens = cu_seqlens.data_ptr()
        p.cu_seqlens_host = host.data_ptr()
    return p, keep


def num_chunks(p):
    return int(lib.gdr_num_chunks(ctypes.byref(p)))


def workspace_size(p):
    return int(lib.gdr_workspace_size(ctypes.byref(p)))


def _dims(q_or_k, v, cu_seqlens, B):
    ntok, HK, K = q_or_k.shape
    _, HV, V = v.shape
    if cu_seqlens is None:
        return B, ntok // B, HK, HV, K, V
    return 1, ntok, HK, HV, K, V


def gdr_chunk_bwd(q, k, v, g_cum, beta, dO, dht=None, h0=None, cu_seqlens=None, B=1, scale=None, BT=64,
                  want_dh0=True, out=None, workspace=None, stream=None, seg_chunks=0):
    """Backward of the chunkwise gated delta rule.  Returns dict dq, dk, dv, dg, dbeta, dh0."""
    check_gdr_args(q, k, v, g_cum, beta, dO, dht, h0, cu_seqlens, B, need_dO=True)
    B, T, HK, HV, K, V = _dims(k, v, cu_seqlens, B)
    p, keep = make_problem(B, T, HK, HV, K, V, v.dtype, BT, cu_seqlens, scale, seg_chunks)
    N = B if cu_seqlens is None else p.N
    dev = v.device
    if out is None:
        out = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
               "dg": torch.empty(g_cum.shape, dtype=torch.float32, device=dev),
               "dbeta": torch.empty(beta.shape, dtype=torch.float32, device=dev),
               "dh0": torch.empty((N, HV, K, V), dtype=torch.float32, device=dev) if want_dh0 else None}
    if workspace is None:
        workspace = torch.empty(max(workspace_size(p), 1), dtype=torch.uint8, device=dev)
    _check(lib.gdr_chunk_bwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g_cum), _ptr(beta), _ptr(h0),
                             _ptr(dO), _ptr(dht), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                             _ptr(out["dg"]), _ptr(out["dbeta"]), _ptr(out["dh0"]), _ptr(workspace),
                             workspace.numel(), _stream(stream)))
    del keep
    return out


def gdr_chunk_bwd_noalloc(q, k, v, g_cum, beta, dO, dht=None, h0=None, cu_seqlens=None, B=1, scale=None, BT=64,
                          want_dh0=True, out=None, stream=None, seg_chunks=0):
    """gdr_chunk_bwd through the entry point that takes no workspace (the
    library's fixed per-GPU scratch array).  `out` (dict of preallocated
    outputs) lets a caller that cannot allocate pass its own buffers."""
    check_gdr_args(q, k, v, g_cum, beta, dO, dht, h0, cu_seqlens, B, need_dO=True)
    B, T, HK, HV, K, V = _dims(k, v, cu_seqlens, B)
    p, keep = make_problem(B, T, HK, HV, K, V, v.dtype, BT, cu_seqlens, scale, seg_chunks)
    N = B if cu_seqlens is None else p.N
    dev = v.device
    if out is None:
        out = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
               "dg": torch.empty(g_cum.shape, dtype=torch.float32, device=dev),
               "dbeta": torch.empty(beta.shape, dtype=torch.float32, device=dev),
               "dh0": torch.empty((N, HV, K, V), dtype=torch.float32, device=dev) if want_dh0 else None}
    _check(lib.gdr_chunk_bwd_noalloc(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g_cum), _ptr(beta), _ptr(h0),
                                     _ptr(dO), _ptr(dht), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                                     _ptr(out["dg"]), _ptr(out["dbeta"]), _ptr(out["dh0"]), _stream(stream)))
    del keep
    return out


def gdr_gate_cumsum(g, cu_seqlens=None, B=1, BT=64, out=None, stream=None):
    """In-chunk cumulative sum of the raw gate g [B*T, HV] fp32 (restarting every BT
    tokens and at every sequence start).  Returns g_cum, same shape, fp32."""
    _need(g, "g", torch.float32)
    if g.dim() != 2:
        raise ValueError("g must be [B*T, HV]")
    ntok, HV = g.shape
    T = ntok // B if cu_seqlens is None else ntok
    if cu_seqlens is None and ntok % B != 0:
        raise ValueError(f"the token count {ntok} is not a multiple of B = {B}")
    _nseq(cu_seqlens, B, True)
    p, keep = make_problem(B if cu_seqlens is None else 1, T, 1, HV, 1, 1, torch.float32, BT, cu_seqlens)
    if out is None:
        out = torch.empty_like(g)
    _check(lib.gdr_gate_cumsum(ctypes.byref(p), _ptr(g), _ptr(out), _stream(stream)))
    del keep
    return out


def gdr_chunk_fwd(q, k, v, g_cum, beta, h0=None, cu_seqlens=None, B=1, scale=None, BT=64, want_ht=True,
                  out=None, workspace=None, stream=None, seg_chunks=0):
    """Chunked forward of the gated delta rule.  Returns dict o [B*T, HV, V] (input
    dtype) and ht [N, HV, K, V] fp32 (or None)."""
    check_gdr_args(q, k, v, g_cum, beta, h0=h0, cu_seqlens=cu_seqlens, B=B)
    B, T, HK, HV, K, V = _dims(k, v, cu_seqlens, B)
    p, keep = make_problem(B, T, HK, HV, K, V, v.dtype, BT, cu_seqlens, scale, seg_chunks)
    N = B if cu_seqlens is None else p.N
    dev = v.device
    if out is None:
        out = {"o": torch.empty_like(v),
               "ht": torch.empty((N, HV, K, V), dtype=torch.float32, device=dev) if want_ht else None}
    if workspace is None:
        workspace = torch.empty(max(workspace_size(p), 1), dtype=torch.uint8, device=dev)
    _check(lib.gdr_chunk_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g_cum), _ptr(beta), _ptr(h0),
                             _ptr(out["o"]), _ptr(out["ht"]), _ptr(workspace), workspace.numel(), _stream(stream)))
    del keep
    return out


def gdr_fwd_states(k, v, g_cum, beta, h0=None, cu_seqlens=None, B=1, BT=64, want_v_new=True, want_ht=True,
                   workspace=None, stream=None, seg_chunks=0):
    """Per-chunk forward states h [NT, HV, K, V] fp32 (state entering each chunk), v_new, ht."""
    check_gdr_args(None, k, v, g_cum, beta, h0=h0, cu_seqlens=cu_seqlens, B=B, need_q=False)
    B, T, HK, HV, K, V = _dims(k, v, cu_seqlens, B)
    p, keep = make_problem(B, T, HK, HV, K, V, v.dtype, BT, cu_seqlens, None, seg_chunks)
    N = B if cu_seqlens is None else p.N
    dev = v.device
    NT = num_chunks(p)
    h = torch.empty((max(NT, 0), HV, K, V), dtype=torch.float32, device=dev)
    vn = torch.empty_like(v) if want_v_new else None
    ht = torch.empty((N, HV, K, V), dtype=torch.float32, device=dev) if want_ht else None
    if workspace is None:
        workspace = torch.empty(max(workspace_size(p), 1), dtype=torch.uint8, device=dev)
    _check(lib.gdr_fwd_states(ctypes.byref(p), _ptr(k), _ptr(v), _ptr(g_cum), _ptr(beta), _ptr(h0), _ptr(h),
                              _ptr(vn), _ptr(ht), _ptr(workspace), workspace.numel(), _stream(stream)))
    del keep
    return {"h": h, "v_new": vn, "ht": ht}


def kda_chunk_bwd(q, k, v, v_new, g, beta, A, h, dO, dh, dv, scale=None, cu_seqlens=None, B=1, BT=64,
                  out=None, stream=None):
    """KDA WY backward stage.  Returns dict dq, dk, dv, db, dg, dA (the page's order)."""
    ntok, H, K = k.shape
    V = v.shape[-1]
    T = ntok // B if cu_seqlens is None else ntok
    if cu_seqlens is None and ntok % B != 0:
        raise ValueError(f"the token count {ntok} is not a multiple of B = {B}")
    _nseq(cu_seqlens, B, True)
    p, keep = make_problem(B if cu_seqlens is None else 1, T, H, H, K, V, v.dtype, BT, cu_seqlens, scale)
    check_kda_stage_args(q, k, v, v_new, g, beta, A, h, dO, dh, dv, BT=BT, NT=num_chunks(p))
    dev = v.device
    if out is None:
        out = {"dq": torch.empty((ntok, H, K), dtype=torch.float32, device=dev),
               "dk": torch.empty((ntok, H, K), dtype=torch.float32, device=dev),
               "dv": torch.empty_like(v),
               "db": torch.empty((ntok, H), dtype=torch.float32, device=dev),
               "dg": torch.empty((ntok, H, K), dtype=torch.float32, device=dev),
               "dA": torch.empty((ntok, H, BT), dtype=torch.float32, device=dev)}
    _check(lib.kda_chunk_bwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(v_new), _ptr(g), _ptr(beta), _ptr(A),
                             _ptr(h), _ptr(dO), _ptr(dh), _ptr(dv), _ptr(out["dq"]), _ptr(out["dk"]),
                             _ptr(out["dv"]), _ptr(out["db"]), _ptr(out["dg"]), _ptr(out["dA"]), _stream(stream)))
    del keep
    return out


def kda_chunk_bwd_full(q, k, v, g_cum, beta, dO, dht=None, h0=None, cu_seqlens=None, B=1, scale=None, BT=64,
                       want_dh0=True, out=None, workspace=None, stream=None):
    """Full chunked KDA backward (per-channel gate).  g_cum [B*T, H, K] fp32 in-chunk
    cumulative log-gate.  Returns dict dq, dk, dv (input dtype), dg [B*T,H,K],
    dbeta [B*T,H], dh0 [N,H,K,V] (fp32)."""
    check_kda_full_args(q, k, v, g_cum, beta, dO, dht, h0, cu_seqlens, B)
    ntok, H, K = k.shape
    V = v.shape[-1]
    T = ntok // B if cu_seqlens is None else ntok
    p, keep = make_problem(B if cu_seqlens is None else 1, T, H, H, K, V, v.dtype, BT, cu_seqlens, scale)
    N = B if cu_seqlens is None else p.N
    dev = v.device
    if out is None:
        out = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
               "dg": torch.empty(g_cum.shape, dtype=torch.float32, device=dev),
               "dbeta": torch.empty(beta.shape, dtype=torch.float32, device=dev),
               "dh0": torch.empty((N, H, K, V), dtype=torch.float32, device=dev) if want_dh0 else None}
    if workspace is None:
        workspace = torch.empty(max(int(lib.kda_workspace_size(ctypes.byref(p))), 1), dtype=torch.uint8, device=dev)
    _check(lib.kda_chunk_bwd_full(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g_cum), _ptr(beta), _ptr(h0),
                                  _ptr(dO), _ptr(dht), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                                  _ptr(out["dg"]), _ptr(out["dbeta"]), _ptr(out["dh0"]), _ptr(workspace),
                                  workspace.numel(), _stream(stream)))
    del keep
    return out


# --------------------------------------------------------------------------
# BiGDN layer (include/bigdn.h).  Layouts: qkv bf16 [B, N, 3, H, D] with
# N = F*S; beta fp32 [B, H, F, S]; decay fp32 [B, H, F]; norm weights fp32
# [H*D]; rope cos/sin fp32 [N, D]; out / dout bf16 [B, N, H, D].

def bigdn_problem(qkv, F, S, k_scale=1.0, norm_eps=1e-5, eps=1e-6):
    if qkv.dim() != 5 or qkv.shape[2] != 3 or qkv.shape[1] != F * S:
        raise ValueError(f"qkv must be [B, F*S, 3, H, D]; got {tuple(qkv.shape)} with F={F}, S={S}")
    B, N, three, H, D = qkv.shape
    return BigdnProblem(B, F, S, H, D, float(k_scale), float(norm_eps), float(eps))


def _bigdn_inputs(qkv, beta, decay, qw, kw, cos, sin, F, S):
    _need(qkv, "qkv", torch.bfloat16)
    if qkv.dim() != 5 or qkv.shape[2] != 3 or qkv.shape[1] != F * S:
        raise ValueError(f"qkv must be [B, F*S, 3, H, D]; got {tuple(qkv.shape)} with F={F}, S={S}")
    B, N, _, H, D = qkv.shape
    for t, n, shape in ((beta, "beta", (B, H, F, S)), (decay, "decay", (B, H, F)), (qw, "qw", (H * D,)),
                        (kw, "kw", (H * D,)), (cos, "cos", (N, D)), (sin, "sin", (N, D))):
        _need(t, n, torch.float32, shape)


def bigdn_workspace_size(p, bwd):
    return int(lib.bigdn_workspace_size(ctypes.byref(p), 1 if bwd else 0))


def bigdn_fwd(qkv, beta, decay, qw, kw, cos, sin, F, S, k_scale=1.0, norm_eps=1e-5, eps=1e-6, out=None,
              workspace=None, stream=None, events=None):
    """BiGDN layer output bf16 [B, N, H, D]."""
    _bigdn_inputs(qkv, beta, decay, qw, kw, cos, sin, F, S)
    p = bigdn_problem(qkv, F, S, k_scale, norm_eps, eps)
    B, N, _, H, D = qkv.shape
    if out is None:
        out = torch.empty((B, N, H, D), dtype=torch.bfloat16, device=qkv.device)
    if workspace is None:
        workspace = torch.empty(max(bigdn_workspace_size(p, False), 1), dtype=torch.uint8, device=qkv.device)
    args = [ctypes.byref(p), _ptr(qkv), _ptr(beta), _ptr(decay), _ptr(qw), _ptr(kw), _ptr(cos), _ptr(sin),
            _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)]
    if events is None:
        _check(lib.bigdn_fwd(*args))
    else:
        _check(lib.bigdn_fwd_events(*args, events))
    return out


def bigdn_bwd(qkv, beta, decay, qw, kw, cos, sin, dout, F, S, k_scale=1.0, norm_eps=1e-5, eps=1e-6, out=None,
              workspace=None, stream=None, events=None):
    """BiGDN layer backward.  Returns dict dqkv (bf16, qkv's shape), dbeta, ddecay,
    dqw, dkw (fp32)."""
    _bigdn_inputs(qkv, beta, decay, qw, kw, cos, sin, F, S)
    B, N, _, H, D = qkv.shape
    _need(dout, "dout", torch.bfloat16, (B, N, H, D))
    p = bigdn_problem(qkv, F, S, k_scale, norm_eps, eps)
    dev = qkv.device
    if out is None:
        out = {"dqkv": torch.empty_like(qkv), "dbeta": torch.empty_like(beta), "ddecay": torch.empty_like(decay),
               "dqw": torch.empty_like(qw), "dkw": torch.empty_like(kw)}
    if workspace is None:
        workspace = torch.empty(max(bigdn_workspace_size(p, True), 1), dtype=torch.uint8, device=dev)
    args = [ctypes.byref(p), _ptr(qkv), _ptr(beta), _ptr(decay), _ptr(qw), _ptr(kw), _ptr(cos), _ptr(sin),
            _ptr(dout), _ptr(out["dqkv"]), _ptr(out["dbeta"]), _ptr(out["ddecay"]), _ptr(out["dqw"]),
            _ptr(out["dkw"]), _ptr(workspace), workspace.numel(), _stream(stream)]
    if events is None:
        _check(lib.bigdn_bwd(*args))
    else:
        _check(lib.bigdn_bwd_events(*args, events))
    return out


# --------------------------------------------------------------------------
# Layer operators (include/gdn_layer.h): gated RMSNorm, residual add with
# RMSNorm, dropout, gated linear recurrence, single-token steps.  Every tensor of a call
# is on one device, which need not be the current one; `stream` (default: that
# device's current stream) belongs to it; where a call allocates its outputs or
# workspace, that stream first waits for the current one, whose memory they may
# reuse (give `out` and `workspace` to overlap the two).  Preallocated outputs are checked like
# inputs; which of them may be an input's own buffer is said in the header.  In `out` an output
# that a call may skip (the header's NULL) is None or not there.

class NormProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("D", ctypes.c_int), ("eps", ctypes.c_float), ("dtype", ctypes.c_int),
                ("res_dtype", ctypes.c_int), ("act", ctypes.c_int)]


class GlrProblem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("D", ctypes.c_int), ("N", ctypes.c_int),
                ("cu_seqlens", ctypes.c_void_p), ("cu_seqlens_host", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("polls", ctypes.c_int)]


class Dropout(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64), ("rng", ctypes.c_void_p)]


GLR_TILE = 16
ACTS = {"silu": 0, "sigmoid": 1}
EXPORTED_LAYER = ["norm_workspace_size", "gated_norm_fwd", "gated_norm_bwd", "add_norm_fwd", "add_norm_bwd",
                  "gdn_dropout_fwd", "dropout_add_norm_fwd", "dropout_add_norm_bwd", "glr_num_states",
                  "glr_workspace_size", "glr_fwd", "glr_bwd", "glr_step", "gdr_step"]
_i, _i64, _f = ctypes.c_int, ctypes.c_int64, ctypes.c_float
_np, _gp = ctypes.POINTER(NormProblem), ctypes.POINTER(GlrProblem)
lib.norm_workspace_size.restype = _sz
lib.norm_workspace_size.argtypes = [_np]
lib.gated_norm_fwd.argtypes = [_np] + [_vp] * 5
lib.gated_norm_bwd.argtypes = [_np] + [_vp] * 8 + [_sz, _vp]
lib.add_norm_fwd.argtypes = [_np] + [_vp] * 7
lib.add_norm_bwd.argtypes = [_np] + [_vp] * 11 + [_sz, _vp]
_dp = ctypes.POINTER(Dropout)
lib.gdn_dropout_fwd.argtypes = [_i64, _i64, _i, _dp] + [_vp] * 3
lib.dropout_add_norm_fwd.argtypes = [_np, _dp] + [_vp] * 7
lib.dropout_add_norm_bwd.argtypes = [_np, _dp] + [_vp] * 11 + [_sz, _vp]
lib.glr_num_states.restype = _i64
lib.glr_num_states.argtypes = [_gp]
lib.glr_workspace_size.restype = _sz
lib.glr_workspace_size.argtypes = [_gp]
lib.glr_fwd.argtypes = [_gp] + [_vp] * 7 + [_sz, _vp]
lib.glr_bwd.argtypes = [_gp] + [_vp] * 10 + [_sz, _vp]
lib.glr_step.argtypes = [_i, _i, _i64, _i] + [_vp] * 6
lib.gdr_step.argtypes = [_i] * 5 + [_i64, _f, _i] + [_vp] * 9


def _same_device(first, *others):
    dev = first.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on {first.device} and {t.device}: one device is needed")


# the current device and its current stream's handle, without the checks and the
# Stream object around them where torch offers that (a GPU tensor is at hand, so
# torch has been initialised)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(dev, stream, temps, call, *args):
    """call(*args, stream handle) with `dev` current.  `temps`: tensors allocated for this
    call on the current stream.  Another one that uses them waits for the current stream,
    which may still work on that memory, and the allocator is told of it."""
    index = dev.index
    handle = _current_stream(index)
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
        if stream.cuda_stream != handle:
            temps = [t for t in temps if t is not None]
            if temps:
                stream.wait_stream(torch.cuda.current_stream(dev))
            for t in temps:
                t.record_stream(stream)
        handle = stream.cuda_stream
    if _current_device() == index:
        code = call(*args, handle)
    else:
        with torch.cuda.device(dev):
            code = call(*args, handle)
    if code != 0:
        _check(code)


def _p(t):
    return None if t is None else t.data_ptr()


def check_gated_norm_args(x, z, w, dy=None, act="silu", need_dy=False, cuda=True):
    """x, z (None: no gate), dy [..., D] of one dtype; w [D] fp32."""
    _need(x, "x", cuda=cuda)
    if x.dtype not in _DT:
        raise TypeError(f"x has dtype {x.dtype}; expected one of {_FLOATS}")
    if x.dim() < 1:
        raise ValueError("x must be [..., D]")
    if act not in ACTS:
        raise ValueError(f"act is {act!r}; expected one of {sorted(ACTS)}")
    _need(z, "z", x.dtype, x.shape, cuda=cuda, optional=True)
    _need(w, "w", torch.float32, x.shape[-1:], cuda=cuda)
    if need_dy:
        _need(dy, "dy", x.dtype, x.shape, cuda=cuda)
    _same_device(x, z, w, dy)


@functools.lru_cache(maxsize=1024)
def _norm_sizes(rows, D, eps, dtype, res_dtype, act):
    """The struct of these sizes (calls only read it) and the workspace it needs."""
    p = NormProblem(rows, D, eps, _DT[dtype], _DT[res_dtype], ACTS[act])
    return p, int(lib.norm_workspace_size(ctypes.byref(p)))


def _norm_problem(x, eps, res_dtype=None, act="silu"):
    D = x.shape[-1]
    return _norm_sizes(x.numel() // D if D else 0, D, eps, x.dtype, res_dtype or x.dtype, act)


def norm_workspace_size(rows, D, dtype):
    """Bytes of workspace gated_norm_bwd and add_norm_bwd need."""
    return _norm_sizes(rows, D, 0.0, dtype, dtype, "silu")[1]


def _workspace(workspace, size, like):
    """(the workspace, its bytes, the tensor allocated for it or None), on the device of
    the tensor `like`; no workspace for a size of 0."""
    if workspace is None:
        ws = like.new_empty(-(-size // like.element_size())) if size else None
        return ws, size, ws
    _need(workspace, "workspace", torch.uint8)
    _same_device(like, workspace)
    return workspace, workspace.numel(), None


def gated_norm_fwd(x, z, w, eps=1e-5, act="silu", out=None, stream=None):
    """y = x rsqrt(mean(x^2) + eps) w act(z) over the last axis; z None: no gate."""
    check_gated_norm_args(x, z, w, act=act)
    if out is None:
        y = torch.empty_like(x)
    else:
        y = out
        _need(y, "out", x.dtype, x.shape)
        _same_device(x, y)
    p, _ = _norm_problem(x, eps, act=act)
    _launch(x.device, stream, (y,) if out is None else (), lib.gated_norm_fwd, p, _p(x), _p(z), _p(w), _p(y))
    return y


def gated_norm_bwd(x, z, w, dy, eps=1e-5, act="silu", out=None, workspace=None, stream=None):
    """Gradients of gated_norm_fwd.  Returns dict dx, dz (None without z), dw (fp32)."""
    check_gated_norm_args(x, z, w, dy, act=act, need_dy=True)
    own = []
    if out is None:
        out = {"dx": torch.empty_like(x), "dz": None if z is None else torch.empty_like(z), "dw": torch.empty_like(w)}
        own += out.values()
    else:
        _need(out.get("dx"), "dx", x.dtype, x.shape)
        _need(out.get("dw"), "dw", torch.float32, w.shape)
        _need(out.get("dz"), "dz", x.dtype, x.shape, optional=z is None)
        _same_device(x, *out.values())
    dz = None if z is None else out["dz"]
    p, size = _norm_problem(x, eps, act=act)
    ws, size, mine = _workspace(workspace, size, w)
    own.append(mine)
    _launch(x.device, stream, own, lib.gated_norm_bwd, p, _p(x), _p(z), _p(w), _p(dy), _p(out["dx"]), _p(dz),
            _p(out["dw"]), _p(ws), size)
    return out


def check_add_norm_args(x, res, w, scale=None, cuda=True):
    """x [..., D]; res of x's shape, in x's dtype or fp32; w, scale (None: 1) [D] fp32."""
    _need(x, "x", cuda=cuda)
    if x.dtype not in _DT:
        raise TypeError(f"x has dtype {x.dtype}; expected one of {_FLOATS}")
    if x.dim() < 1:
        raise ValueError("x must be [..., D]")
    _need(res, "res", shape=x.shape, cuda=cuda)
    if res.dtype not in (x.dtype, torch.float32):
        raise TypeError(f"res has dtype {res.dtype}, expected {x.dtype} or torch.float32")
    _need(w, "w", torch.float32, x.shape[-1:], cuda=cuda)
    _need(scale, "scale", torch.float32, x.shape[-1:], cuda=cuda, optional=True)
    _same_device(x, res, w, scale)


def check_dropout_args(x, p, rng, cuda=True):
    """0 <= p <= 1; rng: (seed, offset), whole numbers taken modulo 2^64, or an int64 tensor [2] on x's device."""
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p is {p}; expected a probability")
    if isinstance(rng, torch.Tensor):
        _need(rng, "rng", torch.int64, (2,), cuda=cuda)
        _same_device(x, rng)
    elif len(rng) != 2:
        raise ValueError("rng must be (seed, offset) or an int64 tensor [2]")


def _dropout(p, rng):
    if isinstance(rng, torch.Tensor):
        return Dropout(p, 0, 0, rng.data_ptr())
    return Dropout(p, int(rng[0]) & 0xFFFFFFFFFFFFFFFF, int(rng[1]) & 0xFFFFFFFFFFFFFFFF, None)


def dropout(x, p, rng, out=None, stream=None):
    """y = x / (1 - p) where the generator keeps the element, else 0; p to the nearest 2^-16.
    The mask is a function of rng = (seed, offset) and of the element's row and column in
    x [..., D]: the gradient is dropout(dy, p, rng).  An rng that is a tensor on the GPU is
    read when the kernel runs, so each replay of a graph may have its own.  out may be x."""
    _need(x, "x")
    if x.dtype not in _DT:
        raise TypeError(f"x has dtype {x.dtype}; expected one of {_FLOATS}")
    if x.dim() < 1:
        raise ValueError("x must be [..., D]")
    check_dropout_args(x, p, rng)
    if out is None:
        y = torch.empty_like(x)
    else:
        y = out
        _need(y, "out", x.dtype, x.shape)
        _same_device(x, y)
    D = x.shape[-1]
    if D:
        _launch(x.device, stream, (y,) if out is None else (), lib.gdn_dropout_fwd, x.numel() // D, D, _DT[x.dtype],
                _dropout(p, rng), _p(x), _p(y))
    return y


def add_norm_fwd(x, res, w, scale=None, eps=1e-5, out=None, stream=None):
    """res' = res + scale x and y = RMSNorm(res') w.  Returns dict y (x's dtype), res
    (res's dtype).  out={"y": ..., "res": res} updates the residual stream in place."""
    return _add_norm_fwd(lib.add_norm_fwd, (), x, res, w, scale, eps, out, stream)


def dropout_add_norm_fwd(x, res, w, p, rng, scale=None, eps=1e-5, out=None, stream=None):
    """add_norm_fwd of dropout(x, p, rng), in one pass."""
    check_dropout_args(x, p, rng)
    return _add_norm_fwd(lib.dropout_add_norm_fwd, (_dropout(p, rng),), x, res, w, scale, eps, out, stream)


def _add_norm_fwd(call, drop, x, res, w, scale, eps, out, stream):
    check_add_norm_args(x, res, w, scale)
    own = ()
    if out is None:
        out = {"y": torch.empty_like(x), "res": torch.empty_like(res)}
        own = out.values()
    else:
        _need(out.get("y"), "y", x.dtype, x.shape)
        _need(out.get("res"), "res", res.dtype, x.shape)
        _same_device(x, *out.values())
    p, _ = _norm_problem(x, eps, res.dtype)
    _launch(x.device, stream, own, call, p, *drop, _p(x), _p(res), _p(w), _p(scale), _p(out["y"]), _p(out["res"]))
    return out


def check_add_norm_bwd_args(dy, dres, res, w, x=None, scale=None, cuda=True):
    """As check_add_norm_args, dy in x's place; dres (None: zero) like res; x and scale both or neither."""
    check_add_norm_args(dy, res, w, scale, cuda=cuda)
    _need(dres, "dres", res.dtype, res.shape, cuda=cuda, optional=True)
    if (x is None) != (scale is None):
        raise ValueError("x and scale come together: the scale's gradient reads x")
    _need(x, "x", dy.dtype, dy.shape, cuda=cuda, optional=True)
    _same_device(dy, dres, x)


def add_norm_bwd(dy, dres, res, w, x=None, scale=None, eps=1e-5, out=None, workspace=None, stream=None):
    """Gradients of add_norm_fwd: dy of y, dres (None: zero) of res', at res = the
    forward's res'.  Returns dict dx (dy's dtype), dres, dw, dscale (None without
    scale).  Without scale and in one dtype, dx is dres, the same tensor."""
    return _add_norm_bwd(lib.add_norm_bwd, (), dy, dres, res, w, x, scale, eps, out, workspace, stream)


def dropout_add_norm_bwd(dy, dres, res, w, p, rng, x=None, scale=None, eps=1e-5, out=None, workspace=None,
                         stream=None):
    """Gradients of dropout_add_norm_fwd, as add_norm_bwd's; dx is always a tensor of its own."""
    check_dropout_args(dy, p, rng)
    return _add_norm_bwd(lib.dropout_add_norm_bwd, (_dropout(p, rng),), dy, dres, res, w, x, scale, eps, out, workspace,
                         stream)


def _add_norm_bwd(call, drop, dy, dres, res, w, x, scale, eps, out, workspace, stream):
    check_add_norm_bwd_args(dy, dres, res, w, x, scale)
    own = []
    if out is None:
        d = torch.empty_like(res)
        out = {"dx": d if scale is None and not drop and dy.dtype == res.dtype else torch.empty_like(dy), "dres": d,
               "dw": torch.empty_like(w), "dscale": None if scale is None else torch.empty_like(scale)}
        own += out.values()
    else:
        _need(out.get("dres"), "dres", res.dtype, res.shape)
        _need(out.get("dx"), "dx", dy.dtype, dy.shape, optional=scale is None and not drop)
        _need(out.get("dw"), "dw", torch.float32, w.shape)
        _need(out.get("dscale"), "dscale", torch.float32, w.shape, optional=scale is None)
        _same_device(dy, *out.values())
    dx = out.get("dx")
    if scale is None and not drop and dx is out["dres"]:
        dx = None
    ds = None if scale is None else out["dscale"]
    p, size = _norm_problem(dy, eps, res.dtype)
    ws, size, mine = _workspace(workspace, size, w)
    own.append(mine)
    _launch(dy.device, stream, own, call, p, *drop, _p(dy), _p(dres), _p(res), _p(w), _p(x), _p(scale), _p(dx),
            _p(out["dres"]), _p(out["dw"]), _p(ds), _p(ws), size)
    return out


def check_glr_args(x, g, h0=None, cu_seqlens=None, cu_seqlens_host=None, B=1, dh=None, dht=None, states=None,
                   bwd=False, cuda=True):
    """x, dh [B*T, D] of one dtype; g [B*T, D] fp32; h0, dht [N, D] fp32; states
    [ceil(B*T / GLR_TILE), D] fp32; cu_seqlens int32 [N+1], cu_seqlens_host the same on the CPU.  Returns N."""
    _need(x, "x", cuda=cuda)
    if x.dtype not in _DT:
        raise TypeError(f"x has dtype {x.dtype}; expected one of {_FLOATS}")
    if x.dim() != 2:
        raise ValueError("x must be [B*T, D]")
    ntok, D = x.shape
    _need(g, "g", torch.float32, x.shape, cuda=cuda)
    if B < 1 or (cu_seqlens is None and ntok % B != 0):
        raise ValueError(f"the token count {ntok} is not a multiple of B = {B}")
    if cu_seqlens is not None and B != 1:
        raise ValueError("B must be 1 with cu_seqlens")
    N = _nseq(cu_seqlens, B, cuda)
    if cu_seqlens_host is not None:
        if cu_seqlens is None:
            raise ValueError("cu_seqlens_host without cu_seqlens")
        _need(cu_seqlens_host, "cu_seqlens_host", torch.int32, cu_seqlens.shape, cuda=False)
        if cu_seqlens_host.is_cuda:
            raise ValueError("cu_seqlens_host must be a CPU tensor")
    _need(h0, "h0", torch.float32, (N, D), cuda=cuda, optional=True)
    if bwd:
        _need(dh, "dh", x.dtype, x.shape, cuda=cuda)
        _need(dht, "dht", torch.float32, (N, D), cuda=cuda, optional=True)
        _need(states, "states", torch.float32, (-(-ntok // GLR_TILE), D), cuda=cuda)
    _same_device(x, g, h0, cu_seqlens, dh, dht, states)
    return N


@functools.lru_cache(maxsize=1024)
def _glr_sizes(B, T, D, dtype, polls):
    """The struct of these dense sizes (calls only read it) and the workspace it needs."""
    p = GlrProblem(B, T, D, 0, None, None, _DT[dtype], polls)
    return p, int(lib.glr_workspace_size(ctypes.byref(p)))


def _glr_problem(x, cu_seqlens, cu_seqlens_host, B, polls=0, stream=None):
    """The problem struct, the workspace it needs and what has to outlive its use.
    Without a host mirror cu_seqlens is copied to the host, which waits for the
    current stream and for a given one, either of which may still write it."""
    ntok, D = x.shape
    if cu_seqlens is None:
        return (*_glr_sizes(B, ntok // B, D, x.dtype, polls), None)
    host = cu_seqlens_host
    if host is None:
        if stream is not None:
            stream.synchronize()
        host = cu_seqlens.detach().cpu()
    p = GlrProblem(1, ntok, D, host.numel() - 1, cu_seqlens.data_ptr(), host.data_ptr(), _DT[x.dtype], polls)
    return p, int(lib.glr_workspace_size(ctypes.byref(p))), host


def glr_workspace_size(ntok, D, dtype, cu_seqlens_host=None, B=1):
    """Bytes of workspace glr_fwd and glr_bwd need."""
    if cu_seqlens_host is None:
        return _glr_sizes(B, ntok // B, D, dtype, 0)[1]
    host = cu_seqlens_host
    p = GlrProblem(1, ntok, D, host.numel() - 1, host.data_ptr(), host.data_ptr(), _DT[dtype], 0)
    return int(lib.glr_workspace_size(ctypes.byref(p)))


def glr_num_states(ntok):
    """Rows of glr_fwd's `states` for ntok = B*T tokens."""
    return -(-ntok // GLR_TILE)


def glr_fwd(x, g, h0=None, cu_seqlens=None, cu_seqlens_host=None, B=1, want_ht=True, want_states=False, out=None,
            workspace=None, stream=None, polls=0):
    """Gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t over [B*T, D].  Returns dict
    h (x's dtype), ht [N, D] fp32, states (for glr_bwd, when wanted).  Sums of g over
    consecutive tokens must stay below 80.  Give
    cu_seqlens_host (the CPU copy of cu_seqlens) to avoid a copy and its wait."""
    N = check_glr_args(x, g, h0, cu_seqlens, cu_seqlens_host, B)
    ntok, D = x.shape
    dev = x.device
    own = []
    if out is None:
        out = {"h": torch.empty_like(x),
               "ht": g.new_empty((N, D)) if want_ht else None,
               "states": g.new_empty((glr_num_states(ntok), D)) if want_states else None}
        own += out.values()
    else:
        _need(out.get("h"), "h", x.dtype, x.shape)
        _need(out.get("ht"), "ht", torch.float32, (N, D), optional=True)
        _need(out.get("states"), "states", torch.float32, (glr_num_states(ntok), D), optional=True)
        _same_device(x, *out.values())
    p, size, keep = _glr_problem(x, cu_seqlens, cu_seqlens_host, B, polls, stream)
    ws, size, mine = _workspace(workspace, size, g)
    own.append(mine)
    _launch(dev, stream, own, lib.glr_fwd, p, _p(x), _p(g), _p(h0), _p(out["h"]), _p(out.get("ht")),
            _p(out.get("states")), _p(ws), size)
    del keep
    return out


def glr_bwd(x, g, dh, states, dht=None, h0=None, cu_seqlens=None, cu_seqlens_host=None, B=1, want_dh0=True, out=None,
            workspace=None, stream=None, polls=0):
    """Gradients of glr_fwd for dh of h and dht of ht; states from glr_fwd(want_states=True).
    Returns dict dx (x's dtype), dg fp32, dh0 [N, D] fp32."""
    N = check_glr_args(x, g, h0, cu_seqlens, cu_seqlens_host, B, dh, dht, states, bwd=True)
    D, dev = x.shape[1], x.device
    own = []
    if out is None:
        out = {"dx": torch.empty_like(x), "dg": torch.empty_like(g),
               "dh0": g.new_empty((N, D)) if want_dh0 else None}
        own += out.values()
    else:
        _need(out.get("dx"), "dx", x.dtype, x.shape)
        _need(out.get("dg"), "dg", torch.float32, x.shape)
        _need(out.get("dh0"), "dh0", torch.float32, (N, D), optional=True)
        _same_device(x, *out.values())
    p, size, keep = _glr_problem(x, cu_seqlens, cu_seqlens_host, B, polls, stream)
    ws, size, mine = _workspace(workspace, size, g)
    own.append(mine)
    _launch(dev, stream, own, lib.glr_bwd, p, _p(x), _p(g), _p(h0), _p(states), _p(dh), _p(dht), _p(out["dx"]),
            _p(out["dg"]), _p(out.get("dh0")), _p(ws), size)
    del keep
    return out


def _check_pool(state, slots, n, shape, cuda):
    _need(state, "state", torch.float32, cuda=cuda)
    if state.shape[1:] != shape:
        raise ValueError(f"state has shape {tuple(state.shape)}, expected [slots, {', '.join(map(str, shape))}]")
    _need(slots, "slots", torch.int32, (n,), cuda=cuda, optional=True)
    if slots is None and n > state.shape[0]:
        raise ValueError(f"{n} rows and {state.shape[0]} states: give slots, or a state for each row")


def check_glr_step_args(x, g, state, slots=None, cuda=True):
    """x [N, D]; g [N, D] fp32; state [slots, D] fp32; slots [N] int32 or None."""
    _need(x, "x", cuda=cuda)
    if x.dtype not in _DT:
        raise TypeError(f"x has dtype {x.dtype}; expected one of {_FLOATS}")
    if x.dim() != 2:
        raise ValueError("x must be [N, D]")
    _need(g, "g", torch.float32, x.shape, cuda=cuda)
    _check_pool(state, slots, x.shape[0], x.shape[1:], cuda)
    _same_device(x, g, state, slots)


def glr_step(x, g, state, slots=None, out=None, stream=None):
    """One token of glr_fwd's recurrence per row, on the states state[slots[n]], updated
    in place.  A row whose slot is outside the pool is padding (its h is zero); rows of
    one slot are successive tokens.  Returns h [N, D] (x's dtype)."""
    check_glr_step_args(x, g, state, slots)
    if out is None:
        h = torch.empty_like(x)
    else:
        h = out
        _need(h, "out", x.dtype, x.shape)
        _same_device(x, h)
    _launch(x.device, stream, (h,) if out is None else (), lib.glr_step, x.shape[0], x.shape[1], state.shape[0],
            _DT[x.dtype], _p(x), _p(g), _p(slots), _p(state), _p(h))
    return h


def check_gdr_step_args(q, k, v, g, beta, state, slots=None, cuda=True):
    """q, k [N, HK, K]; v [N, HV, V]; beta [N, HV] (one dtype); g [N, HV] fp32; state
    [slots, HV, K, V] fp32; slots [N] int32 or None."""
    _need(v, "v", cuda=cuda)
    _need(k, "k", v.dtype, cuda=cuda)
    if v.dtype not in _DT:
        raise TypeError(f"v has dtype {v.dtype}; expected one of {_FLOATS}")
    if k.dim() != 3 or v.dim() != 3 or k.shape[0] != v.shape[0]:
        raise ValueError("k must be [N, HK, K] and v [N, HV, V]")
    N, HV, V = v.shape
    HK, K = k.shape[1:]
    if HK < 1 or HV < 1 or HV % HK != 0:
        raise ValueError(f"HV ({HV}) must be a multiple of HK ({HK})")
    _need(q, "q", v.dtype, k.shape, cuda=cuda)
    _need(beta, "beta", v.dtype, (N, HV), cuda=cuda)
    _need(g, "g", torch.float32, (N, HV), cuda=cuda)
    _check_pool(state, slots, N, (HV, K, V), cuda)
    _same_device(v, q, k, g, beta, state, slots)


def gdr_step(q, k, v, g, beta, state, slots=None, scale=None, out=None, stream=None):
    """One token of the gated delta rule per row, on the states state[slots[n]] (fp32
    [slots, HV, K, V], as gdr_chunk_fwd's ht), updated in place; g is the token's raw
    log-gate.  Slots as for glr_step.  Returns o [N, HV, V] (v's dtype)."""
    check_gdr_step_args(q, k, v, g, beta, state, slots)
    if out is None:
        o = torch.empty_like(v)
    else:
        o = out
        _need(o, "out", v.dtype, v.shape)
        _same_device(v, o)
    (N, HK, K), (_, HV, V) = k.shape, v.shape
    _launch(v.device, stream, (o,) if out is None else (), lib.gdr_step, N, HK, HV, K, V, state.shape[0], scale or 0.0,
            _DT[v.dtype], _p(q), _p(k), _p(v), _p(g), _p(beta), _p(slots), _p(state), _p(o))
    return o


# --------------------------------------------------------------------------
# Gated feed-forward block (include/gdn_ffn.h).  Devices, streams, workspaces and
# preallocated outputs as for the layer operators.

class FfnProblem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("D", ctypes.c_int), ("F", ctypes.c_int), ("dtype", ctypes.c_int),
                ("act", ctypes.c_int)]


FFN_ACTS = {"silu": 0, "sigmoid": 1, "gelu": 2}
EXPORTED_FFN = ["ffn_workspace_size", "ffn_saved_width", "gated_ffn_fwd", "gated_ffn_bwd"]
_fp = ctypes.POINTER(FfnProblem)
lib.ffn_workspace_size.restype = _sz
lib.ffn_workspace_size.argtypes = [_fp, _i]
lib.ffn_saved_width.restype = _i64
lib.ffn_saved_width.argtypes = [_fp]
lib.gated_ffn_fwd.argtypes = [_fp] + [_vp] * 7 + [_sz, _vp]
lib.gated_ffn_bwd.argtypes = [_fp] + [_vp] * 11 + [_sz, _vp]


@functools.lru_cache(maxsize=1024)
def _ffn_sizes(T, D, F, dtype, act):
    """The struct of these sizes (calls only read it) and the workspaces it needs, forward and backward."""
    p = FfnProblem(T, D, F, _DT[dtype], FFN_ACTS[act])
    return p, tuple(int(lib.ffn_workspace_size(ctypes.byref(p), b)) for b in (0, 1))


def ffn_workspace_size(T, D, F, dtype, bwd=False):
    """Bytes of workspace gated_ffn_fwd (gated_ffn_bwd) needs."""
    return _ffn_sizes(T, D, F, dtype, "silu")[1][bool(bwd)]


def ffn_saved_width(F, dtype):
    """Floats that gated_ffn_fwd saves for a token: gate and up in fp32 and their product in the
    type, F rounded up to 16 bytes of the type."""
    piece = 8 if dtype != torch.float32 else 4
    F = -(-F // piece) * piece
    return 2 * F + (F if piece == 4 else F // 2)


def check_gated_ffn_args(x, w_gate, w_up, w_down, act="silu", saved=None, dy=None, bwd=False, cuda=True):
    """x, dy [..., D]; w_gate, w_up [F, D]; w_down [D, F], all of one dtype; saved
    [T, ffn_saved_width(F, dtype)] fp32, T the rows of x.  Returns T, D, F."""
    _need(x, "x", cuda=cuda)
    if x.dtype not in _DT:
        raise TypeError(f"x has dtype {x.dtype}; expected one of {_FLOATS}")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be [..., D]")
    if act not in FFN_ACTS:
        raise ValueError(f"act is {act!r}; expected one of {sorted(FFN_ACTS)}")
    D = x.shape[-1]
    T = x.numel() // D
    _need(w_gate, "w_gate", x.dtype, cuda=cuda)
    if w_gate.dim() != 2 or w_gate.shape[0] < 1 or w_gate.shape[1] != D:
        raise ValueError(f"w_gate has shape {tuple(w_gate.shape)}, expected [F, {D}]")
    F = w_gate.shape[0]
    _need(w_up, "w_up", x.dtype, (F, D), cuda=cuda)
    _need(w_down, "w_down", x.dtype, (D, F), cuda=cuda)
    if bwd:
        _need(saved, "saved", torch.float32, (T, ffn_saved_width(F, x.dtype)), cuda=cuda)
        _need(dy, "dy", x.dtype, x.shape, cuda=cuda)
    _same_device(x, w_gate, w_up, w_down, saved, dy)
    piece = 16 // x.element_size()
    if D % piece == 0 and F % piece == 0:
        for t, name in ((x, "x"), (w_gate, "w_gate"), (w_up, "w_up"), (w_down, "w_down"), (dy, "dy")):
            if t is not None and t.data_ptr() % 16:
                raise ValueError(f"{name} must be aligned to 16 bytes (clone it)")
    return T, D, F


def gated_ffn_fwd(x, w_gate, w_up, w_down, act="silu", want_saved=False, out=None, workspace=None, stream=None):
    """y = (act(x w_gate^T) * (x w_up^T)) w_down^T over the last axis; act is "silu", "gelu"
    (exact) or "sigmoid".  Returns dict y, saved (fp32 [T, ffn_saved_width], what
    gated_ffn_bwd needs, when wanted)."""
    T, D, F = check_gated_ffn_args(x, w_gate, w_up, w_down, act)
    own = []
    if out is None:
        out = {"y": torch.empty_like(x),
               "saved": x.new_empty((T, ffn_saved_width(F, x.dtype)), dtype=torch.float32) if want_saved else None}
        own += out.values()
    else:
        _need(out.get("y"), "y", x.dtype, x.shape)
        _need(out.get("saved"), "saved", torch.float32, (T, ffn_saved_width(F, x.dtype)), optional=True)
        _same_device(x, *out.values())
    p, sizes = _ffn_sizes(T, D, F, x.dtype, act)
    ws, size, mine = _workspace(workspace, sizes[0], x)
    own.append(mine)
    _launch(x.device, stream, own, lib.gated_ffn_fwd, p, _p(x), _p(w_gate), _p(w_up), _p(w_down), _p(out["y"]),
            _p(out.get("saved")), _p(ws), size)
    return out


def gated_ffn_bwd(x, w_gate, w_up, w_down, saved, dy, act="silu", want_dx=True, want_dw=True, out=None,
                  workspace=None, stream=None):
    """Gradients of gated_ffn_fwd for dy of y; saved from gated_ffn_fwd(want_saved=True).
    Returns dict dx, dw_gate, dw_up, dw_down, all in x's dtype (None where not wanted)."""
    T, D, F = check_gated_ffn_args(x, w_gate, w_up, w_down, act, saved, dy, bwd=True)
    own = []
    if out is None:
        out = {"dx": torch.empty_like(x) if want_dx else None,
               "dw_gate": torch.empty_like(w_gate) if want_dw else None,
               "dw_up": torch.empty_like(w_up) if want_dw else None,
               "dw_down": torch.empty_like(w_down) if want_dw else None}
        own += out.values()
    else:
        _need(out.get("dx"), "dx", x.dtype, x.shape, optional=True)
        _need(out.get("dw_gate"), "dw_gate", x.dtype, w_gate.shape, optional=True)
        _need(out.get("dw_up"), "dw_up", x.dtype, w_up.shape, optional=out.get("dw_gate") is None)
        _need(out.get("dw_down"), "dw_down", x.dtype, w_down.shape, optional=True)
        _same_device(x, *out.values())
    p, sizes = _ffn_sizes(T, D, F, x.dtype, act)
    ws, size, mine = _workspace(workspace, sizes[1], x)
    own.append(mine)
    _launch(x.device, stream, own, lib.gated_ffn_bwd, p, _p(x), _p(w_gate), _p(w_up), _p(w_down), _p(saved), _p(dy),
            _p(out.get("dx")), _p(out.get("dw_gate")), _p(out.get("dw_up")), _p(out.get("dw_down")), _p(ws), size)
    return out
