"""Thin ctypes binding of ``include/gdn.h`` (argument marshalling only).

Each function takes CUDA torch tensors, checks dtypes/shapes/contiguity,
passes raw device pointers and the current torch stream to the native entry
point of the same name, and raises ``GdnError`` on a negative status. Output
tensors are allocated with torch when not supplied (torch is the memory and
stream provider; every step of the computation runs in the library's
kernels). There is no CPU fallback: without the built library, or with a
non-CUDA tensor, these functions raise.
"""
from __future__ import annotations

import ctypes
import struct
from pathlib import Path

import torch

from . import build as _build

GDN_OK = 0
GDN_GATE_BEFORE_PREDICT = 0
GDN_GATE_AFTER_PREDICT = 1
GDN_DTYPE_BF16 = 0
GDN_DTYPE_F32 = 1
GDN_DTYPE_F16 = 2
GDN_PATH_AUTO = 0
GDN_PATH_SIMT = 1
GDN_PATH_TCGEN05 = 2
GDN_PATH_TCGEN05_SPLIT = 3
GDN_PATH_TCGEN05_WHOLE = 4
GDN_PATH_TCGEN05_FUSED = 5
GDN_SP_CHAIN = 0x100
GDN_SP_SCAN = 0x200
GDN_PAGED_AUTO = 0
GDN_PAGED_ROWS = 1
GDN_PAGED_TILES = 2
# kernel families for per-kernel timing (gdn_kernel_t)
GDN_KERNEL_CHUNK_PREP = 0
GDN_KERNEL_CHUNK_CHAIN = 1
GDN_KERNEL_CHUNK_SIMT = 2
GDN_KERNEL_SP_CHAIN = 3
GDN_KERNEL_DECODE = 4
GDN_KERNEL_CHUNK_OFFSETS = 5
GDN_KERNEL_CHUNK_CHAIN_WHOLE = 6
GDN_KERNEL_KDA = 7
GDN_KERNEL_KDA_PREP = 8
GDN_KERNEL_BWD = 9
GDN_KERNEL_BWD_FINALIZE = 10
GDN_KERNEL_CBWD_PREP = 11
GDN_KERNEL_CBWD_FWD = 12
GDN_KERNEL_CBWD_REV = 13
GDN_KERNEL_CBWD_GRAD = 14
GDN_KERNEL_CHUNK_FUSED = 15
GDN_KERNEL_PAGED_APPEND = 16
GDN_KERNEL_PAGED_ROWS = 17
GDN_KERNEL_PAGED_MERGE = 18
GDN_KERNEL_PAGED_TILES = 19
GDN_KERNEL_COUNT = 20
KERNEL_NAMES = {
    GDN_KERNEL_CHUNK_PREP: "ut_prep_kernel",
    GDN_KERNEL_CHUNK_CHAIN: "chunk_tc_kernel",
    GDN_KERNEL_CHUNK_SIMT: "chunk_simt_kernel",
    GDN_KERNEL_SP_CHAIN: "sp_chain_kernel",
    GDN_KERNEL_DECODE: "decode_kernel",
    GDN_KERNEL_CHUNK_OFFSETS: "chunk_offsets_kernel",
    GDN_KERNEL_CHUNK_CHAIN_WHOLE: "chain_tx_kernel",
    GDN_KERNEL_KDA: "kda_kernel",
    GDN_KERNEL_KDA_PREP: "kda_prep_kernel",
    GDN_KERNEL_BWD: "bwd_kernel",
    GDN_KERNEL_BWD_FINALIZE: "bwd_finalize_kernel",
    GDN_KERNEL_CBWD_PREP: "cbwd_prep_kernel",
    GDN_KERNEL_CBWD_FWD: "cbwd_fwd_kernel",
    GDN_KERNEL_CBWD_REV: "cbwd_rev_kernel",
    GDN_KERNEL_CBWD_GRAD: "cbwd_grad_kernel",
    GDN_KERNEL_CHUNK_FUSED: "fused_chunk_kernel",
    GDN_KERNEL_PAGED_APPEND: "paged_append_kernel",
    GDN_KERNEL_PAGED_ROWS: "paged_rows_kernel",
    GDN_KERNEL_PAGED_MERGE: "paged_merge_kernel",
    GDN_KERNEL_PAGED_TILES: "paged_tiles_kernel",
}

_lib = None
_current_device = torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {gdn_status_string(status)} ({status})")


# gdn_paged_cache_t of the C ABI, packed field by field (native alignment):
# k, v, six strides, page_table, table_stride, kv_lens, six ints
_PAGED_CACHE = struct.Struct("@PP6qPqP6i")


def library_path() -> Path:
    return _build.LIB


def library():
    """The loaded ``libgdn_gb300.so`` (ctypes.CDLL) with typed entry points."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not path.exists():
        raise RuntimeError(
            f"native library {path} is missing: run "
            "`python -c 'import __graft_entry__ as g; g.build()'` first "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(str(path))
    vp, fp, ip = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
    i = ctypes.c_int
    chunk_args = [vp, vp, vp, fp, fp, fp, vp, fp, ip, i, i, i, i, i, i, vp]
    lib.gdn_chunk_fwd.argtypes = chunk_args
    lib.gdn_chunk_fwd.restype = i
    lib.gdn_chunk_fwd_f32.argtypes = chunk_args
    lib.gdn_chunk_fwd_f32.restype = i
    lib.gdn_chunk_fwd_ex.argtypes = chunk_args[:-1] + [i, i, i, i, vp]
    lib.gdn_chunk_fwd_ex.restype = i
    lib.gdn_recurrent_step.argtypes = [vp, vp, vp, fp, fp, fp, vp, i, i, i, i,
                                       vp]
    lib.gdn_recurrent_step.restype = i
    lib.gdn_kda_fwd.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, ip, i, i, i, i,
                                i, vp]
    lib.gdn_kda_fwd.restype = i
    lib.gdn_kda_fwd_ex.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, ip, i, i, i,
                                   i, i, i, i, vp]
    lib.gdn_kda_fwd_ex.restype = i
    bwd_args = [vp, vp, vp, fp, fp, fp, vp, fp, fp, fp, fp, fp, fp, fp, ip, i,
                i, i, i, i]
    lib.gdn_kda_bwd.argtypes = bwd_args + [vp]
    lib.gdn_kda_bwd.restype = i
    lib.gdn_chunk_bwd.argtypes = bwd_args + [i, vp]
    lib.gdn_chunk_bwd.restype = i
    lib.gdn_chunk_bwd_f32.argtypes = bwd_args + [i, vp]
    lib.gdn_chunk_bwd_f32.restype = i
    lib.gdn_chunk_bwd_chunked.argtypes = bwd_args + [vp]
    lib.gdn_chunk_bwd_chunked.restype = i
    lib.gdn_chunk_bwd_fused.argtypes = [vp, vp, vp, fp, fp, fp, ip, fp, vp,
                                        ctypes.c_float, vp, fp, fp, fp, fp, fp,
                                        fp, fp, fp, fp, i, i, i, i, i, vp]
    lib.gdn_chunk_bwd_fused.restype = i
    lib.gdn_device_status.argtypes = [vp]
    lib.gdn_device_status.restype = i
    lib.gdn_status_string.argtypes = [i]
    lib.gdn_status_string.restype = ctypes.c_char_p
    lib.gdn_version.restype = i
    lib.gdn_kernel_launches.restype = ctypes.c_ulonglong
    lib.gdn_selftest_mma.argtypes = [vp, vp, vp, i, i, i, i, i, i, vp]
    lib.gdn_selftest_mma.restype = i
    lib.gdn_chunk_fwd_fused.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, ip,
                                        fp, vp, ctypes.c_float, i, i, i, i,
                                        i, i, i, vp]
    lib.gdn_chunk_fwd_fused.restype = i
    i64, cache = ctypes.c_int64, ctypes.c_char_p
    lib.gdn_paged_append.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, fp, i,
                                     i, ip, i, ip, i, cache, ip, i, i, i, vp]
    lib.gdn_paged_append.restype = i
    lib.gdn_paged_attn.argtypes = [vp, i64, cache, ip, i, i, i, ctypes.c_float,
                                   i, i, vp, fp, i, vp]
    lib.gdn_paged_attn.restype = i
    lib.gdn_timing_enable.argtypes = [i]
    lib.gdn_timing_enable.restype = i
    lib.gdn_timing_read.argtypes = [i, ctypes.POINTER(ctypes.c_ulonglong),
                                    ctypes.POINTER(ctypes.c_double)]
    lib.gdn_timing_read.restype = i
    _lib = lib
    return lib


def gdn_status_string(status: int) -> str:
    return library().gdn_status_string(int(status)).decode()


def kernel_counters() -> int:
    """Kernels enqueued by the library so far in this process."""
    return int(library().gdn_kernel_launches())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, name, dtype, device):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (no CPU fallback)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _shape(t, name, shape):
    """The kernels index by the sizes passed: a tensor of another shape would
    be read or written out of bounds, so it is refused here."""
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t


def _chunk_call(fn_name, q, k, v, g, beta, h0, cu_seqlens, out, hT,
                output_final_state, C, stream, io_dtype, extra=()):
    fn = getattr(library(), fn_name)
    if extra:
        f0 = fn
        fn = (lambda *a: f0(*a[:-1], *extra, a[-1]))
    return _chunk_call_fn(fn, fn_name, q, k, v, g, beta, h0, cu_seqlens, out,
                          hT, output_final_state, C, stream, io_dtype)


def _chunk_call_fn(fn, fn_name, q, k, v, g, beta, h0, cu_seqlens, out, hT,
                   output_final_state, C, stream, io_dtype):
    dev = q.device
    _need(q, "q", io_dtype, None)
    _need(k, "k", io_dtype, dev)
    _need(v, "v", io_dtype, dev)
    _need(g, "g", torch.float32, dev)
    _need(beta, "beta", torch.float32, dev)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q/k must be [B, T, H, dk] and v [B, T, H, dv]")
    Bt, T, H, dk = q.shape
    dv = v.shape[-1]
    if k.shape != q.shape or v.shape[:3] != (Bt, T, H):
        raise ValueError("q/k/v shapes disagree")
    if g.shape != (Bt, T, H) or beta.shape != (Bt, T, H):
        raise ValueError("g/beta must be [B, T, H]")
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if Bt != 1:
            raise ValueError("packed sequences are passed as [1, T, H, ...]")
        N = cu_seqlens.numel() - 1
    else:
        N = Bt
    if h0 is not None:
        _need(h0, "h0", torch.float32, dev)
        if h0.shape != (N, H, dk, dv):
            raise ValueError(f"h0 must be [{N}, {H}, {dk}, {dv}]")
    if out is None:
        out = torch.empty_like(v)
    else:
        _shape(_need(out, "out", io_dtype, dev), "out", v.shape)
    if hT is None and output_final_state:
        hT = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    elif hT is not None:
        _shape(_need(hT, "hT", torch.float32, dev), "hT", (N, H, dk, dv))
    with torch.cuda.device(dev):
        rc = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                _ptr(out), _ptr(hT), _ptr(cu_seqlens), N, H, T, dk, dv, C,
                _stream(stream))
    if rc != GDN_OK:
        raise GdnError(rc, fn_name)
    return out, hT


def gdn_chunk_fwd(q, k, v, g, beta, h0=None, cu_seqlens=None, *, out=None,
                  hT=None, output_final_state=True, C=64, stream=None):
    """bf16 chunkwise forward; returns (out bf16 like v, hT fp32 or None)."""
    return _chunk_call("gdn_chunk_fwd", q, k, v, g, beta, h0, cu_seqlens, out,
                       hT, output_final_state, C, stream, torch.bfloat16)


def gdn_chunk_fwd_f32(q, k, v, g, beta, h0=None, cu_seqlens=None, *, out=None,
                      hT=None, output_final_state=True, C=64, stream=None):
    """fp32 chunkwise forward; returns (out fp32, hT fp32 or None)."""
    return _chunk_call("gdn_chunk_fwd_f32", q, k, v, g, beta, h0, cu_seqlens,
                       out, hT, output_final_state, C, stream, torch.float32)


def gdn_chunk_fwd_ex(q, k, v, g, beta, h0=None, cu_seqlens=None, *, out=None,
                     hT=None, output_final_state=True, C=64,
                     variant=GDN_GATE_BEFORE_PREDICT, path=GDN_PATH_AUTO,
                     sp_parts=0, stream=None):
    """Chunkwise forward with explicit gate placement, kernel family and
    sequence-parallel split; q/k/v dtype (bf16 or fp32) selects the dtype."""
    dtype = {torch.bfloat16: GDN_DTYPE_BF16, torch.float32: GDN_DTYPE_F32}.get(
        q.dtype)
    if dtype is None:
        raise ValueError("q/k/v must be bf16 or fp32")
    return _chunk_call("gdn_chunk_fwd_ex", q, k, v, g, beta, h0, cu_seqlens,
                       out, hT, output_final_state, C, stream, q.dtype,
                       extra=(dtype, int(variant), int(path), int(sp_parts)))


def gdn_kda_fwd(q, k, v, g, beta, h0=None, cu_seqlens=None, *, out=None,
                hT=None, output_final_state=True, stream=None):
    """The delta rule with a per-channel decay, token by token: q, k bf16
    [B, T, H, dk], v bf16 [B, T, H, dv], g fp32 [B, T, H, dk] log-decays,
    beta fp32 [B, T, H]. Returns (out bf16 like v, hT fp32 [N, H, dk, dv] or
    None); ``hT`` may be ``h0`` (in-place state update)."""
    return _kda("gdn_kda_fwd", q, k, v, g, beta, h0, cu_seqlens, out, hT,
                output_final_state, stream, ())


def gdn_kda_fwd_ex(q, k, v, g, beta, h0=None, cu_seqlens=None, *, out=None,
                   hT=None, output_final_state=True, path=GDN_PATH_AUTO,
                   sp_parts=0, stream=None):
    """gdn_kda_fwd with a choice of kernels: ``path`` GDN_PATH_AUTO (the
    chunk form on the tensor cores where it applies), GDN_PATH_SIMT (token by
    token) or GDN_PATH_TCGEN05 (the chunk form), optionally or-ed with
    GDN_SP_CHAIN / GDN_SP_SCAN; ``sp_parts`` the sequence-parallel split of
    the chunk form (0: automatic)."""
    return _kda("gdn_kda_fwd_ex", q, k, v, g, beta, h0, cu_seqlens, out, hT,
                output_final_state, stream, (int(path), int(sp_parts)))


def gdn_kda_bwd(q, k, v, g, beta, h0, dout, dhT=None, cu_seqlens=None, *,
                want_dh0=True, stream=None):
    """Gradients of gdn_kda_fwd for L = sum(dout * out) + sum(dhT * hT):
    returns dict dq, dk [B, T, H, dk], dv [B, T, H, dv], dg [B, T, H, dk],
    dbeta [B, T, H] (fp32) and dh0 [N, H, dk, dv] (fp32, or None)."""
    return _bwd("gdn_kda_bwd", q, k, v, g, beta, h0, dout, dhT, cu_seqlens,
                want_dh0, stream, per_channel=True)


def gdn_chunk_bwd(q, k, v, g, beta, h0, dout, dhT=None, cu_seqlens=None, *,
                  variant=GDN_GATE_BEFORE_PREDICT, want_dh0=True, stream=None):
    """Gradients of gdn_chunk_fwd_ex (scalar gate; ``variant`` the forward's
    gate placement): as gdn_kda_bwd with g and dg [B, T, H]."""
    return _bwd("gdn_chunk_bwd", q, k, v, g, beta, h0, dout, dhT, cu_seqlens,
                want_dh0, stream, per_channel=False, extra=(int(variant),))


def gdn_chunk_bwd_chunked(q, k, v, g, beta, h0, dout, dhT=None, *,
                          want_dh0=True, stream=None):
    """gdn_chunk_bwd (decay before the prediction) through the chunk form:
    per-chunk UT/WY quantities, the chunks' entry states and exit gradients by
    two chains, then every chunk's gradients in parallel; dense batches only.
    Returns the dict of gdn_chunk_bwd."""
    return _bwd("gdn_chunk_bwd_chunked", q, k, v, g, beta, h0, dout, dhT,
                None, want_dh0, stream, per_channel=False)


def gdn_chunk_bwd_f32(q, k, v, g, beta, h0, dout, dhT=None, cu_seqlens=None,
                      *, variant=GDN_GATE_BEFORE_PREDICT, want_dh0=True,
                      stream=None):
    """gdn_chunk_bwd for fp32 q, k, v and dout."""
    return _bwd("gdn_chunk_bwd_f32", q, k, v, g, beta, h0, dout, dhT,
                cu_seqlens, want_dh0, stream, per_channel=False,
                extra=(int(variant),), in_dtype=torch.float32)


def gdn_chunk_bwd_fused(q, k, v, a, b, h0, dout, dhT=None, cu_seqlens=None, *,
                        norm_weight=None, gate=None, eps=1e-6, want_dh0=True,
                        stream=None):
    """Gradients of gdn_chunk_fwd_fused for L = sum(dout * out) + sum(dhT *
    hT): dict dq, dk, dv, da, db, dh0 (or None), dweight (with norm_weight,
    else None), dgate (with gate, else None); all fp32."""
    dev = q.device
    _need(q, "q", torch.bfloat16, None)
    for name, t in (("k", k), ("v", v), ("dout", dout)):
        _need(t, name, torch.bfloat16, dev)
    _need(a, "a", torch.float32, dev)
    _need(b, "b", torch.float32, dev)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q/k must be [B, T, H, dk] and v/dout [B, T, H, dv]")
    Bt, T, H, dk = q.shape
    dv = v.shape[-1]
    _shape(k, "k", q.shape)
    _shape(v, "v", (Bt, T, H, dv))
    _shape(dout, "dout", v.shape)
    _shape(a, "a", (Bt, T, H))
    _shape(b, "b", (Bt, T, H))
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if Bt != 1:
            raise ValueError("packed sequences are passed as [1, T, H, ...]")
        N = cu_seqlens.numel() - 1
    else:
        N = Bt
    if norm_weight is not None:
        _shape(_need(norm_weight, "norm_weight", torch.float32, dev),
               "norm_weight", (dv,))
    if gate is not None:
        _shape(_need(gate, "gate", torch.bfloat16, dev), "gate", v.shape)
    for name, st in (("h0", h0), ("dhT", dhT)):
        if st is not None:
            _shape(_need(st, name, torch.float32, dev), name, (N, H, dk, dv))
    f32 = dict(dtype=torch.float32, device=dev)
    res = {"dq": torch.empty(q.shape, **f32), "dk": torch.empty(q.shape, **f32),
           "dv": torch.empty(v.shape, **f32), "da": torch.empty(a.shape, **f32),
           "db": torch.empty(b.shape, **f32),
           "dh0": torch.empty((N, H, dk, dv), **f32) if want_dh0 else None,
           "dweight": torch.empty((dv,), **f32) if norm_weight is not None else None,
           "dgate": torch.empty(v.shape, **f32) if gate is not None else None}
    with torch.cuda.device(dev):
        rc = library().gdn_chunk_bwd_fused(
            _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(h0),
            _ptr(cu_seqlens), _ptr(norm_weight), _ptr(gate), float(eps),
            _ptr(dout), _ptr(dhT), _ptr(res["dq"]), _ptr(res["dk"]),
            _ptr(res["dv"]), _ptr(res["da"]), _ptr(res["db"]),
            _ptr(res["dh0"]), _ptr(res["dweight"]), _ptr(res["dgate"]), N, H,
            T, dk, dv, _stream(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_chunk_bwd_fused")
    return res


def _bwd(fn, q, k, v, g, beta, h0, dout, dhT, cu_seqlens, want_dh0, stream,
         per_channel, extra=(), in_dtype=torch.bfloat16):
    dev = q.device
    _need(q, "q", in_dtype, None)
    for name, t in (("k", k), ("v", v), ("dout", dout)):
        _need(t, name, in_dtype, dev)
    _need(g, "g", torch.float32, dev)
    _need(beta, "beta", torch.float32, dev)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q/k must be [B, T, H, dk] and v/dout [B, T, H, dv]")
    Bt, T, H, dk = q.shape
    dv = v.shape[-1]
    gshape = q.shape if per_channel else q.shape[:3]
    if k.shape != q.shape or v.shape[:3] != (Bt, T, H) or dout.shape != v.shape:
        raise ValueError("q/k must be [B, T, H, dk], v/dout [B, T, H, dv]")
    if g.shape != gshape or beta.shape != (Bt, T, H):
        raise ValueError(f"g must be {tuple(gshape)} and beta [B, T, H]")
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if Bt != 1:
            raise ValueError("packed sequences are passed as [1, T, H, ...]")
        N = cu_seqlens.numel() - 1
    else:
        N = Bt
    for name, st in (("h0", h0), ("dhT", dhT)):
        if st is not None:
            _need(st, name, torch.float32, dev)
            if st.shape != (N, H, dk, dv):
                raise ValueError(f"{name} must be [{N}, {H}, {dk}, {dv}]")
    f32 = dict(dtype=torch.float32, device=dev)
    res = {"dq": torch.empty(q.shape, **f32), "dk": torch.empty(q.shape, **f32),
           "dv": torch.empty(v.shape, **f32), "dg": torch.empty(gshape, **f32),
           "dbeta": torch.empty(beta.shape, **f32),
           "dh0": torch.empty((N, H, dk, dv), **f32) if want_dh0 else None}
    with torch.cuda.device(dev):
        rc = getattr(library(), fn)(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
            _ptr(dout), _ptr(dhT), _ptr(res["dq"]), _ptr(res["dk"]),
            _ptr(res["dv"]), _ptr(res["dg"]), _ptr(res["dbeta"]),
            _ptr(res["dh0"]), _ptr(cu_seqlens), N, H, T, dk, dv, *extra,
            _stream(stream))
    if rc != GDN_OK:
        raise GdnError(rc, fn)
    return res


def _kda(fn, q, k, v, g, beta, h0, cu_seqlens, out, hT, output_final_state,
         stream, extra):
    dev = q.device
    _need(q, "q", torch.bfloat16, None)
    _need(k, "k", torch.bfloat16, dev)
    _need(v, "v", torch.bfloat16, dev)
    _need(g, "g", torch.float32, dev)
    _need(beta, "beta", torch.float32, dev)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q/k/g must be [B, T, H, dk] and v [B, T, H, dv]")
    Bt, T, H, dk = q.shape
    dv = v.shape[-1]
    if k.shape != q.shape or v.shape[:3] != (Bt, T, H) or g.shape != q.shape:
        raise ValueError("q/k/g must be [B, T, H, dk] and v [B, T, H, dv]")
    if beta.shape != (Bt, T, H):
        raise ValueError("beta must be [B, T, H]")
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if Bt != 1:
            raise ValueError("packed sequences are passed as [1, T, H, ...]")
        N = cu_seqlens.numel() - 1
    else:
        N = Bt
    for name, st in (("h0", h0), ("hT", hT)):
        if st is not None:
            _need(st, name, torch.float32, dev)
            if st.shape != (N, H, dk, dv):
                raise ValueError(f"{name} must be [{N}, {H}, {dk}, {dv}]")
    if out is None:
        out = torch.empty_like(v)
    else:
        _shape(_need(out, "out", torch.bfloat16, dev), "out", v.shape)
    if hT is None and output_final_state:
        hT = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        rc = getattr(library(), fn)(_ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                      _ptr(beta), _ptr(h0), _ptr(out),
                                      _ptr(hT), _ptr(cu_seqlens), N, H, T, dk,
                                      dv, *extra, _stream(stream))
    if rc != GDN_OK:
        raise GdnError(rc, fn)
    return out, hT


def gdn_chunk_fwd_fused(q, k, v, a, b, h0=None, cu_seqlens=None, *,
                        norm_weight=None, gate=None, eps=1e-6, out=None,
                        hT=None, output_final_state=True, C=64,
                        path=GDN_PATH_AUTO, stream=None):
    """The forward pass with the steps either side fused: raw q, k (L2-
    normalised in the kernels), gate logits a (log alpha = -softplus(a)) and
    step logits b (beta = sigmoid(b)); output RMS-normalised over d_v and
    scaled by ``norm_weight`` [dv] fp32 when given, then gated by
    sigmoid(``gate``) (bf16, like v) when given. Returns (out bf16, hT)."""
    dev = q.device
    if norm_weight is not None:
        _need(norm_weight, "norm_weight", torch.float32, dev)
        if norm_weight.shape != (v.shape[-1],):
            raise ValueError("norm_weight must be [dv]")
    if gate is not None:
        _need(gate, "gate", torch.bfloat16, dev)
        if gate.shape != v.shape:
            raise ValueError("gate must have the shape of v")
    extra_ptrs = (_ptr(norm_weight), _ptr(gate), ctypes.c_float(float(eps)))

    class _Fn:  # argument order of gdn_chunk_fwd_fused
        def __init__(self, f):
            self.f = f

        def __call__(self, q_, k_, v_, a_, b_, h0_, out_, hT_, cu_, N, H, T,
                     dk, dv, C_, stream_):
            return self.f(q_, k_, v_, a_, b_, h0_, out_, hT_, cu_,
                          *extra_ptrs, N, H, T, dk, dv, C_, int(path),
                          stream_)

    lib = library()
    return _chunk_call_fn(_Fn(lib.gdn_chunk_fwd_fused), "gdn_chunk_fwd_fused",
                          q, k, v, a, b, h0, cu_seqlens, out, hT,
                          output_final_state, C, stream, torch.bfloat16)


def gdn_recurrent_step(q, k, v, g, beta, state, *, out=None, stream=None):
    """One decode token per (sequence, head); ``state`` is updated in place.
    q, k [N, H, dk] bf16, v [N, H, dv] bf16, g/beta [N, H] fp32, state
    [N, H, dk, dv] fp32. Returns out [N, H, dv] bf16."""
    dev = q.device
    _need(q, "q", torch.bfloat16, None)
    _need(k, "k", torch.bfloat16, dev)
    _need(v, "v", torch.bfloat16, dev)
    _need(g, "g", torch.float32, dev)
    _need(beta, "beta", torch.float32, dev)
    _need(state, "state", torch.float32, dev)
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q/k must be [N, H, dk] and v [N, H, dv]")
    N, H, dk = q.shape
    dv = v.shape[-1]
    _shape(k, "k", q.shape)
    _shape(v, "v", (N, H, dv))
    _shape(g, "g", (N, H))
    _shape(beta, "beta", (N, H))
    if state.shape != (N, H, dk, dv):
        raise ValueError("state must be [N, H, dk, dv]")
    if out is None:
        out = torch.empty_like(v)
    else:
        _shape(_need(out, "out", torch.bfloat16, dev), "out", v.shape)
    with torch.cuda.device(dev):
        rc = library().gdn_recurrent_step(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state),
            _ptr(out), N, H, dk, dv, _stream(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_recurrent_step")
    return out


_PAGED_DTYPES = {torch.bfloat16: GDN_DTYPE_BF16, torch.float16: GDN_DTYPE_F16}


def _paged_rows(t, name, dtype, device, shape):
    """Token stride of a [B, T, H, d] tensor whose heads are contiguous and
    whose tokens lie a fixed stride apart (a slice of a fused projection)."""
    B, T, H, d = shape
    if t.device != device or t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {[B, T, H, d]} on {device}, "
                         f"got {t.dtype} {list(t.shape)} on {t.device}")
    sb, st, sh, sd = t.stride()
    if B * T * H and (sd != 1 or (H > 1 and sh != d)
                      or (B > 1 and T > 1 and sb != T * st)):
        raise ValueError(f"{name}: heads must be contiguous and tokens one "
                         "stride apart")
    return st if T > 1 else sb if B > 1 else H * d


def _paged_cache(k_cache, v_cache, page_table, kv_lens, N, dev):
    """The packed gdn_paged_cache_t, and (heads, d, dtype) of the cache."""
    if dev.type != "cuda":
        raise ValueError("the tensors must be CUDA tensors (no CPU fallback)")
    dt = k_cache.dtype
    code = _PAGED_DTYPES.get(dt)
    if code is None:
        raise ValueError("k_cache must be bf16 or fp16")
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape or v_cache.dtype != dt:
        raise ValueError("k_cache and v_cache must both be "
                         "[pages, heads, page_size, d] of one type")
    if k_cache.device != dev or v_cache.device != dev:
        raise ValueError(f"the cache must be on {dev}")
    i32 = torch.int32
    if (page_table.dtype != i32 or kv_lens.dtype != i32
            or page_table.device != dev or kv_lens.device != dev):
        raise ValueError(f"page_table and kv_lens must be int32 on {dev}")
    if page_table.dim() != 2 or page_table.shape[0] != N:
        raise ValueError(f"page_table must be [{N}, max_pages]")
    width = page_table.shape[1]
    row, unit = page_table.stride()
    if unit != 1 and width > 1:
        raise ValueError("page_table rows must be contiguous")
    if kv_lens.shape != (N,) or not kv_lens.is_contiguous():
        raise ValueError(f"kv_lens must be [{N}], contiguous")
    pages, heads, page, d = shape
    kp, kh, kt, ks = k_cache.stride()
    vp, vh, vt, vs = v_cache.stride()
    if ks != 1 or vs != 1:
        raise ValueError("the cache's last dimension must be contiguous")
    # strides of dimensions of one element are never used
    if pages == 1:
        kp = vp = 0
    if heads == 1:
        kh = vh = 0
    return _PAGED_CACHE.pack(
        k_cache.data_ptr(), v_cache.data_ptr(), kp, kh, kt, vp, vh, vt,
        page_table.data_ptr(), row if N > 1 else width, kv_lens.data_ptr(),
        pages, page, width, heads, d, code), heads, d, dt


def _paged_batch(B, cu_seqlens, dev):
    """Number of sequences of a packed call."""
    if cu_seqlens.device != dev or cu_seqlens.dtype != torch.int32:
        raise ValueError(f"cu_seqlens must be int32 on {dev}")
    if cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be [N + 1], contiguous")
    if B != 1:
        raise ValueError("packed sequences are passed as [1, T, H, d]")
    return cu_seqlens.numel() - 1


def _paged_stream(stream, dev, tensors):
    """(raw stream, context to leave) of a call: under ``dev``, and under
    ``stream`` if one is given, so that outputs are allocated there; inputs are
    marked as used on it, so that the allocator does not hand their memory out
    before the kernels are done with it. (The usual case, the current stream
    of the current device, has nothing to enter: these calls are short.)"""
    # what may fail comes before the context is entered: callers leave it only
    # if they have got it
    if stream is None:
        raw = _raw_stream(dev.index)
        if _current_device() == dev.index:
            return raw, None
        ctx = torch.cuda.device(dev)
    else:
        raw = stream.cuda_stream
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        ctx = torch.cuda.stream(stream)
    ctx.__enter__()
    return raw, ctx


def gdn_paged_append(q, k, v, k_cache, v_cache, page_table, kv_lens,
                     cu_seqlens=None, *, rope=None, positions=None,
                     sections=None, interleaved=False, q_out=None, stream=None):
    """New tokens' keys and values into the paged cache, queries and keys
    rotated on the way. q [B, T, Hq, d] (or None), k, v [B, T, Hkv, d] bf16 or
    fp16, tokens any stride apart; k_cache, v_cache [pages, Hkv, page_size, d]
    (any strides: pass token-major pages transposed), written in place;
    page_table int32 [N, max_pages]; kv_lens int32 [N], the new tokens counted
    in; ``cu_seqlens`` for a packed batch [1, T, H, d]. ``rope`` fp32
    [rows, rot]: cosines and sines of each position (None: no rotation);
    ``positions`` int32 [B, T] or, with ``sections`` (pairs per axis),
    [axes, B, T]; default the tokens' places in their sequences. Returns the
    rotated queries (``q_out``, which may be ``q`` and spares a short call the
    allocation, 4 us of 16)."""
    dev = k.device
    shape = k.shape
    if len(shape) != 4:
        raise ValueError("k must be [B, T, H, d]")
    B, T, _, _ = shape
    N = B if cu_seqlens is None else _paged_batch(B, cu_seqlens, dev)
    cache, heads, d, dt = _paged_cache(k_cache, v_cache, page_table, kv_lens, N,
                                       dev)
    shape = (B, T, heads, d)
    sk = _paged_rows(k, "k", dt, dev, shape)
    sv = _paged_rows(v, "v", dt, dev, shape)
    sq = so = hq = 0
    if q is not None:
        shape = q.shape
        if len(shape) != 4:
            raise ValueError("q must be [B, T, H, d]")
        hq = shape[2]
        shape = (B, T, hq, d)
        sq = _paged_rows(q, "q", dt, dev, shape)
        if q_out is not None:
            so = _paged_rows(q_out, "q_out", dt, dev, shape)
    elif q_out is not None:
        raise ValueError("q_out without q")
    rot = rows = 0
    rope_at = None
    if rope is not None:
        if (rope.dtype != torch.float32 or rope.device != dev
                or rope.dim() != 2 or not rope.is_contiguous()):
            raise ValueError(f"rope must be fp32 [rows, rot] on {dev}, "
                             "contiguous")
        rows, rot = rope.shape
        rope_at = rope.data_ptr()
    axes, sec = 1, None
    if positions is not None:
        _need(positions, "positions", torch.int32, dev)
        if positions.dim() == 3:
            axes = positions.shape[0]
        if positions.dim() not in (2, 3) or positions.shape[-2:] != (B, T):
            raise ValueError(f"positions must be {[B, T]} or [axes, {B}, {T}]")
        if axes > 1:
            if sections is None or len(sections) != axes:
                raise ValueError(f"sections must hold {axes} pair counts")
            sec = (ctypes.c_int32 * axes)(*[int(x) for x in sections])
    raw, ctx = _paged_stream(stream, dev, stream and (
        q, k, v, k_cache, v_cache, page_table, kv_lens, cu_seqlens, rope,
        positions, q_out))
    try:
        q_at = out_at = None
        if q is not None:
            if q_out is None:
                q_out = torch.empty(shape, dtype=dt, device=dev)
                so = hq * d
            q_at, out_at = q.data_ptr(), q_out.data_ptr()
        rc = (_lib or library()).gdn_paged_append(
            q_at, sq, k.data_ptr(), sk, v.data_ptr(), sv, out_at, so, rope_at,
            rows, rot, positions if positions is None else positions.data_ptr(),
            axes, sec, 1 if interleaved else 0, cache,
            cu_seqlens if cu_seqlens is None else cu_seqlens.data_ptr(), N, T, hq,
            raw)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_paged_append")
    return q_out


def gdn_paged_attn(q, k_cache, v_cache, page_table, kv_lens, cu_seqlens=None, *,
                   scale=None, causal=True, window=0, out=None,
                   return_lse=False, path=GDN_PAGED_AUTO, stream=None):
    """Attention of new tokens over the paged cache that holds their keys and
    values already (gdn_paged_append): q [B, T, Hq, d] (T = 1: a decode step),
    or packed [1, T, Hq, d] with ``cu_seqlens``; the cache as there. ``scale``
    defaults to d ** -0.5; ``window`` > 0 hides keys that far back. Returns
    out like q, contiguous (and lse fp32 [B, T, Hq] with ``return_lse``);
    tokens that see no key get 0 and -inf."""
    dev = q.device
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be [B, T, H, d]")
    B, T, hq, _ = shape
    N = B if cu_seqlens is None else _paged_batch(B, cu_seqlens, dev)
    cache, _, d, dt = _paged_cache(k_cache, v_cache, page_table, kv_lens, N, dev)
    sq = _paged_rows(q, "q", dt, dev, (B, T, hq, d))
    if out is not None:
        _shape(_need(out, "out", dt, dev), "out", shape)
    if scale is None:
        scale = d ** -0.5
    if window:  # (in the range of a C int; from 2^30 on it hides nothing)
        window = min(max(int(window), -1), 1 << 30)
    raw, ctx = _paged_stream(stream, dev, stream and (
        q, k_cache, v_cache, page_table, kv_lens, cu_seqlens, out))
    try:
        if out is None:
            out = torch.empty(shape, dtype=dt, device=dev)
        lse = (torch.empty((B, T, hq), dtype=torch.float32, device=dev)
               if return_lse else None)
        rc = (_lib or library()).gdn_paged_attn(
            q.data_ptr(), sq, cache,
            cu_seqlens if cu_seqlens is None else cu_seqlens.data_ptr(), N, T, hq,
            scale, 1 if causal else 0, window, out.data_ptr(),
            lse if lse is None else lse.data_ptr(), path, raw)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_paged_attn")
    return (out, lse) if return_lse else out


def gdn_selftest_mma(A, B, *, a_mn=False, b_mn=False, b_stacked=False,
                     twice=False, a_tmem=False, stream=None):
    """D = A @ B (x2 when ``twice``) through one tcgen05 MMA sequence with the
    chunk kernel's shared-memory layouts. A bf16 [128, K], B bf16 [K, N];
    ``a_tmem`` places A in TMEM instead of shared memory."""
    dev = A.device
    _need(A, "A", torch.bfloat16, None)
    _need(B, "B", torch.bfloat16, dev)
    K, N = A.shape[1], B.shape[1]
    if A.shape != (128, K) or B.shape != (K, N):
        raise ValueError("A must be [128, K] and B [K, N]")
    D = torch.empty((128, N), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        rc = library().gdn_selftest_mma(_ptr(A), _ptr(B), _ptr(D), K, N,
                                        2 if a_tmem else int(a_mn),
                                        int(b_mn), int(b_stacked),
                                        int(twice), _stream(stream))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_selftest_mma")
    return D


def gdn_device_status(stream=None) -> int:
    """Synchronises ``stream`` and returns/clears the kernels' status word."""
    return int(library().gdn_device_status(_stream(stream)))


def gdn_timing_enable(on: bool) -> None:
    """Per-kernel device timing on/off (resets the accumulated totals)."""
    rc = library().gdn_timing_enable(1 if on else 0)
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_timing_enable")


def gdn_timing_read(kernel: int):
    """(launches, total_ms) of one kernel family since timing was enabled;
    waits for the recorded events."""
    n = ctypes.c_ulonglong(0)
    ms = ctypes.c_double(0.0)
    rc = library().gdn_timing_read(int(kernel), ctypes.byref(n),
                                   ctypes.byref(ms))
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_timing_read")
    return int(n.value), float(ms.value)


def kernel_timings():
    """{kernel name: (launches, total_ms)} for every family timed so far."""
    out = {}
    for k in range(GDN_KERNEL_COUNT):
        n, ms = gdn_timing_read(k)
        if n:
            out[KERNEL_NAMES[k]] = (n, ms)
    return out
