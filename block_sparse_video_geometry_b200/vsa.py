"""ctypes binding of libvsa (C ABI in include/vsa.h).

Argument marshalling only: every step of the computation runs in the CUDA
library. torch tensors are used as device buffers and torch streams as CUDA
streams: `stream` is a torch stream or a CUDA handle (0: the legacy default
stream), None torch's current stream, so that a call stands in order with the
torch operations around it. The library is loaded on first use; if it is missing
the call raises, there is no fallback path.
"""

from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libvsa.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE_TOO_SMALL, ERR_CUDA, ERR_TIMEOUT, ERR_NOT_UPLOADED = range(7)
SEG_TEXT, SEG_REF_IMAGE, SEG_REF_AUDIO, SEG_OTHER_COND, SEG_VIDEO = range(5)
SELECT_TOPK, SELECT_ADAPTIVE = 0, 1
SINK_EXACT_KV, SINK_EXACT_KV_AND_ROWS, SINK_OFF = 0, 1, 2
COARSE_MEAN, COARSE_REWEIGHT = 0, 1
OUT_F32, OUT_BF16 = 0, 1
DTYPE_F32, DTYPE_BF16, DTYPE_F16 = 0, 1, 2
ROPE_ADJACENT, ROPE_HALVES = 0, 1
MASK_FULL, MASK_CAUSAL = 0, 1
TILE, HEAD_DIM = 64, 128
MAX_NORM_WIDTH = 16384
MAX_EXTRA_TOKENS = 64


class VSAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = "%s: %s (status %d)" % (where, status_string(status), status)
        if status == ERR_CUDA:
            msg += ": " + lib().vsa_last_error_detail().decode()
        super().__init__(msg)


class Segment(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("grid_t", ctypes.c_int32), ("grid_h", ctypes.c_int32),
                ("grid_w", ctypes.c_int32), ("start", ctypes.c_int64), ("length", ctypes.c_int64)]


class Params(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("keep", ctypes.c_float), ("tau", ctypes.c_float),
                ("sink", ctypes.c_int32), ("scale", ctypes.c_float), ("coarse", ctypes.c_int32),
                ("extra_tokens", ctypes.c_int32)]


class LayoutInfo(ctypes.Structure):
    _fields_ = [("seq_len", ctypes.c_int64), ("n_cond_tiles", ctypes.c_int32),
                ("n_video_tiles", ctypes.c_int32), ("n_tiles", ctypes.c_int32),
                ("grid_t", ctypes.c_int32), ("grid_h", ctypes.c_int32), ("grid_w", ctypes.c_int32),
                ("video_start", ctypes.c_int64), ("device_bytes", ctypes.c_size_t)]


class Rope(ctypes.Structure):
    _fields_ = [("dim_t", ctypes.c_int32), ("dim_h", ctypes.c_int32), ("dim_w", ctypes.c_int32),
                ("pairing", ctypes.c_int32), ("theta", ctypes.c_double), ("scale_t", ctypes.c_double),
                ("scale_h", ctypes.c_double), ("scale_w", ctypes.c_double)]


class Mask(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("documents", ctypes.c_int32), ("scale", ctypes.c_float),
                ("softcap", ctypes.c_float)]


class MaskTerms(ctypes.Structure):
    _fields_ = [("doc_q", ctypes.c_void_p), ("doc_k", ctypes.c_void_p), ("doc_q_stride_b", ctypes.c_int64),
                ("doc_k_stride_b", ctypes.c_int64), ("prefix", ctypes.c_void_p), ("slopes", ctypes.c_void_p)]


_lib = None
_P = ctypes.c_void_p
_I32, _I64, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_V = ctypes.c_void_p      # a vsa_view, passed as the bytes of the struct

_SIGNATURES = {
    "vsa_layout_build": (_I32, [ctypes.POINTER(Segment), _I32, _I64, _P, _SZ, _P, ctypes.POINTER(_P)]),
    "vsa_layout_upload": (_I32, [_P, _P, _SZ, _P]),
    "vsa_layout_query": (_I32, [_P, ctypes.POINTER(LayoutInfo)]),
    "vsa_layout_copy_tables": (_I32, [_P, _P, _P, _P, _P]),
    "vsa_layout_free": (None, [_P]),
    "vsa_select_kmax": (_I32, [_P, ctypes.POINTER(Params), ctypes.POINTER(_I32)]),
    "vsa_coarse_select_workspace_size": (_I32, [_P, _I32, _I32, ctypes.POINTER(Params), ctypes.POINTER(_SZ)]),
    "vsa_coarse_select": (_I32, [_P, ctypes.POINTER(Params), _I32, _I32, _P, _P, _P, _I64, _I64, _I64,
                                 _P, _P, _P, _P, _SZ, _P]),
    "vsa_coarse_select_noalloc": (_I32, [_P, ctypes.POINTER(Params), _I32, _I32, _P, _P, _P, _I64, _I64, _I64,
                                         _P, _P, _P, _P]),
    "vsa_coarse_select_workspace_init": (_I32, [_P, _P]),
    "vsa_coarse_select_status": (_I32, [_P, _P]),
    "vsa_coarse_select_failed_calls": (_I32, [_P, _P, ctypes.POINTER(ctypes.c_uint32)]),
    "vsa_coarse_select_noalloc_status": (_I32, [_P]),
    "vsa_debug_inject_select_wait_timeout": (_I32, [ctypes.c_uint64]),
    "vsa_sparse_attn_workspace_size": (_I32, [_P, _I32, _I32, ctypes.POINTER(Params), ctypes.POINTER(_SZ)]),
    "vsa_sparse_attn_fwd": (_I32, [_P, ctypes.POINTER(Params), _I32, _I32, _P, _P, _P, _I64, _I64, _I64,
                                   _P, _I64, _I64, _I64, _I64, _P, _P, _I32, _P, _P, _P, _P, _I32, _I64, _I64,
                                   _I64, _P, _SZ, _P]),
    "vsa_extra_tokens_workspace_size": (_I32, [_P, _I32, _I32, ctypes.POINTER(Params), ctypes.POINTER(_SZ)]),
    "vsa_extra_tokens_select": (_I32, [_P, ctypes.POINTER(Params), _I32, _I32, _P, _P, _I64, _I64, _I64,
                                       _P, _P, _I32, _P, _P, _P, _SZ, _P]),
    "vsa_extra_tokens_status": (_I32, [_P, _P]),
    "vsa_sparse_attn_bwd_workspace_size": (_I32, [_P, _I32, _I32, ctypes.POINTER(Params), ctypes.POINTER(_SZ)]),
    "vsa_sparse_attn_bwd": (_I32, [_P, ctypes.POINTER(Params), _I32, _I32, _P, _P, _P, _I64, _I64, _I64,
                                   _P, _I64, _I64, _I64, _I64, _P, _P, _I32, _P, _P, _I64, _I64, _I64,
                                   _P, _P, _P, _I64, _I64, _I64, _P, _I64, _I64, _I64, _I64, _P, _SZ, _P]),
    "vsa_sparse_attn_bwd_status": (_I32, [_P, _P]),
    "vsa_sparse_attn_status": (_I32, [_P, _P]),
    "vsa_sparse_attn_workspace_init": (_I32, [_P, _P]),
    "vsa_sparse_attn_failed_calls": (_I32, [_P, _P, ctypes.POINTER(ctypes.c_uint32)]),
    "vsa_debug_inject_wait_timeout": (_I32, [ctypes.c_uint64]),
    "vsa_rope_positions": (_I32, [_P, _I32, _I32, _I32, _P, _P]),
    "vsa_rope_fwd": (_I32, [ctypes.POINTER(Rope), _I32, _I64, _P, _I64, _V, _V, _V, _V, _P]),
    "vsa_rope_bwd": (_I32, [ctypes.POINTER(Rope), _I32, _I64, _P, _I64, _V, _V, _V, _V, _P]),
    "vsa_layer_norm_fwd": (_I32, [_I32, _I64, _I32, _V, _P, _P, _I32, ctypes.c_float, _V, _P, _P, _P]),
    "vsa_layer_norm_bwd_workspace_size": (_I32, [_I32, _I64, _I32, _I32, ctypes.POINTER(_SZ)]),
    "vsa_layer_norm_bwd": (_I32, [_I32, _I64, _I32, _V, _V, _P, _I32, _P, _P, _V, _P, _P, _P, _SZ, _P]),
    "vsa_masked_attn_workspace_size": (_I32, [ctypes.POINTER(Mask), _I32, _I32, _I32, _I32, _I32,
                                              ctypes.POINTER(_SZ)]),
    "vsa_masked_attn_fwd": (_I32, [ctypes.POINTER(Mask), ctypes.POINTER(MaskTerms), _I32, _I32, _I32, _V, _V, _V, _V,
                                   _P, _P, _SZ, _P]),
    "vsa_masked_attn_bwd_workspace_size": (_I32, [ctypes.POINTER(Mask), _I32, _I32, _I32, _I32, _I32,
                                                  ctypes.POINTER(_SZ)]),
    "vsa_masked_attn_bwd": (_I32, [ctypes.POINTER(Mask), ctypes.POINTER(MaskTerms), _I32, _I32, _I32, _V, _V, _V, _V,
                                   _P, _V, _V, _V, _V, _P, _SZ, _P]),
    "vsa_masked_attn_status": (_I32, [_P, _P]),
    "vsa_status_string": (ctypes.c_char_p, [_I32]),
    "vsa_version": (_I32, []),
    "vsa_last_error_detail": (ctypes.c_char_p, []),
}


def lib() -> ctypes.CDLL:
    """Loads libvsa.so (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libvsa.so is missing: build it with "
                               "`python -m block_sparse_video_geometry_b200.build_ext`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().vsa_status_string(status).decode()


def version() -> int:
    return lib().vsa_version()


def _check(status: int, where: str) -> None:
    if status != OK:
        raise VSAError(status, where)


def make_params(mode: int = SELECT_TOPK, keep: float = 0.1, tau: float = 1.0,
                sink: int = SINK_EXACT_KV, scale: float = 0.0, coarse: int = 0, extra_tokens: int = 0) -> Params:
    return Params(mode, keep, tau, sink, scale, coarse, extra_tokens)


def _stream_handle(stream, index=None) -> int:
    """CUDA stream of a call; None: torch's current stream of device `index` (of the current device)."""
    if stream is None:
        import torch
        if index is None:
            if not torch.cuda.is_initialized():
                return 0             # nothing but the default stream yet
            index = torch.cuda.current_device()
        # the handle alone: torch.cuda.current_stream makes an object of it, 2 us of a call of 10
        return torch._C._cuda_getCurrentRawStream(index)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream        # torch.cuda.Stream


class Layout:
    """Owned vsa_layout handle. `segments` is a list of (kind, start, length,
    (t, h, w) or None) in sequence order."""

    def __init__(self, segments, seq_len: int):
        arr = (Segment * len(segments))()
        for i, (kind, start, length, grid) in enumerate(segments):
            t, h, w = grid if grid is not None else (0, 0, 0)
            arr[i] = Segment(kind, t, h, w, start, length)
        handle = _P()
        _check(lib().vsa_layout_build(arr, len(segments), seq_len, None, 0, None, ctypes.byref(handle)),
               "vsa_layout_build")
        self._h = handle
        self.info = LayoutInfo()
        _check(lib().vsa_layout_query(self._h, ctypes.byref(self.info)), "vsa_layout_query")
        self._dev = None

    @property
    def handle(self):
        return self._h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h and _lib is not None:
            _lib.vsa_layout_free(h)
            self._h = None

    def tables(self):
        """Host copies: perm [n_tiles, 64], inv [S], tile_count [n_tiles], tile_kind [n_tiles]."""
        i = self.info
        perm = np.empty(i.n_tiles * TILE, dtype=np.int32)
        inv = np.empty(i.seq_len, dtype=np.int32)
        cnt = np.empty(i.n_tiles, dtype=np.int32)
        kind = np.empty(i.n_tiles, dtype=np.int32)
        _check(lib().vsa_layout_copy_tables(self._h, perm.ctypes.data, inv.ctypes.data, cnt.ctypes.data,
                                            kind.ctypes.data), "vsa_layout_copy_tables")
        return perm.reshape(-1, TILE), inv, cnt, kind

    def upload(self, dev_buf, stream=None) -> None:
        """Uploads the device tables into `dev_buf` (a torch uint8 CUDA tensor
        of at least info.device_bytes bytes, kept alive by this object)."""
        _check(lib().vsa_layout_upload(self._h, dev_buf.data_ptr(), dev_buf.numel() * dev_buf.element_size(),
                                       _stream_handle(stream)), "vsa_layout_upload")
        self._dev = dev_buf

    def kmax(self, params: Params) -> int:
        k = _I32()
        _check(lib().vsa_select_kmax(self._h, ctypes.byref(params), ctypes.byref(k)), "vsa_select_kmax")
        return k.value

    def coarse_select_workspace_size(self, B: int, H: int, params: Params) -> int:
        n = _SZ()
        _check(lib().vsa_coarse_select_workspace_size(self._h, B, H, ctypes.byref(params), ctypes.byref(n)),
               "vsa_coarse_select_workspace_size")
        return n.value

    def extra_tokens_workspace_size(self, B: int, H: int, params: Params) -> int:
        n = _SZ()
        _check(lib().vsa_extra_tokens_workspace_size(self._h, B, H, ctypes.byref(params), ctypes.byref(n)),
               "vsa_extra_tokens_workspace_size")
        return n.value

    def sparse_attn_bwd_workspace_size(self, B: int, H: int, params: Params) -> int:
        n = _SZ()
        _check(lib().vsa_sparse_attn_bwd_workspace_size(self._h, B, H, ctypes.byref(params), ctypes.byref(n)),
               "vsa_sparse_attn_bwd_workspace_size")
        return n.value

    def sparse_attn_workspace_size(self, B: int, H: int, params: Params) -> int:
        n = _SZ()
        _check(lib().vsa_sparse_attn_workspace_size(self._h, B, H, ctypes.byref(params), ctypes.byref(n)),
               "vsa_sparse_attn_workspace_size")
        return n.value


def _qkv_strides(q, k, v):
    if not (q.stride() == k.stride() == v.stride()):
        raise ValueError("q, k and v must share strides")
    if q.dim() != 4 or q.shape[-1] != HEAD_DIM or q.stride(-1) != 1:
        raise ValueError("q, k, v must be [B, S, H, 128] with a contiguous head dim")
    return q.stride(0), q.stride(1), q.stride(2)


def coarse_select(layout: Layout, params: Params, q, k, v, idx, cnt, o_coarse, workspace, stream=None) -> None:
    """vsa_coarse_select on torch tensors (bf16 q/k/v [B, S, H, 128])."""
    B, S, H, _ = q.shape
    sb, ss, sh = _qkv_strides(q, k, v)
    _check(lib().vsa_coarse_select(layout.handle, ctypes.byref(params), B, H, q.data_ptr(), k.data_ptr(),
                                   v.data_ptr(), sb, ss, sh, idx.data_ptr(), cnt.data_ptr(),
                                   o_coarse.data_ptr(), workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(), _stream_handle(stream)),
           "vsa_coarse_select")


def coarse_select_noalloc(layout: Layout, params: Params, q, k, v, idx, cnt, o_coarse, stream=None) -> None:
    """vsa_coarse_select_noalloc: the selection call for callers that cannot
    provide scratch memory (the library's built-in 32 MiB buffer is used)."""
    B, S, H, _ = q.shape
    sb, ss, sh = _qkv_strides(q, k, v)
    _check(lib().vsa_coarse_select_noalloc(layout.handle, ctypes.byref(params), B, H, q.data_ptr(), k.data_ptr(),
                                           v.data_ptr(), sb, ss, sh, idx.data_ptr(), cnt.data_ptr(),
                                           o_coarse.data_ptr(), _stream_handle(stream)),
           "vsa_coarse_select_noalloc")


def coarse_select_workspace_init(workspace, stream=None) -> None:
    """Zeroes the selection workspace header (and its count of failed calls)."""
    _check(lib().vsa_coarse_select_workspace_init(workspace.data_ptr(), _stream_handle(stream)),
           "vsa_coarse_select_workspace_init")


def coarse_select_status(workspace, stream=None) -> int:
    """Synchronises the stream and returns the selection call's status word (OK or ERR_TIMEOUT)."""
    return lib().vsa_coarse_select_status(workspace.data_ptr(), _stream_handle(stream))


def coarse_select_failed_calls(workspace, stream=None) -> int:
    """Synchronises the stream; selection calls that recorded an error since the header was zeroed."""
    n = ctypes.c_uint32()
    _check(lib().vsa_coarse_select_failed_calls(workspace.data_ptr(), _stream_handle(stream), ctypes.byref(n)),
           "vsa_coarse_select_failed_calls")
    return n.value


def coarse_select_noalloc_status(stream=None) -> int:
    """coarse_select_status of the built-in buffer of coarse_select_noalloc (current device)."""
    return lib().vsa_coarse_select_noalloc_status(_stream_handle(stream))


def extra_tokens_select(layout: Layout, params: Params, q, k, idx, cnt, kmax: int, extra_idx, extra_cnt,
                        workspace, stream=None) -> None:
    """vsa_extra_tokens_select: extra_idx int32 [B, H, n_tiles, E], extra_cnt int32 [B, H, n_tiles] out."""
    B, S, H, _ = q.shape
    sb, ss, sh = _qkv_strides(q, k, k)
    _check(lib().vsa_extra_tokens_select(layout.handle, ctypes.byref(params), B, H, q.data_ptr(), k.data_ptr(),
                                         sb, ss, sh, idx.data_ptr(), cnt.data_ptr(), kmax, extra_idx.data_ptr(),
                                         extra_cnt.data_ptr(), workspace.data_ptr(),
                                         workspace.numel() * workspace.element_size(), _stream_handle(stream)),
           "vsa_extra_tokens_select")


def extra_tokens_status(workspace, stream=None) -> int:
    """Synchronises the stream; the status word of the extra-token selection (OK or ERR_TIMEOUT)."""
    return lib().vsa_extra_tokens_status(workspace.data_ptr(), _stream_handle(stream))


def sparse_attn_fwd(layout: Layout, params: Params, q, k, v, g, idx, cnt, kmax: int, o_coarse, out,
                    workspace, stream=None, extra_idx=None, extra_cnt=None) -> None:
    """vsa_sparse_attn_fwd on torch tensors; out is float32 or bfloat16 [B, S, H, 128];
    g is bf16 [B, S, H] (one gate per token and head) or [B, S, H, 128] (one per channel);
    extra_idx / extra_cnt from extra_tokens_select when params.extra_tokens > 0."""
    import torch
    B, S, H, _ = q.shape
    if g.dim() == 3:
        g_sd = 0
    elif g.dim() == 4 and g.shape[3] == HEAD_DIM:
        g_sd = g.stride(3)
    else:
        raise ValueError("g must be [B, S, H] or [B, S, H, 128]")
    sb, ss, sh = _qkv_strides(q, k, v)
    if out.dtype == torch.float32:
        od = OUT_F32
    elif out.dtype == torch.bfloat16:
        od = OUT_BF16
    else:
        raise ValueError("out must be float32 or bfloat16")
    _check(lib().vsa_sparse_attn_fwd(layout.handle, ctypes.byref(params), B, H, q.data_ptr(), k.data_ptr(),
                                     v.data_ptr(), sb, ss, sh, g.data_ptr(), g.stride(0), g.stride(1),
                                     g.stride(2), g_sd, idx.data_ptr(), cnt.data_ptr(), kmax, o_coarse.data_ptr(),
                                     None if extra_idx is None else extra_idx.data_ptr(),
                                     None if extra_cnt is None else extra_cnt.data_ptr(),
                                     out.data_ptr(), od, out.stride(0), out.stride(1), out.stride(2),
                                     workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                     _stream_handle(stream)), "vsa_sparse_attn_fwd")


def sparse_attn_bwd(layout: Layout, params: Params, q, k, v, g, idx, cnt, kmax: int, o_coarse, dout,
                    dq, dk, dv, dg, workspace, stream=None) -> None:
    """vsa_sparse_attn_bwd on torch tensors: dout bf16 [B, S, H, 128]; dq, dk, dv
    float32 [B, S, H, 128] and dg float32 shaped like g (outputs)."""
    B, S, H, _ = q.shape
    sb, ss, sh = _qkv_strides(q, k, v)
    if dout.dim() != 4 or dout.stride(-1) != 1:
        raise ValueError("dout must be [B, S, H, 128] with a contiguous head dim")
    if not (dq.stride() == dk.stride() == dv.stride()):
        raise ValueError("dq, dk and dv must share strides")
    g_sd = g.stride(3) if g.dim() == 4 else 0
    dg_sd = dg.stride(3) if dg.dim() == 4 else 0
    _check(lib().vsa_sparse_attn_bwd(layout.handle, ctypes.byref(params), B, H, q.data_ptr(), k.data_ptr(),
                                     v.data_ptr(), sb, ss, sh, g.data_ptr(), g.stride(0), g.stride(1), g.stride(2),
                                     g_sd, idx.data_ptr(), cnt.data_ptr(), kmax, o_coarse.data_ptr(),
                                     dout.data_ptr(), dout.stride(0), dout.stride(1), dout.stride(2),
                                     dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dq.stride(0), dq.stride(1),
                                     dq.stride(2), dg.data_ptr(), dg.stride(0), dg.stride(1), dg.stride(2), dg_sd,
                                     workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                     _stream_handle(stream)), "vsa_sparse_attn_bwd")


def sparse_attn_bwd_status(workspace, stream=None) -> int:
    """Synchronises the stream; the backward pass's status (OK or ERR_TIMEOUT)."""
    return lib().vsa_sparse_attn_bwd_status(workspace.data_ptr(), _stream_handle(stream))


def sparse_attn_status(workspace, stream=None) -> int:
    """Synchronises the stream and returns the kernel's status word (OK or ERR_TIMEOUT)."""
    return lib().vsa_sparse_attn_status(workspace.data_ptr(), _stream_handle(stream))


def sparse_attn_workspace_init(workspace, stream=None) -> None:
    """Zeroes the attention workspace header (and its count of failed calls)."""
    _check(lib().vsa_sparse_attn_workspace_init(workspace.data_ptr(), _stream_handle(stream)),
           "vsa_sparse_attn_workspace_init")


def sparse_attn_failed_calls(workspace, stream=None) -> int:
    """Synchronises the stream; number of calls that recorded an error since the header was zeroed."""
    n = ctypes.c_uint32()
    _check(lib().vsa_sparse_attn_failed_calls(workspace.data_ptr(), _stream_handle(stream), ctypes.byref(n)),
           "vsa_sparse_attn_failed_calls")
    return n.value


# ---------------------------------------------------------------- operators around the sparse call
_DTYPES = {}


def _dtype(t) -> int:
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16})
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError("tensors must be float32, bfloat16 or float16, got %s" % t.dtype)
    return code


_VIEW = struct.Struct("@Pqqqii")      # vsa_view: data, stride_b, stride_s, stride_h, heads, dtype


def view_bytes(data: int, stride_b: int, stride_s: int, stride_h: int, heads: int, dtype: int) -> bytes:
    """A vsa_view as bytes, which ctypes passes by address."""
    return _VIEW.pack(data, stride_b, stride_s, stride_h, heads, dtype)


def _view(t) -> bytes:
    """The vsa_view of a [..., width] tensor of 2 ([S, width]), 3 ([B, S, width]) or 4 dimensions."""
    shape, st = t.shape, t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError("the last dimension must be contiguous")
    n = len(st)
    if n == 4:
        return _VIEW.pack(t.data_ptr(), st[0], st[1], st[2], shape[2], _dtype(t))
    if n == 3:
        return _VIEW.pack(t.data_ptr(), st[0], st[1], 0, 1, _dtype(t))
    if n == 2:
        return _VIEW.pack(t.data_ptr(), 0, st[0], 0, 1, _dtype(t))
    raise ValueError("tensors must have 2, 3 or 4 dimensions")


def _run(name, tensors, stream, *args) -> None:
    """Calls a library function with the tensors' device current and the stream as last argument; they must share
    one CUDA device."""
    import torch
    index = tensors[0].get_device()
    if index < 0:
        raise ValueError("tensors must be on a CUDA device, got %s" % tensors[0].device)
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors must be on one device, got %s and %s" % (tensors[0].device, t.device))
    fn, handle = getattr(lib(), name), _stream_handle(stream, index)
    if index == torch.cuda.current_device():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            status = fn(*args, handle)
    if status != OK:
        raise VSAError(status, name)


def make_rope(dims=(44, 42, 42), theta: float = 10000.0, scale=(1.0, 1.0, 1.0),
              pairing: int = ROPE_ADJACENT) -> Rope:
    """Rotary positions with `dims` (time, height, width) channels of the head's 128; see vsa_rope in vsa.h."""
    if len(dims) != 3 or len(scale) != 3:
        raise ValueError("dims and scale hold one value per axis: time, height, width")
    return Rope(*dims, pairing, theta, *scale)


def rope_positions(layout: Layout, pos, origin=(0, 0, 0), stream=None) -> None:
    """vsa_rope_positions: fills pos, int32 [seq_len, 3], with the positions of the layout's tokens."""
    import torch
    if pos.dtype != torch.int32 or tuple(pos.shape) != (layout.info.seq_len, 3) or not pos.is_contiguous():
        raise ValueError("pos must be a contiguous int32 [seq_len, 3] tensor")
    _run("vsa_rope_positions", (pos,), stream, layout.handle, *origin, pos.data_ptr())


def _rope_call(name, rope, pos, q, k, q_out, k_out, stream):
    import torch
    shape = q.shape
    if len(shape) != 4 or shape[3] != HEAD_DIM or q_out.shape != shape:
        raise ValueError("q and its output must be [B, S, H, 128]")
    B, S = shape[0], shape[1]
    if (k is None) != (k_out is None):
        raise ValueError("k and its output come together")
    if k is not None:
        shape = k.shape
        if len(shape) != 4 or shape[0] != B or shape[1] != S or shape[3] != HEAD_DIM or k_out.shape != shape:
            raise ValueError("k and its output must be [B, S, H, 128] with q's B and S")
    shape, strides = pos.shape, pos.stride()
    if pos.dtype != torch.int32 or shape not in ((S, 3), (B, S, 3)) or strides[-1] != 1 or (S > 1 and strides[-2] != 3):
        raise ValueError("pos must be int32 [S, 3] or [B, S, 3], contiguous in its last two dimensions")
    _run(name, (q, pos, k, q_out, k_out), stream, ctypes.byref(rope), B, S, pos.data_ptr(),
         strides[0] if len(strides) == 3 else 0, _view(q), None if k is None else _view(k), _view(q_out),
         None if k is None else _view(k_out))


def rope_fwd(rope: Rope, pos, q, k, q_out, k_out, stream=None) -> None:
    """vsa_rope_fwd on torch tensors: q [B, S, Hq, 128] and k [B, S, Hk, 128] (or None, with k_out None) rotated
    by their positions, int32 [S, 3] or [B, S, 3], into q_out and k_out (which may be q and k)."""
    _rope_call("vsa_rope_fwd", rope, pos, q, k, q_out, k_out, stream)


def rope_bwd(rope: Rope, pos, dq_out, dk_out, dq, dk, stream=None) -> None:
    """vsa_rope_bwd on torch tensors: dq and dk from the gradients of rope_fwd's outputs."""
    _rope_call("vsa_rope_bwd", rope, pos, dq_out, dk_out, dq, dk, stream)


def _norm_shape(x):
    """(B, S, heads, width) of x [S, width], [B, S, width] or [B, S, heads, width]."""
    s = x.shape
    if not 2 <= len(s) <= 4:
        raise ValueError("x must be [S, width], [B, S, width] or [B, S, heads, width]")
    return (1, s[0], 1, s[1]) if len(s) == 2 else (s[0], s[1], 1, s[2]) if len(s) == 3 else s


def _vector(t, n, what, dtypes):
    """Address of a contiguous [n] tensor of one of the types, or None."""
    if t is None:
        return None
    if t.dtype not in dtypes or t.numel() != n or not t.is_contiguous():
        raise ValueError("%s must be contiguous with %d elements of %s" % (what, n, " or ".join(map(str, dtypes))))
    return t.data_ptr()


def layer_norm_fwd(x, weight, bias, eps: float, y, mean=None, rstd=None, stream=None) -> None:
    """vsa_layer_norm_fwd on torch tensors: y = layer norm of x over its last dimension; weight and bias [width]
    in x's type or float32 (both of one type), or None; mean and rstd float32 of x's leading shape, or None."""
    import torch
    B, S, H, N = _norm_shape(x)
    if y.shape != x.shape or y.dtype != x.dtype:
        raise ValueError("y must have x's shape and type")
    wt = weight if weight is not None else bias
    types = (x.dtype, torch.float32)
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError("weight and bias must have one type")
    f32 = (torch.float32,)
    _run("vsa_layer_norm_fwd", (x, weight, bias, y, mean, rstd), stream, B, S, N, _view(x),
         _vector(weight, N, "weight", types), _vector(bias, N, "bias", types), 0 if wt is None else _dtype(wt), eps,
         _view(y), _vector(mean, B * S * H, "mean", f32), _vector(rstd, B * S * H, "rstd", f32))


def layer_norm_bwd_workspace_size(x) -> int:
    """Workspace bytes of layer_norm_bwd for an x of this shape."""
    B, S, H, N = _norm_shape(x)
    n = _SZ()
    _check(lib().vsa_layer_norm_bwd_workspace_size(B, S, H, N, ctypes.byref(n)), "vsa_layer_norm_bwd_workspace_size")
    return n.value


def layer_norm_bwd(dy, x, weight, mean, rstd, dx, dweight, dbias, workspace, stream=None) -> None:
    """vsa_layer_norm_bwd on torch tensors: dx (x's type or float32) from dy (x's type or float32), x, weight and
    the forward's mean and rstd; dweight and dbias float32 [width] out, or None."""
    import torch
    B, S, H, N = _norm_shape(x)
    if dy.shape != x.shape or dx.shape != x.shape:
        raise ValueError("dy and dx must have x's shape")
    f32 = (torch.float32,)
    _run("vsa_layer_norm_bwd", (x, dy, weight, mean, rstd, dx, dweight, dbias, workspace), stream, B, S, N, _view(dy),
         _view(x), _vector(weight, N, "weight", (x.dtype, torch.float32)), 0 if weight is None else _dtype(weight),
         _vector(mean, B * S * H, "mean", f32), _vector(rstd, B * S * H, "rstd", f32), _view(dx),
         _vector(dweight, N, "dweight", f32), _vector(dbias, N, "dbias", f32), workspace.data_ptr(),
         workspace.numel() * workspace.element_size())


def make_mask(causal: bool = False, softcap: float = 0.0, scale: float = 0.0, documents: bool = False) -> Mask:
    """Parameters of the dense masked attention; see vsa_mask in vsa.h. MaskedAttention sets `documents` by itself."""
    return Mask(MASK_CAUSAL if causal else MASK_FULL, int(documents), scale, softcap)


def _mask_terms(mask, B, Sq, Sk, Hq, doc_q, doc_k, prefix, slopes):
    import torch
    if (doc_q is None) != (doc_k is None) or bool(mask.documents) != (doc_q is not None):
        raise ValueError("doc_q and doc_k come together, with a mask of documents")
    t = MaskTerms()
    for name, d, n in (("doc_q", doc_q, Sq), ("doc_k", doc_k, Sk)):
        if d is None:
            continue
        if d.dtype != torch.int32 or tuple(d.shape) != (B, n) or (n > 1 and d.stride(1) != 1):
            raise ValueError("%s must be int32 [B, %d], contiguous in its last dimension" % (name, n))
        setattr(t, name, d.data_ptr())
        setattr(t, name + "_stride_b", d.stride(0))
    t.prefix = _vector(prefix, B, "prefix", (torch.int32,))
    t.slopes = _vector(slopes, Hq, "slopes", (torch.float32,))
    return t


def _attn_shapes(q, k, v):
    if q.dim() != 4 or k.dim() != 4 or k.shape != v.shape or q.shape[-1] != HEAD_DIM or k.shape[-1] != HEAD_DIM \
            or q.shape[0] != k.shape[0] or k.shape[2] == 0 or q.shape[2] % k.shape[2]:
        raise ValueError("q must be [B, Sq, Hq, 128], k and v [B, Sk, Hk, 128] with Hq a multiple of Hk")
    return q.shape[0], q.shape[1], k.shape[1], q.shape[2], k.shape[2]


def masked_attn_workspace_size(mask: Mask, B: int, Sq: int, Sk: int, Hq: int, Hk: int) -> int:
    n = _SZ()
    _check(lib().vsa_masked_attn_workspace_size(ctypes.byref(mask), B, Sq, Sk, Hq, Hk, ctypes.byref(n)),
           "vsa_masked_attn_workspace_size")
    return n.value


def masked_attn_fwd(mask: Mask, q, k, v, out, lse, workspace, doc_q=None, doc_k=None, prefix=None, slopes=None,
                    stream=None) -> None:
    """vsa_masked_attn_fwd on torch tensors: bf16 q, out [B, Sq, Hq, 128], k, v [B, Sk, Hk, 128], lse float32
    [B, Hq, Sq]; doc_q int32 [B, Sq] and doc_k int32 [B, Sk] (mask.documents), prefix int32 [B], slopes float32 [Hq]."""
    import torch
    B, Sq, Sk, Hq, Hk = _attn_shapes(q, k, v)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    terms = _mask_terms(mask, B, Sq, Sk, Hq, doc_q, doc_k, prefix, slopes)
    _run("vsa_masked_attn_fwd", (q, k, v, out, lse, workspace, doc_q, doc_k, prefix, slopes), stream,
         ctypes.byref(mask), ctypes.byref(terms), B, Sq, Sk, _view(q), _view(k), _view(v), _view(out),
         _vector(lse, B * Hq * Sq, "lse", (torch.float32,)), workspace.data_ptr(),
         workspace.numel() * workspace.element_size())


def masked_attn_bwd_workspace_size(mask: Mask, B: int, Sq: int, Sk: int, Hq: int, Hk: int) -> int:
    n = _SZ()
    _check(lib().vsa_masked_attn_bwd_workspace_size(ctypes.byref(mask), B, Sq, Sk, Hq, Hk, ctypes.byref(n)),
           "vsa_masked_attn_bwd_workspace_size")
    return n.value


def masked_attn_bwd(mask: Mask, q, k, v, out, lse, dout, dq, dk, dv, workspace, doc_q=None, doc_k=None, prefix=None,
                    slopes=None, stream=None) -> None:
    """vsa_masked_attn_bwd on torch tensors: bf16 dq, dk, dv shaped like q, k, v from masked_attn_fwd's inputs, its out
    and lse, and dout (bf16, out's shape)."""
    import torch
    B, Sq, Sk, Hq, Hk = _attn_shapes(q, k, v)
    if out.shape != q.shape or dout.shape != q.shape or dq.shape != q.shape:
        raise ValueError("out, dout and dq must have q's shape")
    if dk.shape != k.shape or dv.shape != k.shape:
        raise ValueError("dk and dv must have k's shape")
    terms = _mask_terms(mask, B, Sq, Sk, Hq, doc_q, doc_k, prefix, slopes)
    _run("vsa_masked_attn_bwd", (q, k, v, out, lse, dout, dq, dk, dv, workspace, doc_q, doc_k, prefix, slopes),
         stream, ctypes.byref(mask), ctypes.byref(terms), B, Sq, Sk, _view(q), _view(k), _view(v), _view(out),
         _vector(lse, B * Hq * Sq, "lse", (torch.float32,)), _view(dout), _view(dq), _view(dk), _view(dv),
         workspace.data_ptr(), workspace.numel() * workspace.element_size())


def masked_attn_status(workspace, stream=None) -> int:
    """Synchronises the stream; the status of the latest masked attention call on `workspace` (OK or ERR_TIMEOUT)."""
    import torch
    with torch.cuda.device(workspace.device):
        return lib().vsa_masked_attn_status(workspace.data_ptr(), _stream_handle(stream, workspace.get_device()))


def _torch_stream(handle, device):
    """The torch stream of a CUDA handle."""
    import torch
    here = torch.cuda.current_stream(device)
    if handle == here.cuda_stream:
        return here
    return torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)


def _empty(shape, dtype, device, handle):
    """A tensor that a call on the stream `handle` writes: out of that stream's memory, which nothing queued elsewhere
    still uses, and kept while the current stream, where the caller goes on with it, still reads it."""
    import torch
    if handle == _stream_handle(None, device.index):
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_torch_stream(handle, device)):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


class MaskedAttention:
    """Dense attention of one shape and mask with its workspaces (allocated by the first call that needs them, so
    run one call before a capture, and keep the object while its graph is replayed). Calls of one object share them:
    for calls on two streams, or graphs that may run at once, make one object each. Outputs that a call allocates are
    written on its `stream`: a caller that reads them on another one waits for it, as for any torch operation on a side
    stream. A stream that is given as a handle outlives the object and the outputs."""

    def __init__(self, mask: Mask, B: int, Sq: int, Sk: int, Hq: int, Hk: int, device="cuda"):
        import torch
        self.shape, self.device, self._made = (B, Sq, Sk, Hq, Hk), device, torch.device(device)
        self.masks = [Mask(mask.mode, d, mask.scale, mask.softcap) for d in (0, 1)]
        for m in self.masks:
            masked_attn_workspace_size(m, *self.shape)       # refuses a shape or mask at once
        self.ws_fwd, self.ws_bwd = {}, {}      # by whether documents are given
        self._kept_for = {}                    # id of a workspace -> handles of the streams that it is kept for

    def _begin(self, q, k, v, stream) -> int:
        """Checks a call's tensors; the handle of its stream."""
        if _attn_shapes(q, k, v) != self.shape:
            raise ValueError("made for B, Sq, Sk, Hq, Hk = %s, called with %s" % (self.shape, _attn_shapes(q, k, v)))
        if self._made.type != q.device.type or self._made.index not in (None, q.device.index):
            raise ValueError("made for device %s, called with tensors on %s" % (self.device, q.device))
        return _stream_handle(stream, q.device.index)

    def _workspace(self, held, size, documents, device, handle):
        import torch
        ws = held.get(documents)
        if ws is None:
            ws = held[documents] = _empty(size(self.masks[documents], *self.shape), torch.uint8, device, handle)
            self._kept_for[id(ws)] = {handle}
        elif handle not in self._kept_for[id(ws)]:        # its memory outlives the object while that stream needs it
            ws.record_stream(_torch_stream(handle, device))
            self._kept_for[id(ws)].add(handle)
        return ws

    def forward(self, q, k, v, out=None, lse=None, doc_q=None, doc_k=None, prefix=None, slopes=None, stream=None):
        """masked_attn_fwd; returns (out, lse)."""
        import torch
        handle = self._begin(q, k, v, stream)
        B, Sq, _, Hq, _ = self.shape
        d = int(doc_q is not None)
        ws = self._workspace(self.ws_fwd, masked_attn_workspace_size, d, q.device, handle)
        if out is None:
            out = _empty(q.shape, q.dtype, q.device, handle)
        if lse is None:
            lse = _empty((B, Hq, Sq), torch.float32, q.device, handle)
        masked_attn_fwd(self.masks[d], q, k, v, out, lse, ws, doc_q, doc_k, prefix, slopes, handle)
        return out, lse

    def backward(self, q, k, v, out, lse, dout, dq=None, dk=None, dv=None, doc_q=None, doc_k=None, prefix=None,
                 slopes=None, stream=None):
        """masked_attn_bwd; returns (dq, dk, dv)."""
        handle = self._begin(q, k, v, stream)
        d = int(doc_q is not None)
        ws = self._workspace(self.ws_bwd, masked_attn_bwd_workspace_size, d, q.device, handle)
        dq, dk, dv = (_empty(x.shape, x.dtype, x.device, handle) if g is None else g
                      for g, x in ((dq, q), (dk, k), (dv, v)))
        masked_attn_bwd(self.masks[d], q, k, v, out, lse, dout, dq, dk, dv, ws, doc_q, doc_k, prefix, slopes, handle)
        return dq, dk, dv

    def status(self, stream=None) -> int:
        """Synchronises the stream (the one that the calls ran on); OK, or ERR_TIMEOUT where a bounded wait ran out and
        left the outputs of the latest forward or backward call (with documents or without, each for itself)
        incomplete."""
        for ws in (*self.ws_fwd.values(), *self.ws_bwd.values()):
            status = masked_attn_status(ws, stream)
            if status != OK:
                return status
        return OK


def debug_inject_wait_timeout(timeout_ns):
    """Test hook: while timeout_ns > 0, each sparse_attn_fwd runs into a bounded
    wait that nothing completes and reports ERR_TIMEOUT (see vsa.h); 0 disarms."""
    lib().vsa_debug_inject_wait_timeout(int(timeout_ns))


def debug_inject_select_wait_timeout(timeout_ns):
    """Test hook: while timeout_ns > 0, each coarse_select (mean coarse branch)
    runs into a bounded wait that nothing completes and reports ERR_TIMEOUT
    through coarse_select_status; 0 disarms."""
    lib().vsa_debug_inject_select_wait_timeout(int(timeout_ns))


class Forward:
    """Holds the buffers of one shape and runs the two calls of the forward
    pass (caller-owned torch buffers; no allocation inside the calls)."""

    def __init__(self, layout: Layout, params: Params, B: int, H: int, device="cuda",
                 out_dtype=None, stream=None):
        import torch
        self.layout, self.params, self.B, self.H = layout, params, B, H
        info = layout.info
        if layout._dev is None:
            buf = torch.empty(info.device_bytes, dtype=torch.uint8, device=device)
            layout.upload(buf, stream)
        self.kmax = layout.kmax(params)
        self.idx = torch.empty((B, H, info.n_tiles, self.kmax), dtype=torch.int32, device=device)
        self.cnt = torch.empty((B, H, info.n_tiles), dtype=torch.int32, device=device)
        self.o_coarse = torch.empty((B, H, info.n_tiles, HEAD_DIM), dtype=torch.float32, device=device)
        self.ws_select = torch.empty(layout.coarse_select_workspace_size(B, H, params), dtype=torch.uint8,
                                     device=device)
        self.ws_attn = torch.empty(layout.sparse_attn_workspace_size(B, H, params), dtype=torch.uint8,
                                   device=device)
        sparse_attn_workspace_init(self.ws_attn, stream)
        coarse_select_workspace_init(self.ws_select, stream)
        self.out_dtype = out_dtype or torch.float32
        self.stream = stream
        self.extra_idx = self.extra_cnt = self.ws_extra = None
        if params.extra_tokens > 0:
            self.extra_idx = torch.empty((B, H, info.n_tiles, params.extra_tokens), dtype=torch.int32, device=device)
            self.extra_cnt = torch.empty((B, H, info.n_tiles), dtype=torch.int32, device=device)
            self.ws_extra = torch.empty(layout.extra_tokens_workspace_size(B, H, params), dtype=torch.uint8,
                                        device=device)

    def __call__(self, q, k, v, g, out=None):
        import torch
        if out is None:
            out = torch.empty(q.shape, dtype=self.out_dtype, device=q.device)
        coarse_select(self.layout, self.params, q, k, v, self.idx, self.cnt, self.o_coarse, self.ws_select,
                      self.stream)
        if self.params.extra_tokens > 0:
            extra_tokens_select(self.layout, self.params, q, k, self.idx, self.cnt, self.kmax, self.extra_idx,
                                self.extra_cnt, self.ws_extra, self.stream)
        sparse_attn_fwd(self.layout, self.params, q, k, v, g, self.idx, self.cnt, self.kmax, self.o_coarse,
                        out, self.ws_attn, self.stream, self.extra_idx, self.extra_cnt)
        return out

    def pooled(self):
        """Pooled means [3, B, H, n_tiles, 128] left in the selection workspace (from byte 256)."""
        import torch
        n = 3 * self.B * self.H * self.layout.info.n_tiles * HEAD_DIM
        return self.ws_select[256: 256 + 4 * n].view(torch.float32).view(3, self.B, self.H, self.layout.info.n_tiles,
                                                                HEAD_DIM)
