"""Thin ctypes binding of liblq.so (C ABI declared in include/lq.h).

The functions carry the C names and only marshal arguments: torch device
tensors become device pointers, the current torch stream becomes the HIP
stream.  Before each call the binding checks dtype, device, contiguity and
shape of every tensor against the lq_dims, because the C ABI sees only
pointers.  Every step of the computation runs in the HIP kernels; if the
library is missing, loading fails loudly (there is no fallback).
"""
from __future__ import annotations

import ctypes as ct
import operator
import os
from dataclasses import dataclass

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# LQ_LIB may name another build of the same sources (the host-sanitizer build)
LIB_PATH = os.environ.get("LQ_LIB") or os.path.join(_PKG, "liblq.so")

LQ_OK, LQ_ERR_NULL, LQ_ERR_DIMS, LQ_ERR_UNSUPPORTED, LQ_ERR_WINDOW_FULL, LQ_ERR_POS, \
    LQ_ERR_ALIGN, LQ_ERR_HIP, LQ_ERR_WORKSPACE, LQ_ERR_OVERLAP = range(10)
LQ_DECAY_SCALAR, LQ_DECAY_PER_KEY = 0, 1
LQ_IO_F32, LQ_IO_BF16 = 0, 1
LQ_ALPHA_TOKENS, LQ_ALPHA_HEADS = 0, 1
LQ_ROW_KEEP, LQ_ROW_CLEAR = -1, -2

# every symbol include/lq.h declares
EXPORTS = ("lq_gdn_decode_step", "lq_gdn_window_flush", "lq_gdn_decode_step_ragged",
           "lq_gdn_window_flush_ragged", "lq_gdn_state_quantize",
           "lq_gdn_state_dequantize", "lq_gdn_fp32_recurrence", "lq_state_bytes",
           "lq_buffer_bytes", "lq_status_str", "lq_last_hip_error", "lq_check_dims",
           "lq_timing_enable", "lq_timing_collect", "lq_checkpoint_bytes", "lq_gdn_state_pack",
           "lq_gdn_state_unpack", "lq_gdn_decode_step_flush", "lq_gdn_prefill",
           "lq_gdn_decode_step_flush_ragged", "lq_measure_stream_read", "lq_la_prefill",
           "lq_la_workspace_bytes", "lq_la_decode_step", "lq_la_decode_step_ragged",
           "lq_gdn_tree_step", "lq_la_tree_step", "lq_tree_commit", "lq_gdn_prefill_ragged",
           "lq_gdn_workspace_bytes", "lq_tree_verify", "lq_verify_workspace_bytes", "lq_state_gather")
LQ_KERNEL_DECODE, LQ_KERNEL_FLUSH, LQ_KERNEL_QUANTIZE, LQ_KERNEL_DEQUANTIZE, \
    LQ_KERNEL_FP32_RECURRENCE, LQ_KERNEL_CHECKPOINT, LQ_KERNEL_DECODE_FLUSH, \
    LQ_KERNEL_PREFILL, LQ_KERNEL_MEASURE, LQ_KERNEL_LA_PREFILL, LQ_KERNEL_LA_DECODE, \
    LQ_KERNEL_TREE, LQ_KERNEL_COMMIT, LQ_KERNEL_VERIFY, LQ_KERNEL_GATHER = range(15)


class lq_dims(ct.Structure):
    _fields_ = [(n, ct.c_int32) for n in ("B", "H", "dk", "dv", "W", "C", "decay_mode", "smooth",
                                          "io_dtype")]


class lq_state(ct.Structure):
    _fields_ = [(n, ct.c_void_p) for n in ("sq", "row_scale", "col_scale", "comp_idx", "comp_val",
                                           "buf_k", "buf_m", "buf_g")]


class LQError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = _lib.lq_status_str(status).decode() if _lib is not None else str(status)
        extra = f" (hipError {_lib.lq_last_hip_error()})" if status == LQ_ERR_HIP else ""
        super().__init__(f"{fn}: {msg}{extra} [status {status}]")


_lib = None


def load() -> ct.CDLL:
    """Loads liblq.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m recurrent_state_quant_lq_amd.build`")
        L = ct.CDLL(LIB_PATH)
        D, S, P, I = ct.POINTER(lq_dims), ct.POINTER(lq_state), ct.c_void_p, ct.c_int32
        L.lq_gdn_decode_step.argtypes = [D, S, I, P, P, P, P, P, P, P]
        L.lq_gdn_window_flush.argtypes = [D, S, I, P, P]
        L.lq_gdn_decode_step_flush.argtypes = [D, S, I, P, P, P, P, P, P, P, P]
        L.lq_gdn_prefill.argtypes = [D, S, P, I, P, P, P, P, P, P, P]
        L.lq_gdn_decode_step_flush_ragged.argtypes = [D, S, P, P, P, P, P, P, P, P, P]
        L.lq_gdn_decode_step_ragged.argtypes = [D, S, P, P, P, P, P, P, P, P]
        L.lq_gdn_window_flush_ragged.argtypes = [D, S, P, P, P]
        L.lq_gdn_state_quantize.argtypes = [D, P, S, P]
        L.lq_gdn_state_dequantize.argtypes = [D, S, P, P]
        L.lq_gdn_fp32_recurrence.argtypes = [D, P, I, P, P, P, P, P, P, P]
        L.lq_la_prefill.argtypes = [D, S, P, P, I, P, P, P, P, I, P, P, P, ct.c_size_t, P]
        L.lq_la_workspace_bytes.argtypes = [D, I]
        L.lq_la_workspace_bytes.restype = ct.c_size_t
        L.lq_la_decode_step.argtypes = [D, S, I, P, P, P, P, I, P, P]
        L.lq_la_decode_step_ragged.argtypes = [D, S, P, P, P, P, P, I, P, P]
        L.lq_gdn_tree_step.argtypes = [D, S, P, I, P, P, P, P, P, P, P, P, P, P]
        L.lq_la_tree_step.argtypes = [D, S, P, I, P, P, P, P, P, I, P, P, P, P]
        L.lq_tree_commit.argtypes = [D, S, P, I, P, I, P, P, P, P, P]
        L.lq_gdn_prefill_ragged.argtypes = [D, S, P, P, I, P, P, P, P, P, P, P, P, ct.c_size_t, P]
        L.lq_gdn_workspace_bytes.argtypes = [D, I]
        L.lq_gdn_workspace_bytes.restype = ct.c_size_t
        L.lq_tree_verify.argtypes = [D, P, I, P, P, I, P, P, P, P, I, P, P, I, P, P, P, ct.c_size_t, P]
        L.lq_verify_workspace_bytes.argtypes = [D, I, I]
        L.lq_verify_workspace_bytes.restype = ct.c_size_t
        L.lq_state_gather.argtypes = [D, I, S, S, I, P, P, P, P]
        for f in ("lq_gdn_prefill_ragged", "lq_tree_verify", "lq_state_gather",
                  "lq_gdn_decode_step", "lq_gdn_window_flush", "lq_gdn_decode_step_flush", "lq_gdn_prefill",
                  "lq_la_prefill", "lq_la_decode_step", "lq_la_decode_step_ragged", "lq_gdn_tree_step",
                  "lq_la_tree_step", "lq_tree_commit",
                  "lq_gdn_decode_step_flush_ragged", "lq_gdn_decode_step_ragged",
                  "lq_gdn_window_flush_ragged", "lq_gdn_state_quantize",
                  "lq_gdn_state_dequantize", "lq_gdn_fp32_recurrence", "lq_check_dims",
                  "lq_last_hip_error"):
            getattr(L, f).restype = ct.c_int
        L.lq_check_dims.argtypes = [D]
        L.lq_state_bytes.argtypes = [D]
        L.lq_state_bytes.restype = ct.c_size_t
        L.lq_buffer_bytes.argtypes = [D]
        L.lq_buffer_bytes.restype = ct.c_size_t
        L.lq_status_str.argtypes = [ct.c_int]
        L.lq_status_str.restype = ct.c_char_p
        L.lq_last_hip_error.argtypes = []
        L.lq_checkpoint_bytes.argtypes = [D]
        L.lq_checkpoint_bytes.restype = ct.c_size_t
        L.lq_gdn_state_pack.argtypes = [D, S, P, P]
        L.lq_gdn_state_pack.restype = ct.c_int
        L.lq_gdn_state_unpack.argtypes = [D, P, S, P]
        L.lq_gdn_state_unpack.restype = ct.c_int
        L.lq_measure_stream_read.argtypes = [P, ct.c_size_t, I, I, I, P, ct.c_size_t, P]
        L.lq_measure_stream_read.restype = ct.c_int
        L.lq_timing_enable.argtypes = [ct.c_int32]
        L.lq_timing_enable.restype = ct.c_int
        L.lq_timing_collect.argtypes = [ct.c_int32, ct.POINTER(ct.c_int32), ct.POINTER(ct.c_float),
                                        ct.POINTER(ct.c_int32)]
        L.lq_timing_collect.restype = ct.c_int
        _lib = L
    return _lib


def make_dims(B, H, dk, dv, W, C, decay_mode=LQ_DECAY_SCALAR, smooth=1, io_dtype=LQ_IO_F32) -> lq_dims:
    return lq_dims(B, H, dk, dv, W, C, decay_mode, smooth, io_dtype)


def io_torch_dtype(d: lq_dims):
    """torch dtype of the token vectors q, k, v and outputs o for these dims."""
    return torch.bfloat16 if d.io_dtype == LQ_IO_BF16 else torch.float32


def _dtype_of(d: lq_dims, name: str):
    return io_torch_dtype(d) if name in ("q", "k", "v", "o") else torch.float32


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ct.c_void_p(stream.cuda_stream)


def _check(t: torch.Tensor, name: str, shape, dtype):
    # one fast test of the usual case; the detailed messages below otherwise
    if t is not None and t.dtype == dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _raise(fn, rc):
    if rc != LQ_OK:
        raise LQError(fn, rc)


_data_ptr = torch.Tensor.data_ptr
_STATE_FIELDS = ("sq", "row_scale", "col_scale", "comp_idx", "comp_val", "buf_k", "buf_m", "buf_g")

_SQ_ORDER: dict = {}


def sq_order(dk: int) -> np.ndarray:
    """off[i, j]: where byte (i, j) of a head's int8 state (key channel i,
    value channel j) sits in the head's dk*dv stored bytes (the operand order
    of the int8 matrix cores, as include/lq.h states it)."""
    off = _SQ_ORDER.get(dk)
    if off is None:
        i = np.arange(dk, dtype=np.int64)[:, None]
        j = np.arange(dk, dtype=np.int64)[None, :]
        G, KS = min(4, dk // 16), (dk + 63) // 64
        off = ((((j >> 4) * KS + (i >> 6)) * G + ((i & 63) >> 4)) * 16 + (j & 15)) * 16 + (i & 15)
        off.setflags(write=False)
        _SQ_ORDER[dk] = off
    return off


def sq_to_rows(sq: np.ndarray, dk: int) -> np.ndarray:
    """Stored int8 state [..., dk*dv] -> row-major [..., dk, dv]."""
    return np.ascontiguousarray(np.asarray(sq)[..., sq_order(dk)])


def sq_from_rows(rows: np.ndarray) -> np.ndarray:
    """Row-major int8 state [..., dk, dv] -> stored order [..., dk*dv]."""
    rows = np.asarray(rows)
    dk = rows.shape[-2]
    out = np.empty(rows.shape[:-2] + (rows.shape[-2] * rows.shape[-1],), dtype=rows.dtype)
    out[..., sq_order(dk).ravel()] = rows.reshape(out.shape)
    return out


@dataclass
class LayerState:
    """Device tensors of one layer's codec and window buffer (torch-owned).
    ``sq`` is [B,H,dk*dv], each head's bytes in the library's stored order
    (sq_order; sq_to_rows / sq_from_rows convert)."""
    dims: lq_dims
    sq: torch.Tensor
    row_scale: torch.Tensor
    col_scale: torch.Tensor
    comp_idx: torch.Tensor
    comp_val: torch.Tensor
    buf_k: torch.Tensor
    buf_m: torch.Tensor
    buf_g: torch.Tensor

    def __setattr__(self, name, value):
        """A field set anew drops what ready() keeps."""
        self.__dict__[name] = value
        self.__dict__["_ready"] = self.__dict__["_valid"] = None

    @staticmethod
    def allocate(d: lq_dims, device="cuda") -> "LayerState":
        B, H, dk, dv, W, C = d.B, d.H, d.dk, d.dv, d.W, d.C
        gd = dk if d.decay_mode == LQ_DECAY_PER_KEY else 1
        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=device)
        return LayerState(d, z((B, H, dk * dv), torch.int8), z((B, H, dk), torch.float32),
                          z((B, H, dv), torch.float32), z((B, H, max(C, 1)), torch.int32),
                          z((B, H, max(C, 1), dv), torch.float32),
                          z((B, H, W, dk), torch.float32), z((B, H, W, dv), torch.float32),
                          z((B, H, W, gd), torch.float32))

    def check(self, with_buffer=True):
        d = self.dims
        B, H, dk, dv, W, C = d.B, d.H, d.dk, d.dv, d.W, d.C
        gd = dk if d.decay_mode == LQ_DECAY_PER_KEY else 1
        _check(self.sq, "sq", (B, H, dk * dv), torch.int8)
        _check(self.row_scale, "row_scale", (B, H, dk), torch.float32)
        _check(self.col_scale, "col_scale", (B, H, dv), torch.float32)
        _check(self.comp_idx, "comp_idx", (B, H, max(C, 1)), torch.int32)
        _check(self.comp_val, "comp_val", (B, H, max(C, 1), dv), torch.float32)
        if with_buffer:
            _check(self.buf_k, "buf_k", (B, H, W, dk), torch.float32)
            _check(self.buf_m, "buf_m", (B, H, W, dv), torch.float32)
            _check(self.buf_g, "buf_g", (B, H, W, gd), torch.float32)
        for n in _STATE_FIELDS if with_buffer else _STATE_FIELDS[:5]:
            t = getattr(self, n)
            if t.device != self.sq.device:
                raise ValueError(f"{n} on {t.device}, sq on {self.sq.device}")

    def c_state(self) -> lq_state:
        return lq_state(*[_ptr(getattr(self, n)) for n in _STATE_FIELDS])

    def rows(self, b0: int, b1: int) -> "LayerState":
        """Batch rows b0 .. b1-1 as a state of their own: views of the same device
        memory (no copy) with B = b1 - b0, so that parts of a batch can run as
        separate calls, e.g. as independent chains on separate streams."""
        d = lq_dims.from_buffer_copy(self.dims)
        if not (0 <= b0 < b1 <= d.B):
            raise ValueError(f"rows {b0}..{b1} outside the batch of {d.B}")
        d.B = b1 - b0
        return LayerState(d, *[getattr(self, n)[b0:b1] for n in _STATE_FIELDS])

    def ready(self, with_buffer=True) -> lq_state:
        """The C struct of this state, validated (shapes, dtypes, device) once
        for the dims and the tensors the fields hold; dims changed, a field
        replaced by another tensor or a tensor whose memory was exchanged
        (set_, .data) are validated again.  In-place writes to the tensors need
        no revalidation."""
        try:
            key = (with_buffer, bytes(self.dims), self.sq.data_ptr(), self.row_scale.data_ptr(),
                   self.col_scale.data_ptr(), self.comp_idx.data_ptr(), self.comp_val.data_ptr(),
                   self.buf_k.data_ptr(), self.buf_m.data_ptr(), self.buf_g.data_ptr())
        except AttributeError:                           # a codec without a window buffer
            key = (with_buffer, bytes(self.dims), *(_ptr(getattr(self, n)) for n in _STATE_FIELDS))
        c = self._ready
        if c is None or c[0] != key:
            self.check(with_buffer)
            c = (key, self.c_state())
            self.__dict__["_ready"] = c
        return c[1]

    def codec(self) -> dict:
        """Host copies of the codec arrays, int8 matrix row-major [B,H,dk,dv]
        (comp arrays cut to C)."""
        C = self.dims.C
        return dict(sq=sq_to_rows(self.sq.cpu().numpy(), self.dims.dk),
                    r=self.row_scale.cpu().numpy(),
                    s=self.col_scale.cpu().numpy(), idx=self.comp_idx[..., :C].cpu().numpy(),
                    cv=self.comp_val[..., :C, :].cpu().numpy())

    def load_codec(self, cd: dict):
        """Uploads host codec arrays ([B,H,...], int8 matrix row-major
        [B,H,dk,dv], comp arrays with C entries)."""
        C = self.dims.C
        self.sq.copy_(torch.from_numpy(sq_from_rows(cd["sq"])))
        self.row_scale.copy_(torch.as_tensor(cd["r"]))
        self.col_scale.copy_(torch.as_tensor(cd["s"]))
        if C:
            self.comp_idx[..., :C].copy_(torch.as_tensor(cd["idx"]))
            self.comp_val[..., :C, :].copy_(torch.as_tensor(cd["cv"]))


_SHAPES: dict = {}


def _token_shapes(d: lq_dims, T=None):
    key = (d.B, d.H, d.dk, d.dv, d.decay_mode, T)
    sh = _SHAPES.get(key)
    if sh is None:
        pre = (d.B, d.H) if T is None else (T, d.B, d.H)
        ash = pre + ((d.dk,) if d.decay_mode == LQ_DECAY_PER_KEY else ())
        gd = d.dk if d.decay_mode == LQ_DECAY_PER_KEY else 1
        node = (d.B, d.H, 1 if T is None else T)
        sh = {k: torch.Size(v) for k, v in dict(q=pre + (d.dk,), k=pre + (d.dk,), v=pre + (d.dv,),
                                                alpha=ash, beta=pre, o=pre + (d.dv,), row=(d.B,),
                                                parent=(d.B, node[2]), tree_m=node + (d.dv,),
                                                tree_g=node + (gd,)).items()}
        _SHAPES[key] = sh
    return sh


def lq_gdn_decode_step(st: LayerState, pos: int, q, k, v, alpha, beta, o, stream=None):
    d = st.dims
    sh = _token_shapes(d)
    for name, t in (("q", q), ("k", k), ("v", v), ("alpha", alpha), ("beta", beta), ("o", o)):
        _check(t, name, sh[name], _dtype_of(d, name))
    cs = st.ready()
    rc = load().lq_gdn_decode_step(ct.byref(d), ct.byref(cs), int(pos), _ptr(q), _ptr(k), _ptr(v),
                                   _ptr(alpha), _ptr(beta), _ptr(o), _stream(stream))
    _raise("lq_gdn_decode_step", rc)


def lq_gdn_window_flush(st: LayerState, n_buffered: int, h_out=None, stream=None):
    d = st.dims
    if h_out is not None:
        _check(h_out, "h_out", (d.B, d.H, d.dk, d.dv), torch.float32)
    cs = st.ready()
    rc = load().lq_gdn_window_flush(ct.byref(d), ct.byref(cs), int(n_buffered), _ptr(h_out),
                                    _stream(stream))
    _raise("lq_gdn_window_flush", rc)


def lq_gdn_decode_step_flush(st: LayerState, pos: int, q, k, v, alpha, beta, o, h_out=None,
                             stream=None):
    """Decode of one token into slot pos, then the flush of pos + 1 slots (one launch)."""
    d = st.dims
    sh = _token_shapes(d)
    for name, t in (("q", q), ("k", k), ("v", v), ("alpha", alpha), ("beta", beta), ("o", o)):
        _check(t, name, sh[name], _dtype_of(d, name))
    if h_out is not None:
        _check(h_out, "h_out", (d.B, d.H, d.dk, d.dv), torch.float32)
    cs = st.ready()
    rc = load().lq_gdn_decode_step_flush(ct.byref(d), ct.byref(cs), int(pos), _ptr(q), _ptr(k),
                                         _ptr(v), _ptr(alpha), _ptr(beta), _ptr(o), _ptr(h_out),
                                         _stream(stream))
    _raise("lq_gdn_decode_step_flush", rc)


def lq_gdn_decode_step_flush_ragged(st: LayerState, pos, q, k, v, alpha, beta, o, h_out=None,
                                    stream=None):
    """pos: device int32 [B]; rows with pos in [0, W) decode slot pos and flush pos + 1 slots."""
    d = st.dims
    _check(pos, "pos", (d.B,), torch.int32)
    sh = _token_shapes(d)
    for name, t in (("q", q), ("k", k), ("v", v), ("alpha", alpha), ("beta", beta), ("o", o)):
        _check(t, name, sh[name], _dtype_of(d, name))
    if h_out is not None:
        _check(h_out, "h_out", (d.B, d.H, d.dk, d.dv), torch.float32)
    cs = st.ready()
    rc = load().lq_gdn_decode_step_flush_ragged(ct.byref(d), ct.byref(cs), _ptr(pos), _ptr(q), _ptr(k),
                                                _ptr(v), _ptr(alpha), _ptr(beta), _ptr(o), _ptr(h_out),
                                                _stream(stream))
    _raise("lq_gdn_decode_step_flush_ragged", rc)


def lq_gdn_decode_step_ragged(st: LayerState, pos, q, k, v, alpha, beta, o, stream=None):
    """pos: device int32 [B], the window position of each batch row."""
    d = st.dims
    _check(pos, "pos", (d.B,), torch.int32)
    sh = _token_shapes(d)
    for name, t in (("q", q), ("k", k), ("v", v), ("alpha", alpha), ("beta", beta), ("o", o)):
        _check(t, name, sh[name], _dtype_of(d, name))
    cs = st.ready()
    rc = load().lq_gdn_decode_step_ragged(ct.byref(d), ct.byref(cs), _ptr(pos), _ptr(q), _ptr(k), _ptr(v),
                                          _ptr(alpha), _ptr(beta), _ptr(o), _stream(stream))
    _raise("lq_gdn_decode_step_ragged", rc)


def lq_gdn_window_flush_ragged(st: LayerState, n_buffered, h_out=None, stream=None):
    """n_buffered: device int32 [B], slots to flush per batch row (0 = none)."""
    d = st.dims
    _check(n_buffered, "n_buffered", (d.B,), torch.int32)
    if h_out is not None:
        _check(h_out, "h_out", (d.B, d.H, d.dk, d.dv), torch.float32)
    cs = st.ready()
    rc = load().lq_gdn_window_flush_ragged(ct.byref(d), ct.byref(cs), _ptr(n_buffered), _ptr(h_out),
                                           _stream(stream))
    _raise("lq_gdn_window_flush_ragged", rc)


def lq_gdn_state_quantize(st: LayerState, h, stream=None):
    d = st.dims
    _check(h, "h", (d.B, d.H, d.dk, d.dv), torch.float32)
    cs = st.ready(with_buffer=False)
    rc = load().lq_gdn_state_quantize(ct.byref(d), _ptr(h), ct.byref(cs), _stream(stream))
    _raise("lq_gdn_state_quantize", rc)


def lq_gdn_state_dequantize(st: LayerState, h_out, stream=None):
    d = st.dims
    _check(h_out, "h_out", (d.B, d.H, d.dk, d.dv), torch.float32)
    cs = st.ready(with_buffer=False)
    rc = load().lq_gdn_state_dequantize(ct.byref(d), ct.byref(cs), _ptr(h_out), _stream(stream))
    _raise("lq_gdn_state_dequantize", rc)


def lq_gdn_fp32_recurrence(d: lq_dims, h, T: int, q, k, v, alpha, beta, o=None, stream=None):
    _check(h, "h", (d.B, d.H, d.dk, d.dv), torch.float32)
    sh = _token_shapes(d, T)
    for name, t in (("q", q), ("k", k), ("v", v), ("alpha", alpha), ("beta", beta)):
        _check(t, name, sh[name], _dtype_of(d, name))
    if o is not None:
        _check(o, "o", sh["o"], _dtype_of(d, "o"))
    rc = load().lq_gdn_fp32_recurrence(ct.byref(d), _ptr(h), int(T), _ptr(q), _ptr(k), _ptr(v),
                                       _ptr(alpha), _ptr(beta), _ptr(o), _stream(stream))
    _raise("lq_gdn_fp32_recurrence", rc)


def lq_gdn_prefill(d: lq_dims, st, h, T: int, q, k, v, alpha, beta, o=None, stream=None):
    """Chunked fp32 prefill of T tokens (h in/out), then the codec of the final
    state into st (a LayerState, or None for the fp32 state only)."""
    _check(h, "h", (d.B, d.H, d.dk, d.dv), torch.float32)
    sh = _token_shapes(d, T)
    if T > 0:
        for name, t in (("q", q), ("k", k), ("v", v), ("alpha", alpha), ("beta", beta)):
            _check(t, name, sh[name], _dtype_of(d, name))
    if o is not None:
        _check(o, "o", sh["o"], _dtype_of(d, "o"))
    cs = None
    if st is not None:
        cs = st.ready(with_buffer=False)
    rc = load().lq_gdn_prefill(ct.byref(d), ct.byref(cs) if cs is not None else None, _ptr(h), int(T),
                               _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(o),
                               _stream(stream))
    _raise("lq_gdn_prefill", rc)


def _launch(fn, device, stream, *args):
    """Calls fn with the stream (None: device's current stream) on the device that
    holds its tensors, whichever device is the current one."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(device.index)
    elif stream.device != device:
        raise ValueError(f"stream on {stream.device}, tensors on {device}")
    else:
        raw = stream.cuda_stream
    f = getattr(_lib or load(), fn)
    if device.index == torch.cuda.current_device():
        rc = f(*args, raw)
    else:
        with torch.cuda.device(device):
            rc = f(*args, raw)
    if rc:
        raise LQError(fn, rc)


def _check_all(device, dtype_io, *items):
    """Items (name, tensor, shape, dtype): dtype None is the token dtype.  Every tensor
    of the shape and dtype, contiguous, on device."""
    index = device.index
    for name, t, shape, dtype in items:
        if t is None or t.dtype is not (dtype or dtype_io) or t.shape != shape or t.get_device() != index \
                or not t.is_contiguous():
            _check(t, name, shape, dtype or dtype_io)
            raise ValueError(f"{name} on {t.device}, expected {device}")


def _alpha(d: lq_dims, alpha, shape):
    """LQ_ALPHA_HEADS and the shape [H] for one decay per head, LQ_ALPHA_TOKENS and the
    token shape for one per token."""
    if alpha is not None and alpha.dim() == 1:
        return LQ_ALPHA_HEADS, (d.H,)
    return LQ_ALPHA_TOKENS, shape


def lq_la_workspace_bytes(d: lq_dims, T: int) -> int:
    """Bytes of lq_la_prefill's workspace for prompts of up to T tokens."""
    return int(load().lq_la_workspace_bytes(ct.byref(d), int(T)))


def lq_la_prefill(d: lq_dims, st, h0, h, T: int, q, k, v, alpha, o=None, lens=None, workspace=None,
                  stream=None):
    """Linear attention over a prompt: o (or None) and the state h after T tokens
    from h0 (None: zeros; h0 may be h), then the codec of h into st (or None).
    alpha: [T,B,H], or [H] for one fixed decay per head.  lens: device int32 [B]
    tokens per row, or None.  workspace: device uint8 tensor of at least
    lq_la_workspace_bytes(d, T) bytes (None: allocated for this call)."""
    T = int(T)
    f32 = torch.float32
    hs = (d.B, d.H, d.dk, d.dv)
    _check(h, "h", hs, f32)
    dev = h.device
    items = []
    if h0 is not None:
        items.append(("h0", h0, hs, f32))
        off = abs(h0.data_ptr() - h.data_ptr())
        if 0 < off < h.numel() * 4:
            raise ValueError("h0 and h overlap")
    kind = LQ_ALPHA_TOKENS
    if T > 0:
        sh = _token_shapes(d, T)
        kind, ash = _alpha(d, alpha, sh["alpha"])
        items += [("q", q, sh["q"], None), ("k", k, sh["k"], None), ("v", v, sh["v"], None), ("alpha", alpha, ash, f32)]
        if o is not None:
            items.append(("o", o, sh["o"], None))
    if lens is not None:
        items.append(("lens", lens, (d.B,), torch.int32))
    cs = None
    if st is not None:
        cs = ct.byref(st.ready(with_buffer=False))
        items.append(("the state", st.sq, st.sq.shape, torch.int8))
        if any(getattr(st.dims, n) != getattr(d, n) for n in ("B", "H", "dk", "dv", "C")):
            raise ValueError("the state's dims are not d")
    need = lq_la_workspace_bytes(d, T)
    if workspace is None and need:
        with torch.cuda.stream(stream):              # memory of the stream that uses it
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    size = 0
    if workspace is not None:
        size = workspace.numel()
        items.append(("workspace", workspace, (size,), torch.uint8))
    _check_all(dev, io_torch_dtype(d), *items)
    _launch("lq_la_prefill", dev, stream, ct.byref(d), cs, _ptr(h0), h.data_ptr(), T, _ptr(q), _ptr(k), _ptr(v),
            _ptr(alpha), kind, _ptr(lens), _ptr(o), _ptr(workspace) if size else None, size)


def _la_decode(fn, st, pos_arg, q, k, v, alpha, o, stream, *more):
    d = st.dims
    sh = _token_shapes(d)
    cs = st.ready()
    dev = st.sq.device
    kind, ash = _alpha(d, alpha, sh["alpha"])
    _check_all(dev, io_torch_dtype(d), ("q", q, sh["q"], None), ("k", k, sh["k"], None), ("v", v, sh["v"], None),
               ("alpha", alpha, ash, torch.float32), ("o", o, sh["o"], None), *more)
    _launch(fn, dev, stream, ct.byref(d), ct.byref(cs), pos_arg, q.data_ptr(), k.data_ptr(), v.data_ptr(),
            alpha.data_ptr(), kind, o.data_ptr())


def lq_la_decode_step(st: LayerState, pos: int, q, k, v, alpha, o, stream=None):
    """One token of linear attention into slot pos; alpha [B,H], or [H] (fixed per head)."""
    _la_decode("lq_la_decode_step", st, int(pos), q, k, v, alpha, o, stream)


def lq_la_decode_step_ragged(st: LayerState, pos, q, k, v, alpha, o, stream=None):
    """pos: device int32 [B], the window position of each batch row."""
    _la_decode("lq_la_decode_step_ragged", st, _ptr(pos), q, k, v, alpha, o, stream,
               ("pos", pos, (st.dims.B,), torch.int32))


def _tree_items(d, pos, parent, q, k, v, o, tree_m, tree_g):
    if parent is None or parent.dim() != 2:
        raise ValueError("parent: a [B,N] tensor is required")
    N = parent.shape[1]
    sh = _token_shapes(d, N)
    f32, i32 = torch.float32, torch.int32
    return N, sh, (("pos", pos, sh["row"], i32), ("parent", parent, sh["parent"], i32), ("q", q, sh["q"], None),
                   ("k", k, sh["k"], None), ("v", v, sh["v"], None), ("o", o, sh["o"], None),
                   ("tree_m", tree_m, sh["tree_m"], f32), ("tree_g", tree_g, sh["tree_g"], f32))


def lq_gdn_tree_step(st: LayerState, pos, parent, q, k, v, alpha, beta, o, tree_m, tree_g, stream=None):
    """Outputs of the N drafted tokens of every row's tree (parent: device int32 [B,N])
    after the window's pos (device int32 [B]) slots; state, window and pos are left as
    they are.  tree_m [B,H,N,dv] and tree_g [B,H,N,gd] receive the nodes' slots."""
    d = st.dims
    N, sh, items = _tree_items(d, pos, parent, q, k, v, o, tree_m, tree_g)
    cs = st.ready()
    dev = st.sq.device
    _check_all(dev, io_torch_dtype(d), *items, ("alpha", alpha, sh["alpha"], torch.float32),
               ("beta", beta, sh["beta"], torch.float32))
    _launch("lq_gdn_tree_step", dev, stream, ct.byref(d), ct.byref(cs), pos.data_ptr(), N, parent.data_ptr(),
            q.data_ptr(), k.data_ptr(), v.data_ptr(), alpha.data_ptr(), beta.data_ptr(), o.data_ptr(),
            tree_m.data_ptr(), tree_g.data_ptr())


def lq_la_tree_step(st: LayerState, pos, parent, q, k, v, alpha, o, tree_m, tree_g, stream=None):
    """lq_gdn_tree_step for plain linear attention; alpha [N,B,H], or [H] (fixed per head)."""
    d = st.dims
    N, sh, items = _tree_items(d, pos, parent, q, k, v, o, tree_m, tree_g)
    kind, ash = _alpha(d, alpha, sh["alpha"])
    cs = st.ready()
    dev = st.sq.device
    _check_all(dev, io_torch_dtype(d), *items, ("alpha", alpha, ash, torch.float32))
    _launch("lq_la_tree_step", dev, stream, ct.byref(d), ct.byref(cs), pos.data_ptr(), N, parent.data_ptr(),
            q.data_ptr(), k.data_ptr(), v.data_ptr(), alpha.data_ptr(), kind, o.data_ptr(), tree_m.data_ptr(),
            tree_g.data_ptr())


def lq_tree_commit(st: LayerState, pos, path, n_path, k, tree_m, tree_g, stream=None):
    """Appends the nodes path[b][:n_path[b]] (device int32 [B,P], [B]) of a tree step to
    the windows, slots pos[b] on; the caller then advances pos by n_path."""
    d = st.dims
    if k is None or k.dim() != 4 or path is None or path.dim() != 2:
        raise ValueError("k: the tree's [N,B,H,dk] tensor and path: a [B,P] tensor are required")
    N, P = k.shape[0], path.shape[1]
    sh = _token_shapes(d, N)
    cs = st.ready()
    dev = st.sq.device
    f32, i32 = torch.float32, torch.int32
    _check_all(dev, io_torch_dtype(d), ("pos", pos, sh["row"], i32), ("path", path, (d.B, P), i32),
               ("n_path", n_path, sh["row"], i32), ("k", k, sh["k"], None),
               ("tree_m", tree_m, sh["tree_m"], f32), ("tree_g", tree_g, sh["tree_g"], f32))
    _launch("lq_tree_commit", dev, stream, ct.byref(d), ct.byref(cs), pos.data_ptr(), N, path.data_ptr(), P,
            n_path.data_ptr(), k.data_ptr(), tree_m.data_ptr(), tree_g.data_ptr())


def _workspace(given, need, device, stream):
    """The caller's workspace, or memory of the stream that uses it; and its size."""
    if given is None and need:
        with torch.cuda.stream(stream):
            given = torch.empty(need, dtype=torch.uint8, device=device)
    return given, 0 if given is None else given.numel()


def lq_gdn_workspace_bytes(d: lq_dims, T: int) -> int:
    """Bytes of lq_gdn_prefill_ragged's workspace for prompts of up to T tokens."""
    return int(load().lq_gdn_workspace_bytes(ct.byref(d), int(T)))


def lq_gdn_prefill_ragged(d: lq_dims, st, h0, h, T: int, q, k, v, alpha, beta, o=None, lens=None, workspace=None,
                          stream=None):
    """The gated delta rule over a padded batch of prompts: o (or None) and the state h
    after T tokens from h0 (None: zeros; h0 may be h), then the codec of h into st (or
    None).  lens: device int32 [B] tokens per row, or None.  workspace: device uint8
    tensor of at least lq_gdn_workspace_bytes(d, T) bytes (None: allocated for this call)."""
    T = int(T)
    f32 = torch.float32
    hs = (d.B, d.H, d.dk, d.dv)
    _check(h, "h", hs, f32)
    dev = h.device
    items = []
    if h0 is not None:
        items.append(("h0", h0, hs, f32))
        off = abs(h0.data_ptr() - h.data_ptr())
        if 0 < off < h.numel() * 4:
            raise ValueError("h0 and h overlap")
    if T > 0:
        sh = _token_shapes(d, T)
        items += [("q", q, sh["q"], None), ("k", k, sh["k"], None), ("v", v, sh["v"], None),
                  ("alpha", alpha, sh["alpha"], f32), ("beta", beta, sh["beta"], f32)]
        if o is not None:
            items.append(("o", o, sh["o"], None))
    if lens is not None:
        items.append(("lens", lens, (d.B,), torch.int32))
    cs = None
    if st is not None:
        cs = ct.byref(st.ready(with_buffer=False))
        items.append(("the state", st.sq, st.sq.shape, torch.int8))
        if any(getattr(st.dims, n) != getattr(d, n) for n in ("B", "H", "dk", "dv", "C")):
            raise ValueError("the state's dims are not d")
    workspace, size = _workspace(workspace, lq_gdn_workspace_bytes(d, T), dev, stream)
    if workspace is not None:
        items.append(("workspace", workspace, (size,), torch.uint8))
    _check_all(dev, io_torch_dtype(d), *items)
    _launch("lq_gdn_prefill_ragged", dev, stream, ct.byref(d), cs, _ptr(h0), h.data_ptr(), T, _ptr(q), _ptr(k),
            _ptr(v), _ptr(alpha), _ptr(beta), _ptr(lens), _ptr(o), _ptr(workspace) if size else None, size)


def lq_verify_workspace_bytes(d: lq_dims, N: int, V: int) -> int:
    """Bytes of lq_tree_verify's workspace for N nodes and a vocabulary of V tokens."""
    return int(load().lq_verify_workspace_bytes(ct.byref(d), int(N), int(V)))


def lq_tree_verify(d: lq_dims, pos, parent, token, target, u, path, n_path, next, target0=None, draft=None,
                   draft0=None, replace=True, workspace=None, stream=None):
    """Accepted path and next token of every row's drafted tree (parent, token: device int32
    [B,N]) from the target's probabilities (target fp32 [N,B,V] after each node, target0 [B,V]
    before the first, or None: the first node is already chosen), the draft's (draft, draft0,
    or None) and the random numbers u fp32 [N+1,B].  path int32 [B,P], n_path and next int32
    [B] are written.  replace: a node's children were drawn with replacement."""
    if parent is None or parent.dim() != 2 or target is None or target.dim() != 3 or path is None or path.dim() != 2:
        raise ValueError("parent: a [B,N], target: a [N,B,V] and path: a [B,P] tensor are required")
    N, V, P = parent.shape[1], target.shape[2], path.shape[1]
    if draft is None and draft0 is not None or target0 is None and draft0 is not None:
        raise ValueError("draft0 goes with draft and target0")
    f32, i32, B = torch.float32, torch.int32, d.B
    dev = pos.device if pos is not None else None
    items = [("parent", parent, (B, N), i32), ("token", token, (B, N), i32), ("target", target, (N, B, V), f32),
             ("u", u, (N + 1, B), f32), ("path", path, (B, P), i32), ("n_path", n_path, (B,), i32),
             ("next", next, (B,), i32)]
    if target0 is not None:
        items.append(("target0", target0, (B, V), f32))
    if draft is not None:
        items.append(("draft", draft, (N, B, V), f32))
        if target0 is not None:
            items.append(("draft0", draft0, (B, V), f32))
    _check(pos, "pos", (B,), i32)
    _check_all(dev, f32, *items)
    workspace, size = _workspace(workspace, lq_verify_workspace_bytes(d, N, V), dev, stream)
    if workspace is not None:
        _check_all(dev, f32, ("workspace", workspace, (size,), torch.uint8))
    _launch("lq_tree_verify", dev, stream, ct.byref(d), pos.data_ptr(), N, parent.data_ptr(), token.data_ptr(), V,
            target.data_ptr(), _ptr(target0), _ptr(draft), _ptr(draft0), 1 if replace else 0, u.data_ptr(),
            path.data_ptr(), P, n_path.data_ptr(), next.data_ptr(), _ptr(workspace) if size else None, size)


def _c_states(states, d, rows, dev, with_buffer):
    """The C structs of several layers' states of d's dims but `rows` rows, each validated as
    LayerState.ready does, in one pass over their addresses."""
    want = lq_dims.from_buffer_copy(d)
    want.B = rows
    want = bytes(want)
    structs = bytearray()
    for x in states:
        v = x.__dict__["_valid"]
        if v is None:
            v = x.__dict__["_valid"] = [tuple(t for t in (getattr(x, f) for f in _STATE_FIELDS) if t is not None),
                                        None, None, None]
        now = (with_buffer, bytes(x.dims), *map(_data_ptr, v[0]))
        if now != v[1]:
            x.check(with_buffer)
            v[1:] = now, x.sq.device, bytes(x.c_state())
        if v[2] != dev:
            raise ValueError(f"states on {v[2]} and {dev}")
        if now[1] != want and (x.dims.B != rows or any(
                getattr(x.dims, f) != getattr(d, f) for f in ("H", "dk", "dv", "W", "C", "decay_mode"))):
            raise ValueError("the states of a call differ in their dims")
        structs += v[3]
    return (lq_state * len(states)).from_buffer(structs)


def lq_state_gather(dst, src, index, pos=None, pos_out=None, stream=None):
    """Row b of every state in dst (a LayerState or a list, one a layer) becomes row index[b]
    (device int32 [B]; LQ_ROW_KEEP, LQ_ROW_CLEAR) of the state in src, which may be the same
    ones.  pos: device int32, buffered tokens of src's rows (None: the windows are empty);
    pos_out: device int32 [B], receives those of the rows that moved."""
    dst, src = ([x] if isinstance(x, LayerState) else list(x) for x in (dst, src))
    if not dst or len(dst) != len(src):
        raise ValueError("dst and src: as many states each, one at least")
    d, rows = dst[0].dims, src[0].dims.B
    dev = dst[0].sq.device
    n, buf = len(dst), pos is not None
    cd = _c_states(dst, d, d.B, dev, buf)
    cs = cd if all(map(operator.is_, dst, src)) else _c_states(src, d, rows, dev, buf)
    items = [("index", index, (d.B,), torch.int32)]
    if pos is not None:
        items.append(("pos", pos, (rows,), torch.int32))
    if pos_out is not None:
        items.append(("pos_out", pos_out, (d.B,), torch.int32))
    _check_all(dev, torch.float32, *items)
    _launch("lq_state_gather", dev, stream, ct.byref(d), n, cd, cs, rows, index.data_ptr(), _ptr(pos), _ptr(pos_out))


def lq_checkpoint_bytes(d: lq_dims) -> int:
    return int(load().lq_checkpoint_bytes(ct.byref(d)))


def lq_gdn_state_pack(st: LayerState, blob, stream=None):
    """blob: device uint8 tensor of lq_checkpoint_bytes(st.dims) bytes."""
    d = st.dims
    _check(blob, "blob", (lq_checkpoint_bytes(d),), torch.uint8)
    cs = st.ready(with_buffer=False)
    _raise("lq_gdn_state_pack", load().lq_gdn_state_pack(ct.byref(d), ct.byref(cs), _ptr(blob),
                                                          _stream(stream)))


def lq_gdn_state_unpack(st: LayerState, blob, stream=None):
    d = st.dims
    _check(blob, "blob", (lq_checkpoint_bytes(d),), torch.uint8)
    cs = st.ready(with_buffer=False)
    _raise("lq_gdn_state_unpack", load().lq_gdn_state_unpack(ct.byref(d), _ptr(blob), ct.byref(cs),
                                                              _stream(stream)))


def lq_state_bytes(d: lq_dims) -> int:
    return int(load().lq_state_bytes(ct.byref(d)))


def lq_buffer_bytes(d: lq_dims) -> int:
    return int(load().lq_buffer_bytes(ct.byref(d)))


def lq_check_dims(d: lq_dims) -> int:
    return int(load().lq_check_dims(ct.byref(d)))


def lq_measure_stream_read(src, slice_bytes: int, n_slices: int, mode: int, grid: int = 0,
                           sink=None, write_bytes: int = 0, stream=None):
    """Streaming-read reference (measurement only): src and sink device
    tensors holding n_slices * slice_bytes and n_slices * write_bytes bytes."""
    if src.numel() * src.element_size() < slice_bytes * n_slices or not src.is_cuda:
        raise ValueError("src: a device tensor of n_slices * slice_bytes bytes is required")
    if write_bytes and (sink is None or not sink.is_cuda or
                        sink.numel() * sink.element_size() < write_bytes * n_slices):
        raise ValueError("sink: a device tensor of n_slices * write_bytes bytes is required")
    rc = load().lq_measure_stream_read(_ptr(src), int(slice_bytes), int(n_slices), int(mode), int(grid),
                                       _ptr(sink), int(write_bytes), _stream(stream))
    _raise("lq_measure_stream_read", rc)


def lq_timing_enable(on: bool = True):
    _raise("lq_timing_enable", load().lq_timing_enable(1 if on else 0))


def lq_timing_collect(max_records: int = 65536):
    """Per-launch kernel durations recorded since lq_timing_enable(True), in
    launch order: (families, milliseconds) as lists; drops the records."""
    fam = (ct.c_int32 * max_records)()
    ms = (ct.c_float * max_records)()
    n = ct.c_int32(0)
    _raise("lq_timing_collect", load().lq_timing_collect(max_records, fam, ms, ct.byref(n)))
    k = min(n.value, max_records)
    return list(fam[:k]), list(ms[:k])
