"""ctypes binding of libq8adamw.so: argument marshalling only.

Every function here has the name of the C entry point it calls (see
include/q8adamw.h and include/q8train.h) and takes torch tensors that already live on a CUDA device;
all work runs in the library's kernels.  A missing library is an error: there
is no fallback path.
"""
import ctypes as C
import os
from dataclasses import dataclass
from typing import Optional, Sequence

import numpy as np
import torch

from . import build as _build

SIGNED, UNSIGNED = 0, 1
BLOCK = 2048
SMALL_NUMEL = 4096
MAX_STEP = 0x7FFFFFFF

SILU, GELU_TANH, GELU = 0, 1, 2                     # q8_activation
NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2           # q8_norm_kind
NORM_MAX_DIM = 32768
DISTILL_MAX_K = 1024

Q8_OK = 0
_STATUS = {-1: "Q8_ERR_NULL", -2: "Q8_ERR_SIZE", -3: "Q8_ERR_ALIGN", -4: "Q8_ERR_ARG", -5: "Q8_ERR_CUDA"}

# every symbol the headers declare
EXPORTS = ("q8_codebook_init", "q8_blockwise_quantize", "q8_blockwise_dequantize",
           "adamw8bit_sr_step", "adamw_bf16_sr_step", "momentum8bit_sr_step", "lion8bit_sr_step",
           "q8_philox_fill", "q8_selftest_sqrt_div", "q8_prepare_device", "q8_last_error", "q8_abi_version",
           "q8_gated_ff_workspace", "q8_gated_ff_forward", "q8_gated_ff_backward",
           "q8_block_norm_forward", "q8_block_norm_workspace", "q8_block_norm_backward",
           "q8_distill_topk_forward", "q8_distill_topk_backward")


class Q8Error(RuntimeError):
    """A non-zero status from the library, with its message."""

    def __init__(self, fn, code, msg):
        super().__init__("%s failed: %s (%d): %s" % (fn, _STATUS.get(code, "?"), code, msg))
        self.code = code


class HParams(C.Structure):
    """q8_adamw_hparams."""
    _fields_ = [("lr", C.c_double), ("beta1", C.c_double), ("beta2", C.c_double),
                ("eps", C.c_double), ("weight_decay", C.c_double),
                ("step", C.c_int64), ("seed", C.c_uint64), ("sr", C.c_int32), ("exact", C.c_int32)]


class MomentumHParams(C.Structure):
    """q8_momentum_hparams."""
    _fields_ = [("lr", C.c_double), ("momentum", C.c_double), ("weight_decay", C.c_double),
                ("step", C.c_int64), ("seed", C.c_uint64), ("sr", C.c_int32)]


class LionHParams(C.Structure):
    """q8_lion_hparams."""
    _fields_ = [("lr", C.c_double), ("beta1", C.c_double), ("beta2", C.c_double),
                ("weight_decay", C.c_double), ("step", C.c_int64), ("seed", C.c_uint64), ("sr", C.c_int32)]


class _Tensor8(C.Structure):
    _fields_ = [("param", C.c_void_p), ("grad", C.c_void_p), ("numel", C.c_int64),
                ("philox_offset", C.c_int64), ("m_codes", C.c_void_p), ("v_codes", C.c_void_p),
                ("m_absmax", C.c_void_p), ("v_absmax", C.c_void_p),
                ("m32", C.c_void_p), ("v32", C.c_void_p)]


class _Tensor16(C.Structure):
    _fields_ = [("param", C.c_void_p), ("grad", C.c_void_p), ("m", C.c_void_p),
                ("v", C.c_void_p), ("numel", C.c_int64), ("philox_offset", C.c_int64)]


_P, _I64 = C.c_void_p, C.c_int64


class _GatedFF(C.Structure):
    _fields_ = [("x", _P), ("w_gate", _P), ("w_up", _P), ("tokens", _I64), ("d_model", _I64), ("d_ff", _I64),
                ("x_stride", _I64), ("workspace", _P), ("workspace_bytes", _I64), ("act", C.c_int32)]


class _BlockNorm(C.Structure):
    _fields_ = [("residual", _P), ("y", _P), ("post_weight", _P), ("post_bias", _P), ("pre_weight", _P),
                ("pre_bias", _P), ("gate", _P), ("tokens", _I64), ("dim", _I64), ("gate_tokens", _I64),
                ("residual_stride", _I64), ("y_stride", _I64), ("post_kind", C.c_int32), ("pre_kind", C.c_int32),
                ("residual_dtype", C.c_int32), ("eps", C.c_float), ("residual_scale", C.c_float)]


class _BlockNormGrads(C.Structure):
    _fields_ = [("d_residual_out", _P), ("dz", _P), ("d_residual", _P), ("d_y", _P), ("d_post_weight", _P),
                ("d_post_bias", _P), ("d_pre_weight", _P), ("d_pre_bias", _P), ("d_gate", _P),
                ("d_residual_out_stride", _I64), ("dz_stride", _I64), ("d_residual_stride", _I64),
                ("d_y_stride", _I64), ("workspace", _P), ("workspace_bytes", _I64)]


class _DistillTopk(C.Structure):
    _fields_ = [("logits", _P), ("teacher_ids", _P), ("teacher_logits", _P), ("labels", _P), ("row_weight", _P),
                ("rows", _I64), ("vocab", _I64), ("k", _I64), ("logits_stride", _I64), ("logits_dtype", C.c_int32),
                ("temperature", C.c_float), ("kd_weight", C.c_float), ("ce_weight", C.c_float)]


_lib = None


def library_path():
    return _build.LIB


def load_library(path: Optional[str] = None):
    """Load (once) and type the shared library; raise if it was not built."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or _build.LIB
    if not os.path.exists(path):
        raise RuntimeError("libq8adamw.so is not built (%s); run bit_blockwise_adamw_gb300.build.build()" % path)
    L = C.CDLL(path)
    P, S = C.c_void_p, C.c_void_p
    L.q8_codebook_init.argtypes = [C.c_int, P]
    L.q8_blockwise_quantize.argtypes = [P, P, P, C.c_int64, C.c_int, S]
    L.q8_blockwise_dequantize.argtypes = [P, P, P, C.c_int64, C.c_int, S]
    L.adamw8bit_sr_step.argtypes = [C.POINTER(_Tensor8), C.c_int, C.POINTER(HParams), S]
    L.adamw_bf16_sr_step.argtypes = [C.POINTER(_Tensor16), C.c_int, C.POINTER(HParams), S]
    L.momentum8bit_sr_step.argtypes = [C.POINTER(_Tensor8), C.c_int, C.POINTER(MomentumHParams), S]
    L.lion8bit_sr_step.argtypes = [C.POINTER(_Tensor8), C.c_int, C.POINTER(LionHParams), S]
    L.q8_philox_fill.argtypes = [C.c_uint64, C.c_uint32, C.c_uint32, C.c_uint64, C.c_int64, P, S]
    L.q8_selftest_sqrt_div.argtypes = [P, S]
    L.q8_prepare_device.argtypes = []
    L.q8_last_error.argtypes = []
    L.q8_last_error.restype = C.c_char_p
    L.q8_abi_version.argtypes = []
    # the structures go as addresses (c_void_p): ctypes.byref is accepted
    L.q8_gated_ff_workspace.argtypes = [P, C.c_int]
    L.q8_gated_ff_forward.argtypes = [P, P, C.c_int64, P, S]
    L.q8_gated_ff_backward.argtypes = [P, P, C.c_int64, P, P, C.c_int64, P, P, S]
    L.q8_block_norm_forward.argtypes = [P, P, C.c_int64, P, C.c_int64, S]
    L.q8_block_norm_workspace.argtypes = [P, P]
    L.q8_block_norm_backward.argtypes = [P, P, S]
    L.q8_distill_topk_forward.argtypes = [P, P, P, P, C.c_int64, S]
    L.q8_distill_topk_backward.argtypes = [P, P, P, C.c_int64, S]
    for name in EXPORTS:
        if name.endswith("_workspace"):
            getattr(L, name).restype = C.c_int64
        elif name not in ("q8_last_error",):
            getattr(L, name).restype = C.c_int
    _lib = L
    return L


def _check(fn, rc):
    if rc != Q8_OK:
        raise Q8Error(fn, rc, load_library().q8_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return C.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return C.c_void_p(stream.cuda_stream)
    return C.c_void_p(int(stream))


def hparams(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1, seed=0, sr=1, exact=0):
    """q8_adamw_hparams; exact=0 is the fast mode (approximate square root and
    reciprocal in the parameter update of full blocks), exact=1 the bit-exact one."""
    return HParams(lr, beta1, beta2, eps, weight_decay, step, seed, sr, int(exact))


def momentum_hparams(lr=1e-2, momentum=0.9, weight_decay=0.0, step=1, seed=0, sr=1):
    return MomentumHParams(lr, momentum, weight_decay, step, seed, sr)


def lion_hparams(lr=1e-4, beta1=0.9, beta2=0.99, weight_decay=0.0, step=1, seed=0, sr=1):
    return LionHParams(lr, beta1, beta2, weight_decay, step, seed, sr)


# ---------------------------------------------------------------- entry points

def q8_abi_version() -> int:
    return load_library().q8_abi_version()


def q8_last_error() -> str:
    return load_library().q8_last_error().decode()


def q8_prepare_device() -> None:
    _check("q8_prepare_device", load_library().q8_prepare_device())


def q8_codebook_init(kind: int) -> np.ndarray:
    out = np.zeros(256, np.float32)
    _check("q8_codebook_init", load_library().q8_codebook_init(kind, out.ctypes.data))
    return out


def q8_blockwise_quantize(x: torch.Tensor, codes: torch.Tensor, absmax: torch.Tensor, kind: int,
                          stream=None) -> None:
    assert x.dtype == torch.float32 and codes.dtype == torch.uint8 and absmax.dtype == torch.float32
    n = x.numel()
    assert codes.numel() >= n and absmax.numel() >= (n + BLOCK - 1) // BLOCK
    _check("q8_blockwise_quantize", load_library().q8_blockwise_quantize(
        _ptr(x), _ptr(codes), _ptr(absmax), n, kind, _stream(stream)))


def q8_blockwise_dequantize(codes: torch.Tensor, absmax: torch.Tensor, x: torch.Tensor, kind: int,
                            stream=None) -> None:
    assert x.dtype == torch.float32 and codes.dtype == torch.uint8 and absmax.dtype == torch.float32
    n = x.numel()
    assert codes.numel() >= n and absmax.numel() >= (n + BLOCK - 1) // BLOCK
    _check("q8_blockwise_dequantize", load_library().q8_blockwise_dequantize(
        _ptr(codes), _ptr(absmax), _ptr(x), n, kind, _stream(stream)))


def q8_philox_fill(seed: int, step: int, stream_id: int, offset: int, out: torch.Tensor,
                   stream=None) -> None:
    assert out.element_size() == 2, "out holds 16-bit draws (int16 or uint16)"
    _check("q8_philox_fill", load_library().q8_philox_fill(
        seed, step, stream_id, offset, out.numel(), _ptr(out), _stream(stream)))


def q8_selftest_sqrt_div(counts: torch.Tensor, stream=None) -> None:
    """Device self-test of the packed square root and division; counts:
    int64[8] on the GPU (reciprocal mismatches, d values checked, quotient
    mismatches, pairs checked, square-root mismatches, v values checked, and
    the largest relative errors of the fast mode's approximate square root and
    reciprocal as float bit patterns)."""
    assert counts.dtype == torch.int64 and counts.numel() >= 8 and counts.is_contiguous()
    _check("q8_selftest_sqrt_div", load_library().q8_selftest_sqrt_div(_ptr(counts), _stream(stream)))


@dataclass
class Tensor8:
    """One tensor of the 8-bit step: bf16 param/grad plus its optimizer state
    (uint8 codes + float32 block absmax when numel >= 4096, else float32
    m32/v32).  philox_offset < 0 means the running element count."""
    param: torch.Tensor
    grad: torch.Tensor
    m_codes: Optional[torch.Tensor] = None
    v_codes: Optional[torch.Tensor] = None
    m_absmax: Optional[torch.Tensor] = None
    v_absmax: Optional[torch.Tensor] = None
    m32: Optional[torch.Tensor] = None
    v32: Optional[torch.Tensor] = None
    philox_offset: int = -1

    @classmethod
    def zeros_like(cls, param: torch.Tensor, grad: Optional[torch.Tensor] = None, philox_offset=-1,
                   moments: int = 2):
        """Fresh (all-zero) state for `param` on its device: first and second
        moment (AdamW) or, with moments=1, the first only (Momentum, Lion)."""
        n = param.numel()
        dev = param.device
        two = moments == 2
        if n >= SMALL_NUMEL:
            nb = (n + BLOCK - 1) // BLOCK
            return cls(param, grad, torch.full((n,), 127, dtype=torch.uint8, device=dev),
                       torch.zeros(n, dtype=torch.uint8, device=dev) if two else None,
                       torch.zeros(nb, dtype=torch.float32, device=dev),
                       torch.zeros(nb, dtype=torch.float32, device=dev) if two else None,
                       philox_offset=philox_offset)
        return cls(param, grad, m32=torch.zeros(n, dtype=torch.float32, device=dev),
                   v32=torch.zeros(n, dtype=torch.float32, device=dev) if two else None,
                   philox_offset=philox_offset)

    def slice(self, start: int, count: int, philox_offset: int):
        """Block-aligned slice [start, start + count) of this tensor with the
        given global Philox offset (the 8-bit state stays on the 8-bit path)."""
        assert self.m_codes is not None, "slices are taken of 8-bit state"
        assert start % BLOCK == 0 and 0 <= start and start + count <= self.param.numel()
        b0, b1 = start // BLOCK, (start + count + BLOCK - 1) // BLOCK
        sl = slice(start, start + count)
        opt = lambda t, s: None if t is None else t[s]
        return Tensor8(self.param[sl], opt(self.grad, sl), self.m_codes[sl], opt(self.v_codes, sl),
                       self.m_absmax[b0:b1], opt(self.v_absmax, slice(b0, b1)), philox_offset=philox_offset)

    def _struct(self):
        assert self.param.dtype == torch.bfloat16 and self.grad.dtype == torch.bfloat16
        assert self.grad.numel() == self.param.numel()
        return _Tensor8(_ptr(self.param), _ptr(self.grad), self.param.numel(), self.philox_offset,
                        _ptr(self.m_codes), _ptr(self.v_codes), _ptr(self.m_absmax),
                        _ptr(self.v_absmax), _ptr(self.m32), _ptr(self.v32))


@dataclass
class Tensor16:
    """One tensor of the BF16-state step (all bf16)."""
    param: torch.Tensor
    grad: torch.Tensor
    m: torch.Tensor
    v: torch.Tensor
    philox_offset: int = -1

    def _struct(self):
        for t in (self.param, self.grad, self.m, self.v):
            assert t.dtype == torch.bfloat16 and t.numel() == self.param.numel()
        return _Tensor16(_ptr(self.param), _ptr(self.grad), _ptr(self.m), _ptr(self.v),
                         self.param.numel(), self.philox_offset)


def pack_tensor8(tensors: Sequence[Tensor8]):
    """ctypes array for adamw8bit_sr_step (keep it to re-issue the same list)."""
    return (_Tensor8 * len(tensors))(*[t._struct() for t in tensors])


def pack_tensor16(tensors: Sequence[Tensor16]):
    return (_Tensor16 * len(tensors))(*[t._struct() for t in tensors])


def adamw8bit_sr_step(tensors, hp: HParams, stream=None) -> None:
    """Fused 8-bit blockwise AdamW + SR step over a list of Tensor8 (or a list
    already packed by pack_tensor8)."""
    arr = tensors if isinstance(tensors, C.Array) else pack_tensor8(tensors)
    _check("adamw8bit_sr_step", load_library().adamw8bit_sr_step(arr, len(arr), C.byref(hp), _stream(stream)))


def adamw_bf16_sr_step(tensors, hp: HParams, stream=None) -> None:
    """BF16-state AdamW + SR step over a list of Tensor16 (or a packed list)."""
    arr = tensors if isinstance(tensors, C.Array) else pack_tensor16(tensors)
    _check("adamw_bf16_sr_step", load_library().adamw_bf16_sr_step(arr, len(arr), C.byref(hp), _stream(stream)))


def momentum8bit_sr_step(tensors, hp: MomentumHParams, stream=None) -> None:
    """8-bit SGD-with-momentum step with SR parameter write over a list of
    Tensor8 holding first-moment state only (see Tensor8.zeros_like(moments=1))."""
    arr = tensors if isinstance(tensors, C.Array) else pack_tensor8(tensors)
    _check("momentum8bit_sr_step", load_library().momentum8bit_sr_step(arr, len(arr), C.byref(hp), _stream(stream)))


def lion8bit_sr_step(tensors, hp: LionHParams, stream=None) -> None:
    """8-bit Lion step with SR parameter write (first-moment state only)."""
    arr = tensors if isinstance(tensors, C.Array) else pack_tensor8(tensors)
    _check("lion8bit_sr_step", load_library().lion8bit_sr_step(arr, len(arr), C.byref(hp), _stream(stream)))


# ------------------------------------------------- training-step operators

def _rows(t: torch.Tensor, name: str, dtype, cols=None, rows=None):
    """(address, row stride) of a [rows, cols] matrix whose rows are contiguous."""
    shape = t.shape
    if t.dtype != dtype or not t.is_cuda or len(shape) != 2 or (cols is not None and shape[1] != cols) or \
            (rows is not None and shape[0] != rows):
        raise ValueError("%s must be a %s CUDA matrix%s" % (name, dtype, "" if cols is None else " of the matching size"))
    row, col = t.stride()
    if col != 1 and shape[1] != 1:
        raise ValueError("%s's rows must be contiguous" % name)
    return t.data_ptr(), row if shape[0] > 1 else shape[1]


def _array(t: Optional[torch.Tensor], name: str, dtype, shape):
    """Address of a contiguous array of that type and shape, or None."""
    if t is None:
        return None
    if t.dtype != dtype or not t.is_cuda or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s CUDA array of shape %s" % (name, dtype, tuple(shape)))
    return t.data_ptr()


def _opt_rows(t, name, dtype, cols, rows):
    return (None, 0) if t is None else _rows(t, name, dtype, cols, rows)


def _workspace(fn, bytes_, workspace, device, stream):
    """(address, bytes, the tensor that holds it): the caller's workspace, or
    one from torch's allocator for the stream that the call runs on."""
    if bytes_ < 0:
        _check(fn, bytes_)
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    if bytes_ == 0:
        return None, 0, None
    if stream is None:
        t = torch.empty(bytes_, dtype=torch.uint8, device=device)
    else:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else \
                torch.cuda.default_stream(device)
        with torch.cuda.stream(stream):
            t = torch.empty(bytes_, dtype=torch.uint8, device=device)
    return t.data_ptr(), bytes_, t


def _gated_ff(x, w_gate, w_up, act):
    xp, xs = _rows(x, "x", torch.bfloat16)
    tokens, d_model = x.shape
    d_ff = w_gate.shape[0]
    wg = _array(w_gate, "w_gate", torch.bfloat16, (d_ff, d_model))
    wu = _array(w_up, "w_up", torch.bfloat16, (d_ff, d_model))
    return _GatedFF(xp, wg, wu, tokens, d_model, d_ff, xs, None, 0, act)


def q8_gated_ff_workspace(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, backward=False) -> int:
    """Bytes of workspace of q8_gated_ff_forward (backward: of ..._backward)."""
    n = load_library().q8_gated_ff_workspace(C.byref(_gated_ff(x, w_gate, w_up, SILU)), int(backward))
    if n < 0:
        _check("q8_gated_ff_workspace", n)
    return n


def q8_gated_ff_forward(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, h: torch.Tensor, act: int = SILU,
                        saved: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        stream=None) -> None:
    """h = act(x w_gate^T) * (x w_up^T); saved: float32 [2, tokens, d_ff] that
    receives both projections for the backward call.  Without a workspace the
    binding allocates one (from torch's caching allocator) where it is needed."""
    L = load_library()
    f = _gated_ff(x, w_gate, w_up, act)
    hp, hs = _rows(h, "h", torch.bfloat16, f.d_ff, f.tokens)
    sp = _array(saved, "saved", torch.float32, (2, f.tokens, f.d_ff))
    need = L.q8_gated_ff_workspace(C.byref(f), 0)
    f.workspace, f.workspace_bytes, keep = _workspace("q8_gated_ff_forward", need, workspace, x.device, stream)
    _check("q8_gated_ff_forward", L.q8_gated_ff_forward(C.byref(f), hp, hs, sp, _stream(stream)))


def q8_gated_ff_backward(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, dh: torch.Tensor,
                         dx: Optional[torch.Tensor], dw_gate: Optional[torch.Tensor],
                         dw_up: Optional[torch.Tensor], act: int = SILU, saved: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """dx, dw_gate, dw_up (each may be None) from dh; saved as the forward call
    wrote it, or None to compute both projections again."""
    L = load_library()
    f = _gated_ff(x, w_gate, w_up, act)
    dhp, dhs = _rows(dh, "dh", torch.bfloat16, f.d_ff, f.tokens)
    sp = _array(saved, "saved", torch.float32, (2, f.tokens, f.d_ff))
    dxp, dxs = _opt_rows(dx, "dx", torch.bfloat16, f.d_model, f.tokens)
    gp = _array(dw_gate, "dw_gate", torch.bfloat16, w_gate.shape)
    up = _array(dw_up, "dw_up", torch.bfloat16, w_up.shape)
    need = L.q8_gated_ff_workspace(C.byref(f), 1)
    f.workspace, f.workspace_bytes, keep = _workspace("q8_gated_ff_backward", need, workspace, x.device, stream)
    _check("q8_gated_ff_backward", L.q8_gated_ff_backward(C.byref(f), dhp, dhs, sp, dxp, dxs, gp, up, _stream(stream)))


_DTYPES = {torch.bfloat16: 0, torch.float32: 1}     # q8_dtype


def _dtype(t, name):
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError("%s must be bfloat16 or float32" % name)
    return d


def _block_norm(residual, y, post_kind, pre_kind, post_weight, post_bias, pre_weight, pre_bias, gate, gate_tokens,
                residual_scale, eps):
    bf = torch.bfloat16
    yp, ys = _rows(y, "y", bf)
    tokens, dim = y.shape
    rp, rs = _rows(residual, "residual", residual.dtype, dim, tokens)
    vec = (dim,)
    gp = None
    if gate is not None:
        rows = gate.numel() // dim
        if gate_tokens is None:
            if rows < 1 or tokens % rows:
                raise ValueError("gate's rows must divide the tokens (or give gate_tokens)")
            gate_tokens = max(1, tokens // rows)
        elif gate_tokens > 0 and rows < -(-tokens // gate_tokens):
            raise ValueError("gate has fewer rows than ceil(tokens / gate_tokens)")
        gp = _array(gate, "gate", bf, vec if gate.dim() == 1 else (rows, dim))
    return _BlockNorm(rp, yp, _array(post_weight, "post_weight", bf, vec), _array(post_bias, "post_bias", bf, vec),
                      _array(pre_weight, "pre_weight", bf, vec), _array(pre_bias, "pre_bias", bf, vec), gp, tokens, dim,
                      gate_tokens or 0, rs, ys, post_kind, pre_kind, _dtype(residual, "residual"), eps, residual_scale)


def q8_block_norm_forward(residual: torch.Tensor, y: torch.Tensor, residual_out: Optional[torch.Tensor],
                          z: Optional[torch.Tensor], post_kind: int, pre_kind: int, post_weight=None, post_bias=None,
                          pre_weight=None, pre_bias=None, gate=None, gate_tokens: Optional[int] = None,
                          residual_scale: float = 1.0, eps: float = 1e-5, stream=None) -> None:
    """residual_out = residual_scale * residual + gate * N_post(y) and
    z = N_pre(residual_out).  gate: [dim] or [rows, dim], a row for each
    gate_tokens consecutive tokens (by default tokens / rows)."""
    n = _block_norm(residual, y, post_kind, pre_kind, post_weight, post_bias, pre_weight, pre_bias, gate, gate_tokens,
                    residual_scale, eps)
    op, os_ = _opt_rows(residual_out, "residual_out", residual.dtype, n.dim, n.tokens)
    zp, zs = _opt_rows(z, "z", torch.bfloat16, n.dim, n.tokens)
    _check("q8_block_norm_forward",
           load_library().q8_block_norm_forward(C.byref(n), op, os_, zp, zs, _stream(stream)))


def q8_block_norm_backward(residual: torch.Tensor, y: torch.Tensor, dresidual_out: Optional[torch.Tensor],
                           dz: Optional[torch.Tensor], dresidual: Optional[torch.Tensor],
                           dy: Optional[torch.Tensor], post_kind: int, pre_kind: int, post_weight=None,
                           post_bias=None, pre_weight=None, pre_bias=None, gate=None,
                           gate_tokens: Optional[int] = None, residual_scale: float = 1.0, eps: float = 1e-5,
                           dpost_weight=None, dpost_bias=None, dpre_weight=None, dpre_bias=None, dgate=None,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """The gradients of q8_block_norm_forward's inputs (each output may be
    None) from those of its outputs (None: zeros)."""
    L = load_library()
    n = _block_norm(residual, y, post_kind, pre_kind, post_weight, post_bias, pre_weight, pre_bias, gate, gate_tokens,
                    residual_scale, eps)
    bf, vec = torch.bfloat16, (n.dim,)
    rop, ros = _opt_rows(dresidual_out, "dresidual_out", residual.dtype, n.dim, n.tokens)
    dzp, dzs = _opt_rows(dz, "dz", bf, n.dim, n.tokens)
    drp, drs = _opt_rows(dresidual, "dresidual", residual.dtype, n.dim, n.tokens)
    dyp, dys = _opt_rows(dy, "dy", bf, n.dim, n.tokens)
    if dgate is not None and gate is None:
        raise ValueError("dgate without a gate")
    g = _BlockNormGrads(rop, dzp, drp, dyp, _array(dpost_weight, "dpost_weight", bf, vec),
                        _array(dpost_bias, "dpost_bias", bf, vec), _array(dpre_weight, "dpre_weight", bf, vec),
                        _array(dpre_bias, "dpre_bias", bf, vec),
                        None if dgate is None else _array(dgate, "dgate", bf, gate.shape), ros, dzs, drs, dys, None, 0)
    need = L.q8_block_norm_workspace(C.byref(n), C.byref(g))
    g.workspace, g.workspace_bytes, keep = _workspace("q8_block_norm_backward", need, workspace, y.device, stream)
    _check("q8_block_norm_backward", L.q8_block_norm_backward(C.byref(n), C.byref(g), _stream(stream)))


def _distill(logits, teacher_ids, teacher_logits, labels, row_weight, temperature, kd_weight, ce_weight):
    zp, zs = _rows(logits, "logits", logits.dtype)
    rows, vocab = logits.shape
    k = teacher_ids.shape[1] if teacher_ids is not None else 0
    return _DistillTopk(zp, _array(teacher_ids, "teacher_ids", torch.int64, (rows, k)),
                        _array(teacher_logits, "teacher_logits", torch.float32, (rows, k)),
                        _array(labels, "labels", torch.int64, (rows,)),
                        _array(row_weight, "row_weight", torch.float32, (rows,)), rows, vocab, k, zs,
                        _dtype(logits, "logits"), temperature, kd_weight, ce_weight)


def q8_distill_topk_forward(logits: torch.Tensor, teacher_ids: Optional[torch.Tensor],
                            teacher_logits: Optional[torch.Tensor], loss: torch.Tensor,
                            stats: Optional[torch.Tensor] = None, labels: Optional[torch.Tensor] = None,
                            row_weight: Optional[torch.Tensor] = None, dlogits: Optional[torch.Tensor] = None,
                            temperature: float = 1.0, kd_weight: float = 1.0, ce_weight: float = 0.0,
                            stream=None) -> None:
    """Each row's distillation loss (float32 [rows]); stats: float32 [rows, 2]
    for the backward call; dlogits: the gradient of sum(row_weight * loss) in
    the same pass (it may be the logits themselves)."""
    d = _distill(logits, teacher_ids, teacher_logits, labels, row_weight, temperature, kd_weight, ce_weight)
    lp = _array(loss, "loss", torch.float32, (d.rows,))
    sp = _array(stats, "stats", torch.float32, (d.rows, 2))
    gp, gs = _opt_rows(dlogits, "dlogits", logits.dtype, d.vocab, d.rows)
    _check("q8_distill_topk_forward",
           load_library().q8_distill_topk_forward(C.byref(d), lp, sp, gp, gs, _stream(stream)))


def q8_distill_topk_backward(logits: torch.Tensor, teacher_ids: Optional[torch.Tensor],
                             teacher_logits: Optional[torch.Tensor], stats: torch.Tensor, dlogits: torch.Tensor,
                             labels: Optional[torch.Tensor] = None, row_weight: Optional[torch.Tensor] = None,
                             temperature: float = 1.0, kd_weight: float = 1.0, ce_weight: float = 0.0,
                             stream=None) -> None:
    """The logits' gradient from the forward call's stats; row_weight: the
    gradient of the losses."""
    d = _distill(logits, teacher_ids, teacher_logits, labels, row_weight, temperature, kd_weight, ce_weight)
    sp = _array(stats, "stats", torch.float32, (d.rows, 2))
    gp, gs = _rows(dlogits, "dlogits", logits.dtype, d.vocab, d.rows)
    _check("q8_distill_topk_backward",
           load_library().q8_distill_topk_backward(C.byref(d), sp, gp, gs, _stream(stream)))
