"""ctypes binding of libq8adamw.so: argument marshalling only.

Every function here has the name of the C entry point it calls (see
include/q8adamw.h and include/q8train.h) and takes torch tensors that already live on a CUDA device;
all work runs in the library's kernels.  A missing library is an error: there
is no fallback path.
"""
import ctypes as C
import os
import struct
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


# The argument structures of include/q8train.h.  These calls are short, and what
# goes before the launch is a good part of the smallest ones: their structures
# are packed as bytes (native alignment, as the C compiler lays them out), which
# takes half the time of filling a ctypes.Structure.
_GATED_FF = struct.Struct("PPPqqqqPqi4x")
_BLOCK_NORM = struct.Struct("PPPPPPPqqqqqiiiff4x")
_BLOCK_NORM_GRADS = struct.Struct("PPPPPPPPPqqqqPq")
_DISTILL_TOPK = struct.Struct("PPPPPqqqqifff")


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
    # the structures go as the addresses of their bytes
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

_raw_stream = torch._C._cuda_getCurrentRawStream
_BF, _F32, _I64 = torch.bfloat16, torch.float32, torch.int64
_DTYPES = {_BF: 0, _F32: 1}                          # q8_dtype


def _on(stream, t):
    """The stream's address: the given one, or the current one of t's device."""
    if stream is None:
        return _raw_stream(t.get_device())
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _rows(t: torch.Tensor, name: str, dtype, shape):
    """(address, row stride) of a [rows, cols] matrix whose rows are contiguous."""
    if t.dtype is not dtype or not t.is_cuda or t.shape != shape:
        raise ValueError("%s must be a %s CUDA matrix of shape %s" % (name, dtype, tuple(shape)))
    if t.is_contiguous():
        return t.data_ptr(), shape[1]
    row, col = t.stride()
    if col != 1 and shape[1] != 1:
        raise ValueError("%s's rows must be contiguous" % name)
    return t.data_ptr(), row if shape[0] > 1 else shape[1]


def _first(t: torch.Tensor, name: str, dtype):
    """_rows of the matrix that the others' sizes follow from."""
    if t.dim() != 2:
        raise ValueError("%s must be a %s CUDA matrix" % (name, dtype))
    return _rows(t, name, dtype, t.shape)


def _array(t: Optional[torch.Tensor], name: str, dtype, shape):
    """Address of a contiguous array of that type and shape, or 0."""
    if t is None:
        return 0
    if t.dtype is not dtype or not t.is_cuda or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s CUDA array of shape %s" % (name, dtype, tuple(shape)))
    return t.data_ptr()


def _torch_stream(stream, like):
    """The given stream for torch.cuda.stream(); None is the current one."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream), device=like.device) if int(stream) else torch.cuda.default_stream(like.device)


def _workspace(fn, need, workspace, like, stream):
    """(address, bytes, the tensor that holds it): the caller's workspace, or
    one from torch's allocator for the stream that the call runs on."""
    if need < 0:
        _check(fn, need)
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    if need == 0:
        return 0, 0, None
    with torch.cuda.stream(_torch_stream(stream, like)):
        t = torch.empty(need, dtype=torch.uint8, device=like.device)
    return t.data_ptr(), need, t


def _gated_ff(x, w_gate, w_up, act):
    xp, xs = _first(x, "x", _BF)
    tokens, d_model = x.shape
    d_ff = w_gate.shape[0]
    shape = (d_ff, d_model)
    return (xp, _array(w_gate, "w_gate", _BF, shape), _array(w_up, "w_up", _BF, shape), tokens, d_model, d_ff, xs), act


def q8_gated_ff_workspace(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, backward=False) -> int:
    """Bytes of workspace of q8_gated_ff_forward (backward: of ..._backward)."""
    f, act = _gated_ff(x, w_gate, w_up, SILU)
    n = load_library().q8_gated_ff_workspace(_GATED_FF.pack(*f, 0, 0, act), int(backward))
    if n < 0:
        _check("q8_gated_ff_workspace", n)
    return n


def q8_gated_ff_forward(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, h: torch.Tensor, act: int = SILU,
                        saved: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        stream=None) -> None:
    """h = act(x w_gate^T) * (x w_up^T); saved: float32 [2, tokens, d_ff] that
    receives both projections for the backward call.  Without a workspace the
    binding allocates one (from torch's caching allocator) where it is needed."""
    L = _lib or load_library()
    f, act = _gated_ff(x, w_gate, w_up, act)
    tokens, d_ff = f[3], f[5]
    hp, hs = _rows(h, "h", _BF, (tokens, d_ff))
    sp = _array(saved, "saved", _F32, (2, tokens, d_ff))
    need = L.q8_gated_ff_workspace(_GATED_FF.pack(*f, 0, 0, act), 0)
    wp, wb, keep = (0, 0, None) if need == 0 else _workspace("q8_gated_ff_forward", need, workspace, x, stream)
    rc = L.q8_gated_ff_forward(_GATED_FF.pack(*f, wp, wb, act), hp, hs, sp, _on(stream, x))
    if rc:
        _check("q8_gated_ff_forward", rc)


def q8_gated_ff_backward(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, dh: torch.Tensor,
                         dx: Optional[torch.Tensor], dw_gate: Optional[torch.Tensor],
                         dw_up: Optional[torch.Tensor], act: int = SILU, saved: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """dx, dw_gate, dw_up (each may be None) from dh; saved as the forward call
    wrote it, or None to compute both projections again."""
    L = _lib or load_library()
    f, act = _gated_ff(x, w_gate, w_up, act)
    tokens, d_model, d_ff = f[3:6]
    dhp, dhs = _rows(dh, "dh", _BF, (tokens, d_ff))
    sp = _array(saved, "saved", _F32, (2, tokens, d_ff))
    dxp, dxs = (0, 0) if dx is None else _rows(dx, "dx", _BF, (tokens, d_model))
    gp = _array(dw_gate, "dw_gate", _BF, (d_ff, d_model))
    up = _array(dw_up, "dw_up", _BF, (d_ff, d_model))
    need = L.q8_gated_ff_workspace(_GATED_FF.pack(*f, 0, 0, act), 1)
    wp, wb, keep = _workspace("q8_gated_ff_backward", need, workspace, x, stream)
    rc = L.q8_gated_ff_backward(_GATED_FF.pack(*f, wp, wb, act), dhp, dhs, sp, dxp, dxs, gp, up, _on(stream, x))
    if rc:
        _check("q8_gated_ff_backward", rc)


def _dtype(t, name):
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError("%s must be bfloat16 or float32" % name)
    return d


def _block_norm(residual, y, post_kind, pre_kind, post_weight, post_bias, pre_weight, pre_bias, gate, gate_tokens,
                residual_scale, eps):
    yp, ys = _first(y, "y", _BF)
    shape = y.shape
    tokens, dim = shape
    dtype = _dtype(residual, "residual")
    rp, rs = _rows(residual, "residual", residual.dtype, shape)
    vec = (dim,)
    gp = 0
    if gate is not None:
        if gate.dim() == 1:
            rows, gp = 1, _array(gate, "gate", _BF, vec)
        else:
            rows = gate.shape[0]
            gp = _array(gate, "gate", _BF, (rows, dim))
        if gate_tokens is None:
            if rows < 1 or tokens % rows:
                raise ValueError("gate's rows must divide the tokens (or give gate_tokens)")
            gate_tokens = max(1, tokens // rows)
        elif gate_tokens > 0 and rows < -(-tokens // gate_tokens):
            raise ValueError("gate has fewer rows than ceil(tokens / gate_tokens)")
    return _BLOCK_NORM.pack(rp, yp, _array(post_weight, "post_weight", _BF, vec), _array(post_bias, "post_bias", _BF, vec),
                            _array(pre_weight, "pre_weight", _BF, vec), _array(pre_bias, "pre_bias", _BF, vec), gp,
                            tokens, dim, gate_tokens or 0, rs, ys, post_kind, pre_kind, dtype, eps, residual_scale)


def q8_block_norm_forward(residual: torch.Tensor, y: torch.Tensor, residual_out: Optional[torch.Tensor],
                          z: Optional[torch.Tensor], post_kind: int, pre_kind: int, post_weight=None, post_bias=None,
                          pre_weight=None, pre_bias=None, gate=None, gate_tokens: Optional[int] = None,
                          residual_scale: float = 1.0, eps: float = 1e-5, stream=None) -> None:
    """residual_out = residual_scale * residual + gate * N_post(y) and
    z = N_pre(residual_out).  gate: [dim] or [rows, dim], a row for each
    gate_tokens consecutive tokens (by default tokens / rows)."""
    L = _lib or load_library()
    n = _block_norm(residual, y, post_kind, pre_kind, post_weight, post_bias, pre_weight, pre_bias, gate, gate_tokens,
                    residual_scale, eps)
    shape = y.shape
    op, os_ = (0, 0) if residual_out is None else _rows(residual_out, "residual_out", residual.dtype, shape)
    zp, zs = (0, 0) if z is None else _rows(z, "z", _BF, shape)
    rc = L.q8_block_norm_forward(n, op, os_, zp, zs, _on(stream, y))
    if rc:
        _check("q8_block_norm_forward", rc)


def _block_norm_backward(residual, y, dresidual_out, dz, dresidual, dy, post_kind, pre_kind, post_weight, post_bias, pre_weight,
                         pre_bias, gate, gate_tokens, residual_scale, eps, dpost_weight, dpost_bias, dpre_weight, dpre_bias,
                         dgate):
    """The norm's structure, and the fields of the gradients' before the workspace."""
    n = _block_norm(residual, y, post_kind, pre_kind, post_weight, post_bias, pre_weight, pre_bias, gate, gate_tokens,
                    residual_scale, eps)
    shape, dtype = y.shape, residual.dtype
    vec = (shape[1],)
    rop, ros = (0, 0) if dresidual_out is None else _rows(dresidual_out, "dresidual_out", dtype, shape)
    dzp, dzs = (0, 0) if dz is None else _rows(dz, "dz", _BF, shape)
    drp, drs = (0, 0) if dresidual is None else _rows(dresidual, "dresidual", dtype, shape)
    dyp, dys = (0, 0) if dy is None else _rows(dy, "dy", _BF, shape)
    if dgate is not None and gate is None:
        raise ValueError("dgate without a gate")
    return n, (rop, dzp, drp, dyp, _array(dpost_weight, "dpost_weight", _BF, vec), _array(dpost_bias, "dpost_bias", _BF, vec),
               _array(dpre_weight, "dpre_weight", _BF, vec), _array(dpre_bias, "dpre_bias", _BF, vec),
               0 if dgate is None else _array(dgate, "dgate", _BF, gate.shape), ros, dzs, drs, dys)


def q8_block_norm_workspace(residual: torch.Tensor, y: torch.Tensor, dresidual_out: Optional[torch.Tensor],
                            dz: Optional[torch.Tensor], dresidual: Optional[torch.Tensor], dy: Optional[torch.Tensor],
                            post_kind: int, pre_kind: int, post_weight=None, post_bias=None, pre_weight=None,
                            pre_bias=None, gate=None, gate_tokens: Optional[int] = None, residual_scale: float = 1.0,
                            eps: float = 1e-5, dpost_weight=None, dpost_bias=None, dpre_weight=None, dpre_bias=None,
                            dgate=None) -> int:
    """Bytes of workspace of q8_block_norm_backward with these arguments."""
    n, g = _block_norm_backward(residual, y, dresidual_out, dz, dresidual, dy, post_kind, pre_kind, post_weight, post_bias,
                                pre_weight, pre_bias, gate, gate_tokens, residual_scale, eps, dpost_weight, dpost_bias,
                                dpre_weight, dpre_bias, dgate)
    need = load_library().q8_block_norm_workspace(n, _BLOCK_NORM_GRADS.pack(*g, 0, 0))
    if need < 0:
        _check("q8_block_norm_workspace", need)
    return need


def q8_block_norm_backward(residual: torch.Tensor, y: torch.Tensor, dresidual_out: Optional[torch.Tensor],
                           dz: Optional[torch.Tensor], dresidual: Optional[torch.Tensor],
                           dy: Optional[torch.Tensor], post_kind: int, pre_kind: int, post_weight=None,
                           post_bias=None, pre_weight=None, pre_bias=None, gate=None,
                           gate_tokens: Optional[int] = None, residual_scale: float = 1.0, eps: float = 1e-5,
                           dpost_weight=None, dpost_bias=None, dpre_weight=None, dpre_bias=None, dgate=None,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """The gradients of q8_block_norm_forward's inputs (each output may be
    None) from those of its outputs (None: zeros).  Rows of a gate that no
    token has get a gradient of zeros: all of them where there are no tokens."""
    L = _lib or load_library()
    n, g = _block_norm_backward(residual, y, dresidual_out, dz, dresidual, dy, post_kind, pre_kind, post_weight, post_bias,
                                pre_weight, pre_bias, gate, gate_tokens, residual_scale, eps, dpost_weight, dpost_bias,
                                dpre_weight, dpre_bias, dgate)
    need = L.q8_block_norm_workspace(n, _BLOCK_NORM_GRADS.pack(*g, 0, 0))
    wp, wb, keep = _workspace("q8_block_norm_backward", need, workspace, y, stream)
    rc = L.q8_block_norm_backward(n, _BLOCK_NORM_GRADS.pack(*g, wp, wb), _on(stream, y))
    if rc:
        _check("q8_block_norm_backward", rc)
    if dgate is not None:
        (tokens, dim), rows = y.shape, 1 if gate.dim() == 1 else gate.shape[0]
        used = -(-tokens // gate_tokens) if gate_tokens else rows if tokens else 0       # what the call writes
        if used < rows:
            with torch.cuda.stream(_torch_stream(stream, y)):
                dgate.view(rows, dim)[used:].zero_()


def _distill(logits, teacher_ids, teacher_logits, labels, row_weight, temperature, kd_weight, ce_weight):
    dtype = _dtype(logits, "logits")
    zp, zs = _first(logits, "logits", logits.dtype)
    rows, vocab = logits.shape
    k = teacher_ids.shape[1] if teacher_ids is not None else 0
    vec = (rows,)
    return _DISTILL_TOPK.pack(zp, _array(teacher_ids, "teacher_ids", _I64, (rows, k)),
                              _array(teacher_logits, "teacher_logits", _F32, (rows, k)),
                              _array(labels, "labels", _I64, vec), _array(row_weight, "row_weight", _F32, vec),
                              rows, vocab, k, zs, dtype, temperature, kd_weight, ce_weight)


def q8_distill_topk_forward(logits: torch.Tensor, teacher_ids: Optional[torch.Tensor],
                            teacher_logits: Optional[torch.Tensor], loss: torch.Tensor,
                            stats: Optional[torch.Tensor] = None, labels: Optional[torch.Tensor] = None,
                            row_weight: Optional[torch.Tensor] = None, dlogits: Optional[torch.Tensor] = None,
                            temperature: float = 1.0, kd_weight: float = 1.0, ce_weight: float = 0.0,
                            stream=None) -> None:
    """Each row's distillation loss (float32 [rows]); stats: float32 [rows, 2]
    for the backward call; dlogits: the gradient of sum(row_weight * loss) in
    the same pass (it may be the logits themselves)."""
    L = _lib or load_library()
    d = _distill(logits, teacher_ids, teacher_logits, labels, row_weight, temperature, kd_weight, ce_weight)
    rows = logits.shape[0]
    lp = _array(loss, "loss", _F32, (rows,))
    sp = _array(stats, "stats", _F32, (rows, 2))
    gp, gs = (0, 0) if dlogits is None else _rows(dlogits, "dlogits", logits.dtype, logits.shape)
    rc = L.q8_distill_topk_forward(d, lp, sp, gp, gs, _on(stream, logits))
    if rc:
        _check("q8_distill_topk_forward", rc)


def q8_distill_topk_backward(logits: torch.Tensor, teacher_ids: Optional[torch.Tensor],
                             teacher_logits: Optional[torch.Tensor], stats: torch.Tensor, dlogits: torch.Tensor,
                             labels: Optional[torch.Tensor] = None, row_weight: Optional[torch.Tensor] = None,
                             temperature: float = 1.0, kd_weight: float = 1.0, ce_weight: float = 0.0,
                             stream=None) -> None:
    """The logits' gradient from the forward call's stats; row_weight: the
    gradient of the losses."""
    L = _lib or load_library()
    d = _distill(logits, teacher_ids, teacher_logits, labels, row_weight, temperature, kd_weight, ce_weight)
    sp = _array(stats, "stats", _F32, (logits.shape[0], 2))
    gp, gs = _rows(dlogits, "dlogits", logits.dtype, logits.shape)
    rc = L.q8_distill_topk_backward(d, sp, gp, gs, _on(stream, logits))
    if rc:
        _check("q8_distill_topk_backward", rc)
