"""Thin Python binding of libqlora_nf4 (ctypes over the C ABI in include/qlora_nf4.h).

Argument marshalling only: every step of the computation runs in the library's CUDA kernels.
PyTorch supplies device memory (including the caller-owned workspace) and the current stream.
There is no fallback: if the library is missing or the device is not an sm_100 GPU, the
calls raise.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

from . import build as _build

QLORA_OK = 0
QLORA_ERR_INVALID_ARG = -1
QLORA_ERR_BAD_SHAPE = -2
QLORA_ERR_MISALIGNED = -3
QLORA_ERR_WORKSPACE = -4
QLORA_ERR_CUDA = -5
QLORA_ERR_UNSUPPORTED_DEVICE = -6
QLORA_ERR_SCRATCH_LIMIT = -7
QLORA_STATIC_SCRATCH_BYTES = 8 << 20
QLORA_DEV_NONFINITE = 1
QLORA_DEV_TIMEOUT = 2
QLORA_DEV_LAUNCH = 4
QLORA_DEV_TARGET = 8

# Every symbol the header declares, with its ctypes signature.
_PTR = ctypes.c_void_p
_I64 = ctypes.c_int64
SIGNATURES = {
    "qlora_nf4_codebook": (ctypes.c_int, [_PTR, _PTR]),
    "nf4_quantize": (ctypes.c_int, [_PTR, _PTR, _PTR]),
    "nf4_dequantize": (ctypes.c_int, [_PTR, _PTR, _PTR]),
    "qlora_linear_fwd": (ctypes.c_int, [_PTR, _I64, _PTR, _PTR, _PTR, _I64, ctypes.c_float,
                                        _PTR, _PTR, _PTR, ctypes.c_size_t, _PTR]),
    "qlora_linear_bwd": (ctypes.c_int, [_PTR, _PTR, _I64, _PTR, _PTR, _PTR, _I64, ctypes.c_float,
                                        _PTR, _PTR, _PTR, _PTR, _PTR, ctypes.c_size_t, _PTR]),
    "qlora_fwd_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64, _I64]),
    "qlora_bwd_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64, _I64]),
    "qlora_get_last_status": (ctypes.c_int, [_PTR]),
    "qlora_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "qlora_set_gemv_max_ctas": (ctypes.c_int, [ctypes.c_int]),
    "qlora_selftest_wait_timeout": (ctypes.c_int, [_I64, _PTR]),
    "qlora_merge_adapters": (ctypes.c_int, [_PTR, _PTR, _PTR, _I64, ctypes.c_float, _PTR, _PTR]),
    "qlora_codebook": (ctypes.c_int, [ctypes.c_int, _PTR, _PTR]),
    "qlora_adamw_step": (ctypes.c_int, [_PTR, _PTR, _PTR, _PTR, _PTR, _I64, ctypes.c_float,
                                        ctypes.c_float, ctypes.c_float, ctypes.c_float,
                                        ctypes.c_float, _I64, ctypes.c_uint, _PTR]),
    "qlora_adamw_step_multi": (ctypes.c_int, [ctypes.c_int, _PTR, _PTR, _PTR, _PTR, _PTR, _PTR,
                                              ctypes.c_float, ctypes.c_float, ctypes.c_float,
                                              ctypes.c_float, ctypes.c_float, _I64, ctypes.c_uint,
                                              _PTR]),
    "qlora_quantize_codebook": (ctypes.c_int, [_PTR, _PTR, ctypes.c_int, _PTR]),
    "qlora_dequantize_codebook": (ctypes.c_int, [_PTR, ctypes.c_int, _PTR, _PTR]),
    "qlora_quantize_format": (ctypes.c_int, [_PTR, _PTR, ctypes.c_int, ctypes.c_int, _PTR]),
    "qlora_dequantize_format": (ctypes.c_int, [_PTR, ctypes.c_int, ctypes.c_int, _PTR, _PTR]),
    "qlora_profile_begin": (ctypes.c_int, [ctypes.c_int]),
    "qlora_profile_end": (ctypes.c_int, [_PTR, _PTR, ctypes.c_int]),
    "qlora_kernel_name": (ctypes.c_char_p, [ctypes.c_int]),
    "qlora_linear_fwd_noalloc": (ctypes.c_int, [_PTR, _I64, _PTR, _PTR, _PTR, _I64,
                                                ctypes.c_float, _PTR, _PTR, _PTR]),
    "qlora_linear_fwd_dropout": (ctypes.c_int, [_PTR, _I64, _PTR, _PTR, _PTR, _I64, ctypes.c_float,
                                                ctypes.c_float, ctypes.c_uint64, _PTR, _PTR, _PTR,
                                                _PTR, ctypes.c_size_t, _PTR]),
    "qlora_linear_bwd_dropout": (ctypes.c_int, [_PTR, _PTR, _I64, _PTR, _PTR, _PTR, _I64,
                                                ctypes.c_float, ctypes.c_float, ctypes.c_uint64,
                                                _PTR, _PTR, _PTR, _PTR, _PTR, _PTR, ctypes.c_size_t,
                                                _PTR]),
    "qlora_fwd_dropout_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64, _I64]),
    "qlora_bwd_dropout_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64, _I64]),
    "qlora_dropout_apply": (ctypes.c_int, [_PTR, _I64, _I64, ctypes.c_float, ctypes.c_uint64, _PTR,
                                           _PTR]),
    "qlora_linear_fwd_epilogue": (ctypes.c_int, [_PTR, _I64, _PTR, _PTR, _PTR, _I64, ctypes.c_float,
                                                 _PTR, ctypes.c_int, _PTR, _PTR, _PTR, _PTR, _PTR,
                                                 ctypes.c_size_t, _PTR]),
    "qlora_fwd_epilogue_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64, _I64]),
    "qlora_epilogue_bwd": (ctypes.c_int, [_PTR, _PTR, _I64, _I64, ctypes.c_int, _PTR, _PTR, _PTR,
                                          ctypes.c_size_t, _PTR]),
    "qlora_epilogue_bwd_workspace_bytes": (ctypes.c_size_t, [_I64, _I64]),
    "qlora_norm_residual_fwd": (ctypes.c_int, [_PTR, _PTR, _I64, _I64, _PTR, _PTR, _I64,
                                               ctypes.c_float, _PTR, ctypes.c_float, _PTR, _PTR,
                                               _PTR, _PTR, _PTR]),
    "qlora_norm_residual_bwd": (ctypes.c_int, [_PTR, _PTR, _PTR, _PTR, _I64, _I64, _PTR, _PTR, _I64,
                                               ctypes.c_float, _PTR, _PTR, _PTR, _PTR, _PTR, _PTR,
                                               _PTR, _PTR, _PTR, ctypes.c_size_t, _PTR]),
    "qlora_norm_residual_bwd_workspace_bytes": (ctypes.c_size_t, [_I64, _I64]),
    "qlora_vocab_loss_fwd": (ctypes.c_int, [_PTR, _PTR, _I64, _I64, _I64, _PTR, _I64, _PTR, _PTR, _PTR,
                                            ctypes.c_size_t, _PTR]),
    "qlora_vocab_loss_bwd": (ctypes.c_int, [_PTR, _PTR, _I64, _I64, _I64, _PTR, _I64, _PTR, _PTR, _PTR,
                                            _PTR, _PTR, ctypes.c_size_t, _PTR]),
    "qlora_vocab_loss_fwd_bwd": (ctypes.c_int, [_PTR, _PTR, _I64, _I64, _I64, _PTR, _I64, _PTR, _PTR,
                                                _PTR, _PTR, _PTR, ctypes.c_size_t, _PTR]),
    "qlora_vocab_loss_fwd_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64]),
    "qlora_vocab_loss_bwd_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64]),
    "qlora_vocab_loss_fwd_bwd_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64]),
}
KERNEL_KINDS = 13


class NF4WeightDesc(ctypes.Structure):
    """ctypes mirror of `nf4_weight`."""
    _fields_ = [("codes", _PTR), ("absmax_q8", _PTR), ("absmax_s2", _PTR),
                ("out_features", _I64), ("in_features", _I64)]


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return _build.LIB_PATH


def lib() -> ctypes.CDLL:
    """Load the in-tree library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: build it with "
                                   "`python -m bit_quantized_lora_03_b200.build`")
            cdll = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(cdll, name)
                fn.restype = res
                fn.argtypes = args
            _lib = cdll
        return _lib


def status_string(code: int) -> str:
    return lib().qlora_status_string(int(code)).decode()


def _check(rc: int, what: str) -> None:
    if rc != QLORA_OK:
        raise RuntimeError(f"{what} failed: {status_string(rc)} ({rc})")


def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _used_on(stream, *tensors) -> None:
    """Notes that work on `stream` (None: the current one) uses the tensors, which the caller may free as
    soon as the call returns: their memory is then not given out again before that work is done."""
    if stream is None:
        return
    for t in tensors:
        if isinstance(t, PackedNF4):
            _used_on(stream, t.codes, t.absmax_q8, t.absmax_s2)
        elif t is not None:
            t.record_stream(stream)


CODEBOOK_NF4, CODEBOOK_FP4, CODEBOOK_INT4 = 0, 1, 2
SCALES_U8, SCALES_S8, SCALES_E4M3 = 0, 1, 2


def codebook(codebook_id: int | None = None):
    """(levels[16], midpoints[15]) as derived by the library (host call, no GPU needed);
    the NF4 codebook unless another id is given."""
    lv = (ctypes.c_float * 16)()
    md = (ctypes.c_float * 15)()
    if codebook_id is None:
        _check(lib().qlora_nf4_codebook(ctypes.cast(lv, _PTR), ctypes.cast(md, _PTR)), "codebook")
    else:
        _check(lib().qlora_codebook(int(codebook_id), ctypes.cast(lv, _PTR), ctypes.cast(md, _PTR)),
               "codebook")
    return list(lv), list(md)


class PackedNF4:
    """A packed NF4 weight held in caller-owned torch device tensors (Wt is o x h)."""

    def __init__(self, out_features: int, in_features: int, device="cuda"):
        if in_features % 64:
            raise ValueError("in_features must be a multiple of 64")
        n = out_features * in_features
        self.out_features = out_features
        self.in_features = in_features
        self.codes = torch.empty(n // 2, dtype=torch.uint8, device=device)
        self.absmax_q8 = torch.empty(n // 64, dtype=torch.uint8, device=device)
        self.absmax_s2 = torch.empty((n // 64 + 255) // 256, dtype=torch.float32, device=device)

    def desc(self) -> NF4WeightDesc:
        return NF4WeightDesc(self.codes.data_ptr(), self.absmax_q8.data_ptr(),
                             self.absmax_s2.data_ptr(), self.out_features, self.in_features)

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.absmax_q8.numel() + 4 * self.absmax_s2.numel()


def _require(t: torch.Tensor, dtype, shape, name: str) -> None:
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous CUDA {dtype} {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def nf4_quantize(Wt: torch.Tensor, out: PackedNF4 | None = None, stream=None,
                 codebook_id: int = CODEBOOK_NF4, scale_format: int = SCALES_U8) -> PackedNF4:
    """Quantize an fp32 CUDA weight Wt (o x h) to packed 4-bit codes with double-quantized
    scales (NF4 and unsigned 8-bit scales unless another codebook or scale format is given)."""
    o, h = Wt.shape
    _require(Wt, torch.float32, (o, h), "Wt")
    p = out if out is not None else PackedNF4(o, h, Wt.device)
    d = p.desc()
    if scale_format != SCALES_U8:
        _check(lib().qlora_quantize_format(Wt.data_ptr(), ctypes.byref(d), int(codebook_id),
                                           int(scale_format), _stream(stream)),
               "qlora_quantize_format")
    elif codebook_id == CODEBOOK_NF4:
        _check(lib().nf4_quantize(Wt.data_ptr(), ctypes.byref(d), _stream(stream)), "nf4_quantize")
    else:
        _check(lib().qlora_quantize_codebook(Wt.data_ptr(), ctypes.byref(d), int(codebook_id),
                                             _stream(stream)), "qlora_quantize_codebook")
    _used_on(stream, Wt, p)
    return p


def nf4_dequantize(p: PackedNF4, out: torch.Tensor | None = None, stream=None,
                   codebook_id: int = CODEBOOK_NF4, scale_format: int = SCALES_U8) -> torch.Tensor:
    """The bf16 weight Wt' (o x h) reconstructed from a packed weight (with the codebook and
    scale format it was packed with)."""
    if out is None:
        out = torch.empty(p.out_features, p.in_features, dtype=torch.bfloat16,
                          device=p.codes.device)
    _require(out, torch.bfloat16, (p.out_features, p.in_features), "out")
    d = p.desc()
    if scale_format != SCALES_U8:
        _check(lib().qlora_dequantize_format(ctypes.byref(d), int(codebook_id), int(scale_format),
                                             out.data_ptr(), _stream(stream)),
               "qlora_dequantize_format")
    elif codebook_id == CODEBOOK_NF4:
        _check(lib().nf4_dequantize(ctypes.byref(d), out.data_ptr(), _stream(stream)),
               "nf4_dequantize")
    else:
        _check(lib().qlora_dequantize_codebook(ctypes.byref(d), int(codebook_id), out.data_ptr(),
                                               _stream(stream)), "qlora_dequantize_codebook")
    _used_on(stream, p, out)
    return out


_ws_cache: dict = {}


def workspace(nbytes: int, device) -> torch.Tensor:
    """A cached caller-owned scratch buffer of at least nbytes on `device`."""
    key = (str(device), threading.get_ident())
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


def fwd_workspace_bytes(t: int, h: int, o: int, r: int) -> int:
    return int(lib().qlora_fwd_workspace_bytes(t, h, o, r))


def bwd_workspace_bytes(t: int, h: int, o: int, r: int) -> int:
    return int(lib().qlora_bwd_workspace_bytes(t, h, o, r))


def qlora_linear_fwd(X: torch.Tensor, p: PackedNF4, L1: torch.Tensor, L2: torch.Tensor, s: float,
                     Y: torch.Tensor | None = None, sT: torch.Tensor | None = None,
                     want_sT: bool = True, ws: torch.Tensor | None = None, stream=None):
    """Y = X.W' + s.X.L1.L2. Returns (Y t x o bf16, sT t x r bf16 or None)."""
    t, h = X.shape
    o, r = p.out_features, L1.shape[1]
    _require(X, torch.bfloat16, (t, h), "X")
    _require(L1, torch.bfloat16, (h, r), "L1")
    _require(L2, torch.bfloat16, (r, o), "L2")
    if h != p.in_features:
        raise ValueError("X and W disagree on in_features")
    if Y is None:
        Y = torch.empty(t, o, dtype=torch.bfloat16, device=X.device)
    if sT is None and want_sT:
        sT = torch.empty(t, r, dtype=torch.bfloat16, device=X.device)
    need = fwd_workspace_bytes(t, h, o, r)
    if ws is None:
        ws = workspace(need, X.device)
    d = p.desc()
    rc = lib().qlora_linear_fwd(X.data_ptr(), t, ctypes.byref(d), L1.data_ptr(), L2.data_ptr(), r,
                                float(s), Y.data_ptr(), _ptr(sT), ws.data_ptr(), ws.numel(),
                                _stream(stream))
    _check(rc, "qlora_linear_fwd")
    _used_on(stream, X, p, L1, L2, Y, sT, ws)
    return Y, sT


def qlora_linear_bwd(dY: torch.Tensor, X: torch.Tensor, p: PackedNF4, L1: torch.Tensor,
                     L2: torch.Tensor, s: float, sT: torch.Tensor | None = None,
                     dX: torch.Tensor | None = None, dL1: torch.Tensor | None = None,
                     dL2: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                     stream=None):
    """Returns (dX t x h bf16, dL1 h x r fp32, dL2 r x o fp32); W gets no gradient."""
    t, h = X.shape
    o, r = p.out_features, L1.shape[1]
    _require(dY, torch.bfloat16, (t, o), "dY")
    _require(X, torch.bfloat16, (t, h), "X")
    _require(L1, torch.bfloat16, (h, r), "L1")
    _require(L2, torch.bfloat16, (r, o), "L2")
    if sT is not None:
        _require(sT, torch.bfloat16, (t, r), "sT")
    dev = X.device
    dX = torch.empty(t, h, dtype=torch.bfloat16, device=dev) if dX is None else dX
    dL1 = torch.empty(h, r, dtype=torch.float32, device=dev) if dL1 is None else dL1
    dL2 = torch.empty(r, o, dtype=torch.float32, device=dev) if dL2 is None else dL2
    need = bwd_workspace_bytes(t, h, o, r)
    if ws is None:
        ws = workspace(need, dev)
    d = p.desc()
    rc = lib().qlora_linear_bwd(dY.data_ptr(), X.data_ptr(), t, ctypes.byref(d), L1.data_ptr(),
                                L2.data_ptr(), r, float(s), _ptr(sT), dX.data_ptr(),
                                dL1.data_ptr(), dL2.data_ptr(), ws.data_ptr(), ws.numel(),
                                _stream(stream))
    _check(rc, "qlora_linear_bwd")
    _used_on(stream, dY, X, p, L1, L2, sT, dX, dL1, dL2, ws)
    return dX, dL1, dL2


def _dropout_args(dropout_p: float, seed: int):
    p32 = float(dropout_p)
    if not (0.0 <= p32 < 1.0):
        raise ValueError("dropout probability must lie in [0, 1)")
    return ctypes.c_float(p32), ctypes.c_uint64(int(seed) & 0xFFFFFFFFFFFFFFFF)


def qlora_dropout_apply(X: torch.Tensor, dropout_p: float, seed: int,
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """X (.) M for the LoRA-dropout keep mask M of (dropout_p, seed); dropped elements are +0."""
    t, h = X.shape
    _require(X, torch.bfloat16, (t, h), "X")
    out = torch.empty_like(X) if out is None else out
    _require(out, torch.bfloat16, (t, h), "out")
    pf, sd = _dropout_args(dropout_p, seed)
    _check(lib().qlora_dropout_apply(X.data_ptr(), t, h, pf, sd, out.data_ptr(), _stream(stream)),
           "qlora_dropout_apply")
    _used_on(stream, X, out)
    return out


def dropout_mask_bytes(t: int, h: int) -> int:
    """Bytes of a keep mask stored as bits (bit e mod 8 of byte e / 8)."""
    return t * h // 8


def qlora_linear_fwd_dropout(X: torch.Tensor, p: PackedNF4, L1: torch.Tensor, L2: torch.Tensor,
                             s: float, dropout_p: float, seed: int, Y: torch.Tensor | None = None,
                             sT: torch.Tensor | None = None, want_sT: bool = True,
                             mask: torch.Tensor | None = None, want_mask: bool = False,
                             ws: torch.Tensor | None = None, stream=None):
    """Y = X.W' + s.((X (.) M / (1 - p)).L1).L2 with the keep mask M of (dropout_p, seed).
    Returns (Y, sT or None, mask bits or None); pass the mask to the backward to spare it the
    generator calls."""
    t, h = X.shape
    o, r = p.out_features, L1.shape[1]
    _require(X, torch.bfloat16, (t, h), "X")
    _require(L1, torch.bfloat16, (h, r), "L1")
    _require(L2, torch.bfloat16, (r, o), "L2")
    if h != p.in_features:
        raise ValueError("X and W disagree on in_features")
    Y = torch.empty(t, o, dtype=torch.bfloat16, device=X.device) if Y is None else Y
    if sT is None and want_sT:
        sT = torch.empty(t, r, dtype=torch.bfloat16, device=X.device)
    if mask is None and want_mask:
        mask = torch.empty(dropout_mask_bytes(t, h), dtype=torch.uint8, device=X.device)
    if mask is not None:
        _require(mask, torch.uint8, (dropout_mask_bytes(t, h),), "mask")
    if ws is None:
        ws = workspace(int(lib().qlora_fwd_dropout_workspace_bytes(t, h, o, r)), X.device)
    pf, sd = _dropout_args(dropout_p, seed)
    d = p.desc()
    rc = lib().qlora_linear_fwd_dropout(X.data_ptr(), t, ctypes.byref(d), L1.data_ptr(),
                                        L2.data_ptr(), r, float(s), pf, sd, Y.data_ptr(), _ptr(sT),
                                        _ptr(mask), ws.data_ptr(), ws.numel(), _stream(stream))
    _check(rc, "qlora_linear_fwd_dropout")
    _used_on(stream, X, p, L1, L2, Y, sT, mask, ws)
    return Y, sT, mask


def qlora_linear_bwd_dropout(dY: torch.Tensor, X: torch.Tensor, p: PackedNF4, L1: torch.Tensor,
                             L2: torch.Tensor, s: float, dropout_p: float, seed: int,
                             sT: torch.Tensor | None = None, mask: torch.Tensor | None = None,
                             dX: torch.Tensor | None = None,
                             dL1: torch.Tensor | None = None, dL2: torch.Tensor | None = None,
                             ws: torch.Tensor | None = None, stream=None):
    """Gradients for qlora_linear_fwd_dropout with the same (dropout_p, seed) (and, optionally,
    the forward's mask bits)."""
    t, h = X.shape
    o, r = p.out_features, L1.shape[1]
    _require(dY, torch.bfloat16, (t, o), "dY")
    _require(X, torch.bfloat16, (t, h), "X")
    _require(L1, torch.bfloat16, (h, r), "L1")
    _require(L2, torch.bfloat16, (r, o), "L2")
    if sT is not None:
        _require(sT, torch.bfloat16, (t, r), "sT")
    if mask is not None:
        _require(mask, torch.uint8, (dropout_mask_bytes(t, h),), "mask")
    dev = X.device
    dX = torch.empty(t, h, dtype=torch.bfloat16, device=dev) if dX is None else dX
    dL1 = torch.empty(h, r, dtype=torch.float32, device=dev) if dL1 is None else dL1
    dL2 = torch.empty(r, o, dtype=torch.float32, device=dev) if dL2 is None else dL2
    if ws is None:
        ws = workspace(int(lib().qlora_bwd_dropout_workspace_bytes(t, h, o, r)), dev)
    pf, sd = _dropout_args(dropout_p, seed)
    d = p.desc()
    rc = lib().qlora_linear_bwd_dropout(dY.data_ptr(), X.data_ptr(), t, ctypes.byref(d),
                                        L1.data_ptr(), L2.data_ptr(), r, float(s), pf, sd, _ptr(sT),
                                        _ptr(mask), dX.data_ptr(), dL1.data_ptr(), dL2.data_ptr(),
                                        ws.data_ptr(), ws.numel(), _stream(stream))
    _check(rc, "qlora_linear_bwd_dropout")
    _used_on(stream, dY, X, p, L1, L2, sT, mask, dX, dL1, dL2, ws)
    return dX, dL1, dL2


# ------------------------------------------------------------------------------------------
# The operators around the linear. They run on the device of their tensors (all on one) and on the
# current stream there, or on `stream`; what they allocate (outputs, workspace) is allocated on
# that stream, one workspace per call, so that calls on two streams, and graphs captured from them,
# share none. Their inputs may be freed as soon as they return.
# ------------------------------------------------------------------------------------------
_NO_GUARD = contextlib.nullcontext()


def _current(dev) -> int:
    """The current stream of `dev` as a handle (without building a torch.cuda.Stream, which took a
    quarter of a short call's host time)."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _guard(t: torch.Tensor, stream):
    """Makes the device of `t`, and `stream` if given, current for the call."""
    if not t.is_cuda:
        raise ValueError(f"expected CUDA tensors, got one on {t.device}")
    if stream is not None:
        if stream.device != t.device:
            raise ValueError(f"stream of {stream.device} for tensors on {t.device}")
        return torch.cuda.stream(stream)
    return _NO_GUARD if torch._C._cuda_getDevice() == t.device.index else torch.cuda.device(t.device)


def _on(dev, t: torch.Tensor | None, dtype, shape, name: str) -> int | None:
    """The address of t, checked to be a contiguous dtype tensor of `shape` on `dev`; None for None."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on {dev}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}"
                         f"{'' if t.is_contiguous() else ', not contiguous'}")
    return t.data_ptr()


def _out(dev, t: torch.Tensor | None, dtype, shape, name: str, want: bool = True, like: torch.Tensor | None = None):
    """An output: t, checked, or a new tensor where one is wanted (the quicker way where a checked
    tensor of its type and shape is at hand: `like`)."""
    if t is None:
        if not want:
            return None
        return torch.empty(shape, dtype=dtype, device=dev) if like is None else torch.empty_like(like)
    _on(dev, t, dtype, shape, name)
    return t


def _scratch(dev, ws: torch.Tensor | None, nbytes: int) -> torch.Tensor:
    if ws is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
    _on(dev, ws, torch.uint8, ws.shape, "ws")
    return ws


def _matrix(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D tensor, got {tuple(t.shape)}")
    return t.shape


ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = 0, 1, 2, 3, 4
ACTIVATIONS = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH,
               "silu": ACT_SILU}


def _act_id(act) -> int:
    """An activation's id from its name or id (the library checks ids)."""
    if isinstance(act, str):
        if act not in ACTIVATIONS:
            raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACTIVATIONS)}")
        return ACTIVATIONS[act]
    return int(act)


def qlora_linear_fwd_epilogue(X: torch.Tensor, p: PackedNF4, L1: torch.Tensor, L2: torch.Tensor,
                              s: float, bias: torch.Tensor | None = None, act="none",
                              residual: torch.Tensor | None = None, Y: torch.Tensor | None = None,
                              Z: torch.Tensor | None = None, want_Z: bool = False,
                              sT: torch.Tensor | None = None, want_sT: bool = True,
                              ws: torch.Tensor | None = None, stream=None):
    """Z = X.W' + s.X.L1.L2 + bias, Y = act(Z) + residual. act: a name of ACTIVATIONS or its id.
    residual may be Y itself. Returns (Y t x o bf16, Z t x o bf16 or None, sT t x r bf16 or None);
    keep Z for qlora_epilogue_bwd and sT for qlora_linear_bwd."""
    (t, h), (_, r), o, dev = _matrix(X, "X"), _matrix(L1, "L1"), p.out_features, X.device
    with _guard(X, stream):
        if h != p.in_features:
            raise ValueError("X and W disagree on in_features")
        if p.codes.device != dev:
            raise ValueError(f"the packed weight is on {p.codes.device}, X on {dev}")
        bf16 = torch.bfloat16
        ins = (_on(dev, X, bf16, (t, h), "X"), _on(dev, L1, bf16, (h, r), "L1"),
               _on(dev, L2, bf16, (r, o), "L2"), _on(dev, bias, bf16, (o,), "bias"),
               _on(dev, residual, bf16, (t, o), "residual"))
        Y = _out(dev, Y, bf16, (t, o), "Y")
        Z = _out(dev, Z, bf16, (t, o), "Z", want_Z, like=Y)
        sT = _out(dev, sT, bf16, (t, r), "sT", want_sT)
        ws = _scratch(dev, ws, int(lib().qlora_fwd_epilogue_workspace_bytes(t, h, o, r)))
        d = p.desc()
        _check(lib().qlora_linear_fwd_epilogue(
            ins[0], t, ctypes.byref(d), ins[1], ins[2], r, float(s), ins[3], _act_id(act), ins[4],
            Y.data_ptr(), _ptr(Z), _ptr(sT), ws.data_ptr(), ws.numel(), _current(dev)),
            "qlora_linear_fwd_epilogue")
    _used_on(stream, X, p, L1, L2, bias, residual, Y, Z, sT, ws)
    return Y, Z, sT


def qlora_epilogue_bwd(dY: torch.Tensor, Z: torch.Tensor | None, act="none",
                       dZ: torch.Tensor | None = None, dbias: torch.Tensor | None = None,
                       want_dZ: bool = True, want_dbias: bool = True,
                       ws: torch.Tensor | None = None, stream=None):
    """dZ = dY . act'(Z) (bf16) and dbias = its sum over tokens (fp32), either one None if not
    wanted. Pass dZ on to qlora_linear_bwd; the residual's gradient is dY. dZ may be dY itself."""
    (t, o), dev = _matrix(dY, "dY"), dY.device
    with _guard(dY, stream):
        a, z = (_on(dev, x, torch.bfloat16, (t, o), n) for x, n in ((dY, "dY"), (Z, "Z")))
        dZ = _out(dev, dZ, torch.bfloat16, (t, o), "dZ", want_dZ, like=dY)
        dbias = _out(dev, dbias, torch.float32, (o,), "dbias", want_dbias)
        if dbias is not None:
            ws = _scratch(dev, ws, int(lib().qlora_epilogue_bwd_workspace_bytes(t, o)))
        _check(lib().qlora_epilogue_bwd(a, z, t, o, _act_id(act), _ptr(dZ), _ptr(dbias), _ptr(ws),
                                        0 if ws is None else ws.numel(), _current(dev)),
               "qlora_epilogue_bwd")
    _used_on(stream, dY, Z, dZ, dbias, ws)
    return dZ, dbias


def _gate_shape(gate: torch.Tensor | None, rows_per_gate, t: int, h: int):
    """(rows_per_gate, the gate's shape): one row for all tokens unless rows_per_gate is given."""
    if gate is None:
        return 0, None
    rows = t if rows_per_gate is None else int(rows_per_gate)
    return rows, (-(-t // rows) if rows > 0 else 0, h)


def qlora_norm_residual_fwd(x: torch.Tensor, y: torch.Tensor | None = None,
                            w_post: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                            w_pre: torch.Tensor | None = None, scale: float = 1.0, eps: float = 1e-6,
                            rows_per_gate: int | None = None, x_out: torch.Tensor | None = None,
                            n: torch.Tensor | None = None, want_rstd: bool = True, stream=None):
    """u = y.rstd(y).w_post, x' = x + scale.gate.u, n = x'.rstd(x').w_pre; without y, x' = x.
    gate: ceil(t / rows_per_gate) rows of h (one for all tokens by default). Returns
    (x' t x h bf16, n t x h bf16 or None, rstd_post t fp32 or None, rstd_pre t fp32 or None)."""
    (t, h), dev, bf16 = _matrix(x, "x"), x.device, torch.bfloat16
    rows, gshape = _gate_shape(gate, rows_per_gate, t, h)
    with _guard(x, stream):
        xp, yp = _on(dev, x, bf16, (t, h), "x"), _on(dev, y, bf16, (t, h), "y")
        wo, gp = _on(dev, w_post, bf16, (h,), "w_post"), _on(dev, gate, bf16, gshape, "gate")
        wi = _on(dev, w_pre, bf16, (h,), "w_pre")
        x_out = _out(dev, x_out, bf16, (t, h), "x_out", like=x)
        n = _out(dev, n, bf16, (t, h), "n", wi is not None, like=x)
        ro = torch.empty(t, dtype=torch.float32, device=dev) if want_rstd and wo else None
        ri = torch.empty(t, dtype=torch.float32, device=dev) if want_rstd and wi else None
        _check(lib().qlora_norm_residual_fwd(xp, yp, t, h, wo, gp, rows, float(scale), wi, float(eps),
                                             x_out.data_ptr(), _ptr(n), _ptr(ro), _ptr(ri), _current(dev)),
               "qlora_norm_residual_fwd")
    _used_on(stream, x, y, w_post, gate, w_pre, x_out, n)
    return x_out, n, ro, ri


def qlora_norm_residual_bwd(dx_out: torch.Tensor | None, dn: torch.Tensor | None, x_out: torch.Tensor | None,
                            y: torch.Tensor | None, rstd_post: torch.Tensor | None,
                            rstd_pre: torch.Tensor | None, w_post: torch.Tensor | None = None,
                            gate: torch.Tensor | None = None, w_pre: torch.Tensor | None = None,
                            scale: float = 1.0, rows_per_gate: int | None = None,
                            ws: torch.Tensor | None = None, stream=None):
    """Gradients of qlora_norm_residual_fwd from those of x' and n (either may be None: zero), with
    the forward's x', y, rstd_post and rstd_pre. Returns (dx t x h bf16, dy t x h bf16, dw_post h
    fp32, dgate fp32 of the gate's shape, dw_pre h fp32), None where there is no such input."""
    like = dx_out if dx_out is not None else dn
    if like is None:
        raise ValueError("one of dx_out and dn is needed")
    (t, h), dev, bf16, f32 = _matrix(like, "dx_out or dn"), like.device, torch.bfloat16, torch.float32
    rows, gshape = _gate_shape(gate, rows_per_gate, t, h)
    with _guard(like, stream):
        if dn is None:      # n's gradient is zero: nothing of the second norm is needed
            x_out = rstd_pre = w_pre_used = None
        else:
            w_pre_used = w_pre
        g = [_on(dev, v, bf16, (t, h), s) for v, s in ((dx_out, "dx_out"), (dn, "dn"), (x_out, "x_out"), (y, "y"))]
        wo, gp = _on(dev, w_post, bf16, (h,), "w_post"), _on(dev, gate, bf16, gshape, "gate")
        wi = _on(dev, w_pre_used, bf16, (h,), "w_pre")
        ro, ri = _on(dev, rstd_post, f32, (t,), "rstd_post"), _on(dev, rstd_pre, f32, (t,), "rstd_pre")
        dx = torch.empty_like(like)
        dy = torch.empty_like(y) if y is not None else None
        dwo = torch.empty(h, dtype=f32, device=dev) if wo else None
        dg = torch.empty(gshape, dtype=f32, device=dev) if gp else None
        dwi = torch.empty(h, dtype=f32, device=dev) if wi else None
        ws = _scratch(dev, ws, int(lib().qlora_norm_residual_bwd_workspace_bytes(t, h)))
        _check(lib().qlora_norm_residual_bwd(*g, t, h, wo, gp, rows, float(scale), wi, ro, ri, dx.data_ptr(),
                                             _ptr(dy), _ptr(dwo), _ptr(dg), _ptr(dwi), ws.data_ptr(),
                                             ws.numel(), _current(dev)),
               "qlora_norm_residual_bwd")
        if dn is None and w_pre is not None:
            dwi = torch.zeros(h, dtype=f32, device=dev)
    _used_on(stream, dx_out, dn, x_out, y, rstd_post, rstd_pre, w_post, gate, w_pre, ws)
    return dx, dy, dwo, dg, dwi


def _vocab(X, W, targets):
    """(t, h, v) and the addresses of the loss's inputs, checked."""
    (t, h), (v, _), dev = _matrix(X, "X"), _matrix(W, "W"), X.device
    return (t, h, v), (_on(dev, X, torch.bfloat16, (t, h), "X"), _on(dev, W, torch.bfloat16, (v, h), "W"), t, h, v,
                       _on(dev, targets, torch.int64, (t,), "targets"))


def qlora_vocab_loss_fwd(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
                         loss: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                         ws: torch.Tensor | None = None, stream=None):
    """Cross entropy of X.W^T (t x v, never stored) against int64 targets: (loss t fp32, lse t fp32).
    Targets equal to ignore_index are not counted (loss 0)."""
    with _guard(X, stream):
        (t, h, v), args = _vocab(X, W, targets)
        dev, f32 = X.device, torch.float32
        loss = _out(dev, loss, f32, (t,), "loss")
        lse = _out(dev, lse, f32, (t,), "lse", like=loss)
        ws = _scratch(dev, ws, int(lib().qlora_vocab_loss_fwd_workspace_bytes(t, h, v)))
        _check(lib().qlora_vocab_loss_fwd(*args, int(ignore_index), loss.data_ptr(), lse.data_ptr(),
                                          ws.data_ptr(), ws.numel(), _current(dev)), "qlora_vocab_loss_fwd")
    _used_on(stream, X, W, targets, loss, lse, ws)
    return loss, lse


def qlora_vocab_loss_bwd(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                         dloss: torch.Tensor, dlse: torch.Tensor | None = None, ignore_index: int = -100,
                         dX: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    """dX (t x h bf16) from the gradients of loss (and of lse, if given; t fp32 each) and the
    forward's lse; W is frozen."""
    with _guard(X, stream):
        (t, h, v), args = _vocab(X, W, targets)
        dev, f32 = X.device, torch.float32
        grads = (_on(dev, lse, f32, (t,), "lse"), _on(dev, dloss, f32, (t,), "dloss"), _on(dev, dlse, f32, (t,), "dlse"))
        dX = _out(dev, dX, torch.bfloat16, (t, h), "dX", like=X)
        ws = _scratch(dev, ws, int(lib().qlora_vocab_loss_bwd_workspace_bytes(t, h, v)))
        _check(lib().qlora_vocab_loss_bwd(*args, int(ignore_index), *grads, dX.data_ptr(), ws.data_ptr(),
                                          ws.numel(), _current(dev)), "qlora_vocab_loss_bwd")
    _used_on(stream, X, W, targets, lse, dloss, dlse, dX, ws)
    return dX


def qlora_vocab_loss_fwd_bwd(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, dloss: torch.Tensor,
                             ignore_index: int = -100, loss: torch.Tensor | None = None,
                             lse: torch.Tensor | None = None, dX: torch.Tensor | None = None,
                             ws: torch.Tensor | None = None, stream=None):
    """(loss, lse, dX) in one call for a dloss (t fp32) known beforehand, such as 1 / count for the
    mean: the logits are formed once."""
    with _guard(X, stream):
        (t, h, v), args = _vocab(X, W, targets)
        dev, f32 = X.device, torch.float32
        d = _on(dev, dloss, f32, (t,), "dloss")
        loss = _out(dev, loss, f32, (t,), "loss")
        lse = _out(dev, lse, f32, (t,), "lse", like=loss)
        dX = _out(dev, dX, torch.bfloat16, (t, h), "dX", like=X)
        ws = _scratch(dev, ws, int(lib().qlora_vocab_loss_fwd_bwd_workspace_bytes(t, h, v)))
        _check(lib().qlora_vocab_loss_fwd_bwd(*args, int(ignore_index), d, loss.data_ptr(), lse.data_ptr(),
                                              dX.data_ptr(), ws.data_ptr(), ws.numel(), _current(dev)),
               "qlora_vocab_loss_fwd_bwd")
    _used_on(stream, X, W, targets, dloss, loss, lse, dX, ws)
    return loss, lse, dX


class KernelProfile:
    """Per-kernel device time and launch counts, from CUDA events the library records around
    each of its launches while the profile is open (``with KernelProfile() as p: ...``)."""

    def __init__(self, capacity: int = 65536):
        self.capacity = capacity
        self.ms = {}
        self.launches = {}
        self.recorded = 0

    def __enter__(self):
        _check(lib().qlora_profile_begin(self.capacity), "qlora_profile_begin")
        return self

    def __exit__(self, *exc):
        ms = (ctypes.c_double * KERNEL_KINDS)()
        n = (ctypes.c_int64 * KERNEL_KINDS)()
        rc = lib().qlora_profile_end(ctypes.cast(ms, _PTR), ctypes.cast(n, _PTR), KERNEL_KINDS)
        if rc < 0:
            raise RuntimeError(f"qlora_profile_end: {status_string(rc)}")
        self.recorded = rc
        for k in range(KERNEL_KINDS):
            name = lib().qlora_kernel_name(k).decode()
            self.ms[name] = ms[k]
            self.launches[name] = n[k]
        return False


def merge_adapters(p: PackedNF4, L1: torch.Tensor, L2: torch.Tensor, s: float,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Wt_merged (o x h fp32) = W'^T + s.(L1.L2)^T: the adapters merged into the dequantized
    base (re-quantize it with nf4_quantize for a merged packed weight)."""
    o, h, r = p.out_features, p.in_features, L1.shape[1]
    _require(L1, torch.bfloat16, (h, r), "L1")
    _require(L2, torch.bfloat16, (r, o), "L2")
    if out is None:
        out = torch.empty(o, h, dtype=torch.float32, device=L1.device)
    _require(out, torch.float32, (o, h), "out")
    d = p.desc()
    _check(lib().qlora_merge_adapters(ctypes.byref(d), L1.data_ptr(), L2.data_ptr(), r,
                                      float(s), out.data_ptr(), _stream(stream)),
           "qlora_merge_adapters")
    _used_on(stream, p, L1, L2, out)
    return out


ADAMW_PREFETCH = 1


def adamw_step_ptr(p: int, p16: int, g: int, m: int, v: int, n: int, lr: float, beta1: float,
                   beta2: float, eps: float, weight_decay: float, step: int, flags: int = 0,
                   stream=None) -> None:
    """qlora_adamw_step on raw device (or unified-memory) pointers."""
    _check(lib().qlora_adamw_step(p, p16, g, m, v, int(n), float(lr), float(beta1), float(beta2),
                                  float(eps), float(weight_decay), int(step), int(flags),
                                  _stream(stream)),
           "qlora_adamw_step")


def adamw_step(p: torch.Tensor, g: torch.Tensor, m: torch.Tensor, v: torch.Tensor, step: int,
               lr: float = 1e-4, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
               weight_decay: float = 0.0, p16: torch.Tensor | None = None, stream=None) -> None:
    """One fused AdamW step on fp32 CUDA tensors of equal shape (in place); p16, if given, gets
    the bf16 copy of the updated parameters."""
    for t, name in ((p, "p"), (g, "g"), (m, "m"), (v, "v")):
        _require(t, torch.float32, p.shape, name)
    if p16 is not None:
        _require(p16, torch.bfloat16, p.shape, "p16")
    adamw_step_ptr(p.data_ptr(), p16.data_ptr() if p16 is not None else 0, g.data_ptr(),
                   m.data_ptr(), v.data_ptr(), p.numel(), lr, beta1, beta2, eps, weight_decay,
                   step, 0, stream)
    _used_on(stream, p, g, m, v, p16)


ADAMW_MAX_TENSORS = 64


def adamw_step_multi_ptr(params, params_bf16, grads, m, v, counts, lr: float, beta1: float,
                         beta2: float, eps: float, weight_decay: float, step: int, flags: int = 0,
                         stream=None) -> None:
    """qlora_adamw_step_multi on lists of raw device pointers (params_bf16 may be None, or hold
    0 for tensors without a bf16 copy) and parameter counts."""
    n = len(params)
    if not (len(grads) == len(m) == len(v) == len(counts) == n) or (
            params_bf16 is not None and len(params_bf16) != n):
        raise ValueError("adamw_step_multi: pointer lists of different lengths")
    P = ctypes.c_void_p * max(n, 1)
    p16 = P(*params_bf16) if params_bf16 is not None else None
    _check(lib().qlora_adamw_step_multi(
        n, P(*params), p16, P(*grads), P(*m), P(*v), (ctypes.c_int64 * max(n, 1))(*counts),
        float(lr), float(beta1), float(beta2), float(eps), float(weight_decay), int(step),
        int(flags), _stream(stream)), "qlora_adamw_step_multi")


def adamw_step_multi(params, grads, ms, vs, step: int, lr: float = 1e-4, beta1: float = 0.9,
                     beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0,
                     params_bf16=None, stream=None) -> None:
    """One fused AdamW step over several fp32 CUDA tensors in one launch (in place); each
    tensor's grad and moments match its shape; params_bf16, if given, is a list holding a bf16
    tensor (or None) per parameter tensor."""
    for p, g, m, v in zip(params, grads, ms, vs, strict=True):
        for t, name in ((p, "p"), (g, "g"), (m, "m"), (v, "v")):
            _require(t, torch.float32, p.shape, name)
    ptr16 = None
    if params_bf16 is not None:
        ptr16 = []
        for p, q in zip(params, params_bf16, strict=True):
            if q is not None:
                _require(q, torch.bfloat16, p.shape, "p16")
            ptr16.append(q.data_ptr() if q is not None else 0)
    adamw_step_multi_ptr([p.data_ptr() for p in params], ptr16, [g.data_ptr() for g in grads],
                         [m.data_ptr() for m in ms], [v.data_ptr() for v in vs],
                         [p.numel() for p in params], lr, beta1, beta2, eps, weight_decay, step, 0,
                         stream)
    _used_on(stream, *params, *grads, *ms, *vs, *(params_bf16 or ()))


def selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    """Launch the bounded-wait self-test (a wait nothing completes, given up after limit_ns)."""
    _check(lib().qlora_selftest_wait_timeout(int(limit_ns), _stream(stream)),
           "qlora_selftest_wait_timeout")


def set_gemv_max_ctas(n: int) -> int:
    """Cap the decode GEMV's CTA count (n <= 0: one per SM); returns the previous cap."""
    return int(lib().qlora_set_gemv_max_ctas(int(n)))


def last_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return int(lib().qlora_get_last_status(_stream(stream)))
