"""packed_xor_popcount_amd -- Python binding of libbnn.so (include/bnn.h).

Packed binary (+1/-1) matrix products on MI355X (gfx950): sign projection and
packing along K, and <x, w> = K - 2 * popcount(x XOR w) with int32,
alpha-scaled fp32 or sign -> repack outputs ("Binary Math Effectiveness --
why / how / when", section 1).

This module only marshals arguments: it checks tensor devices, dtypes and
shapes, allocates outputs with PyTorch (device memory is PyTorch's; the
library allocates nothing), and passes raw device pointers and the current
HIP stream to the C entry points of the same names.  Every step of the
computation runs in the HIP kernels of libbnn.so; there is no CPU path.  If
libbnn.so is missing this module raises instead of falling back.

Packed matrices are ``torch.int64`` tensors of shape ``(rows, words(K))``
holding the uint64 words bit for bit (bit k%64 of word k/64 is element k,
least significant bit first; bit 1 means -1).
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

__all__ = [
    "BnnError", "EPI_I32", "EPI_SCALED", "EPI_REPACK", "ALGO_AUTO", "ALGO_GEMV", "ALGO_TILED",
    "ALGO_MFMA",
    "library", "library_path", "words", "pack_signs", "gemm_u64", "gemm_u64_scaled",
    "gemm_sign_repack", "gemm_sign_repack_thr", "flip_words", "gemm_signw_bf16", "chain3",
    "gemm_ex", "gemv_act", "version", "layernorm_fwd", "layernorm_bwd",
    "f8_row_bytes", "f8_scale_bytes", "quant_f8", "gemm_f8",
    "gemm_signw_grouped", "Routing", "route_fwd", "route_bwd", "combine_fwd", "combine_bwd",
    "adapter_fwd", "adapter_bwd",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libbnn.so")

BNN_FP32, BNN_BF16, BNN_F8 = 0, 1, 2
EPI_I32, EPI_SCALED, EPI_REPACK = 0, 1, 2
ALGO_AUTO, ALGO_GEMV, ALGO_TILED, ALGO_MFMA = 0, 1, 2, 3

EXPORTED = ("bnn_words", "bnn_status_str", "bnn_version", "bnn_pack_signs", "bnn_gemm_u64",
            "bnn_gemm_u64_scaled", "bnn_gemm_sign_repack", "bnn_gemm_ex", "bnn_gemv_act",
            "bnn_gemm_sign_repack_thr", "bnn_gemm_signw_bf16", "bnn_chain3",
            "bnn_layernorm_fwd", "bnn_layernorm_bwd_workspace", "bnn_layernorm_bwd",
            "bnn_f8_row_bytes", "bnn_f8_scale_bytes", "bnn_quant_f8", "bnn_gemm_f8",
            "bnn_gemm_f8_fast", "bnn_gemm_signw_grouped", "bnn_route_fwd_workspace", "bnn_route_fwd",
            "bnn_route_bwd", "bnn_combine_fwd", "bnn_combine_bwd", "bnn_adapter_fwd_workspace",
            "bnn_adapter_fwd", "bnn_adapter_bwd_workspace", "bnn_adapter_bwd")


class BnnError(RuntimeError):
    """A non-zero bnn_status returned by libbnn.so."""

    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_status_str(status)} (status {status})")


_lib = None
_raw_stream = None  # device index -> handle of its current stream, found at the first call


def library():
    """The loaded libbnn.so (built in-tree first if it does not exist yet)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        from . import build as _build
        _build.build()
    lib = ctypes.CDLL(library_path)
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.bnn_words.argtypes, lib.bnn_words.restype = [I64], I64
    lib.bnn_status_str.argtypes, lib.bnn_status_str.restype = [I], ctypes.c_char_p
    lib.bnn_version.argtypes, lib.bnn_version.restype = [], ctypes.c_char_p
    lib.bnn_pack_signs.argtypes = [P, I, I64, I64, I64, P, P]
    lib.bnn_gemm_u64.argtypes = [P, P, P, I64, I64, I64, P]
    lib.bnn_gemm_u64_scaled.argtypes = [P, P, P, P, I64, I64, I64, P]
    lib.bnn_gemm_sign_repack.argtypes = [P, P, P, I64, I64, I64, P]
    lib.bnn_gemm_ex.argtypes = [P, P, P, P, I64, I64, I64, I, I, P]
    lib.bnn_gemv_act.argtypes = [P, I, I64, P, P, P, I64, I64, I64, I, P]
    lib.bnn_gemm_sign_repack_thr.argtypes = [P, P, P, P, P, I64, I64, I64, I, P]
    lib.bnn_gemm_signw_bf16.argtypes = [P, I64, P, P, P, I64, I64, I64, I, P]
    lib.bnn_chain3.argtypes = [P, I, I64, P, P, P, P, P, P, P, P, P, I64, I64, I64, I64, I64, P]
    F = ctypes.c_float
    lib.bnn_layernorm_fwd.argtypes = [P, I, I64, P, P, P, I64, P, P, I64, I64, F, P]
    lib.bnn_layernorm_bwd.argtypes = [P, I64, P, I64, I, P, P, P, P, I64, P, P, P, I64, I64, I64, P]
    lib.bnn_layernorm_bwd_workspace.argtypes = [I64, I64]
    lib.bnn_layernorm_bwd_workspace.restype = I64
    lib.bnn_f8_row_bytes.argtypes, lib.bnn_f8_row_bytes.restype = [I64], I64
    lib.bnn_f8_scale_bytes.argtypes, lib.bnn_f8_scale_bytes.restype = [I64], I64
    lib.bnn_quant_f8.argtypes = [P, I, I64, I64, I64, I, P, P, P]
    lib.bnn_gemm_f8.argtypes = [P, P, P, P, P, I, I64, I64, I64, P]
    lib.bnn_gemm_f8_fast.argtypes = [P, P, P, P, P, I64, I64, I64, P]
    lib.bnn_gemm_signw_grouped.argtypes = [P, I64, I64, P, P, P, P, P, P, I, I64, I64, I64, I64, I, P]
    lib.bnn_route_fwd.argtypes = [P, I, I64] + [P] * 11 + [I64] * 4 + [I, P]
    lib.bnn_route_bwd.argtypes = [P, I, I64] + [P] * 7 + [I64] * 4 + [I, P]
    lib.bnn_combine_fwd.argtypes = [P, I, I64, I64, P, P, P, I64, P, I, I64, I64, I64, I64, P]
    lib.bnn_combine_bwd.argtypes = [P, I, I64, P, P, I, I64, I64, P, P, P, I, I64, P, I64, I64, I64, P]
    lib.bnn_adapter_fwd.argtypes = [P, I64, P, P, P, P, P, I64, P, I64, I, P, P] + [I64] * 6 + [P]
    lib.bnn_adapter_bwd.argtypes = ([P, I64, P, P, I, I64] + [P] * 6 + [I64, P, I64, I, P, P, P] + [I64] * 6
                                    + [P])
    for name, n in (("bnn_route_fwd_workspace", 3), ("bnn_adapter_fwd_workspace", 5),
                    ("bnn_adapter_bwd_workspace", 5)):
        getattr(lib, name).argtypes, getattr(lib, name).restype = [I64] * n, I64
    for name in ("bnn_route_fwd", "bnn_route_bwd", "bnn_combine_fwd", "bnn_combine_bwd", "bnn_adapter_fwd",
                 "bnn_adapter_bwd"):
        getattr(lib, name).restype = I
    for name in ("bnn_pack_signs", "bnn_gemm_u64", "bnn_gemm_u64_scaled", "bnn_gemm_sign_repack",
                 "bnn_gemm_ex", "bnn_gemv_act", "bnn_gemm_sign_repack_thr", "bnn_gemm_signw_bf16",
                 "bnn_chain3", "bnn_layernorm_fwd", "bnn_layernorm_bwd", "bnn_quant_f8",
                 "bnn_gemm_f8", "bnn_gemm_f8_fast", "bnn_gemm_signw_grouped"):
        getattr(lib, name).restype = I
    _lib = lib
    return lib


def _status_str(status: int) -> str:
    return library().bnn_status_str(int(status)).decode()


def version() -> str:
    return library().bnn_version().decode()


def words(k: int) -> int:
    """ceil(k/64): 64-bit words per packed row of k logical values."""
    return int(library().bnn_words(int(k)))


def _check(status: int, where: str) -> None:
    if status != 0:
        raise BnnError(status, where)


def _stream(t: torch.Tensor) -> int:
    # the current stream's handle, without building a Stream object (a
    # microsecond of a decode step's host time) where torch has that lookup
    global _raw_stream
    if _raw_stream is None:
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
    return _raw_stream(t.device.index)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need_cuda(name: str, t: torch.Tensor) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")


def _packed(name: str, t: torch.Tensor, k: int) -> int:
    _need_cuda(name, t)
    if t.dtype != torch.int64 or t.dim() != 2 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous 2-D int64 tensor of packed words")
    if t.shape[1] != words(k):
        raise ValueError(f"{name} has {t.shape[1]} words per row, K={k} needs {words(k)}")
    return t.shape[0]


def pack_signs(src: torch.Tensor, k: int | None = None, out: torch.Tensor | None = None):
    """Sign-project and pack a 2-D fp32 or bf16 CUDA tensor along its last
    dimension (the first ``k`` columns, default all).  Rows may be strided
    (``src.stride(1)`` must be 1).  Returns int64 ``(rows, words(k))``."""
    _need_cuda("src", src)
    if src.dim() != 2 or (src.shape[1] > 1 and src.stride(1) != 1):
        raise ValueError("src must be 2-D with unit stride along its last dimension")
    if src.dtype == torch.float32:
        dt = BNN_FP32
    elif src.dtype == torch.bfloat16:
        dt = BNN_BF16
    else:
        raise TypeError("src must be float32 or bfloat16")
    rows, cols = src.shape
    k = cols if k is None else int(k)
    ld = src.stride(0) if rows > 1 else max(cols, 1)
    if out is None:
        out = torch.empty((rows, words(k)), dtype=torch.int64, device=src.device)
    else:
        _packed("out", out, k)
    st = library().bnn_pack_signs(_ptr(src), dt, rows, k, ld, _ptr(out), _stream(src))
    _check(st, "bnn_pack_signs")
    return out


def gemm_ex(xp: torch.Tensor, wp: torch.Tensor, K: int, epilogue: int = EPI_I32,
            algo: int = ALGO_AUTO, alpha: torch.Tensor | None = None,
            out: torch.Tensor | None = None):
    """General packed product (bnn_gemm_ex): int32 (EPI_I32), alpha-scaled
    fp32 (EPI_SCALED) or packed signs (EPI_REPACK), with an explicit kernel
    family (ALGO_AUTO, ALGO_GEMV, ALGO_TILED, ALGO_MFMA)."""
    M = _packed("xp", xp, K)
    N = _packed("wp", wp, K)
    if wp.device != xp.device:
        raise ValueError("xp and wp must be on the same device")
    if epilogue == EPI_SCALED:
        _need_cuda("alpha", alpha)
        if alpha.dtype != torch.float32 or alpha.shape != (N,) or not alpha.is_contiguous():
            raise ValueError("alpha must be a contiguous float32 tensor of shape (N,)")
    out = _out_for(epilogue, M, N, xp.device, out)
    st = library().bnn_gemm_ex(_ptr(xp), _ptr(wp), _ptr(alpha) if epilogue == EPI_SCALED else None,
                               _ptr(out), M, N, int(K), int(epilogue), int(algo), _stream(xp))
    _check(st, "bnn_gemm_ex")
    return out


def _out_for(epilogue: int, M: int, N: int, device, out):
    if epilogue == EPI_I32:
        shape, dtype = (M, N), torch.int32
    elif epilogue == EPI_SCALED:
        shape, dtype = (M, N), torch.float32
    elif epilogue == EPI_REPACK:
        shape, dtype = (M, words(N)), torch.int64
    else:
        raise ValueError(f"unknown epilogue {epilogue}")
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(out.shape) != shape or out.dtype != dtype or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {dtype} tensor of shape {shape}")
    return out


def gemv_act(x: torch.Tensor, wp: torch.Tensor, K: int | None = None, epilogue: int = EPI_I32,
             alpha: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """Product of real-valued activation rows ``x`` (fp32 or bf16, 2-D, unit
    stride along the last dimension; the first ``K`` columns are used) with
    packed weights ``wp``; the kernel packs ``x`` itself (bnn_gemv_act).
    Meant for small M (batch-1 decode)."""
    _need_cuda("x", x)
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x must be 2-D with unit stride along its last dimension")
    if x.dtype == torch.float32:
        dt = BNN_FP32
    elif x.dtype == torch.bfloat16:
        dt = BNN_BF16
    else:
        raise TypeError("x must be float32 or bfloat16")
    M, cols = x.shape
    K = cols if K is None else int(K)
    N = _packed("wp", wp, K)
    if epilogue == EPI_SCALED:
        _need_cuda("alpha", alpha)
        if alpha.dtype != torch.float32 or alpha.shape != (N,) or not alpha.is_contiguous():
            raise ValueError("alpha must be a contiguous float32 tensor of shape (N,)")
    out = _out_for(epilogue, M, N, x.device, out)
    ldx = x.stride(0) if M > 1 else max(cols, 1)
    st = library().bnn_gemv_act(_ptr(x), dt, ldx, _ptr(wp),
                                _ptr(alpha) if epilogue == EPI_SCALED else None, _ptr(out),
                                M, N, K, int(epilogue), _stream(x))
    _check(st, "bnn_gemv_act")
    return out


def _named(name: str, xp, wp, K, epilogue: int, alpha, out):
    """Marshal one of the three named products (same checks as gemm_ex) and
    call its own C entry point."""
    M = _packed("xp", xp, K)
    N = _packed("wp", wp, K)
    if wp.device != xp.device:
        raise ValueError("xp and wp must be on the same device")
    if epilogue == EPI_SCALED:
        _need_cuda("alpha", alpha)
        if alpha.dtype != torch.float32 or alpha.shape != (N,) or not alpha.is_contiguous():
            raise ValueError("alpha must be a contiguous float32 tensor of shape (N,)")
    out = _out_for(epilogue, M, N, xp.device, out)
    fn = getattr(library(), name)
    if epilogue == EPI_SCALED:
        st = fn(_ptr(xp), _ptr(wp), _ptr(alpha), _ptr(out), M, N, int(K), _stream(xp))
    else:
        st = fn(_ptr(xp), _ptr(wp), _ptr(out), M, N, int(K), _stream(xp))
    _check(st, name)
    return out


def gemm_u64(xp, wp, K, out=None):
    """int32 ``(M, N)``: ``<x_m, w_n> = K - 2 * popcount(x_m XOR w_n)`` (bnn_gemm_u64)."""
    return _named("bnn_gemm_u64", xp, wp, K, EPI_I32, None, out)


def gemm_u64_scaled(xp, wp, alpha, K, out=None):
    """fp32 ``(M, N)``: ``(float)<x_m, w_n> * alpha[n]`` (bnn_gemm_u64_scaled)."""
    return _named("bnn_gemm_u64_scaled", xp, wp, K, EPI_SCALED, alpha, out)


def gemm_sign_repack(xp, wp, K, out=None):
    """int64 ``(M, words(N))``: projected signs of ``<x_m, w_n>`` packed along N
    (bnn_gemm_sign_repack)."""
    return _named("bnn_gemm_sign_repack", xp, wp, K, EPI_REPACK, None, out)


def gemm_sign_repack_thr(xp, wp, thr, K, flip=None, algo=ALGO_AUTO, out=None):
    """int64 ``(M, words(N))``: bit n of row m is 1 when ``<x_m, w_n> <= thr[n]``,
    inverted where bit n of the packed ``flip`` mask is 1
    (bnn_gemm_sign_repack_thr; the folded form of a BatchNorm after a binary
    layer, see ``fold.bn_fold``).  ``thr`` is a contiguous int32 CUDA tensor
    ``(N,)``; ``flip`` is None or a contiguous int64 CUDA tensor
    ``(words(N),)`` (``flip_words`` builds one from per-channel flags)."""
    M = _packed("xp", xp, K)
    N = _packed("wp", wp, K)
    if wp.device != xp.device:
        raise ValueError("xp and wp must be on the same device")
    _need_cuda("thr", thr)
    if thr.dtype != torch.int32 or tuple(thr.shape) != (N,) or not thr.is_contiguous():
        raise ValueError("thr must be a contiguous int32 tensor of shape (N,)")
    if flip is not None:
        _need_cuda("flip", flip)
        if (flip.dtype != torch.int64 or tuple(flip.shape) != (words(N),)
                or not flip.is_contiguous()):
            raise ValueError("flip must be a contiguous int64 tensor of shape (words(N),)")
    out = _out_for(EPI_REPACK, M, N, xp.device, out)
    st = library().bnn_gemm_sign_repack_thr(_ptr(xp), _ptr(wp), _ptr(thr), _ptr(flip), _ptr(out),
                                            M, N, int(K), int(algo), _stream(xp))
    _check(st, "bnn_gemm_sign_repack_thr")
    return out


def flip_words(flags: torch.Tensor) -> torch.Tensor:
    """Packed flip mask ``(words(N),)`` from N per-channel flags on a CUDA
    device (non-zero = flip), packed by the library's sign packer: a flag
    maps to -1 (bit 1), no flag to +1 (bit 0)."""
    _need_cuda("flags", flags)
    if flags.dim() != 1:
        raise ValueError("flags must be 1-D")
    signs = torch.where(flags != 0, -1.0, 1.0).to(torch.float32).reshape(1, -1)
    return pack_signs(signs)[0]


def gemm_signw_bf16(x, wp, K=None, alpha=None, algo=ALGO_AUTO, out=None):
    """fp32 ``(M, N)``: ``alpha[n] * sum_k x[m, k] * w_n[k]`` for real-valued
    bf16 activations ``x`` (2-D CUDA tensor, unit stride along the last
    dimension; the first ``K`` columns are used) and packed sign weights
    ``wp`` (bnn_gemm_signw_bf16).  ``alpha`` is None (no scale) or a
    contiguous float32 ``(N,)``; ``algo`` is ALGO_AUTO, ALGO_GEMV or ALGO_MFMA."""
    _need_cuda("x", x)
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16")
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x must be 2-D with unit stride along its last dimension")
    M, cols = x.shape
    K = cols if K is None else int(K)
    N = _packed("wp", wp, K)
    if alpha is not None:
        _need_cuda("alpha", alpha)
        if alpha.dtype != torch.float32 or alpha.shape != (N,) or not alpha.is_contiguous():
            raise ValueError("alpha must be a contiguous float32 tensor of shape (N,)")
    out = _out_for(EPI_SCALED, M, N, x.device, out)
    ldx = x.stride(0) if M > 1 else max(cols, 1)
    st = library().bnn_gemm_signw_bf16(_ptr(x), ldx, _ptr(wp), _ptr(alpha), _ptr(out), M, N, K,
                                       int(algo), _stream(x))
    _check(st, "bnn_gemm_signw_bf16")
    return out


def chain3(x, w1, w2, w3, alpha3=None, out=None, thr1=None, flip1=None, thr2=None, flip2=None):
    """fp32 ``(M, N3)``: three chained binary layers in one launch
    (bnn_chain3).  ``x`` is a 2-D fp32 or bf16 CUDA tensor (unit stride along
    its last dimension, K0 columns); ``w1``, ``w2``, ``w3`` are packed weights
    ``(N1, words(K0))``, ``(N2, words(N1))``, ``(N3, words(N2))``; ``alpha3`` is
    None or a contiguous float32 ``(N3,)``.  ``thr1``/``flip1`` and
    ``thr2``/``flip2`` optionally make the hidden layers threshold repacks
    (as gemm_sign_repack_thr).  Equal, bit for bit, to pack_signs ->
    gemm_sign_repack(_thr) -> gemm_sign_repack(_thr) -> gemm_u64_scaled."""
    _need_cuda("x", x)
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x must be 2-D with unit stride along its last dimension")
    if x.dtype == torch.float32:
        dt = BNN_FP32
    elif x.dtype == torch.bfloat16:
        dt = BNN_BF16
    else:
        raise TypeError("x must be float32 or bfloat16")
    M, K0 = x.shape
    N1 = _packed("w1", w1, K0)
    N2 = _packed("w2", w2, N1)
    N3 = _packed("w3", w3, N2)
    if alpha3 is not None:
        _need_cuda("alpha3", alpha3)
        if alpha3.dtype != torch.float32 or alpha3.shape != (N3,) or not alpha3.is_contiguous():
            raise ValueError("alpha3 must be a contiguous float32 tensor of shape (N3,)")
    for name, t, n in (("thr1", thr1, N1), ("thr2", thr2, N2)):
        if t is not None:
            _need_cuda(name, t)
            if t.dtype != torch.int32 or tuple(t.shape) != (n,) or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 tensor of shape ({n},)")
    for name, f, n in (("flip1", flip1, N1), ("flip2", flip2, N2)):
        if f is not None:
            _need_cuda(name, f)
            if f.dtype != torch.int64 or tuple(f.shape) != (words(n),) or not f.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int64 tensor of shape ({words(n)},)")
    out = _out_for(EPI_SCALED, M, N3, x.device, out)
    ldx = x.stride(0) if M > 1 else max(K0, 1)
    st = library().bnn_chain3(_ptr(x), dt, ldx, _ptr(w1), _ptr(thr1), _ptr(flip1), _ptr(w2),
                              _ptr(thr2), _ptr(flip2), _ptr(w3), _ptr(alpha3), _ptr(out), M, K0, N1,
                              N2, N3, _stream(x))
    _check(st, "bnn_chain3")
    return out


def _real_rows(name: str, t: torch.Tensor):
    """(dtype code, rows, columns, row stride) of a 2-D fp32 / bf16 CUDA
    tensor with unit stride along its last dimension."""
    _need_cuda(name, t)
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D with unit stride along its last dimension")
    if t.dtype == torch.float32:
        dt = BNN_FP32
    elif t.dtype == torch.bfloat16:
        dt = BNN_BF16
    else:
        raise TypeError(f"{name} must be float32 or bfloat16")
    rows, cols = t.shape
    return dt, rows, cols, (t.stride(0) if rows > 1 else max(cols, 1))


def _vector(name: str, t, n: int, device, dtype=torch.float32):
    _need_cuda(name, t)
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape ({n},)")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")


def layernorm_fwd(x, gamma=None, beta=None, eps=1e-5, stats=True, out=None):
    """Layer norm of the rows of ``x`` (2-D fp32 or bf16 CUDA tensor, rows may
    be strided): ``(y, mean, rstd)`` with ``y`` of x's type and fp32 ``mean``
    and ``rstd`` of shape ``(M,)``, or None for both with ``stats=False``
    (bnn_layernorm_fwd).  ``gamma`` and ``beta`` are None or contiguous
    float32 ``(N,)``; ``out`` may be a tensor of x's shape and type with unit
    stride along its last dimension."""
    dt, M, N, ldx = _real_rows("x", x)
    if gamma is not None:
        _vector("gamma", gamma, N, x.device)
    if beta is not None:
        _vector("beta", beta, N, x.device)
    if out is None:
        out = torch.empty((M, N), dtype=x.dtype, device=x.device)
        ldy = max(N, 1)
    else:
        dto, Mo, No, ldy = _real_rows("out", out)
        if (dto, Mo, No) != (dt, M, N) or out.device != x.device:
            raise ValueError("out must have x's shape, type and device")
    mean = rstd = None
    if stats:
        mean, rstd = torch.empty((2, M), dtype=torch.float32, device=x.device).unbind(0)
    st = library().bnn_layernorm_fwd(_ptr(x), dt, ldx, _ptr(gamma), _ptr(beta), _ptr(out), ldy,
                                     _ptr(mean), _ptr(rstd), M, N, float(eps), _stream(x))
    _check(st, "bnn_layernorm_fwd")
    return out, mean, rstd


def layernorm_bwd(dy, x, mean, rstd, gamma=None, params=True):
    """Gradient of layernorm_fwd: ``(dx, dgamma, dbeta)`` from the output's
    gradient ``dy`` (x's shape and type), the forward pass's ``x``, ``mean``
    and ``rstd`` and its ``gamma`` (bnn_layernorm_bwd).  ``params=False``
    leaves out the sums over the rows (None for dgamma and dbeta)."""
    dt, M, N, ldx = _real_rows("x", x)
    dtd, Md, Nd, lddy = _real_rows("dy", dy)
    if (dtd, Md, Nd) != (dt, M, N) or dy.device != x.device:
        raise ValueError("dy must have x's shape, type and device")
    _vector("mean", mean, M, x.device)
    _vector("rstd", rstd, M, x.device)
    if gamma is not None:
        _vector("gamma", gamma, N, x.device)
    dx = torch.empty((M, N), dtype=x.dtype, device=x.device)
    dgamma = dbeta = ws = None
    need = 0
    if params:
        dgamma, dbeta = torch.empty((2, N), dtype=torch.float32, device=x.device).unbind(0)
        need = library().bnn_layernorm_bwd_workspace(M, N)
        if need > 0:
            ws = torch.empty((need,), dtype=torch.uint8, device=x.device)
    st = library().bnn_layernorm_bwd(_ptr(dy), lddy, _ptr(x), ldx, dt, _ptr(gamma), _ptr(mean),
                                     _ptr(rstd), _ptr(dx), max(N, 1), _ptr(dgamma), _ptr(dbeta),
                                     _ptr(ws), need, M, N, _stream(x))
    _check(st, "bnn_layernorm_bwd")
    return dx, dgamma, dbeta


def f8_row_bytes(k: int) -> int:
    """Bytes of 8-bit values per row of k columns: 128 * ceil(k / 128)."""
    return max(0, -(-int(k) // 128) * 128)


def f8_scale_bytes(k: int) -> int:
    """Scale bytes per row of k columns: 4 * ceil(k / 512), one per block of
    128 columns and unused ones up to a multiple of four."""
    return max(0, -(-int(k) // 512) * 4)


def quant_f8(x, transpose=False):
    """Block-scaled 8-bit form of ``x`` (2-D fp32 or bf16 CUDA tensor, rows may
    be strided), or of its transpose: ``(q, s)``, two uint8 tensors of shapes
    ``(R, f8_row_bytes(K))`` (e4m3 values, zeros past K; view them as
    ``torch.float8_e4m3fn``) and ``(R, f8_scale_bytes(K))`` (biased exponents of
    the blocks of 128 columns) (bnn_quant_f8)."""
    dt, rows, k, ld = _real_rows("x", x)
    R, K = (k, rows) if transpose else (rows, k)
    q = torch.empty((R, f8_row_bytes(K)), dtype=torch.uint8, device=x.device)
    s = torch.empty((R, f8_scale_bytes(K)), dtype=torch.uint8, device=x.device)
    st = library().bnn_quant_f8(_ptr(x), dt, rows, k, ld, int(bool(transpose)), _ptr(q), _ptr(s),
                                _stream(x))
    _check(st, "bnn_quant_f8")
    return q, s


def _quantised(name: str, q, s, k: int) -> int:
    for t in (q, s):
        _need_cuda(name, t)
        if t.dtype != torch.uint8 or t.dim() != 2 or not t.is_contiguous():
            raise TypeError(f"{name} must be two contiguous 2-D uint8 tensors (values, scales)")
    if (q.shape[1] != f8_row_bytes(k) or s.shape[1] != f8_scale_bytes(k)
            or q.shape[0] != s.shape[0] or q.device != s.device):
        raise ValueError(f"{name} does not have the block-scaled form of K={k} columns")
    return q.shape[0]


def gemm_f8(xq, xs, wq, ws, K, dtype=torch.float32, out=None, fast=False):
    """``(M, N)`` product of two block-scaled 8-bit matrices of K columns (as
    quant_f8 makes them): ``x @ w.T`` with fp32 sums, rounded once to ``dtype``
    (float32 or bfloat16) (bnn_gemm_f8).  ``fast=True``, for bfloat16 outputs:
    the 8-bit matrix instructions, which drop what a product has below 2^-13 of
    the largest among eight neighbours along K (bnn_gemm_f8_fast)."""
    K = int(K)
    M = _quantised("x", xq, xs, K)
    N = _quantised("w", wq, ws, K)
    if wq.device != xq.device:
        raise ValueError("x and w must be on the same device")
    out, dt = _real_out(M, N, dtype, xq.device, out)
    if fast:
        if dt != BNN_BF16:
            raise TypeError("fast products have bfloat16 outputs")
        st = library().bnn_gemm_f8_fast(_ptr(xq), _ptr(xs), _ptr(wq), _ptr(ws), _ptr(out), M, N, K,
                                        _stream(xq))
        _check(st, "bnn_gemm_f8_fast")
        return out
    st = library().bnn_gemm_f8(_ptr(xq), _ptr(xs), _ptr(wq), _ptr(ws), _ptr(out), dt, M, N, K,
                               _stream(xq))
    _check(st, "bnn_gemm_f8")
    return out


def _real_out(M: int, N: int, dtype, device, out):
    """Output tensor and dtype code of a product that stores real values."""
    if out is not None:
        dtype = out.dtype
    if dtype == torch.float32:
        dt = BNN_FP32
    elif dtype == torch.bfloat16:
        dt = BNN_BF16
    else:
        raise TypeError("dtype must be float32 or bfloat16")
    if out is None:
        return torch.empty((M, N), dtype=dtype, device=device), dt
    if tuple(out.shape) != (M, N) or not out.is_contiguous() or out.device != device:
        raise ValueError(f"out must be a contiguous tensor of shape ({M}, {N}) on {device}")
    return out, dt


def gemm_signw_grouped(x, wp, offsets, K=None, alpha=None, rows=None, row_scale=None,
                       dtype=torch.float32, algo=ALGO_AUTO, out=None):
    """``(R, N)`` sign-weight products grouped by expert
    (bnn_gemm_signw_grouped): row r, ``offsets[e] <= r < offsets[e + 1]``, is
    ``row_scale[r] * alpha[e] * (x[rows[r]] @ w[e].T)`` with real bf16
    activations ``x`` (2-D CUDA tensor, unit stride along the last dimension;
    the first ``K`` columns are used) and packed sign weights ``wp``, a
    contiguous int64 tensor ``(E, N, words(K))``.  ``offsets`` is a contiguous
    int32 CUDA tensor ``(E + 1,)``, non-decreasing (it is not read on the
    host); ``rows`` None (row r is x's row r) or contiguous int32 ``(R,)``;
    ``alpha`` None or contiguous float32 ``(E, N)``; ``row_scale`` None or
    contiguous float32 ``(R,)``; ``dtype`` float32 or bfloat16; ``algo``
    ALGO_AUTO, ALGO_GEMV or ALGO_MFMA.  Rows outside the groups are not
    written."""
    dt, xrows, cols, ldx = _real_rows("x", x)
    if dt != BNN_BF16:
        raise TypeError("x must be bfloat16")
    K = cols if K is None else int(K)
    if K > cols:
        raise ValueError(f"x has {cols} columns, K={K}")
    _need_cuda("wp", wp)
    if wp.dtype != torch.int64 or wp.dim() != 3 or not wp.is_contiguous():
        raise TypeError("wp must be a contiguous 3-D int64 tensor of packed words")
    E, N, kw = wp.shape
    if kw != -(-K // 64):
        raise ValueError(f"wp has {kw} words per row, K={K} needs {words(K)}")
    if wp.device != x.device:
        raise ValueError("x and wp must be on the same device")
    _vector("offsets", offsets, E + 1, x.device, torch.int32)
    R = xrows
    if rows is not None:
        R = rows.shape[0] if isinstance(rows, torch.Tensor) and rows.dim() == 1 else -1
        _vector("rows", rows, R, x.device, torch.int32)
    if alpha is not None:
        _need_cuda("alpha", alpha)
        if (alpha.dtype != torch.float32 or tuple(alpha.shape) != (E, N)
                or not alpha.is_contiguous() or alpha.device != x.device):
            raise ValueError(f"alpha must be a contiguous float32 tensor of shape ({E}, {N})")
    if row_scale is not None:
        _vector("row_scale", row_scale, R, x.device)
    out, dto = _real_out(R, N, dtype, x.device, out)
    st = library().bnn_gemm_signw_grouped(_ptr(x), ldx, xrows, _ptr(rows), _ptr(offsets), _ptr(wp),
                                          _ptr(alpha), _ptr(row_scale), _ptr(out), dto, R, E, N, K,
                                          int(algo), _stream(x))
    _check(st, "bnn_gemm_signw_grouped")
    return out


def _call(name: str, t: torch.Tensor, *args) -> None:
    """One C call on the current stream of t's device, with that device current."""
    fn = getattr(library(), name)
    if torch.cuda.current_device() == t.device.index:
        st = fn(*args, _stream(t))
    else:
        with torch.cuda.device(t.device):
            st = fn(*args, _stream(t))
    _check(st, name)


def _matrix(name: str, t, shape, dtype, device) -> None:
    _need_cuda(name, t)
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def _new(rows: int, cols: int, dtype, device):
    # a third of a microsecond less than torch.empty
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _new_vector(n: int, dtype, device):
    return torch.empty_strided((n,), (1,), dtype=dtype, device=device)


def _workspace(need: int, device):
    return torch.empty_strided((need,), (1,), dtype=torch.uint8, device=device) if need > 0 else None


class Routing(NamedTuple):
    """What route_fwd makes of T tokens' logits (bnn_route_fwd)."""
    experts: torch.Tensor  # int32 (T, k): the choices, largest logit first; -1 without an expert
    weights: torch.Tensor  # float32 (T, k)
    place: torch.Tensor    # int32 (T, k): each choice's row in the experts' order; -2 - row without an expert
    rows: torch.Tensor     # int32 (T k,): each row's token; -1 behind the last group
    offsets: torch.Tensor  # int32 (E + 1,): each expert's range of rows
    counts: torch.Tensor   # int32 (E,)
    stats: torch.Tensor    # float32 (T, 2): the row's maximum, 1 / sum exp(z - maximum)
    slope: torch.Tensor | None  # float32 (E,): derivative of the loss by a token's probability
    loss: torch.Tensor | None   # float32 (1,): the balance loss


def route_fwd(logits, k, valid=None, normalise=True, loss=True) -> Routing:
    """Top-``k`` router of a mixture of experts (bnn_route_fwd): choices,
    weights, rows in the experts' order (``rows`` and ``offsets`` are what
    gemm_signw_grouped takes, ``place`` and ``weights`` what combine_fwd takes),
    counts and, with ``loss``, the balance loss.  ``logits``: 2-D fp32 or bf16
    CUDA tensor (T, E), rows may be strided, E <= 1024; -inf switches an expert
    off for a token.  ``valid``: None or a contiguous bool or uint8 tensor (T,);
    a token that is not valid is not routed.  ``normalise``: the weights of a
    token's choices add up to 1."""
    dt, T, E, ldz = _real_rows("logits", logits)
    dev = logits.device
    k = int(k)
    if valid is not None:
        _need_cuda("valid", valid)
        if (valid.dtype not in (torch.bool, torch.uint8) or tuple(valid.shape) != (T,)
                or not valid.is_contiguous() or valid.device != dev):
            raise ValueError(f"valid must be a contiguous bool or uint8 tensor of shape ({T},) on {dev}")
    if not (1 <= k <= E <= 1024 and k <= 32):
        raise BnnError(2, "bnn_route_fwd")
    i32, f32 = torch.int32, torch.float32
    experts, place, weights = _new(T, k, i32, dev), _new(T, k, i32, dev), _new(T, k, f32, dev)
    rows, offsets, counts = _new_vector(T * k, i32, dev), _new_vector(E + 1, i32, dev), _new_vector(E, i32, dev)
    stats = _new(T, 2, f32, dev)
    slope = total = None
    if loss:
        slope, total = _new_vector(E, f32, dev), _new_vector(1, f32, dev)
    need = library().bnn_route_fwd_workspace(T, E, k)
    ws = _workspace(need, dev)
    _call("bnn_route_fwd", logits, _ptr(logits), dt, ldz, _ptr(valid), _ptr(experts), _ptr(weights), _ptr(place),
          _ptr(rows), _ptr(offsets), _ptr(counts), _ptr(stats), _ptr(slope), _ptr(total), _ptr(ws), need, T, E, k,
          int(bool(normalise)))
    return Routing(experts, weights, place, rows, offsets, counts, stats, slope, total)


def route_bwd(logits, experts, weights, stats, slope=None, dweights=None, dloss=None, normalise=True):
    """Gradient of route_fwd by its logits (their shape and type)
    (bnn_route_bwd), from its ``experts``, ``weights``, ``stats`` and ``slope``:
    ``dweights`` (T, k) is the weights' gradient or None, ``dloss`` (a float32
    tensor of one element) the balance loss's or None.  Every tensor but the
    logits is contiguous; ``normalise`` as in the forward pass."""
    dt, T, E, ldz = _real_rows("logits", logits)
    dev = logits.device
    _need_cuda("experts", experts)
    k = experts.shape[1] if experts.dim() == 2 else -1
    _matrix("experts", experts, (T, k), torch.int32, dev)
    _matrix("weights", weights, (T, k), torch.float32, dev)
    _matrix("stats", stats, (T, 2), torch.float32, dev)
    if dweights is not None:
        _matrix("dweights", dweights, (T, k), torch.float32, dev)
    if dloss is not None:
        _vector("slope", slope, E, dev)
        _need_cuda("dloss", dloss)
        if dloss.dtype != torch.float32 or dloss.numel() != 1 or dloss.device != dev:
            raise ValueError(f"dloss must be a float32 tensor of one element on {dev}")
    dz = _new(T, E, logits.dtype, dev)
    _call("bnn_route_bwd", logits, _ptr(logits), dt, ldz, _ptr(experts), _ptr(weights), _ptr(stats),
          None if dloss is None else _ptr(slope), _ptr(dweights), _ptr(dloss), _ptr(dz), max(E, 1), T, E, k,
          int(bool(normalise)))
    return dz


def combine_fwd(y, place, weights=None, residual=None, dtype=None, out=None):
    """``out[t] = residual[t] + sum_j weights[t, j] * y[place[t, j]]``, the sum of
    the experts' outputs at each token (bnn_combine_fwd).  ``y``: 2-D fp32 or
    bf16 CUDA tensor (R, N), rows may be strided; ``place``: contiguous int32
    (T, k) as route_fwd makes it (negative: no expert); ``weights`` None (1)
    or contiguous float32 (T, k); ``residual`` None or (T, N) of the output's
    type.  ``dtype`` of the output: float32 or bfloat16, the residual's or y's
    by default; ``out`` may be the residual itself."""
    dty, R, N, ldy = _real_rows("y", y)
    dev = y.device
    _need_cuda("place", place)
    if place.dim() != 2:
        raise ValueError("place must be 2-D")
    T, k = place.shape
    _matrix("place", place, (T, k), torch.int32, dev)
    if weights is not None:
        _matrix("weights", weights, (T, k), torch.float32, dev)
    if dtype is None:
        dtype = out.dtype if out is not None else residual.dtype if residual is not None else y.dtype
    out, dt, ldo = _rows_out("out", out, T, N, dtype, dev)
    ldr = 0
    if residual is not None:
        ldr = _same_rows("residual", residual, T, N, dt, dev)
    _call("bnn_combine_fwd", y, _ptr(y), dty, ldy, R, _ptr(place), _ptr(weights), _ptr(residual), ldr, _ptr(out), dt,
          ldo, T, N, k)
    return out


def combine_bwd(dout, place, weights=None, y=None, rows=None, dtype=None):
    """Gradient of combine_fwd: ``(dy, dweights)`` (bnn_combine_bwd).  ``dout``:
    2-D fp32 or bf16 CUDA tensor (T, N).  ``y`` is what the forward pass summed,
    or its block-scaled 8-bit form ``(q, s)`` (quant_f8); without it only ``dy``
    is computed (None for dweights) and ``rows`` says how many rows that has.
    ``dy`` has the type ``dtype``: y's by default, dout's where y is in 8 bits
    or missing.  Every row of dy is written if ``place`` names each row once,
    as route_fwd's does (rows without an expert: zeros); others are left
    undefined.  The residual's gradient is dout itself."""
    dt, T, N, lddo = _real_rows("dout", dout)
    dev = dout.device
    _need_cuda("place", place)
    k = place.shape[1] if place.dim() == 2 else -1
    _matrix("place", place, (T, k), torch.int32, dev)
    if weights is not None:
        _matrix("weights", weights, (T, k), torch.float32, dev)
    data = ys = None
    dty, ldy = BNN_BF16, N
    if y is None:
        R = T * k if rows is None else int(rows)
    elif isinstance(y, (tuple, list)):
        data, ys = y
        R = _quantised("y", data, ys, N)
        dty = BNN_F8
    else:
        data = y
        dty, R, Ny, ldy = _real_rows("y", y)
        if Ny != N:
            raise ValueError(f"y has {Ny} columns, dout {N}")
        dtype = y.dtype if dtype is None else dtype
    if data is not None and data.device != dev:
        raise ValueError(f"y must be on {dev}")
    dy, dtd = _real_out(R, N, dout.dtype if dtype is None else dtype, dev, None)
    dw = None if y is None else _new(T, k, torch.float32, dev)
    _call("bnn_combine_bwd", dout, _ptr(dout), dt, lddo, _ptr(data), _ptr(ys), dty, ldy, R, _ptr(place), _ptr(weights),
          _ptr(dy), dtd, max(N, 1), _ptr(dw), T, N, k)
    return dy, dw


def _rows_out(name: str, out, M: int, N: int, dtype, device):
    """(tensor, dtype code, row stride) of an output whose rows may be strided."""
    if out is None:
        out, dt = _real_out(M, N, dtype, device, None)
        return out, dt, max(N, 1)
    dt, Mo, No, ld = _real_rows(name, out)
    if (Mo, No) != (M, N) or out.dtype != dtype or out.device != device:
        raise ValueError(f"{name} must be a {dtype} tensor of shape ({M}, {N}) on {device}")
    return out, dt, ld


def _same_rows(name: str, t, M: int, N: int, dt: int, device) -> int:
    """Row stride of an input of the output's shape and type."""
    d, Mt, Nt, ld = _real_rows(name, t)
    if (d, Mt, Nt) != (dt, M, N) or t.device != device:
        raise ValueError(f"{name} must have the output's shape ({M}, {N}), type and device")
    return ld


def _factors(ids, a, b, scale, T: int, K: int, N: int, device):
    """(adapters, rank) of checked adapter factors."""
    _vector("ids", ids, T, device, torch.int32)
    _need_cuda("a", a)
    if a.dim() != 3:
        raise ValueError("a must be 3-D: (adapters, rank, K)")
    L, r = a.shape[0], a.shape[1]
    _matrix("a", a, (L, r, K), torch.bfloat16, device)
    _matrix("b", b, (L, r, N), torch.bfloat16, device)
    if scale is not None:
        _vector("scale", scale, L, device)
    return L, r


def adapter_fwd(x, ids, a, b, scale=None, base=None, dtype=None, out=None):
    """Low-rank adapters of many requests beside a shared projection
    (bnn_adapter_fwd): ``(out, u)`` with ``u[t] = a[ids[t]] @ x[t]`` (float32
    (T, r)) and ``out[t] = base[t] + scale[ids[t]] * (u[t] @ b[ids[t]])``.  ``x``:
    2-D bf16 CUDA tensor (T, K), rows may be strided; ``ids``: contiguous int32
    (T,), an id outside [0, L) has no adapter; ``a`` and ``b``: contiguous
    bfloat16 (L, r, K) and (L, r, N), r <= 128; ``scale`` None (1) or contiguous
    float32 (L,); ``base`` None (0) or (T, N), the projection's output, of type
    ``dtype`` (float32 or bfloat16; the base's by default, else float32).
    ``out`` may be the base itself: rows without an adapter stay as they are."""
    dtx, T, K, ldx = _real_rows("x", x)
    if dtx != BNN_BF16:
        raise TypeError("x must be bfloat16")
    dev = x.device
    _need_cuda("b", b)
    N = b.shape[2] if b.dim() == 3 else -1
    L, r = _factors(ids, a, b, scale, T, K, N, dev)
    if dtype is None:
        dtype = out.dtype if out is not None else base.dtype if base is not None else torch.float32
    out, dt, ldo = _rows_out("out", out, T, N, dtype, dev)
    ldb = _same_rows("base", base, T, N, dt, dev) if base is not None else 0
    u = _new(T, r, torch.float32, dev)
    need = library().bnn_adapter_fwd_workspace(T, K, N, r, L)
    ws = _workspace(need, dev)
    _call("bnn_adapter_fwd", x, _ptr(x), ldx, _ptr(ids), _ptr(a), _ptr(b), _ptr(scale), _ptr(base), ldb, _ptr(out),
          ldo, dt, _ptr(u), _ptr(ws), need, T, K, N, r, L)
    return out, u


def adapter_bwd(dy, x, u, ids, a, b, scale=None, base=None, dtype=None, dx=True, params=True):
    """Gradient of adapter_fwd: ``(dx, da, db)`` (bnn_adapter_bwd) from the
    output's gradient ``dy`` (2-D bf16 CUDA tensor (T, N)), the forward pass's
    ``x`` (bf16, or its block-scaled 8-bit form ``(q, s)``, quant_f8) and ``u``:
    with ``v[t] = b[ids[t]] @ dy[t]``
    ``dx[t] = base[t] + scale * (v[t] @ a[ids[t]])``,
    ``da[l] = scale[l] * sum_t outer(v[t], x[t])`` and
    ``db[l] = scale[l] * sum_t outer(u[t], dy[t])`` over l's rows (float32).
    ``base`` None (0) or (T, K): the gradient that reaches x by the shared
    projection, of type ``dtype`` (the base's by default, else float32).
    ``dx=False`` and ``params=False`` leave those out (None).  With ``params``
    at most 1024 adapters."""
    dtd, T, N, lddy = _real_rows("dy", dy)
    if dtd != BNN_BF16:
        raise TypeError("dy must be bfloat16")
    dev = dy.device
    _need_cuda("a", a)
    K = a.shape[2] if a.dim() == 3 else -1
    L, r = _factors(ids, a, b, scale, T, K, N, dev)
    data = xs = None
    dtx, ldx = BNN_BF16, max(K, 1)
    if params:
        _matrix("u", u, (T, r), torch.float32, dev)
        if isinstance(x, (tuple, list)):
            data, xs = x
            if _quantised("x", data, xs, K) != T:
                raise ValueError(f"x must have {T} rows")
            dtx = BNN_F8
        else:
            data = x
            dtx, Tx, Kx, ldx = _real_rows("x", x)
            if dtx != BNN_BF16:
                raise TypeError("x must be bfloat16")
            if (Tx, Kx) != (T, K):
                raise ValueError(f"x must have shape ({T}, {K})")
        if data.device != dev:
            raise ValueError(f"x must be on {dev}")
    out, dt, ldo, ldb = None, BNN_FP32, max(K, 1), 0
    if dx:
        if dtype is None:
            dtype = base.dtype if base is not None else torch.float32
        out, dt, ldo = _rows_out("dx", None, T, K, dtype, dev)
        if base is not None:
            ldb = _same_rows("base", base, T, K, dt, dev)
    else:
        base = None
    da = db = None
    need = 0
    ws = None
    if dx or params:
        need = library().bnn_adapter_bwd_workspace(T, K, N, r, L)
        ws = _workspace(need, dev)
    if params:
        da = torch.empty((L, r, K), dtype=torch.float32, device=dev)
        db = torch.empty((L, r, N), dtype=torch.float32, device=dev)
    _call("bnn_adapter_bwd", dy, _ptr(dy), lddy, _ptr(data), _ptr(xs), dtx, ldx, _ptr(u) if params else None,
          _ptr(ids), _ptr(a), _ptr(b), _ptr(scale), _ptr(base), ldb, _ptr(out), ldo, dt, _ptr(da), _ptr(db), _ptr(ws),
          need, T, K, N, r, L)
    return out, da, db
