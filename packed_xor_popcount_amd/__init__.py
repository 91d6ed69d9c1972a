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


# The calls below take a few microseconds on the device, so their checks are
# written for few Python operations, and outputs are allocated by
# torch.empty_strided (a third of a microsecond less than torch.empty).

_CODES = {torch.float32: BNN_FP32, torch.bfloat16: BNN_BF16}


def _index(name: str, t) -> int:
    """Device index of a CUDA tensor."""
    index = t.get_device() if isinstance(t, torch.Tensor) else -1
    if index < 0:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    return index


def _rows_of(name: str, t, index: int):
    """As _real_rows, of a tensor on device ``index``."""
    if _index(name, t) != index:
        raise ValueError(f"{name} must be on cuda:{index}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D with unit stride along its last dimension")
    rows, cols = t.shape
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name} must be 2-D with unit stride along its last dimension")
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16")
    return code, rows, cols, (ld if rows > 1 else max(cols, 1))


def _matrix(name: str, t, shape, dtype, index: int) -> int:
    """Pointer of a contiguous tensor of this shape and type on device ``index``."""
    if _index(name, t) != index or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}")
    return t.data_ptr()


def _same_rows(name: str, t, M: int, N: int, code: int, index: int):
    """(pointer, row stride) of an input of the output's shape and type."""
    d, Mt, Nt, ld = _rows_of(name, t, index)
    if d != code or Mt != M or Nt != N:
        raise ValueError(f"{name} must have the output's shape ({M}, {N}) and type")
    return t.data_ptr(), ld


def _out_rows(name: str, out, M: int, N: int, dtype, device, index: int):
    """(tensor, type code, row stride) of an output, whose rows may be strided where it is given."""
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError("dtype must be float32 or bfloat16")
    if out is None:
        return _new(M, N, dtype, device), code, max(N, 1)
    d, Mo, No, ld = _rows_of(name, out, index)
    if d != code or Mo != M or No != N:
        raise ValueError(f"{name} must be a {dtype} tensor of shape ({M}, {N})")
    return out, code, ld


def _new(rows: int, cols: int, dtype, device):
    return torch.empty_strided((rows, cols), (max(cols, 1), 1), dtype=dtype, device=device)


def _new_vector(n: int, dtype, device):
    return torch.empty_strided((n,), (1,), dtype=dtype, device=device)


def _workspace(need: int, device):
    """(tensor to keep until the call, pointer)."""
    if need <= 0:
        return None, None
    ws = torch.empty_strided((need,), (1,), dtype=torch.uint8, device=device)
    return ws, ws.data_ptr()


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
    index = _index("logits", logits)
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return route_fwd(logits, k, valid, normalise, loss)
    dt, T, E, ldz = _rows_of("logits", logits, index)
    dev = logits.device
    k = int(k)
    if not (1 <= k <= E <= 1024 and k <= 32):
        raise BnnError(2, "bnn_route_fwd")
    mask = None
    if valid is not None:
        _index("valid", valid)
        mask = _matrix("valid", valid, (T,), torch.uint8 if valid.dtype is torch.uint8 else torch.bool, index)
    i32, f32 = torch.int32, torch.float32
    experts, place, weights = _new(T, k, i32, dev), _new(T, k, i32, dev), _new(T, k, f32, dev)
    rows, offsets, counts = _new_vector(T * k, i32, dev), _new_vector(E + 1, i32, dev), _new_vector(E, i32, dev)
    stats = _new(T, 2, f32, dev)
    slope = total = None
    if loss:
        slope, total = _new_vector(E, f32, dev), _new_vector(1, f32, dev)
    lib = library()
    need = lib.bnn_route_fwd_workspace(T, E, k)
    ws, wp = _workspace(need, dev)
    st = lib.bnn_route_fwd(logits.data_ptr(), dt, ldz, mask, experts.data_ptr(), weights.data_ptr(), place.data_ptr(),
                           rows.data_ptr(), offsets.data_ptr(), counts.data_ptr(), stats.data_ptr(), _ptr(slope),
                           _ptr(total), wp, need, T, E, k, 1 if normalise else 0, _stream(logits))
    _check(st, "bnn_route_fwd")
    return Routing(experts, weights, place, rows, offsets, counts, stats, slope, total)


def route_bwd(logits, experts, weights, stats, slope=None, dweights=None, dloss=None, normalise=True):
    """Gradient of route_fwd by its logits (their shape and type)
    (bnn_route_bwd), from its ``experts``, ``weights``, ``stats`` and ``slope``:
    ``dweights`` (T, k) is the weights' gradient or None, ``dloss`` (a float32
    tensor of one element) the balance loss's or None.  Every tensor but the
    logits is contiguous; ``normalise`` as in the forward pass."""
    index = _index("logits", logits)
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return route_bwd(logits, experts, weights, stats, slope, dweights, dloss, normalise)
    dt, T, E, ldz = _rows_of("logits", logits, index)
    _index("experts", experts)
    k = experts.shape[1] if experts.dim() == 2 else -1
    pe = _matrix("experts", experts, (T, k), torch.int32, index)
    pw = _matrix("weights", weights, (T, k), torch.float32, index)
    ps = _matrix("stats", stats, (T, 2), torch.float32, index)
    pd = _matrix("dweights", dweights, (T, k), torch.float32, index) if dweights is not None else None
    sl = dl = None
    if dloss is not None:
        sl = _matrix("slope", slope, (E,), torch.float32, index)
        if _index("dloss", dloss) != index or dloss.dtype is not torch.float32 or dloss.numel() != 1:
            raise ValueError(f"dloss must be a float32 tensor of one element on cuda:{index}")
        dl = dloss.data_ptr()
    dz = _new(T, E, logits.dtype, logits.device)
    st = library().bnn_route_bwd(logits.data_ptr(), dt, ldz, pe, pw, ps, sl, pd, dl, dz.data_ptr(), max(E, 1), T, E, k,
                                 1 if normalise else 0, _stream(logits))
    _check(st, "bnn_route_bwd")
    return dz


def combine_fwd(y, place, weights=None, residual=None, dtype=None, out=None):
    """``out[t] = residual[t] + sum_j weights[t, j] * y[place[t, j]]``, the sum of
    the experts' outputs at each token (bnn_combine_fwd).  ``y``: 2-D fp32 or
    bf16 CUDA tensor (R, N), rows may be strided; ``place``: contiguous int32
    (T, k) as route_fwd makes it (negative: no expert); ``weights`` None (1)
    or contiguous float32 (T, k); ``residual`` None or (T, N) of the output's
    type.  ``dtype`` of the output: float32 or bfloat16, the residual's or y's
    by default; ``out`` may be the residual itself (the same rows, stride
    included)."""
    index = _index("y", y)
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return combine_fwd(y, place, weights, residual, dtype, out)
    dty, R, N, ldy = _rows_of("y", y, index)
    _index("place", place)
    if place.dim() != 2:
        raise ValueError("place must be 2-D")
    T, k = place.shape
    pp = _matrix("place", place, (T, k), torch.int32, index)
    pw = _matrix("weights", weights, (T, k), torch.float32, index) if weights is not None else None
    if dtype is None:
        dtype = out.dtype if out is not None else residual.dtype if residual is not None else y.dtype
    out, dt, ldo = _out_rows("out", out, T, N, dtype, y.device, index)
    pr, ldr = None, 0
    if residual is not None:
        pr, ldr = _same_rows("residual", residual, T, N, dt, index)
    st = library().bnn_combine_fwd(y.data_ptr(), dty, ldy, R, pp, pw, pr, ldr, out.data_ptr(), dt, ldo, T, N, k,
                                   _stream(y))
    _check(st, "bnn_combine_fwd")
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
    index = _index("dout", dout)
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return combine_bwd(dout, place, weights, y, rows, dtype)
    dt, T, N, lddo = _rows_of("dout", dout, index)
    dev = dout.device
    _index("place", place)
    k = place.shape[1] if place.dim() == 2 else -1
    pp = _matrix("place", place, (T, k), torch.int32, index)
    pw = _matrix("weights", weights, (T, k), torch.float32, index) if weights is not None else None
    py = ys = None
    dty, ldy = BNN_BF16, N
    if y is None:
        R = T * k if rows is None else int(rows)
    elif isinstance(y, (tuple, list)):
        q, s = y
        R = _quantised("y", q, s, N)
        if q.get_device() != index:
            raise ValueError(f"y must be on cuda:{index}")
        py, ys, dty = q.data_ptr(), s.data_ptr(), BNN_F8
    else:
        dty, R, Ny, ldy = _rows_of("y", y, index)
        if Ny != N:
            raise ValueError(f"y has {Ny} columns, dout {N}")
        py = y.data_ptr()
        dtype = y.dtype if dtype is None else dtype
    dy, dtd, lddy = _out_rows("dy", None, R, N, dout.dtype if dtype is None else dtype, dev, index)
    dw = None if y is None else _new(T, k, torch.float32, dev)
    st = library().bnn_combine_bwd(dout.data_ptr(), dt, lddo, py, ys, dty, ldy, R, pp, pw, dy.data_ptr(), dtd, lddy,
                                   _ptr(dw), T, N, k, _stream(dout))
    _check(st, "bnn_combine_bwd")
    return dy, dw


def _factors(ids, a, b, scale, T: int, K: int, N: int, index: int):
    """(adapters, rank, pointers of ids, a, b and scale) of checked adapter factors."""
    pi = _matrix("ids", ids, (T,), torch.int32, index)
    _index("a", a)
    if a.dim() != 3:
        raise ValueError("a must be 3-D: (adapters, rank, K)")
    L, r, _ = a.shape
    pa = _matrix("a", a, (L, r, K), torch.bfloat16, index)
    pb = _matrix("b", b, (L, r, N), torch.bfloat16, index)
    return L, r, pi, pa, pb, (_matrix("scale", scale, (L,), torch.float32, index) if scale is not None else None)


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
    index = _index("x", x)
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return adapter_fwd(x, ids, a, b, scale, base, dtype, out)
    dtx, T, K, ldx = _rows_of("x", x, index)
    if dtx != BNN_BF16:
        raise TypeError("x must be bfloat16")
    dev = x.device
    _index("b", b)
    N = b.shape[2] if b.dim() == 3 else -1
    L, r, pi, pa, pb, ps = _factors(ids, a, b, scale, T, K, N, index)
    if dtype is None:
        dtype = out.dtype if out is not None else base.dtype if base is not None else torch.float32
    out, dt, ldo = _out_rows("out", out, T, N, dtype, dev, index)
    pbase, ldb = None, 0
    if base is not None:
        pbase, ldb = _same_rows("base", base, T, N, dt, index)
    u = _new(T, r, torch.float32, dev)
    lib = library()
    need = lib.bnn_adapter_fwd_workspace(T, K, N, r, L)
    ws, wp = _workspace(need, dev)
    st = lib.bnn_adapter_fwd(x.data_ptr(), ldx, pi, pa, pb, ps, pbase, ldb, out.data_ptr(), ldo, dt, u.data_ptr(), wp,
                             need, T, K, N, r, L, _stream(x))
    _check(st, "bnn_adapter_fwd")
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
    ``dx=False`` and ``params=False`` leave those out (None).  At most 1024
    adapters."""
    index = _index("dy", dy)
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return adapter_bwd(dy, x, u, ids, a, b, scale, base, dtype, dx, params)
    dtd, T, N, lddy = _rows_of("dy", dy, index)
    if dtd != BNN_BF16:
        raise TypeError("dy must be bfloat16")
    dev = dy.device
    _index("a", a)
    K = a.shape[2] if a.dim() == 3 else -1
    L, r, pi, pa, pb, ps = _factors(ids, a, b, scale, T, K, N, index)
    px = pxs = pu = None
    dtx, ldx = BNN_BF16, max(K, 1)
    if params:
        pu = _matrix("u", u, (T, r), torch.float32, index)
        if isinstance(x, (tuple, list)):
            q, s = x
            if _quantised("x", q, s, K) != T:
                raise ValueError(f"x must have {T} rows")
            if q.get_device() != index:
                raise ValueError(f"x must be on cuda:{index}")
            px, pxs, dtx = q.data_ptr(), s.data_ptr(), BNN_F8
        else:
            dtx, Tx, Kx, ldx = _rows_of("x", x, index)
            if dtx != BNN_BF16:
                raise TypeError("x must be bfloat16")
            if (Tx, Kx) != (T, K):
                raise ValueError(f"x must have shape ({T}, {K})")
            px = x.data_ptr()
    out, dt, ldo = None, BNN_FP32, max(K, 1)
    pbase, ldb = None, 0
    if dx:
        if dtype is None:
            dtype = base.dtype if base is not None else torch.float32
        out, dt, ldo = _out_rows("dx", None, T, K, dtype, dev, index)
        if base is not None:
            pbase, ldb = _same_rows("base", base, T, K, dt, index)
    da = db = None
    if params:
        da = torch.empty((L, r, K), dtype=torch.float32, device=dev)
        db = torch.empty((L, r, N), dtype=torch.float32, device=dev)
    lib = library()
    need = lib.bnn_adapter_bwd_workspace(T, K, N, r, L)
    ws, wp = _workspace(need, dev)
    st = lib.bnn_adapter_bwd(dy.data_ptr(), lddy, px, pxs, dtx, ldx, pu, pi, pa, pb, ps, pbase, ldb, _ptr(out), ldo, dt,
                             _ptr(da), _ptr(db), wp, need, T, K, N, r, L, _stream(dy))
    _check(st, "bnn_adapter_bwd")
    return out, da, db
