"""Python binding of the gfx950 GPTQ layer library (libgptq_mi355x.so).

The functions here have the names of the C entry points declared in
``include/gptq_mi355x.h`` and only marshal arguments: they check tensor
devices, dtypes and shapes, allocate outputs and workspaces with torch, and
pass raw device pointers plus torch's current HIP stream to the library.
Every step of the computation runs in the library's HIP kernels; there is no
fallback path, and loading fails loudly if the library is missing.
"""

from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgptq_mi355x.so")

GPTQ_OK, GPTQ_E_INVALID_ARG, GPTQ_E_UNSUPPORTED, GPTQ_E_WORKSPACE, GPTQ_E_HIP, GPTQ_E_TOO_LARGE = range(6)
GPTQ_NOALLOC_MAX_WEIGHTS, GPTQ_NOALLOC_MAX_ROWS = 1 << 24, 65536
GPTQ_F16, GPTQ_F32, GPTQ_BF16 = 0, 1, 2

_lib: Optional[ctypes.CDLL] = None

_c_size, _c_i64, _c_int, _c_dbl, _c_ptr = ctypes.c_size_t, ctypes.c_int64, ctypes.c_int, ctypes.c_double, ctypes.c_void_p


class _KvCacheStruct(ctypes.Structure):  # gptq_kv_cache
    _fields_ = [("k_codes", _c_ptr), ("v_codes", _c_ptr), ("k_grid", _c_ptr), ("v_grid", _c_ptr), ("n_pages", _c_i64),
                ("page_size", _c_i64), ("kv_heads", _c_i64), ("head_dim", _c_i64), ("bits", _c_int)]


class _KvBatchStruct(ctypes.Structure):  # gptq_kv_batch
    _fields_ = [("table", _c_ptr), ("ld_table", _c_i64), ("max_pages", _c_i64), ("lens", _c_ptr), ("starts", _c_ptr),
                ("batch", _c_i64), ("n_tokens", _c_i64)]


_SIGNATURES = {
    "gptq_status_string": (ctypes.c_char_p, [_c_int]),
    "gptq_version": (ctypes.c_char_p, []),
    "gptq_hessian_workspace_size": (_c_size, [_c_i64, _c_i64, _c_int]),
    "gptq_hessian_accumulate": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_i64, _c_ptr, _c_int, _c_ptr, _c_size, _c_ptr]),
    "gptq_prepare_hinv_workspace_size": (_c_size, [_c_i64]),
    "gptq_prepare_hinv": (_c_int, [_c_ptr, _c_i64, _c_dbl, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_size, _c_ptr]),
    "gptq_quantize_layer_workspace_size": (_c_size, [_c_i64, _c_i64, _c_int, _c_i64, _c_i64]),
    "gptq_quantize_layer": (
        _c_int,
        [_c_ptr, _c_int, _c_i64, _c_i64, _c_ptr, _c_int, _c_i64, _c_i64, _c_int, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_size, _c_ptr],
    ),
    "gptq_quantize_layer_noalloc": (
        _c_int,
        [_c_ptr, _c_int, _c_i64, _c_i64, _c_ptr, _c_int, _c_i64, _c_i64, _c_int, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr],
    ),
    "gptq_pack_codes": (_c_int, [_c_ptr, _c_i64, _c_i64, _c_int, _c_ptr, _c_ptr]),
    "gptq_dequantize": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_int, _c_i64, _c_ptr, _c_int, _c_i64, _c_ptr]),
    "gptq_act_order_perm": (_c_int, [_c_ptr, _c_i64, _c_i64, _c_ptr, _c_ptr, _c_ptr]),
    "gptq_gather": (
        _c_int,
        [_c_ptr, _c_int, _c_i64, _c_i64, _c_i64, _c_ptr, _c_i64, _c_ptr, _c_i64, _c_ptr, _c_i64, _c_ptr, _c_ptr],
    ),
    "gptq_dequant_gemm": (
        _c_int,
        [_c_ptr, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_int, _c_i64, _c_ptr, _c_i64, _c_i64, _c_ptr, _c_i64, _c_int, _c_ptr,
         _c_size, _c_ptr],
    ),
    "gptq_dequant_gemm_workspace_size": (_c_size, [_c_i64, _c_i64, _c_i64]),
    "gptq_kv_cache_write": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int, _c_i64, _c_i64, _c_ptr, _c_ptr]),
    "gptq_kv_cache_read": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int, _c_i64, _c_i64, _c_ptr, _c_ptr]),
    "gptq_kv_attention_workspace_size": (_c_size, [_c_ptr, _c_ptr, _c_i64]),
    "gptq_kv_attention": (
        _c_int,
        [_c_ptr, _c_ptr, _c_ptr, _c_int, _c_i64, _c_i64, _c_dbl, _c_ptr, _c_ptr, _c_int, _c_i64, _c_ptr, _c_size, _c_ptr,
         _c_ptr],
    ),
    "gptq_dequant_matvec": (
        _c_int,
        [_c_ptr, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_int, _c_i64, _c_ptr, _c_i64, _c_i64, _c_ptr, _c_ptr],
    ),
}


class GptqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} (status {status})")


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} not found: build the HIP library first "
            "(python -m post_weight_quantization_17_amd.build)"
        )
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().gptq_status_string(status).decode()


def version() -> str:
    return load().gptq_version().decode()


def _check(fn: str, status: int) -> None:
    if status != GPTQ_OK:
        raise GptqError(fn, status)


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return GPTQ_F16
    if t.dtype == torch.float32:
        return GPTQ_F32
    raise TypeError(f"unsupported dtype {t.dtype} (float16 or float32)")


def _on_gpu(name: str, t: torch.Tensor) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")


def _workspace(nbytes: int, device, ws: Optional[torch.Tensor]) -> torch.Tensor:
    if ws is not None and ws.numel() * ws.element_size() >= nbytes:
        return ws
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------- stage 1
def gptq_hessian_workspace_size(n_tokens: int, d: int, dtype: torch.dtype) -> int:
    return load().gptq_hessian_workspace_size(n_tokens, d, GPTQ_F16 if dtype == torch.float16 else GPTQ_F32)


def gptq_hessian_accumulate(
    X: torch.Tensor, H: Optional[torch.Tensor] = None, accumulate: bool = False, ws: Optional[torch.Tensor] = None
) -> torch.Tensor:
    """H (+)= 2 X^T X for X [n_tokens, d] (fp16/fp32, rows may be strided)."""
    _on_gpu("X", X)
    if X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be 2-D with unit column stride")
    n, d = X.shape
    if H is None:
        if accumulate:
            raise ValueError("accumulate needs an existing H")
        H = torch.empty((d, d), dtype=torch.float32, device=X.device)
    if H.shape != (d, d) or H.dtype != torch.float32 or not H.is_contiguous():
        raise ValueError("H must be a contiguous float32 [d, d] tensor")
    lib = load()
    code = _dtype_code(X)
    need = lib.gptq_hessian_workspace_size(n, d, code)
    ws = _workspace(need, X.device, ws)
    ldx = X.stride(0) if n > 1 else d
    _check(
        "gptq_hessian_accumulate",
        lib.gptq_hessian_accumulate(_ptr(X), code, n, d, ldx, _ptr(H), int(accumulate), _ptr(ws), ws.numel(), _stream()),
    )
    return H


# ---------------------------------------------------------------- stage 2
@dataclasses.dataclass
class Hinv:
    U: torch.Tensor  # fp32 [d, d] upper triangular, H_d^-1 = U^T U
    lam: torch.Tensor  # fp32 scalar (device)
    info: torch.Tensor  # int32 scalar (device), 0 = success


def gptq_prepare_hinv_workspace_size(d: int) -> int:
    return load().gptq_prepare_hinv_workspace_size(d)


def gptq_prepare_hinv(
    H: torch.Tensor,
    damp: float = 0.01,
    U: Optional[torch.Tensor] = None,
    ws: Optional[torch.Tensor] = None,
    out: Optional[Hinv] = None,
) -> Hinv:
    """Upper Cholesky factor U of (H + damp*mean(diag H) I)^-1."""
    _on_gpu("H", H)
    if H.dim() != 2 or H.shape[0] != H.shape[1] or H.dtype != torch.float32 or not H.is_contiguous():
        raise ValueError("H must be a contiguous float32 square tensor")
    d = H.shape[0]
    if out is not None:
        U, lam, info = out.U, out.lam, out.info
    else:
        if U is None:
            U = torch.empty((d, d), dtype=torch.float32, device=H.device)
        lam = torch.empty((), dtype=torch.float32, device=H.device)
        info = torch.empty((), dtype=torch.int32, device=H.device)
    lib = load()
    ws = _workspace(lib.gptq_prepare_hinv_workspace_size(d), H.device, ws)
    _check(
        "gptq_prepare_hinv",
        lib.gptq_prepare_hinv(_ptr(H), d, float(damp), _ptr(U), _ptr(lam), _ptr(info), _ptr(ws), ws.numel(), _stream()),
    )
    return Hinv(U, lam, info)


# ---------------------------------------------------------------- stage 3
@dataclasses.dataclass
class Quantized:
    codes: torch.Tensor  # uint8 [d_row, d_col]
    scales: torch.Tensor  # fp32 [d_row, n_groups]
    zeros: torch.Tensor  # int32 [d_row, n_groups]
    packed: torch.Tensor  # int32 view of the uint32 words [d_row, ceil(d_col*bits/32)]
    loss: torch.Tensor  # fp64 scalar
    row_loss: Optional[torch.Tensor]  # fp32 [d_row]


def n_groups(d_col: int, group_size: int) -> int:
    return 1 if group_size == -1 else -(-d_col // group_size)


def words_per_row(d_col: int, bits: int) -> int:
    return -(-d_col * bits // 32)


def gptq_quantize_layer_workspace_size(d_row: int, d_col: int, bits: int, group_size: int, block: int = 128) -> int:
    return load().gptq_quantize_layer_workspace_size(d_row, d_col, bits, group_size, block)


def gptq_quantize_layer(
    W: torch.Tensor,
    U: torch.Tensor,
    bits: int,
    group_size: int,
    block: int = 128,
    want_row_loss: bool = True,
    ws: Optional[torch.Tensor] = None,
    out: Optional[Quantized] = None,
    symmetric: bool = False,
) -> Quantized:
    """GPTQ sweep of W [d_row, d_col] (fp16/fp32) with the factor U
    (min-max grid, or the symmetric grid with ``symmetric``)."""
    _on_gpu("W", W)
    _on_gpu("U", U)
    if W.dim() != 2 or not W.is_contiguous():
        raise ValueError("W must be a contiguous 2-D tensor")
    d_row, d_col = W.shape
    if U.shape != (d_col, d_col) or U.dtype != torch.float32 or not U.is_contiguous():
        raise ValueError("U must be a contiguous float32 [d_col, d_col] tensor")
    dev = W.device
    if out is None:
        ng = n_groups(d_col, group_size) if group_size == -1 or group_size > 0 else 1
        out = Quantized(
            codes=torch.empty((d_row, d_col), dtype=torch.uint8, device=dev),
            scales=torch.empty((d_row, ng), dtype=torch.float32, device=dev),
            zeros=torch.empty((d_row, ng), dtype=torch.int32, device=dev),
            packed=torch.empty((d_row, words_per_row(d_col, bits)), dtype=torch.int32, device=dev),
            loss=torch.empty((), dtype=torch.float64, device=dev),
            row_loss=torch.empty((d_row,), dtype=torch.float32, device=dev) if want_row_loss else None,
        )
    lib = load()
    ws = _workspace(lib.gptq_quantize_layer_workspace_size(d_row, d_col, bits, group_size, block), dev, ws)
    _check(
        "gptq_quantize_layer",
        lib.gptq_quantize_layer(
            _ptr(W), _dtype_code(W), d_row, d_col, _ptr(U), bits, group_size, block, int(bool(symmetric)),
            _ptr(out.codes), _ptr(out.scales), _ptr(out.zeros), _ptr(out.packed), _ptr(out.loss),
            _ptr(out.row_loss), _ptr(ws), ws.numel(), _stream(),
        ),
    )
    return out


def _quantized_like(d_row: int, d_col: int, bits: int, group_size: int, want_row_loss: bool, dev) -> Quantized:
    ng = n_groups(d_col, group_size) if group_size == -1 or group_size > 0 else 1
    return Quantized(
        codes=torch.empty((d_row, d_col), dtype=torch.uint8, device=dev),
        scales=torch.empty((d_row, ng), dtype=torch.float32, device=dev),
        zeros=torch.empty((d_row, ng), dtype=torch.int32, device=dev),
        packed=torch.empty((d_row, words_per_row(d_col, bits)), dtype=torch.int32, device=dev),
        loss=torch.empty((), dtype=torch.float64, device=dev),
        row_loss=torch.empty((d_row,), dtype=torch.float32, device=dev) if want_row_loss else None,
    )


def gptq_quantize_layer_noalloc(
    W: torch.Tensor,
    U: torch.Tensor,
    bits: int,
    group_size: int,
    block: int = 128,
    out: Optional[Quantized] = None,
    symmetric: bool = False,
) -> Quantized:
    """gptq_quantize_layer without a workspace: the library's static scratch
    holds the working copy (at most GPTQ_NOALLOC_MAX_WEIGHTS weights and
    GPTQ_NOALLOC_MAX_ROWS rows). Pass ``out`` to allocate nothing here either;
    calls that overlap on one GPU race."""
    _on_gpu("W", W)
    _on_gpu("U", U)
    if W.dim() != 2 or not W.is_contiguous():
        raise ValueError("W must be a contiguous 2-D tensor")
    d_row, d_col = W.shape
    if U.shape != (d_col, d_col) or U.dtype != torch.float32 or not U.is_contiguous():
        raise ValueError("U must be a contiguous float32 [d_col, d_col] tensor")
    if out is None:
        out = _quantized_like(d_row, d_col, bits, group_size, True, W.device)
    _check(
        "gptq_quantize_layer_noalloc",
        load().gptq_quantize_layer_noalloc(
            _ptr(W), _dtype_code(W), d_row, d_col, _ptr(U), bits, group_size, block, int(bool(symmetric)),
            _ptr(out.codes), _ptr(out.scales), _ptr(out.zeros), _ptr(out.packed), _ptr(out.loss),
            _ptr(out.row_loss), _stream(),
        ),
    )
    return out


def gptq_pack_codes(codes: torch.Tensor, bits: int, packed: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Pack uint8 codes [d_row, d_col] into int32 (bit pattern uint32) words."""
    _on_gpu("codes", codes)
    if codes.dtype != torch.uint8 or codes.dim() != 2 or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous uint8 2-D tensor")
    d_row, d_col = codes.shape
    if packed is None:
        packed = torch.empty((d_row, words_per_row(d_col, bits)), dtype=torch.int32, device=codes.device)
    _check("gptq_pack_codes", load().gptq_pack_codes(_ptr(codes), d_row, d_col, bits, _ptr(packed), _stream()))
    return packed


def gptq_dequantize(packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, d_col: int, bits: int,
                    group_size: int, dtype: torch.dtype = torch.float16,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """What [d_row, d_col] = s (code - z), computed in fp32 and rounded to
    ``dtype`` (float16 or float32)."""
    for name, t in (("packed", packed), ("scales", scales), ("zeros", zeros)):
        _on_gpu(name, t)
    d_row = packed.shape[0]
    if (packed.dim() != 2 or packed.shape[1] != words_per_row(d_col, bits) or not packed.is_contiguous()
            or packed.dtype not in (torch.int32, torch.uint32)):
        raise ValueError("packed must be a contiguous [d_row, words_per_row] 32-bit tensor")
    ng = n_groups(d_col, group_size) if group_size == -1 or group_size > 0 else 1
    if scales.shape != (d_row, ng) or scales.dtype != torch.float32 or not scales.is_contiguous():
        raise ValueError("scales must be a contiguous float32 [d_row, n_groups] tensor")
    if zeros.shape != (d_row, ng) or zeros.dtype != torch.int32 or not zeros.is_contiguous():
        raise ValueError("zeros must be a contiguous int32 [d_row, n_groups] tensor")
    if out is None:
        out = torch.empty((d_row, d_col), dtype=dtype, device=packed.device)
    if out.shape != (d_row, d_col) or out.stride(1) != 1 or out.dtype not in (torch.float16, torch.float32):
        raise ValueError("out must be float16/float32 [d_row, d_col] with unit column stride")
    _check(
        "gptq_dequantize",
        load().gptq_dequantize(_ptr(packed), _ptr(scales), _ptr(zeros), d_row, d_col, bits, group_size, _ptr(out),
                               _dtype_code(out), max(out.stride(0), d_col), _stream()),
    )
    return out


# ------------------------------------------------------------ column order
def gptq_act_order_perm(H: torch.Tensor, perm: Optional[torch.Tensor] = None,
                        invperm: Optional[torch.Tensor] = None):
    """(perm, invperm), int32 [d]: columns by descending diag(H) (ties by
    index, NaN last); perm[q] is the original column taken q-th."""
    _on_gpu("H", H)
    if H.dtype != torch.float32 or H.dim() != 2 or H.shape[0] != H.shape[1] or H.stride(1) != 1:
        raise ValueError("H must be a float32 [d, d] tensor with unit column stride")
    d = H.shape[0]
    if perm is None:
        perm = torch.empty(d, dtype=torch.int32, device=H.device)
    if invperm is None:
        invperm = torch.empty(d, dtype=torch.int32, device=H.device)
    _check("gptq_act_order_perm", load().gptq_act_order_perm(_ptr(H), d, H.stride(0), _ptr(perm), _ptr(invperm),
                                                             _stream()))
    return perm, invperm


def gptq_gather(src: torch.Tensor, row_idx: Optional[torch.Tensor] = None, col_idx: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, info: Optional[torch.Tensor] = None):
    """out[i][q] = src[row_idx[i]][col_idx[q]] (identity where an index is
    None) for 2-D src with 1-, 2- or 4-byte elements; returns (out, info),
    info[0] = 1 if an index was out of range."""
    _on_gpu("src", src)
    if src.dim() != 2 or src.stride(1) != 1 or src.element_size() not in (1, 2, 4):
        raise ValueError("src must be 2-D with unit column stride and 1-, 2- or 4-byte elements")
    for name, t in (("row_idx", row_idx), ("col_idx", col_idx)):
        if t is not None:
            _on_gpu(name, t)
            if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 vector")
    rows = src.shape[0] if row_idx is None else row_idx.shape[0]
    cols = src.shape[1] if col_idx is None else col_idx.shape[0]
    if out is None:
        out = torch.empty((rows, cols), dtype=src.dtype, device=src.device)
    if out.shape != (rows, cols) or out.dtype != src.dtype or out.stride(1) != 1:
        raise ValueError("out has the wrong shape, dtype or layout")
    if info is None:
        info = torch.empty(1, dtype=torch.int32, device=src.device)
    _check(
        "gptq_gather",
        load().gptq_gather(
            _ptr(src), src.element_size(), src.shape[0], src.shape[1], max(src.stride(0), src.shape[1]),
            _ptr(row_idx), rows, _ptr(col_idx), cols, _ptr(out), max(out.stride(0), cols), _ptr(info), _stream(),
        ),
    )
    return out, info


# ------------------------------------------------------------ packed use
def gptq_dequant_matvec(
    packed: torch.Tensor,
    scales: torch.Tensor,
    zeros: torch.Tensor,
    d_col: int,
    bits: int,
    group_size: int,
    x: torch.Tensor,
    y: Optional[torch.Tensor] = None,
) -> torch.Tensor:
    """y [batch, d_row] = x [batch, d_col] (fp16) times the dequantized
    packed matrix, transposed."""
    for name, t in (("packed", packed), ("scales", scales), ("zeros", zeros), ("x", x)):
        _on_gpu(name, t)
    if x.dtype != torch.float16 or x.dim() not in (1, 2) or x.stride(-1) != 1:
        raise ValueError("x must be a float16 [d_col] or [batch, d_col] tensor with unit column stride")
    x2 = x.unsqueeze(0) if x.dim() == 1 else x
    batch = x2.shape[0]
    if x2.shape[1] != d_col:
        raise ValueError("x has the wrong width")
    d_row = packed.shape[0]
    if (packed.shape[1] != words_per_row(d_col, bits) or not packed.is_contiguous()
            or packed.dtype not in (torch.int32, torch.uint32)):
        raise ValueError("packed must be a contiguous [d_row, words_per_row] 32-bit tensor")
    ng = n_groups(d_col, group_size) if group_size == -1 or group_size > 0 else 1
    if scales.shape != (d_row, ng) or scales.dtype != torch.float32 or not scales.is_contiguous():
        raise ValueError("scales must be a contiguous float32 [d_row, n_groups] tensor")
    if zeros.shape != (d_row, ng) or zeros.dtype != torch.int32 or not zeros.is_contiguous():
        raise ValueError("zeros must be a contiguous int32 [d_row, n_groups] tensor")
    if y is None:
        y = torch.empty((batch, d_row), dtype=torch.float32, device=x.device)
    ldx = x2.stride(0) if batch > 1 else d_col
    _check(
        "gptq_dequant_matvec",
        load().gptq_dequant_matvec(
            _ptr(packed), _ptr(scales), _ptr(zeros), d_row, d_col, bits, group_size, _ptr(x2), batch, ldx,
            _ptr(y), _stream(),
        ),
    )
    return y.squeeze(0) if x.dim() == 1 else y


def gptq_dequant_gemm_workspace_size(d_out: int, d_in: int, n_tokens: int) -> int:
    return load().gptq_dequant_gemm_workspace_size(d_out, d_in, n_tokens)


def gptq_dequant_gemm(packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, d_in: int, bits: int,
                      group_size: int, X: torch.Tensor, relu: bool = False,
                      Y: Optional[torch.Tensor] = None, fused: bool = False,
                      ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y = act(X What^T) (fp16) for the packed layer [d_out rows] and fp16
    tokens X [n, d_in]; act is ReLU with ``relu``. By default a workspace is
    passed (weights dequantized once, K-major operands); ``fused`` runs the
    per-tile dequantizing kernel without one. Both give the same bits."""
    for n, t in (("packed", packed), ("scales", scales), ("zeros", zeros), ("X", X)):
        _on_gpu(n, t)
    if X.dtype != torch.float16 or X.dim() != 2 or X.stride(1) != 1 or X.shape[1] != d_in:
        raise ValueError("X must be a 2-D fp16 tensor [n, d_in] with unit column stride")
    d_out = packed.shape[0]
    n = X.shape[0]
    if Y is None:
        Y = torch.empty((n, d_out), dtype=torch.float16, device=X.device)
    if Y.dtype != torch.float16 or Y.shape != (n, d_out) or Y.stride(1) != 1:
        raise ValueError("Y must be fp16 [n, d_out] with unit column stride")
    ldx = X.stride(0) if n > 1 else d_in
    ldy = Y.stride(0) if n > 1 else d_out
    lib = load()
    wsp, wsb = None, 0
    if not fused and n > 0:
        wsb = lib.gptq_dequant_gemm_workspace_size(d_out, d_in, n)
        ws = _workspace(wsb, X.device, ws)
        wsp, wsb = _ptr(ws), ws.numel() * ws.element_size()
    _check(
        "gptq_dequant_gemm",
        lib.gptq_dequant_gemm(_ptr(packed), _ptr(scales), _ptr(zeros), d_out, d_in, bits, group_size, _ptr(X), n,
                              ldx, _ptr(Y), ldy, int(bool(relu)), wsp, wsb, _stream()),
    )
    return Y


# ------------------------------------------------- quantised key-value cache
@dataclasses.dataclass
class KVCache:
    """A paged cache of 4- or 8-bit keys and values (``gptq_kv_cache_alloc``
    makes one). ``info`` collects over all calls on the cache: it becomes 1
    when a call met a position past its table or on no page of the cache."""

    k_codes: torch.Tensor  # int32 view of the uint32 words [n_pages, kv_heads, page_size, head_dim*bits/32]
    v_codes: torch.Tensor
    k_grid: torch.Tensor  # int32 view of the grid words [n_pages, kv_heads, page_size]: fp32 scale | zero
    v_grid: torch.Tensor
    head_dim: int
    bits: int
    info: torch.Tensor  # int32 [1] (device)


def gptq_kv_cache_alloc(n_pages: int, page_size: int, kv_heads: int, head_dim: int, bits: int, device) -> KVCache:
    """A zero-filled cache of n_pages pages of page_size tokens."""
    if bits not in (4, 8):
        raise ValueError("bits must be 4 or 8")
    if head_dim % 16 != 0 or not 16 <= head_dim <= 256:
        raise ValueError("head_dim must be a multiple of 16, 16 to 256")
    if page_size & (page_size - 1) or not 16 <= page_size <= 1024:
        raise ValueError("page_size must be a power of two, 16 to 1024")
    if n_pages < 1 or kv_heads < 1:
        raise ValueError("n_pages and kv_heads must be at least 1")
    rows = (n_pages, kv_heads, page_size)
    z = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)
    return KVCache(k_codes=z(*rows, head_dim * bits // 32), v_codes=z(*rows, head_dim * bits // 32), k_grid=z(*rows),
                   v_grid=z(*rows), head_dim=head_dim, bits=bits, info=z(1))


def _kv_structs(cache: KVCache, table: torch.Tensor, lens: torch.Tensor, starts: Optional[torch.Tensor],
                n_tokens: int):
    """The two structs of a call, after the checks of shapes and devices."""
    dev = cache.k_codes.device
    tensors = [("cache.k_codes", cache.k_codes), ("cache.v_codes", cache.v_codes), ("cache.k_grid", cache.k_grid),
               ("cache.v_grid", cache.v_grid), ("cache.info", cache.info), ("table", table), ("lens", lens)]
    if starts is not None:
        tensors.append(("starts", starts))
    for name, t in tensors:
        _on_gpu(name, t)
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the cache on {dev}")
        if t.dtype != torch.int32:
            raise ValueError(f"{name} must be int32")
        if name != "table" and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    grid = cache.k_grid.shape
    if len(grid) != 3 or cache.v_grid.shape != grid:
        raise ValueError("cache grids must be [n_pages, kv_heads, page_size]")
    codes = (*grid, cache.head_dim * cache.bits // 32)
    if cache.k_codes.shape != codes or cache.v_codes.shape != codes:
        raise ValueError("cache codes must be [n_pages, kv_heads, page_size, head_dim * bits / 32]")
    if cache.info.numel() != 1:
        raise ValueError("cache.info must hold one element")
    if lens.dim() != 1:
        raise ValueError("lens must be a vector")
    batch = lens.shape[0]
    if table.dim() != 2 or table.shape[0] != batch or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError("table must be [batch, max_pages] with unit column stride")
    if starts is not None and starts.shape != (batch + 1,):
        raise ValueError("starts must be [batch + 1]")
    if starts is None and n_tokens != batch:
        raise ValueError("without starts there is one token a sequence")
    c = _KvCacheStruct(_ptr(cache.k_codes), _ptr(cache.v_codes), _ptr(cache.k_grid), _ptr(cache.v_grid), grid[0],
                       grid[2], grid[1], cache.head_dim, cache.bits)
    ld = table.stride(0) if batch > 1 else table.shape[1]
    b = _KvBatchStruct(_ptr(table), ld, table.shape[1], _ptr(lens), _ptr(starts), batch, n_tokens)
    return c, b


def _kv_dtype(name: str, dtype: torch.dtype) -> int:
    codes = {torch.float16: GPTQ_F16, torch.float32: GPTQ_F32, torch.bfloat16: GPTQ_BF16}
    if dtype not in codes:
        raise TypeError(f"{name}: unsupported dtype {dtype} (float16, bfloat16 or float32)")
    return codes[dtype]


def _kv_rows(name: str, t: torch.Tensor, n: Optional[int], heads: Optional[int], dim: int, dev) -> int:
    """Checks [n_tokens, heads, dim] with heads and elements contiguous; returns the token stride."""
    _on_gpu(name, t)
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the cache on {dev}")
    if (t.dim() != 3 or t.shape[2] != dim or (heads is not None and t.shape[1] != heads)
            or (n is not None and t.shape[0] != n)):
        raise ValueError(f"{name} must be [n_tokens, heads, head_dim] of the call and its cache")
    if t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != dim):
        raise ValueError(f"{name} must have its heads and their elements contiguous")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * dim


def gptq_kv_cache_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                        starts: Optional[torch.Tensor] = None) -> None:
    """Quantise and store k, v [n_tokens, kv_heads, head_dim] (fp16, bf16 or
    fp32; rows may be strided) as the last tokens of their sequences:
    ``lens`` [batch] counts each sequence's tokens with these, rows
    ``starts[b]:starts[b + 1]`` are sequence b's (None: one each), ``table``
    [batch, max_pages] holds its pages."""
    dev = cache.k_codes.device
    n = k.shape[0]
    c, b = _kv_structs(cache, table, lens, starts, n)
    heads = cache.k_grid.shape[1]
    ldk, ldv = (_kv_rows(name, t, n, heads, cache.head_dim, dev) for name, t in (("k", k), ("v", v)))
    if v.dtype != k.dtype:
        raise ValueError("k and v must have the same dtype")
    lib = load()
    with torch.cuda.device(dev):
        _check("gptq_kv_cache_write",
               lib.gptq_kv_cache_write(ctypes.byref(c), ctypes.byref(b), _ptr(k), _ptr(v), _kv_dtype("k", k.dtype), ldk,
                                       ldv, _ptr(cache.info), _stream()))


def gptq_kv_cache_read(cache: KVCache, table: torch.Tensor, lens: torch.Tensor, starts: Optional[torch.Tensor] = None,
                       n_tokens: Optional[int] = None, dtype: torch.dtype = torch.float16, out=None):
    """(k, v) [n_tokens, kv_heads, head_dim]: what the cache holds of the
    last tokens of the sequences (arguments as in gptq_kv_cache_write;
    ``n_tokens`` rows in all, needed with ``starts`` unless ``out`` = (k, v)
    is given). Rows past ``starts[batch]`` are left as they are (unspecified
    in new tensors)."""
    dev = cache.k_codes.device
    heads = cache.k_grid.shape[1]
    if out is None:
        if n_tokens is None:
            if starts is not None:
                raise ValueError("n_tokens is needed with starts")
            n_tokens = lens.shape[0]
        out = tuple(torch.empty((n_tokens, heads, cache.head_dim), dtype=dtype, device=dev) for _ in range(2))
    k, v = out
    n = k.shape[0]
    if n_tokens is not None and n_tokens != n:
        raise ValueError("out has another number of rows than n_tokens")
    c, b = _kv_structs(cache, table, lens, starts, n)
    ldk, ldv = (_kv_rows(name, t, n, heads, cache.head_dim, dev) for name, t in (("k", k), ("v", v)))
    if v.dtype != k.dtype:
        raise ValueError("k and v must have the same dtype")
    lib = load()
    with torch.cuda.device(dev):
        _check("gptq_kv_cache_read",
               lib.gptq_kv_cache_read(ctypes.byref(c), ctypes.byref(b), _ptr(k), _ptr(v), _kv_dtype("out", k.dtype),
                                      ldk, ldv, _ptr(cache.info), _stream()))
    return k, v


def gptq_kv_attention_workspace_size(cache: KVCache, table: torch.Tensor, n_tokens: int, q_heads: int,
                                     ragged: Optional[bool] = None) -> int:
    """Bytes of workspace that gptq_kv_attention takes for n_tokens rows of
    q_heads heads over the sequences of ``table`` (``ragged``: with starts;
    None: the larger of both where both are possible)."""
    grid = cache.k_grid.shape
    c = _KvCacheStruct(_ptr(cache.k_codes), _ptr(cache.v_codes), _ptr(cache.k_grid), _ptr(cache.v_grid), grid[0],
                       grid[2], grid[1], cache.head_dim, cache.bits)
    lib = load()
    sizes = []
    p = _ptr(table)
    for r in (True, False) if ragged is None else (ragged,):
        if r or n_tokens == table.shape[0]:
            b = _KvBatchStruct(p, table.shape[1], table.shape[1], p, p if r else None, table.shape[0], n_tokens)
            sizes.append(lib.gptq_kv_attention_workspace_size(ctypes.byref(c), ctypes.byref(b), q_heads))
    return max(sizes, default=0)


def gptq_kv_attention(q: torch.Tensor, cache: KVCache, table: torch.Tensor, lens: torch.Tensor,
                      starts: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                      slopes: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
                      out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [n_tokens, q_heads, head_dim] (``dtype``, by default q's): causal
    attention of q [n_tokens, q_heads, head_dim] (fp16, bf16 or fp32) over
    the cached tokens of its sequences, its own among them. ``scale``: by
    default 1 / sqrt(head_dim); ``slopes`` fp32 [q_heads]: linear position
    biases. Rows past ``starts[batch]`` are left as they are (unspecified in
    a new tensor)."""
    dev = cache.k_codes.device
    n = q.shape[0]
    c, b = _kv_structs(cache, table, lens, starts, n)
    ldq = _kv_rows("q", q, n, None, cache.head_dim, dev)
    hq = q.shape[1]
    if hq % cache.k_grid.shape[1] != 0:
        raise ValueError("q's heads must be a multiple of the cache's")
    if slopes is not None:
        _on_gpu("slopes", slopes)
        if slopes.device != dev or slopes.dtype != torch.float32 or slopes.shape != (hq,) or not slopes.is_contiguous():
            raise ValueError("slopes must be a contiguous float32 [q_heads] vector on the cache's device")
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype if dtype is None else dtype, device=dev)
    elif dtype is not None and out.dtype != dtype:
        raise ValueError("out has another dtype than asked for")
    ldo = _kv_rows("out", out, n, hq, cache.head_dim, dev)
    lib = load()
    with torch.cuda.device(dev):
        need = lib.gptq_kv_attention_workspace_size(ctypes.byref(c), ctypes.byref(b), hq)
        if ws is not None and (ws.device != dev or not ws.is_contiguous()):
            raise ValueError("ws must be contiguous and on the cache's device")
        ws = _workspace(need, dev, ws)
        _check("gptq_kv_attention",
               lib.gptq_kv_attention(ctypes.byref(c), ctypes.byref(b), _ptr(q), _kv_dtype("q", q.dtype), hq, ldq,
                                     cache.head_dim ** -0.5 if scale is None else float(scale), _ptr(slopes), _ptr(out),
                                     _kv_dtype("out", out.dtype), ldo, _ptr(ws), ws.numel() * ws.element_size(),
                                     _ptr(cache.info), _stream()))
    return out
