"""LLM.int8() vector-wise mixed-precision linear for AMD MI355X (gfx950).

Thin Python binding of libi8mp.so.  Every step of the computation runs in the
library's HIP kernels; this module checks devices, dtypes and layouts (all
non-None tensors on one GPU, as the bitsandbytes pre-call check requires),
allocates outputs and workspaces with PyTorch, and passes the current stream.
There is no CPU fallback: calling an op without the built library, or on
tensors that are not on a GPU, raises.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

from ._lib import (  # noqa: F401
    EXPORTS,
    BackwardWorkspaceLayout,
    Fp4AppendStruct,
    Fp4AttentionStruct,
    Fp4CacheStruct,
    I8MP_MAX_K,
    I8MP_NOALLOC_SCRATCH_BYTES,
    I8mpError,
    LinearWorkspaceLayout,
    Mx4Struct,
    check,
    lib,
    status_string,
)
from .serialize import load_int8_weights, save_int8_weights  # noqa: F401

__all__ = [
    "quantize_weight",
    "save_int8_weights",
    "load_int8_weights",
    "vectorwise_quant",
    "outlier_extract",
    "linear_matmul",
    "mm_dequant",
    "vectorwise_dequant",
    "linear",
    "linear_forward_noalloc",
    "linear_quantize",
    "linear_matmul_dequant",
    "LinearWorkspace",
    "colwise_quant",
    "linear_backward",
    "BackwardWorkspace",
    "Fp4Weight",
    "fp4_quantize",
    "fp4_double_quant",
    "fp4_dequantize",
    "fp4_linear",
    "Fp4Cache",
    "fp4_cache_write",
    "fp4_cache_read",
    "fp4_cache_attention",
    "fp4_cache_append",
    "Mx4Tensor",
    "mx4_quantize",
    "mx4_dequantize",
    "mx4_matmul",
    "mx4_linear",
    "mx4_linear_backward",
    "I8mpError",
]

DEFAULT_THRESHOLD = 6.0
DEFAULT_CAP = 256


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _device_of(*tensors) -> torch.device:
    first = index = None
    for t in tensors:
        if t is not None:
            if first is None:
                first, index = t, t.get_device()
            elif t.get_device() != index or (index < 0 and t.device != first.device):
                raise ValueError("all tensors must be on one device, got "
                                 f"{sorted({str(x.device) for x in tensors if x is not None})}")
    if first is None or not first.is_cuda:
        raise ValueError(f"tensors must be on a GPU (got {None if first is None else first.device}); there is no CPU path")
    return first.device


def _rowmajor(t: torch.Tensor, name: str, dtype: torch.dtype) -> int:
    """Leading dimension of a row-major 2-D tensor with unit column stride."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = shape
    ld, unit = t.stride()
    if unit != 1 and cols > 1 and rows > 0:
        raise ValueError(f"{name} must have unit column stride")
    if rows > 1 and ld < cols:
        raise ValueError(f"{name} must not have rows that overlap (an expanded tensor: make it contiguous)")
    return max(ld, cols, 1)


def _vec(t: torch.Tensor, name: str, dtype: torch.dtype, n: int) -> None:
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous {dtype} vector of length {n}")


def _bytes(t: torch.Tensor, name: str) -> None:
    """t can be written as a run of t.numel() bytes."""
    if t.dtype != torch.uint8 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {torch.uint8} tensor")


def vectorwise_quant(x: torch.Tensor, threshold: float = DEFAULT_THRESHOLD,
                     ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """int8_vectorwise_quant: (codes int8 [m,k], row absmax fp32 [m], outlier bitmap uint32-as-int32)."""
    dev = _device_of(x)
    ldx = _rowmajor(x, "x", torch.float16)
    m, k = x.shape
    q = torch.empty((m, k), dtype=torch.int8, device=dev)
    absmax = torch.empty(m, dtype=torch.float32, device=dev)
    bitmap = torch.empty((k + 31) // 32, dtype=torch.int32, device=dev)
    L = lib()
    wsb = L.i8mp_quant_workspace_bytes(m, k) if threshold > 0 else 0
    ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        check(L.i8mp_int8_vectorwise_quant(_ptr(x), m, k, ldx, threshold, _ptr(q), k, _ptr(absmax),
                                           _ptr(bitmap), _ptr(ws), wsb, _stream(dev)),
              "i8mp_int8_vectorwise_quant")
    return q, absmax, bitmap


def quantize_weight(w: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Row-wise int8 weight state (codes, per-row absmax) of an fp16 weight [n, k]."""
    q, absmax, _ = vectorwise_quant(w, 0.0)
    return q, absmax


def outlier_extract(x: torch.Tensor, bitmap: torch.Tensor, cap: Optional[int] = None, strict: bool = True
                    ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """extract_outliers: (idx int32 [cap], count int32 [1], x_out fp16 [m, cap]).

    ``cap`` defaults to k, which holds every outlier column.  With a smaller
    cap and more outlier columns than it, only the first cap are listed;
    ``strict`` (default) then raises instead, reading the count back (a
    synchronization), since the sparse decomposition built from such a list
    would drop columns.
    """
    dev = _device_of(x, bitmap)
    ldx = _rowmajor(x, "x", torch.float16)
    m, k = x.shape
    _vec(bitmap, "bitmap", torch.int32, (k + 31) // 32)
    if cap is None:
        cap = k
    idx = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
    count = torch.empty(1, dtype=torch.int32, device=dev)
    xo = torch.empty((m, max(cap, 1)), dtype=torch.float16, device=dev)
    with torch.cuda.device(dev):
        check(lib().i8mp_outlier_extract(_ptr(x), m, k, ldx, _ptr(bitmap), cap, _ptr(idx), _ptr(count),
                                         _ptr(xo), max(cap, 1), _stream(dev)),
              "i8mp_outlier_extract")
    if strict and cap < k:
        found = int(count.item())
        if found > cap:
            raise ValueError(f"{found} outlier columns found, more than cap={cap}: extract with a larger cap")
    return idx[:cap], count, xo[:, :cap]


def linear_matmul(a: torch.Tensor, b: torch.Tensor) -> torch.Tensor:
    """int8_linear_matmul: C = A . B^T, exact int32 [m, n]."""
    dev = _device_of(a, b)
    lda = _rowmajor(a, "a", torch.int8)
    ldb = _rowmajor(b, "b", torch.int8)
    m, k = a.shape
    n, kb = b.shape
    if kb != k:
        raise ValueError("inner dimensions differ")
    c = torch.empty((m, n), dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        check(lib().i8mp_int8_linear_matmul(_ptr(a), lda, _ptr(b), ldb, m, n, k, _ptr(c), max(n, 1),
                                            _stream(dev)),
              "i8mp_int8_linear_matmul")
    return c


def mm_dequant(c: torch.Tensor, row_absmax: torch.Tensor, col_absmax: torch.Tensor,
               bias: Optional[torch.Tensor] = None,
               outliers: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]] = None,
               ) -> torch.Tensor:
    """int8_mm_dequant (+ bias, + the sparse-decomposition term).

    ``outliers`` = (x_out fp16 [m, cap], idx int32 [cap], count int32 [1], w_q int8 [n, k]).
    """
    xo = idx = count = wq = None
    if outliers is not None:
        xo, idx, count, wq = outliers
    dev = _device_of(c, row_absmax, col_absmax, bias, xo, idx, count, wq)
    ldc = _rowmajor(c, "c", torch.int32)
    m, n = c.shape
    _vec(row_absmax, "row_absmax", torch.float32, m)
    _vec(col_absmax, "col_absmax", torch.float32, n)
    if bias is not None:
        _vec(bias, "bias", torch.float16, n)
    cap, ldo, ldb, k = 0, 0, 0, 1
    if outliers is not None:
        ldo = _rowmajor(xo, "x_out", torch.float16)
        cap = xo.shape[1]
        ldb = _rowmajor(wq, "w_q", torch.int8)
        k = wq.shape[1]
    out = torch.empty((m, n), dtype=torch.float16, device=dev)
    with torch.cuda.device(dev):
        check(lib().i8mp_int8_mm_dequant(_ptr(c), ldc, _ptr(row_absmax), _ptr(col_absmax), _ptr(bias), m, n,
                                         _ptr(xo), ldo, _ptr(idx), _ptr(count), cap, _ptr(wq), ldb, k,
                                         _ptr(out), max(n, 1), _stream(dev)),
              "i8mp_int8_mm_dequant")
    return out


@dataclass
class LinearWorkspace:
    """Device workspace of i8mp_linear_forward plus views of its intermediates."""

    m: int
    n: int
    k: int
    cap: int
    layout: LinearWorkspaceLayout
    buf: torch.Tensor

    @classmethod
    def create(cls, m: int, n: int, k: int, cap: int, device) -> "LinearWorkspace":
        L = LinearWorkspaceLayout()
        check(lib().i8mp_linear_workspace_query(m, n, k, cap, ctypes.byref(L)), "i8mp_linear_workspace_query")
        buf = torch.empty(max(L.bytes, 1), dtype=torch.uint8, device=device)
        return cls(m, n, k, cap, L, buf)

    def fits(self, m: int, n: int, k: int, cap: int) -> bool:
        L = LinearWorkspaceLayout()
        check(lib().i8mp_linear_workspace_query(m, n, k, cap, ctypes.byref(L)), "i8mp_linear_workspace_query")
        return L.bytes <= self.buf.numel() and (m, k, cap) == (self.m, self.k, self.cap)

    def _view(self, off: int, count: int, dtype: torch.dtype) -> torch.Tensor:
        nbytes = count * torch.tensor([], dtype=dtype).element_size()
        return self.buf[off:off + nbytes].view(dtype)

    # intermediates left by the last forward call (for tests and inspection)
    def codes(self) -> torch.Tensor:
        return self._view(self.layout.q_offset, self.m * self.layout.ldq, torch.int8).view(
            self.m, self.layout.ldq)[:, : self.k]

    def absmax(self) -> torch.Tensor:
        return self._view(self.layout.absmax_offset, self.m, torch.float32)

    def bitmap(self) -> torch.Tensor:
        return self._view(self.layout.bitmap_offset, (self.k + 31) // 32, torch.int32)

    def idx(self) -> torch.Tensor:
        """Every outlier column, ascending, -1 past the count (idx_len entries)."""
        return self._view(self.layout.idx_offset, self.layout.idx_len, torch.int32)

    def count(self) -> torch.Tensor:
        return self._view(self.layout.count_offset, 1, torch.int32)

    def x_out(self) -> torch.Tensor:
        cp = self.layout.cap_pad
        return self._view(self.layout.xo_offset, self.m * cp, torch.float16).view(self.m, cp)[:, : self.cap]

    def outliers_past_cap(self) -> bool:
        """True if the last call found more outlier columns than cap (synchronizes).

        The output is the method's either way; the columns past cap read their
        x values through the index list, which is slower."""
        return int(self.count().item()) > self.cap


def vectorwise_dequant(q: torch.Tensor, absmax: torch.Tensor, dtype: torch.dtype = torch.float16,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """int8 vectorwise dequantize: q[i, j] * (absmax[i] / 127) in fp32, as fp16 or fp32."""
    if dtype not in (torch.float16, torch.float32):
        raise ValueError("dtype must be torch.float16 or torch.float32")
    dev = _device_of(q, absmax, out)
    ldq = _rowmajor(q, "q", torch.int8)
    m, k = q.shape
    _vec(absmax, "absmax", torch.float32, m)
    if out is None:
        out = torch.empty((m, k), dtype=dtype, device=dev)
    ldout = _rowmajor(out, "out", dtype)
    if tuple(out.shape) != (m, k):
        raise ValueError("out has the wrong shape")
    code = 0 if dtype == torch.float16 else 1
    with torch.cuda.device(dev):
        check(lib().i8mp_int8_vectorwise_dequant(_ptr(q), ldq, m, k, _ptr(absmax), code, _ptr(out), ldout,
                                                 _stream(dev)),
              "i8mp_int8_vectorwise_dequant")
    return out


def linear(x: torch.Tensor, w_q: torch.Tensor, w_absmax: torch.Tensor,
           bias: Optional[torch.Tensor] = None, threshold: float = DEFAULT_THRESHOLD,
           cap: int = DEFAULT_CAP, workspace: Optional[LinearWorkspace] = None,
           out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The fused mixed-precision linear: fp16 out [m, n] = x . dequant(w)^T + bias.

    Every outlier column takes the fp16 path for any count; ``cap`` sizes the
    workspace's gathered copy of the outlier columns (the fast path)."""
    dev = _device_of(x, w_q, w_absmax, bias, out)
    ldx = _rowmajor(x, "x", torch.float16)
    ldw = _rowmajor(w_q, "w_q", torch.int8)
    m, k = x.shape
    n, kw = w_q.shape
    if kw != k:
        raise ValueError("x and w_q differ in k")
    _vec(w_absmax, "w_absmax", torch.float32, n)
    if bias is not None:
        _vec(bias, "bias", torch.float16, n)
    if out is None:
        out = torch.empty((m, n), dtype=torch.float16, device=dev)
    ldout = _rowmajor(out, "out", torch.float16)
    if tuple(out.shape) != (m, n):
        raise ValueError("out has the wrong shape")
    if workspace is None:
        workspace = LinearWorkspace.create(m, n, k, cap, dev)
    elif not workspace.fits(m, n, k, cap):
        raise ValueError("workspace was created for another shape or capacity")
    with torch.cuda.device(dev):
        check(lib().i8mp_linear_forward(_ptr(x), m, k, ldx, _ptr(w_q), ldw, _ptr(w_absmax), n, _ptr(bias),
                                        threshold, cap, _ptr(out), ldout, _ptr(workspace.buf),
                                        workspace.buf.numel(), _stream(dev)),
              "i8mp_linear_forward")
    return out


def linear_forward_noalloc(x: torch.Tensor, w_q: torch.Tensor, w_absmax: torch.Tensor, out: torch.Tensor,
                           bias: Optional[torch.Tensor] = None, threshold: float = DEFAULT_THRESHOLD,
                           cap: int = DEFAULT_CAP) -> torch.Tensor:
    """``linear`` into a caller-owned ``out`` with the library's fixed scratch
    array as workspace: the call allocates nothing (for graph capture and
    serving loops).  Shapes whose workspace exceeds the array raise; calls
    that overlap on one GPU share the array and race."""
    dev = _device_of(x, w_q, w_absmax, bias, out)
    ldx = _rowmajor(x, "x", torch.float16)
    ldw = _rowmajor(w_q, "w_q", torch.int8)
    m, k = x.shape
    n, kw = w_q.shape
    if kw != k:
        raise ValueError("x and w_q differ in k")
    _vec(w_absmax, "w_absmax", torch.float32, n)
    if bias is not None:
        _vec(bias, "bias", torch.float16, n)
    ldout = _rowmajor(out, "out", torch.float16)
    if tuple(out.shape) != (m, n):
        raise ValueError("out has the wrong shape")
    with torch.cuda.device(dev):
        check(lib().i8mp_linear_forward_noalloc(_ptr(x), m, k, ldx, _ptr(w_q), ldw, _ptr(w_absmax), n, _ptr(bias),
                                                threshold, cap, _ptr(out), ldout, _stream(dev)),
              "i8mp_linear_forward_noalloc")
    return out


def linear_quantize(x: torch.Tensor, workspace: LinearWorkspace,
                    threshold: float = DEFAULT_THRESHOLD) -> None:
    """First half of ``linear``: detect, calibrate, quantize and extract into the workspace."""
    dev = _device_of(x, workspace.buf)
    ldx = _rowmajor(x, "x", torch.float16)
    m, k = x.shape
    if (m, k) != (workspace.m, workspace.k):
        raise ValueError("workspace was created for another shape")
    with torch.cuda.device(dev):
        check(lib().i8mp_linear_quantize(_ptr(x), m, k, ldx, threshold, workspace.cap, _ptr(workspace.buf),
                                         workspace.buf.numel(), _stream(dev)),
              "i8mp_linear_quantize")


def linear_matmul_dequant(x: torch.Tensor, workspace: LinearWorkspace, w_q: torch.Tensor,
                          w_absmax: torch.Tensor, bias: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Second half of ``linear``: fused int8 GEMM + dequant epilogue from the
    workspace that ``linear_quantize(x, workspace)`` filled (x is read for
    outlier columns past the workspace's cap)."""
    dev = _device_of(x, workspace.buf, w_q, w_absmax, bias, out)
    ldx = _rowmajor(x, "x", torch.float16)
    ldw = _rowmajor(w_q, "w_q", torch.int8)
    n, k = w_q.shape
    if k != workspace.k or tuple(x.shape) != (workspace.m, workspace.k):
        raise ValueError("x, w_q and the workspace differ in shape")
    _vec(w_absmax, "w_absmax", torch.float32, n)
    if bias is not None:
        _vec(bias, "bias", torch.float16, n)
    m = workspace.m
    if out is None:
        out = torch.empty((m, n), dtype=torch.float16, device=dev)
    ldout = _rowmajor(out, "out", torch.float16)
    with torch.cuda.device(dev):
        check(lib().i8mp_linear_matmul_dequant(_ptr(x), ldx, _ptr(workspace.buf), workspace.buf.numel(), m, k,
                                               workspace.cap,
                                               _ptr(w_q), ldw, _ptr(w_absmax), n, _ptr(bias), _ptr(out),
                                               ldout, _stream(dev)),
              "i8mp_linear_matmul_dequant")
    return out


def colwise_quant(a: torch.Tensor, zero_idx: Optional[torch.Tensor] = None,
                  zero_count: Optional[torch.Tensor] = None, ldqt: Optional[int] = None
                  ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Column-wise (transposed) int8 quantization: (qt int8 [cols, ldqt], col absmax fp32 [cols]).

    qt[j, i] is the code of a[i, j] under column j's absmax; columns listed in
    zero_idx[:min(zero_count, len)] get zero codes; rows >= a.shape[0] of qt are 0.
    """
    dev = _device_of(a, zero_idx, zero_count)
    lda = _rowmajor(a, "a", torch.float16)
    rows, cols = a.shape
    if (zero_idx is None) != (zero_count is None):
        raise ValueError("zero_idx and zero_count go together")
    cap = 0
    if zero_idx is not None:
        if zero_idx.dtype != torch.int32 or zero_idx.dim() != 1 or not zero_idx.is_contiguous():
            raise ValueError("zero_idx must be a contiguous int32 vector")
        _vec(zero_count, "zero_count", torch.int32, 1)
        cap = zero_idx.shape[0]
    ldqt = rows if ldqt is None else ldqt
    qt = torch.empty((cols, max(ldqt, 1)), dtype=torch.int8, device=dev)
    absmax = torch.empty(cols, dtype=torch.float32, device=dev)
    L = lib()
    wsb = L.i8mp_colwise_quant_workspace_bytes(rows, max(cols, 1))
    ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        check(L.i8mp_int8_colwise_quant(_ptr(a), rows, cols, lda, _ptr(zero_idx), _ptr(zero_count), cap, _ptr(qt),
                                        ldqt, _ptr(absmax), _ptr(ws), wsb, _stream(dev)),
              "i8mp_int8_colwise_quant")
    return qt[:, :ldqt], absmax


@dataclass
class BackwardWorkspace:
    """Device workspace of i8mp_linear_backward plus views of the GEMM operands it holds."""

    m: int
    n: int
    k: int
    cap: int
    layout: BackwardWorkspaceLayout
    buf: torch.Tensor

    @classmethod
    def create(cls, m: int, n: int, k: int, cap: int, device) -> "BackwardWorkspace":
        L = BackwardWorkspaceLayout()
        check(lib().i8mp_linear_backward_workspace_query(m, n, k, cap, ctypes.byref(L)),
              "i8mp_linear_backward_workspace_query")
        return cls(m, n, k, cap, L, torch.empty(max(L.bytes, 1), dtype=torch.uint8, device=device))

    def _mat(self, off: int, rows: int, ld: int, cols: int) -> torch.Tensor:
        return self.buf[off:off + rows * ld].view(rows, ld)[:, :cols]

    def _f32(self, off: int, count: int) -> torch.Tensor:
        return self.buf[off:off + 4 * count].view(torch.float32)

    # operands left by the last call (for tests and inspection)
    def g_q(self):
        return self._mat(self.layout.gq_offset, self.m, self.layout.ld_n, self.n).view(torch.int8)

    def g_s(self):
        return self._f32(self.layout.gs_offset, self.m)

    def wt_q(self):
        return self._mat(self.layout.wtq_offset, self.k, self.layout.ld_n, self.n).view(torch.int8)

    def wt_s(self):
        return self._f32(self.layout.wts_offset, self.k)

    def gt_q(self):
        return self._mat(self.layout.gtq_offset, self.n, self.layout.ld_m, self.m).view(torch.int8)

    def gt_s(self):
        return self._f32(self.layout.gts_offset, self.n)

    def xt_q(self):
        return self._mat(self.layout.xtq_offset, self.k, self.layout.ld_m, self.m).view(torch.int8)

    def xt_s(self):
        return self._f32(self.layout.xts_offset, self.k)


def linear_backward(grad_out: torch.Tensor, x: torch.Tensor, w: Optional[torch.Tensor],
                    forward_workspace: Optional[LinearWorkspace] = None,
                    need_grad_x: bool = True, need_grad_w: bool = True,
                    workspace: Optional[BackwardWorkspace] = None,
                    out_x: Optional[torch.Tensor] = None, out_w: Optional[torch.Tensor] = None,
                    ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Both gradients of ``linear`` for dL/dout = grad_out: (grad_x fp16 [m, k], grad_w fp16 [n, k]).

    w is the fp16 weight kept for training (needed for grad_x).  The outlier
    columns are those the forward left in ``forward_workspace`` (None: none).
    """
    dev = _device_of(grad_out, x, w, None if forward_workspace is None else forward_workspace.buf)
    ldg = _rowmajor(grad_out, "grad_out", torch.float16)
    ldx = _rowmajor(x, "x", torch.float16)
    m, n = grad_out.shape
    mx, k = x.shape
    if mx != m:
        raise ValueError("grad_out and x differ in rows")
    ldw = k
    if need_grad_x:
        if w is None:
            raise ValueError("grad_x needs the fp16 weight")
        ldw = _rowmajor(w, "w", torch.float16)
        if tuple(w.shape) != (n, k):
            raise ValueError("w must be [n, k]")
    cap = 0
    if forward_workspace is not None:
        if (forward_workspace.m, forward_workspace.k) != (m, k):
            raise ValueError("forward workspace was made for another shape")
        cap = forward_workspace.cap
    if workspace is None:
        workspace = BackwardWorkspace.create(m, n, k, cap, dev)
    elif (workspace.m, workspace.n, workspace.k, workspace.cap) != (m, n, k, cap):
        raise ValueError("backward workspace was created for another shape or capacity")
    gx = gw = None
    if need_grad_x:
        gx = torch.empty((m, k), dtype=torch.float16, device=dev) if out_x is None else out_x
        if tuple(gx.shape) != (m, k) or not gx.is_contiguous() or gx.dtype != torch.float16:
            raise ValueError("out_x must be a contiguous fp16 [m, k] tensor")
    if need_grad_w:
        gw = torch.empty((n, k), dtype=torch.float16, device=dev) if out_w is None else out_w
        if tuple(gw.shape) != (n, k) or not gw.is_contiguous() or gw.dtype != torch.float16:
            raise ValueError("out_w must be a contiguous fp16 [n, k] tensor")
    fws = None if forward_workspace is None else forward_workspace.buf
    with torch.cuda.device(dev):
        check(lib().i8mp_linear_backward(_ptr(grad_out), ldg, _ptr(x), ldx, _ptr(w if need_grad_x else None), ldw,
                                         m, n, k, cap, _ptr(fws), 0 if fws is None else fws.numel(),
                                         _ptr(gx), k, _ptr(gw), k, _ptr(workspace.buf), workspace.buf.numel(),
                                         _stream(dev)),
              "i8mp_linear_backward")
    return gx, gw


@dataclass
class Fp4Weight:
    """A weight in blockwise 4-bit E2M1 form: packed codes [n, ldc] (ldc = k/2
    rounded up to 16 bytes), and either fp32 block scales [n, k/64] or their
    8-bit double quantization (c8 [n * k/64], s2 [ceil(n * k/64 / 256)])."""

    codes: torch.Tensor
    k: int
    absmax: Optional[torch.Tensor] = None
    c8: Optional[torch.Tensor] = None
    s2: Optional[torch.Tensor] = None

    @property
    def n(self) -> int:
        return self.codes.shape[0]

    def scale_ptrs(self):
        if self.absmax is not None:
            return _ptr(self.absmax), None, None
        return None, _ptr(self.c8), _ptr(self.s2)


def fp4_quantize(w: torch.Tensor, double_quant: bool = False) -> Fp4Weight:
    """Blockwise 4-bit E2M1 quantization of an fp16 weight [n, k] (k a multiple of 64)."""
    dev = _device_of(w)
    ldw = _rowmajor(w, "w", torch.float16)
    n, k = w.shape
    if k % 64 or k == 0:
        raise ValueError("k must be a positive multiple of 64")
    ldc = (k // 2 + 15) // 16 * 16
    codes = torch.zeros((n, ldc), dtype=torch.uint8, device=dev)
    absmax = torch.empty((n, k // 64), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        check(lib().i8mp_fp4_quantize(_ptr(w), n, k, ldw, _ptr(codes), ldc, _ptr(absmax), _stream(dev)),
              "i8mp_fp4_quantize")
    fw = Fp4Weight(codes, k, absmax)
    return fp4_double_quant(fw) if double_quant else fw


def fp4_double_quant(fw: Fp4Weight) -> Fp4Weight:
    """The same weight with its block scales quantized to 8 bits in groups of 256."""
    if fw.absmax is None:
        raise ValueError("already double-quantized")
    dev = _device_of(fw.codes, fw.absmax)
    nb = fw.absmax.numel()
    c8 = torch.empty(nb, dtype=torch.uint8, device=dev)
    s2 = torch.empty(max((nb + 255) // 256, 1), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        check(lib().i8mp_fp4_double_quant(_ptr(fw.absmax), nb, _ptr(c8), _ptr(s2), _stream(dev)),
              "i8mp_fp4_double_quant")
    return Fp4Weight(fw.codes, fw.k, None, c8, s2[: (nb + 255) // 256])


def fp4_dequantize(fw: Fp4Weight, dtype: torch.dtype = torch.float16) -> torch.Tensor:
    """w' [n, k] = E2M1 value * (block scale / 6), as fp16 or fp32."""
    if dtype not in (torch.float16, torch.float32):
        raise ValueError("dtype must be torch.float16 or torch.float32")
    dev = _device_of(fw.codes)
    out = torch.empty((fw.n, fw.k), dtype=dtype, device=dev)
    a, c8, s2 = fw.scale_ptrs()
    with torch.cuda.device(dev):
        check(lib().i8mp_fp4_dequantize(_ptr(fw.codes), fw.codes.stride(0), fw.n, fw.k, a, c8, s2,
                                        0 if dtype == torch.float16 else 1, _ptr(out), fw.k, _stream(dev)),
              "i8mp_fp4_dequantize")
    return out


def fp4_linear(x: torch.Tensor, fw: Fp4Weight, bias: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The 4-bit linear for decode-sized batches: fp16 out [m, n] = x . w'^T + bias."""
    dev = _device_of(x, fw.codes, bias, out)
    ldx = _rowmajor(x, "x", torch.float16)
    m, k = x.shape
    if k != fw.k:
        raise ValueError("x and the weight differ in k")
    if bias is not None:
        _vec(bias, "bias", torch.float16, fw.n)
    if out is None:
        out = torch.empty((m, fw.n), dtype=torch.float16, device=dev)
    ldout = _rowmajor(out, "out", torch.float16)
    a, c8, s2 = fw.scale_ptrs()
    with torch.cuda.device(dev):
        check(lib().i8mp_fp4_linear(_ptr(x), m, k, ldx, _ptr(fw.codes), fw.codes.stride(0), a, c8, s2, fw.n,
                                    _ptr(bias), _ptr(out), ldout, _stream(dev)),
              "i8mp_fp4_linear")
    return out


_DTYPE_CODE = {torch.float16: 0, torch.float32: 1, torch.bfloat16: 2}
_CACHE_CODE = {torch.float16: 0, torch.bfloat16: 2}
# the handle of a device's current stream, without a Stream object around it (2 us a call);
# a torch built without GPU support has none, and no tensor that would need it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


@dataclass
class Fp4Cache:
    """A paged 4-bit key/value cache: ``data`` uint8 [pages, kv_heads, slab] in the
    layout of include/i8mp.h (``create`` allocates it), pages of ``page_size``
    tokens, beside keys, values and queries of ``dtype`` (fp16 or bfloat16).
    Slot ``page * page_size + i`` is place i of a page."""

    data: torch.Tensor
    page_size: int
    head_dim: int
    dtype: torch.dtype = torch.float16

    @classmethod
    def create(cls, pages: int, kv_heads: int, head_dim: int, page_size: int = 64,
               dtype: torch.dtype = torch.float16, device="cuda") -> "Fp4Cache":
        nbytes = page_size * (head_dim + 4 * (head_dim // 64))
        cache = cls(torch.zeros((pages, kv_heads, nbytes), dtype=torch.uint8, device=device), page_size, head_dim, dtype)
        if lib().i8mp_fp4_cache_bytes(ctypes.byref(cache.struct())) == 0:
            raise ValueError("a cache has page_size 16, 32, 64, 128 or 256 and head_dim 64, 128 or 256")
        return cache

    @property
    def pages(self) -> int:
        return self.data.shape[0]

    @property
    def kv_heads(self) -> int:
        return self.data.shape[1]

    def struct(self) -> Fp4CacheStruct:
        """The C form, after checking that the fields go together (the library checks their ranges)."""
        d = self.data
        dtype = _CACHE_CODE.get(self.dtype)
        if dtype is None:
            raise TypeError(f"a cache's dtype is torch.float16 or torch.bfloat16, got {self.dtype}")
        if d.dtype != torch.uint8 or d.dim() != 3 or not d.is_contiguous():
            raise ValueError("data must be a contiguous uint8 [pages, kv_heads, slab] tensor")
        pages, heads, slab = d.shape
        if slab != self.page_size * (self.head_dim + 4 * (self.head_dim // 64)):
            raise ValueError("data's last axis must be page_size * (head_dim + head_dim / 16) bytes")
        return Fp4CacheStruct(d.data_ptr(), pages, heads, self.page_size, self.head_dim, dtype)


def _run(dev: torch.device, what: str, *args) -> None:
    """Calls a library entry point on dev with its current stream as the last argument."""
    f, i = getattr(lib(), what), dev.index
    if i == torch.cuda.current_device():
        status = f(*args, _raw_stream(i))
    else:
        with torch.cuda.device(dev):
            status = f(*args, _raw_stream(i))
    if status:
        check(status, what)


def _heads(t: torch.Tensor, name: str, dtype: torch.dtype, heads: Optional[int], head_dim: int) -> Tuple[int, int]:
    """Token and head strides of a [tokens, heads, head_dim] tensor with unit stride within a head."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != head_dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [tokens, {'heads' if heads is None else heads}, {head_dim}]")
    ld, hs, unit = t.stride()
    if unit != 1:
        raise ValueError(f"{name} must have unit stride within a head")
    # the stride of an axis of one element is never taken: any that the library accepts will do
    return (ld if shape[0] > 1 else head_dim), (hs if shape[1] > 1 else head_dim)


def _int32(**values: int) -> None:
    """The values are whole in an int32 of a C structure (ctypes keeps the low 32 bits of others)."""
    for name, value in values.items():
        if not -1 << 31 <= value < 1 << 31:
            raise ValueError(f"{name} is out of range: {value}")


def _float32(**values: float) -> None:
    """The values that are not 0 are not 0 in fp32 either."""
    for name, value in values.items():
        if value != 0.0 and ctypes.c_float(value).value == 0.0:
            raise ValueError(f"{name} is less than any fp32 number: {value}")


def fp4_cache_write(cache: Fp4Cache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
    """Quantizes k and v [tokens, kv_heads, head_dim] into the cache's slots (int64 [tokens], distinct).

    A slot outside the cache (-1) is skipped."""
    dev = _device_of(cache.data, k, v, slots)
    c = cache.struct()
    ldk, hsk = _heads(k, "k", cache.dtype, c.kv_heads, c.head_dim)
    ldv, hsv = _heads(v, "v", cache.dtype, c.kv_heads, c.head_dim)
    n = k.shape[0]
    if v.shape[0] != n:
        raise ValueError("k and v differ in tokens")
    _vec(slots, "slots", torch.int64, n)
    _run(dev, "i8mp_fp4_cache_write", ctypes.byref(c), k.data_ptr(), ldk, hsk, v.data_ptr(), ldv, hsv,
         slots.data_ptr(), n)


def fp4_cache_read(cache: Fp4Cache, slots: torch.Tensor, dtype: Optional[torch.dtype] = None
                   ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(k, v) [tokens, kv_heads, head_dim] held at the slots, as the cache's type or ``dtype``
    (fp16, bfloat16 or fp32).  A slot outside the cache reads as zeros."""
    dtype = cache.dtype if dtype is None else dtype
    if dtype not in _DTYPE_CODE:
        raise ValueError("dtype must be torch.float16, torch.bfloat16 or torch.float32")
    dev = _device_of(cache.data, slots)
    c = cache.struct()
    n = slots.shape[0]
    _vec(slots, "slots", torch.int64, n)
    k = slots.new_empty((n, c.kv_heads, c.head_dim), dtype=dtype)
    v = torch.empty_like(k)
    ld, hs = c.kv_heads * c.head_dim, c.head_dim
    _run(dev, "i8mp_fp4_cache_read", ctypes.byref(c), slots.data_ptr(), n, _DTYPE_CODE[dtype], k.data_ptr(), ld, hs,
         v.data_ptr(), ld, hs)
    return k, v


def fp4_cache_attention(q: torch.Tensor, cache: Fp4Cache, table: torch.Tensor, lengths: torch.Tensor,
                        q_offsets: Optional[torch.Tensor] = None, max_q: Optional[int] = None,
                        max_len: Optional[int] = None, scale: Optional[float] = None, window: int = 0,
                        softcap: float = 0.0, alibi: Optional[torch.Tensor] = None,
                        prefix: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                        return_lse: bool = False, workspace: Optional[torch.Tensor] = None):
    """Attention of q [tokens, q_heads, head_dim] over the 4-bit cache: out, or (out, lse fp32 [tokens, q_heads]).

    ``lengths`` int32 [batch] counts each sequence's cached tokens, its queries' own
    included (write them first); ``table`` int32 [batch, n] names its pages.  The rows
    of q are ``max_q`` queries a sequence (default: tokens / batch), or, with
    ``q_offsets`` int32 [batch + 1], rows q_offsets[b] .. q_offsets[b + 1] (``max_q``
    then bounds them; default: tokens).  Query i of n is at position lengths - n + i
    and sees tokens up to it, within ``window`` (0: all), and the first ``prefix``
    (int32 [batch]) tokens.  ``softcap`` > 0 caps scores by a tanh; ``alibi`` (fp32
    [q_heads]) subtracts alibi * distance.  ``scale`` defaults to head_dim ** -0.5,
    ``max_len`` (a bound on the lengths) to the table's width.  A row that sees
    nothing is zeros, its lse -inf; so are rows of q that are no sequence's queries
    (before the first offset, past the last, past ``max_q``), but those of a given
    ``out`` keep what they hold.  No gradient is recorded.  ``workspace``: contiguous uint8, reused by the
    caller (default: allocated here)."""
    dev = _device_of(q, cache.data, table, lengths, q_offsets, alibi, prefix, out, workspace)
    c = cache.struct()
    ldq, hsq = _heads(q, "q", cache.dtype, None, c.head_dim)
    tokens, q_heads = q.shape[:2]
    batch = lengths.shape[0]
    _vec(lengths, "lengths", torch.int32, batch)
    ldt = _rowmajor(table, "table", torch.int32)
    cols = table.shape[1]
    if table.shape[0] != batch:
        raise ValueError("table and lengths differ in sequences")
    if q_offsets is not None:
        _vec(q_offsets, "q_offsets", torch.int32, batch + 1)
    if alibi is not None:
        _vec(alibi, "alibi", torch.float32, q_heads)
    if prefix is not None:
        _vec(prefix, "prefix", torch.int32, batch)
    if max_q is None:
        max_q = tokens if q_offsets is not None else tokens // max(batch, 1)
    if q_offsets is None and max_q * batch != tokens:
        raise ValueError("without q_offsets every sequence has max_q queries: tokens must be batch * max_q")
    fill = out is None
    if fill:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        if batch == 0:                                  # no launch
            out.zero_()
    ldo, hso = _heads(out, "out", cache.dtype, q_heads, c.head_dim)
    if out.shape[0] != tokens:
        raise ValueError("out has the wrong shape")
    lse = None
    if return_lse:
        lse = q.new_empty((tokens, q_heads), dtype=torch.float32)
        if q_offsets is not None and not (fill and batch):
            lse.fill_(float("-inf"))
    max_len = cols * cache.page_size if max_len is None else max_len
    if (max_q | max_len | window) >> 31:                # not all of them in 0 .. 2^31 - 1
        _int32(max_q=max_q, max_len=max_len, window=window)
    if softcap:
        _float32(softcap=softcap)
    call = Fp4AttentionStruct(
        q.data_ptr(), ldq, hsq, out.data_ptr(), ldo, hso, None if lse is None else lse.data_ptr(), table.data_ptr(), ldt,
        cols, lengths.data_ptr(), None if q_offsets is None else q_offsets.data_ptr(),
        None if alibi is None else alibi.data_ptr(), None if prefix is None else prefix.data_ptr(), tokens, batch,
        q_heads, max(max_q, 1), max_len, window, c.head_dim ** -0.5 if scale is None else scale, softcap, fill)
    if workspace is not None:
        _bytes(workspace, "workspace")
    else:
        need = lib().i8mp_fp4_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(call))
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _run(dev, "i8mp_fp4_cache_attention", ctypes.byref(c), ctypes.byref(call),
         None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel())
    return out if lse is None else (out, lse)


def fp4_cache_append(cache: Fp4Cache, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                     positions: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor, interleaved: bool = False,
                     out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Rotates q [tokens, q_heads, head_dim] and k by position, writes k and v [tokens, kv_heads,
    head_dim] into the cache's slots, and returns the rotated q (None for q None).

    Row positions[t] (int64 [tokens]) of ``cos`` and ``sin`` (fp32 [rows, rotary / 2]) turns token t:
    dims (i, i + rotary / 2) of a head, or (2 i, 2 i + 1) if ``interleaved``, for the first ``rotary`` dims (a
    multiple of 16).  A position is taken into the tables' rows; a slot (int64 [tokens], distinct) outside
    the cache (-1) is skipped.  ``out`` may be q itself; other tensors must not share elements with it.  No
    gradient is recorded."""
    dev = _device_of(cache.data, q, k, v, slots, positions, cos, sin, out)
    c = cache.struct()
    ldk, hsk = _heads(k, "k", cache.dtype, c.kv_heads, c.head_dim)
    ldv, hsv = _heads(v, "v", cache.dtype, c.kv_heads, c.head_dim)
    n = k.shape[0]
    if v.shape[0] != n:
        raise ValueError("k and v differ in tokens")
    _vec(slots, "slots", torch.int64, n)
    _vec(positions, "positions", torch.int64, n)
    ldcos, ldsin = _rowmajor(cos, "cos", torch.float32), _rowmajor(sin, "sin", torch.float32)
    rows, half = cos.shape
    if sin.shape != cos.shape:
        raise ValueError("cos and sin differ in shape")
    if rows == 0:
        raise ValueError("cos and sin have no rows")
    _int32(rotary=2 * half)
    ldq = hsq = ldo = hso = heads = 0
    if q is not None:
        ldq, hsq = _heads(q, "q", cache.dtype, None, c.head_dim)
        if q.shape[0] != n:
            raise ValueError("q and k differ in tokens")
        heads = q.shape[1]
        if out is None:
            out = q.new_empty(q.shape)
            ldo, hso = heads * c.head_dim, c.head_dim
        else:
            ldo, hso = _heads(out, "out", cache.dtype, heads, c.head_dim)
            if out.shape[0] != n:
                raise ValueError("out has the wrong shape")
    elif out is not None:
        raise ValueError("out without q")
    call = Fp4AppendStruct(k.data_ptr(), ldk, hsk, v.data_ptr(), ldv, hsv, slots.data_ptr(), positions.data_ptr(),
                           cos.data_ptr(), sin.data_ptr(), ldcos, ldsin, rows,
                           q.data_ptr() if heads else None, ldq, hsq, out.data_ptr() if heads else None, ldo, hso, n, heads,
                           2 * half, bool(interleaved))
    _run(dev, "i8mp_fp4_cache_append", ctypes.byref(c), ctypes.byref(call))
    return out


@dataclass
class Mx4Tensor:
    """A microscaled 4-bit matrix [rows, k] in the layout of include/i8mp.h: packed E2M1 ``codes`` uint8
    [rows, kp / 2] and E8M0 ``scales`` uint8 [rows, kp / 32], kp = k rounded up to 128 (``create`` allocates them).
    An ``out`` of the calls that take one shares no memory with their inputs."""

    codes: torch.Tensor
    scales: torch.Tensor
    k: int

    @classmethod
    def create(cls, rows: int, k: int, device="cuda") -> "Mx4Tensor":
        kp = (k + 127) // 128 * 128
        return cls(torch.empty((rows, kp // 2), dtype=torch.uint8, device=device),
                   torch.empty((rows, kp // 32), dtype=torch.uint8, device=device), k)

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    @property
    def shape(self) -> Tuple[int, int]:
        return self.codes.shape[0], self.k

    def struct(self) -> Mx4Struct:
        """The C form, after checking that the fields go together (the library checks ranges and alignment)."""
        codes, scales, k = self.codes, self.scales, self.k
        ldc, lds = _rowmajor(codes, "codes", torch.uint8), _rowmajor(scales, "scales", torch.uint8)
        rows, width = codes.shape
        held, scale_width = scales.shape
        units = -(-k // 128)
        if held != rows or width < units * 64 or scale_width < units * 4:
            raise ValueError(f"codes and scales must hold [{rows}, {units * 64}] and [{rows}, {units * 4}] bytes for k = {k}")
        if rows <= 1 or units == 0:     # a stride that is never taken: any that the library accepts
            ldc, lds = units * 64, units * 4
        return Mx4Struct(codes.data_ptr(), scales.data_ptr(), rows, k, ldc, lds)


def _half(t: torch.Tensor, name: str) -> int:
    """The code of a 16-bit type."""
    code = _CACHE_CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be torch.float16 or torch.bfloat16, got {t.dtype}")
    return code


def _space(need: int, workspace: Optional[torch.Tensor], like: torch.Tensor) -> Optional[torch.Tensor]:
    """A call's workspace: the caller's, or one of ``need`` bytes (none for 0)."""
    if workspace is not None:
        _bytes(workspace, "workspace")
        return workspace
    return like.new_empty(need, dtype=torch.uint8) if need else None


def _run_of(ws: Optional[torch.Tensor]) -> Tuple[Optional[int], int]:
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel())


def mx4_quantize(x: torch.Tensor, columns: bool = False, out: Optional[Mx4Tensor] = None) -> Mx4Tensor:
    """Microscaled 4-bit form of a 16-bit matrix x [m, k]: blocks of 32 along its rows, or with ``columns`` along
    its columns, which gives the transpose [k, m]."""
    dev = _device_of(x, None if out is None else out.codes, None if out is None else out.scales)
    ldx = _rowmajor(x, "x", x.dtype)
    code = _half(x, "x")
    m, k = x.shape
    rows, length = (k, m) if columns else (m, k)
    if out is None:
        kp = -(-length // 128) * 128
        codes = x.new_empty((rows, kp // 2), dtype=torch.uint8)
        scales = x.new_empty((rows, kp // 32), dtype=torch.uint8)
        out = Mx4Tensor(codes, scales, length)
        c = Mx4Struct(codes.data_ptr(), scales.data_ptr(), rows, length, kp // 2, kp // 32)
    elif out.shape != (rows, length):
        raise ValueError("out has the wrong shape")
    else:
        c = out.struct()
    _run(dev, "i8mp_mx4_quantize", x.data_ptr(), code, m, k, ldx, bool(columns), ctypes.byref(c))
    return out


def mx4_dequantize(t: Mx4Tensor, dtype: torch.dtype = torch.float16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """E2M1 value * 2^(scale - 127) [rows, k], as fp16, bfloat16 or fp32."""
    if dtype not in _DTYPE_CODE:
        raise ValueError("dtype must be torch.float16, torch.bfloat16 or torch.float32")
    dev = _device_of(t.codes, t.scales, out)
    if out is None:
        out = t.codes.new_empty((t.codes.shape[0], t.k), dtype=dtype)
        ldout = t.k
    else:
        ldout = _rowmajor(out, "out", dtype)
        if tuple(out.shape) != t.shape:
            raise ValueError("out has the wrong shape")
    _run(dev, "i8mp_mx4_dequantize", ctypes.byref(t.struct()), _DTYPE_CODE[dtype], out.data_ptr(), ldout)
    return out


def mx4_matmul(a: Mx4Tensor, b: Mx4Tensor, bias: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.float16,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """a . b^T + bias of two microscaled matrices: out [a.rows, b.rows] in ``dtype`` (fp16, bfloat16 or fp32, the
    bias too), sums in fp32.  ``workspace``: contiguous uint8, reused by the caller (default: allocated here)."""
    if dtype not in _DTYPE_CODE:
        raise ValueError("dtype must be torch.float16, torch.bfloat16 or torch.float32")
    dev = _device_of(a.codes, a.scales, b.codes, b.scales, bias, out, workspace)
    m, n, k = a.rows, b.rows, a.k
    if b.k != k:
        raise ValueError("a and b differ in k")
    if bias is not None:
        _vec(bias, "bias", dtype, n)
    if out is None:
        out = a.codes.new_empty((m, n), dtype=dtype)
        ldout = n
    else:
        ldout = _rowmajor(out, "out", dtype)
        if tuple(out.shape) != (m, n):
            raise ValueError("out has the wrong shape")
    ws = _space(lib().i8mp_mx4_matmul_workspace_bytes(m, n, k), workspace, a.codes)
    _run(dev, "i8mp_mx4_matmul", ctypes.byref(a.struct()), ctypes.byref(b.struct()),
         None if bias is None else bias.data_ptr(), _DTYPE_CODE[dtype], out.data_ptr(), ldout, *_run_of(ws))
    return out


def mx4_linear(x: torch.Tensor, w: Mx4Tensor, bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The linear with 4-bit weights and activations: mx4(x) . w^T + bias for x [m, k] of a 16-bit type, which out
    [m, n] and the bias share.  No gradient is recorded: ``mx4_linear_backward`` computes both."""
    dev = _device_of(x, w.codes, w.scales, bias, out, workspace)
    ldx = _rowmajor(x, "x", x.dtype)
    code = _half(x, "x")
    m, k = x.shape
    n = w.rows
    if w.k != k:
        raise ValueError("x and w differ in k")
    if bias is not None:
        _vec(bias, "bias", x.dtype, n)
    if out is None:
        out = x.new_empty((m, n))
        ldout = n
    else:
        ldout = _rowmajor(out, "out", x.dtype)
        if tuple(out.shape) != (m, n):
            raise ValueError("out has the wrong shape")
    ws = _space(lib().i8mp_mx4_linear_workspace_bytes(m, n, k), workspace, x)
    _run(dev, "i8mp_mx4_linear", x.data_ptr(), code, m, ldx, ctypes.byref(w.struct()),
         None if bias is None else bias.data_ptr(), out.data_ptr(), ldout, *_run_of(ws))
    return out


def mx4_linear_backward(grad_out: torch.Tensor, x: Optional[torch.Tensor], w: Optional[torch.Tensor],
                        need_grad_x: bool = True, need_grad_w: bool = True, workspace: Optional[torch.Tensor] = None,
                        out_x: Optional[torch.Tensor] = None, out_w: Optional[torch.Tensor] = None,
                        ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Both gradients of x [m, k] . w^T for dL/dout = grad_out [m, n], w [n, k] the 16-bit weight kept for training:
    (grad_x [m, k], grad_w [n, k]), products of operands quantized along what they sum over.  grad_x needs w, grad_w
    needs x; all tensors share one 16-bit type."""
    need_x, need_w = bool(need_grad_x), bool(need_grad_w)
    dev = _device_of(grad_out, x, w, workspace, out_x, out_w)
    dtype = grad_out.dtype
    ldg = _rowmajor(grad_out, "grad_out", dtype)
    code = _half(grad_out, "grad_out")
    m, n = grad_out.shape
    if (need_x and w is None) or (need_w and x is None):
        raise ValueError("grad_x needs w, grad_w needs x")
    if not (need_x or need_w):
        return None, None
    ldx = ldw = 0
    if need_x:
        ldw = _rowmajor(w, "w", dtype)
    if need_w:
        ldx = _rowmajor(x, "x", dtype)
    k = w.shape[1] if need_x else x.shape[1]
    if (need_x and tuple(w.shape) != (n, k)) or (need_w and tuple(x.shape) != (m, k)):
        raise ValueError("grad_out, x and w must be [m, n], [m, k] and [n, k]")
    ldgx = ldgw = 0
    if need_x:
        if out_x is None:
            out_x, ldgx = grad_out.new_empty((m, k)), k
        else:
            ldgx = _rowmajor(out_x, "out_x", dtype)
            if tuple(out_x.shape) != (m, k):
                raise ValueError("out_x has the wrong shape")
    if need_w:
        if out_w is None:
            out_w, ldgw = grad_out.new_empty((n, k)), k
        else:
            ldgw = _rowmajor(out_w, "out_w", dtype)
            if tuple(out_w.shape) != (n, k):
                raise ValueError("out_w has the wrong shape")
    ws = _space(lib().i8mp_mx4_linear_backward_workspace_bytes(m, n, k), workspace, grad_out)
    _run(dev, "i8mp_mx4_linear_backward", grad_out.data_ptr(), ldg, x.data_ptr() if need_w else None, ldx,
         w.data_ptr() if need_x else None, ldw, code, m, n, k, out_x.data_ptr() if need_x else None, ldgx,
         out_w.data_ptr() if need_w else None, ldgw, *_run_of(ws))
    return out_x if need_x else None, out_w if need_w else None
