"""4-bit whole-number weights with group scales: quantisation, dequantisation
and products, plain and by expert (binding of ``liboptimizer_experts.so``,
``include/optimizer_experts.h``).

    q = int4_quantize(w, group=128)           Int4: codes, scales, zeros, group
    q = Int4(codes, scales, zeros, group)     of a checkpoint's own tensors
    w4 = int4_dequantize(q, torch.bfloat16)   the values: (code - zero) * scale
    y = int4_matmul(x, q)                     x q^T
    y = int4_grouped_matmul(x, qe, offsets)   rows offsets[e]:offsets[e + 1] of x against expert e

Made for the few rows of serving.  No gradients are recorded; the products
refuse operands that ask for them.  Streams, checks and ownership are those of
the other 4-bit operators (``mx4``); copies that views take are made on the
call's stream, and a result that is given counts as written for autograd.
"""
from __future__ import annotations

import math

import torch

from . import DTYPES
from .mx4 import _offsets, _output, _result_type, _row_stride, _rows_apart, _run, _same, _values
from .route import _fail, _written, load_experts


class Int4:
    """A matrix [N, K], or a batch [E, N, K], in 4-bit whole numbers:
    ``codes`` uint8 [..., N, K / 2] (the even column in the low four bits),
    ``scales`` [..., N, K / group] and ``zeros`` of the same shape and dtype,
    or None for 8 everywhere; value = (code - zero) * scale.  ``group`` is a
    multiple of 32, K one of group."""

    __slots__ = ("codes", "scales", "zeros", "group")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None, group: int):
        if codes.dtype != torch.uint8 or codes.dim() not in (2, 3):
            raise ValueError("codes must be uint8 [N, K / 2] or [E, N, K / 2]")
        k = codes.shape[-1] * 2
        if group < 32 or group % 32 or k % group:
            raise ValueError(f"group must be a multiple of 32 that divides K = {k}: got {group}")
        for t, name in ((scales, "scales"), (zeros, "zeros")):
            if t is None and name == "zeros":
                continue
            if t.dtype not in DTYPES or t.dtype != scales.dtype:
                raise ValueError("scales and zeros must be float32, float16 or bfloat16, of one type")
            if tuple(t.shape) != (*codes.shape[:-1], k // group):
                raise ValueError(f"{name} must be {[*codes.shape[:-1], k // group]}: got {list(t.shape)}")
            if t.get_device() != codes.get_device() or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous and on the codes' device")
        if not codes.is_contiguous():
            raise ValueError("codes must be contiguous")
        self.codes, self.scales, self.zeros, self.group = codes, scales, zeros, int(group)

    @property
    def k(self) -> int:
        return self.codes.shape[-1] * 2

    @property
    def shape(self) -> torch.Size:
        return torch.Size((*self.codes.shape[:-1], self.k))

    @property
    def device(self) -> torch.device:
        return self.codes.device

    def __getitem__(self, i: int) -> "Int4":
        """Matrix i of a batch."""
        if self.codes.dim() < 3:
            raise ValueError("not a batch of matrices")
        return Int4(self.codes[i], self.scales[i], None if self.zeros is None else self.zeros[i], self.group)

    def __repr__(self) -> str:
        return f"Int4(shape={list(self.shape)}, group={self.group}, device={self.device})"


def _weights(q, dims: int | None = None) -> int:
    """Device index of an Int4."""
    if not isinstance(q, Int4) or dims is not None and q.codes.dim() != dims:
        raise ValueError("expected an Int4" + ("" if dims is None else " matrix" if dims == 2 else " batch of matrices"))
    index = q.codes.get_device()
    if index < 0:
        raise ValueError("the weights must be on a HIP device")
    return index


def _ptrs(q: Int4) -> tuple:
    return (q.codes.data_ptr(), DTYPES[q.scales.dtype], q.scales.data_ptr(),
            None if q.zeros is None else q.zeros.data_ptr())


def _do_quantize(x, lead, rows, k, group, dtype, zeros, handle):
    device = x.device
    x = _rows_apart(x.reshape(rows, k))   # a copy, where it takes one, is made on the call's stream
    codes = torch.empty((*lead, k // 2), dtype=torch.uint8, device=device)
    scales = torch.empty((*lead, k // group), dtype=dtype, device=device)
    z = torch.empty_like(scales) if zeros else None
    st = load_experts().ou_int4_quantize(DTYPES[x.dtype], x.data_ptr(), rows, k, _row_stride(x, "x"), group, DTYPES[dtype],
                                         codes.data_ptr(), scales.data_ptr(), None if z is None else z.data_ptr(), handle)
    if st:
        _fail(st)
    return Int4(codes, scales, z, group)


def int4_quantize(x: torch.Tensor, group: int = 128, zeros: bool = True, dtype: torch.dtype | None = None,
                  stream=None) -> Int4:
    """x [N, K] or [E, N, K] by groups of ``group`` columns, each with the
    smallest scale whose 16 steps hold its values (and 0) and a whole zero;
    without ``zeros``, around code 8.  Scales (of ``dtype``, x's by default)
    are rounded first, codes to the nearest, ties to even.  Finite values only."""
    _values(x, "x")
    if x.dim() not in (2, 3):
        raise ValueError("x must be [N, K] or [E, N, K]")
    *lead, k = x.shape
    dtype = dtype or x.dtype
    _result_type(dtype)
    group = int(group)
    if group < 32 or group % 32 or k % group:
        raise ValueError(f"group must be a multiple of 32 that divides K = {k}: got {group}")
    return _run(x.get_device(), stream, _do_quantize, x.detach(), lead, math.prod(lead), k, group, dtype, bool(zeros))


def _do_dequantize(q, dtype, out, handle):
    given = out is not None
    if not given:
        out = torch.empty(q.shape, dtype=dtype, device=q.device)
    st = load_experts().ou_int4_dequantize(DTYPES[out.dtype], *_ptrs(q), math.prod(q.codes.shape[:-1]), q.k, q.group,
                                           out.data_ptr(), q.k, handle)
    if st:
        _fail(st)
    return _written(out) if given else out


def int4_dequantize(q: Int4, dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """The values of q in ``dtype`` (or in ``out``, contiguous), computed in
    binary32 and rounded once."""
    index = _weights(q)
    if out is None:
        _result_type(dtype)
    else:
        _values(out, "out")
        _same(index, out.get_device(), "out")
        if out.shape != q.shape or not out.is_contiguous():
            raise ValueError(f"out must be contiguous, of shape {list(q.shape)}")
    return _run(index, stream, _do_dequantize, q, dtype, out)


def _do_matmul(x, dt, rs, q, m, n, k, dtype, od, out, stride, offsets, groups, handle):
    rest = 0 if out is not None else 1
    if rest:
        out = x.new_empty((m, n), dtype=dtype)
    codes, scales, zeros = q.codes, q.scales, q.zeros
    sd, zp = DTYPES[scales.dtype], None if zeros is None else zeros.data_ptr()
    lib = load_experts()
    if offsets is None:
        st = lib.ou_int4_matmul(dt, x.data_ptr(), m, rs, od, codes.data_ptr(), sd, scales.data_ptr(), zp, n, k, q.group,
                                out.data_ptr(), stride, handle)
    else:
        st = lib.ou_int4_grouped_matmul(dt, x.data_ptr(), m, rs, od, codes.data_ptr(), sd, scales.data_ptr(), zp, n, k,
                                        q.group, offsets.data_ptr(), groups, out.data_ptr(), stride, rest, handle)
    if st:
        _fail(st)
    return out if rest else _written(out)


def _matmul(x, q, offsets, dims, dtype, out, stream):
    on = _weights(q, dims)
    n, k = q.codes.shape[-2], q.codes.shape[-1] * 2
    dt = _values(x, "the left operand", 2)
    index = x.get_device()
    _same(index, on, "the weights")
    if (x.requires_grad or out is not None and out.requires_grad) and torch.is_grad_enabled():
        raise ValueError("gradients are not recorded through 4-bit whole numbers: detach x, or call under no_grad()")
    m, have = x.shape
    if have != k:
        raise ValueError(f"the operands contract {have} and {k} columns")
    groups = 0
    if offsets is not None:
        groups = _offsets(offsets, index)
        if groups != q.codes.shape[0]:
            raise ValueError(f"offsets name {groups} groups, the weights hold {q.codes.shape[0]}")
    if dtype is None:
        dtype = x.dtype
    od, stride = _output(out, m, n, dtype, index)
    return _run(index, stream, _do_matmul, x, dt, _row_stride(x, "the left operand"), q, m, n, k, dtype, od, out, stride,
                offsets, groups)


def int4_matmul(x: torch.Tensor, q: Int4, dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """x q^T for x [M, K] (any row stride) and an Int4 [N, K]: [M, N] of
    ``dtype`` (x's by default), or ``out`` (any row stride).  Products are exact
    but for what lies below 2^-133 of a float32 x; a group's columns are summed
    in binary32, the codes (less 7.5 with a float32 x) and x apart, so that a
    result's error goes by |x| (code + |zero|) |scale| (less 7.5 each with
    float32) rather than by its own terms, and may be infinite or NaN where
    these sums are; rounded once.  For many rows (a prompt), ``int4_dequantize``
    and a library product are faster."""
    return _matmul(x, q, None, 2, dtype, out, stream)


def int4_grouped_matmul(x: torch.Tensor, q: Int4, offsets: torch.Tensor, dtype: torch.dtype | None = None,
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rows offsets[e]:offsets[e + 1] of x [T, K] times matrix e of an Int4
    [E, N, K], transposed; ``offsets`` as in ``mx4_grouped_matmul`` (of a
    ``RouteOrder``, say).  Rows of no group are 0 in a new result and left as
    they were in ``out``."""
    if offsets is None:
        raise ValueError("offsets must be a contiguous int32 tensor of groups + 1 values")
    return _matmul(x, q, offsets, 3, dtype, out, stream)
