"""Microscaled 4-bit floats: quantisation, products of quantised matrices and
products grouped by expert (binding of ``liboptimizer_mx4.so``,
``include/optimizer_mx4.h``).

    q = mx4_quantize(w)                       Mx4: codes, scales, k
    q, qt = mx4_quantize_both(w)              along the columns and along the rows, one read
    w4 = mx4_dequantize(q, torch.bfloat16)    the values held
    y = mx4_matmul(x, q)                      x q^T; x as values (quantised on the way) or Mx4
    y = mx4_grouped_matmul(x, qe, offsets)    rows offsets[e]:offsets[e+1] of x against expert e
    y = mx4_linear(x, w)                      the layer with its gradients (straight through
    y = mx4_grouped_linear(x, w, offsets)     the roundings), all three products in 4 bits
    Mx4Weight(w)                              both 4-bit forms of a weight, refreshed by its
                                              optimizer's steps (``attach_mx4``)

As in the rest of the package, functions check and marshal arguments; all
arithmetic runs in the HIP kernels.  Every call goes to the current stream of
the operands' device, or to ``stream`` (a stream of that device or its handle,
0 being the default stream); results and workspaces are allocated on that
stream.  As elsewhere in torch, an operand of another stream must stay until
the call's work is done (``record_stream``).  The functions other than the two
layers do not record gradients.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import warnings
import weakref

import torch

from . import DTYPES, _GET_DEVICE, _lib, _raw_stream

HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(HERE, "liboptimizer_mx4.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "optimizer_mx4.h")

MX4_BLOCK = 32     # values that share a scale
MX4_PAD = 128      # columns of a held matrix are padded to this
_mx4 = None


def load_mx4(path: str = LIBRARY) -> ctypes.CDLL:
    """Load the library of the 4-bit operators (raises if it is missing)."""
    global _mx4
    if _mx4 is not None and path == LIBRARY:
        return _mx4
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built; run __graft_entry__.build() "
                          "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    i32, i64, vp = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p
    for name, res, args in (
            ("ou_mx4_columns", i64, [i64]),
            ("ou_mx4_grouped_columns", i64, [i64, i32]),
            ("ou_mx4_quantize", i32, [i32, vp, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp]),
            ("ou_mx4_quantize_grouped", i32, [i32, vp, i64, i64, i64, vp, i32, vp, vp, vp, vp, vp]),
            ("ou_mx4_dequantize", i32, [i32, vp, vp, i64, i64, vp, i64, vp]),
            ("ou_mx4_matmul_workspace_bytes", i64, [i64, i64, i64, i32]),
            ("ou_mx4_grouped_workspace_bytes", i64, [i64, i64, i64, i32, i32]),
            ("ou_mx4_matmul", i32, [i32, vp, vp, i64, vp, vp, i64, i64, vp, i64, vp, i64, vp]),
            ("ou_mx4_matmul_values", i32, [i32, vp, i64, i64, i32, vp, vp, i64, i64, vp, i64, vp, i64, vp]),
            ("ou_mx4_grouped_matmul", i32, [i32, vp, vp, i64, vp, vp, i64, i64, vp, i32, vp, i64, i32, vp, i64, vp]),
            ("ou_mx4_grouped_matmul_values", i32, [i32, vp, i64, i64, i32, vp, vp, i64, i64, vp, i32, vp, i64, i32,
                                                   vp, i64, vp]),
            ("ou_mx4_grouped_outer", i32, [i32, vp, vp, i64, vp, vp, i64, i64, vp, i32, vp, vp]),
            ("ou_mx4_last_error", ctypes.c_char_p, [])):
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    if path == LIBRARY:
        _mx4 = lib
    return lib


def _fail(status: int) -> None:
    raise _lib.OptimizerUpdateError(status, load_mx4().ou_mx4_last_error().decode(errors="replace"))


def _columns(k: int) -> int:
    return -(-k // MX4_PAD) * MX4_PAD


class Mx4:
    """A matrix, or a batch of them, held in 4 bits: ``codes`` uint8
    [..., R, P / 2], ``scales`` uint8 [..., R, P / 32], ``k`` columns, P = k
    rounded up to 128 (the layout of ``include/optimizer_mx4.h``)."""

    __slots__ = ("codes", "scales", "k")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, k: int):
        p = _columns(k)
        if k < 0 or codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise ValueError("codes and scales are uint8 tensors, k >= 0")
        if codes.dim() < 2 or codes.shape[:-1] != scales.shape[:-1] or codes.shape[-1] * 2 != p \
                or scales.shape[-1] * MX4_BLOCK != p:
            raise ValueError(f"k = {k} wants codes [..., {p // 2}] and scales [..., {p // MX4_BLOCK}]: "
                             f"got {list(codes.shape)} and {list(scales.shape)}")
        if not codes.is_contiguous() or not scales.is_contiguous() or codes.device != scales.device:
            raise ValueError("codes and scales must be contiguous and on one device")
        self.codes, self.scales, self.k = codes, scales, k

    @property
    def shape(self) -> torch.Size:
        return torch.Size((*self.codes.shape[:-1], self.k))

    @property
    def device(self) -> torch.device:
        return self.codes.device

    def __getitem__(self, i: int) -> "Mx4":
        """Matrix i of a batch."""
        if self.codes.dim() < 3:
            raise ValueError("not a batch of matrices")
        return Mx4(self.codes[i], self.scales[i], self.k)

    def __repr__(self) -> str:
        return f"Mx4(shape={list(self.shape)}, device={self.device})"


def _held(codes, scales, k) -> Mx4:
    """An Mx4 of tensors made here."""
    q = Mx4.__new__(Mx4)
    q.codes, q.scales, q.k = codes, scales, k
    return q


def _empty(lead, k, device) -> Mx4:
    p = _columns(k)
    return _held(torch.empty((*lead, p // 2), dtype=torch.uint8, device=device),
                 torch.empty((*lead, p // MX4_BLOCK), dtype=torch.uint8, device=device), k)


class _Call:
    """Makes a device, or a given stream of it, current for a call: what is
    allocated inside belongs to that stream; ``handle`` is the stream's."""

    __slots__ = ("handle", "_ctx")

    def __init__(self, index: int, stream):
        if stream is None:
            self._ctx = torch.cuda.device(index)
        else:
            if not isinstance(stream, torch.cuda.Stream):
                handle = int(stream)   # 0: the default stream, for which ExternalStream makes another
                stream = (torch.cuda.ExternalStream(handle, device=torch.device("cuda", index)) if handle
                          else torch.cuda.default_stream(index))
            if stream.device_index != index:
                raise ValueError(f"the stream is on device {stream.device_index}, the operands on {index}")
            self._ctx = torch.cuda.stream(stream)
            self.handle = stream.cuda_stream
        if stream is None:
            self.handle = _raw_stream(index)

    def __enter__(self) -> int:
        self._ctx.__enter__()
        return self.handle

    def __exit__(self, *exc):
        return self._ctx.__exit__(*exc)


def _run(index: int, stream, fn, *args):
    """fn(*args, stream handle) on device `index`, switching to it (or to the
    stream) only when it is not the current one."""
    if stream is None and _GET_DEVICE() == index:
        return fn(*args, _raw_stream(index))
    with _Call(index, stream) as handle:
        return fn(*args, handle)


def _values(x, name: str, dims: int | None = None) -> int:
    """dtype code of a tensor of values."""
    if not isinstance(x, torch.Tensor) or x.get_device() < 0:
        raise ValueError(f"{name} must be a tensor on a HIP device")
    dt = DTYPES.get(x.dtype)
    if dt is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16")
    if dims is not None and x.dim() != dims:
        raise ValueError(f"{name} must have {dims} axes, got {x.dim()}")
    return dt


def _result_type(dtype) -> int:
    dt = DTYPES.get(dtype)
    if dt is None:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    return dt


def _held_on(q, name: str, dims: int | None = None) -> int:
    """Device index of an Mx4."""
    if not isinstance(q, Mx4) or dims is not None and q.codes.dim() != dims:
        raise ValueError(f"{name} must be an Mx4" + ("" if dims is None else
                                                     " matrix" if dims == 2 else " batch of matrices"))
    index = q.codes.get_device()
    if index < 0:
        raise ValueError(f"{name} must be on a HIP device")
    return index


def _same(index: int, other: int, name: str) -> None:
    if index != other:
        raise ValueError(f"{name} is on another device than the first operand")


def _row_stride(x: torch.Tensor, name: str) -> int:
    """Elements between the rows of x [R, C], its columns being neighbours."""
    r, c = x.shape
    if x.is_contiguous():
        return c
    rs, cs = x.stride()
    if c > 1 and cs != 1 or r > 1 and rs < c:
        raise ValueError(f"the last axis of {name} must be contiguous and its rows apart")
    return rs if r > 1 else c


def _offsets(offsets, index: int) -> int:
    """Groups of an offsets tensor."""
    if not isinstance(offsets, torch.Tensor) or offsets.dtype != torch.int32 or offsets.dim() != 1 \
            or offsets.shape[0] < 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous int32 tensor of groups + 1 values")
    _same(index, offsets.get_device(), "offsets")
    return offsets.shape[0] - 1


# The workspaces' sizes are the library's to say, and go by sizes alone.
@functools.lru_cache(maxsize=4096)
def _matmul_workspace(m: int, n: int, k: int, values: bool) -> int:
    return int(load_mx4().ou_mx4_matmul_workspace_bytes(m, n, k, values))


@functools.lru_cache(maxsize=4096)
def _grouped_workspace(m: int, n: int, k: int, groups: int, values: bool) -> int:
    return int(load_mx4().ou_mx4_grouped_workspace_bytes(m, n, k, groups, values))


@functools.lru_cache(maxsize=4096)
def _grouped_columns(rows: int, groups: int) -> int:
    return int(load_mx4().ou_mx4_grouped_columns(rows, groups))


def _ptrs(q: Mx4 | None) -> tuple:
    return (None, None) if q is None else (q.codes.data_ptr(), q.scales.data_ptr())


def _do_quantize(x, dt, lead, batch, r, c, rs, bs, rows, transposed, handle):
    q = _empty((*lead, r), c, x.device) if rows else None
    qt = _empty((*lead, c), r, x.device) if transposed else None
    st = load_mx4().ou_mx4_quantize(dt, x.data_ptr(), batch, r, c, rs, bs, *_ptrs(q), *_ptrs(qt), handle)
    if st:
        _fail(st)
    return q, qt


def _quantize(x: torch.Tensor, rows: bool, transposed: bool, stream) -> tuple[Mx4 | None, Mx4 | None]:
    dt = _values(x, "x")
    if x.dim() < 2:
        raise ValueError("x must have two axes at least")
    *lead, r, c = x.shape
    if lead:
        if not x.is_contiguous():
            raise ValueError("a batch of matrices must be contiguous")
        return _run(x.get_device(), stream, _do_quantize, x, dt, lead, math.prod(lead), r, c, c, r * c, rows, transposed)
    if c > 1 and x.stride(1) != 1 and x.stride(0) == 1:
        # a transposed view: its rows are the columns of what lies in memory
        qt, q = _quantize(x.t(), transposed, rows, stream)
        return q, qt
    return _run(x.get_device(), stream, _do_quantize, x, dt, lead, 1, r, c, _row_stride(x, "x"), 0, rows, transposed)


def mx4_quantize(x: torch.Tensor, stream=None) -> Mx4:
    """x [..., R, C] (float32, float16 or bfloat16) in 4 bits along its last
    axis.  A matrix may have any row stride, or be the transposed view of
    one; a batch must be contiguous."""
    return _quantize(x, True, False, stream)[0]


def mx4_quantize_both(x: torch.Tensor, stream=None) -> tuple[Mx4, Mx4]:
    """(x along its last axis, x transposed along its rows): [..., R, C] and
    [..., C, R] in 4 bits, with one read of x."""
    return _quantize(x, True, True, stream)


def _do_quantize_grouped(x, dt, t, c, rs, offsets, groups, rows, handle):
    q = _empty((t,), c, x.device) if rows else None
    qt = _empty((c,), _grouped_columns(t, groups), x.device)
    st = load_mx4().ou_mx4_quantize_grouped(dt, x.data_ptr(), t, c, rs, offsets.data_ptr(), groups, *_ptrs(q),
                                            *_ptrs(qt), handle)
    if st:
        _fail(st)
    return q, qt


def mx4_quantize_grouped(x: torch.Tensor, offsets: torch.Tensor, rows: bool = True,
                         stream=None) -> tuple[Mx4 | None, Mx4]:
    """x [T, C] along its columns (None with rows=False) and, group by group,
    along its rows: group e is rows offsets[e]:offsets[e + 1] (int32, on the
    device), a matrix of its own padded to 128 rows (``ou_mx4_quantize_grouped``).
    Rows of no group are not quantised.  The operands of ``mx4_grouped_outer``."""
    dt = _values(x, "x", 2)
    index = x.get_device()
    groups = _offsets(offsets, index)
    t, c = x.shape
    return _run(index, stream, _do_quantize_grouped, x, dt, t, c, _row_stride(x, "x"), offsets, groups, rows)


def _do_dequantize(q, dtype, dt, out, handle):
    if out is None:
        out = torch.empty(q.shape, dtype=dtype, device=q.codes.device)
    rows = out.numel() // q.k if q.k else 0
    st = load_mx4().ou_mx4_dequantize(dt, q.codes.data_ptr(), q.scales.data_ptr(), rows, q.k, out.data_ptr(), q.k,
                                      handle)
    if st:
        _fail(st)
    return out


def mx4_dequantize(q: Mx4, dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """The values that q holds, in ``dtype`` (or in ``out``, contiguous)."""
    index = _held_on(q, "q")
    if out is None:
        dt = _result_type(dtype)
    else:
        dt = _values(out, "out")
        _same(index, out.get_device(), "out")
        if out.shape != q.shape or not out.is_contiguous():
            raise ValueError(f"out must be contiguous, of shape {list(q.shape)}")
    return _run(index, stream, _do_dequantize, q, dtype, dt, out)


def _output(out, rows: int, n: int, dtype, index: int) -> tuple[int, int]:
    """dtype code and row stride of a result, given or to be made."""
    if out is None:
        return _result_type(dtype), n
    dt = _values(out, "out", 2)
    _same(index, out.get_device(), "out")
    if tuple(out.shape) != (rows, n):
        raise ValueError(f"out must have shape [{rows}, {n}], got {list(out.shape)}")
    return dt, _row_stride(out, "out")


def _left(a, k: int) -> tuple[bool, int, torch.dtype, int, int, int]:
    """(given as values, device index, default dtype of a result, rows, dtype
    code, row stride) of a left operand."""
    if isinstance(a, Mx4):
        index = _held_on(a, "the left operand", 2)
        m, have, values, dtype, dt, rs = a.codes.shape[0], a.k, False, torch.bfloat16, 0, 0
    else:
        dt = _values(a, "the left operand", 2)
        m, have = a.shape
        index, values, dtype, rs = a.get_device(), True, a.dtype, _row_stride(a, "the left operand")
    if have != k:
        raise ValueError(f"the operands contract {have} and {k} columns")
    return values, index, dtype, m, dt, rs


def _do_matmul(a, values, dt, rs, m, b, n, k, dtype, od, out, stride, offsets, groups, handle):
    """Both products: grouped with offsets."""
    lib = load_mx4()
    device = b.codes.device
    zero_rest = out is None
    if out is None:
        out = torch.empty((m, n), dtype=dtype, device=device)
    need = (_matmul_workspace(m, n, k, values) if offsets is None else _grouped_workspace(m, n, k, groups, values))
    ws = torch.empty(need, dtype=torch.uint8, device=device) if need > 0 else None
    tail = (ws.data_ptr() if ws is not None else None, need, handle)
    right = (b.codes.data_ptr(), b.scales.data_ptr(), n, k)
    if offsets is None:
        if values:
            st = lib.ou_mx4_matmul_values(dt, a.data_ptr(), m, rs, od, *right, out.data_ptr(), stride, *tail)
        else:
            st = lib.ou_mx4_matmul(od, a.codes.data_ptr(), a.scales.data_ptr(), m, *right, out.data_ptr(), stride, *tail)
    else:
        by = (offsets.data_ptr(), groups, out.data_ptr(), stride, zero_rest)
        if values:
            st = lib.ou_mx4_grouped_matmul_values(dt, a.data_ptr(), m, rs, od, *right, *by, *tail)
        else:
            st = lib.ou_mx4_grouped_matmul(od, a.codes.data_ptr(), a.scales.data_ptr(), m, *right, *by, *tail)
    if st:
        _fail(st)
    return out


def mx4_matmul(a, b: Mx4, dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """a b^T: a [M, K] as values (quantised along K on the way, in the same
    call) or as Mx4, b an Mx4 [N, K].  The result is [M, N] of ``dtype``
    (default: a's, bfloat16 for an Mx4), or ``out`` (any row stride)."""
    on = _held_on(b, "b", 2)
    n, k = b.codes.shape[0], b.k
    values, index, default, m, dt, rs = _left(a, k)
    _same(index, on, "b")
    dtype = dtype or default
    od, stride = _output(out, m, n, dtype, index)
    return _run(index, stream, _do_matmul, a, values, dt, rs, m, b, n, k, dtype, od, out, stride, None, 0)


def mx4_grouped_matmul(a, b: Mx4, offsets: torch.Tensor, dtype: torch.dtype | None = None,
                       out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rows of a [T, K] (values or Mx4) by groups: rows offsets[e]:offsets[e + 1]
    times matrix e of b [E, N, K], transposed.  ``offsets``: E + 1 rising int32
    on the device, read there.  Rows of no group are 0 in a new result and left
    as they were in ``out``."""
    on = _held_on(b, "b", 3)
    (e, n), k = b.codes.shape[:2], b.k
    values, index, default, m, dt, rs = _left(a, k)
    _same(index, on, "b")
    groups = _offsets(offsets, index)
    if groups != e:
        raise ValueError(f"offsets name {groups} groups, b holds {e}")
    dtype = dtype or default
    od, stride = _output(out, m, n, dtype, index)
    return _run(index, stream, _do_matmul, a, values, dt, rs, m, b, n, k, dtype, od, out, stride, offsets, groups)


def _do_outer(at, bt, offsets, groups, rows, dtype, dt, handle):
    m, n = at.codes.shape[0], bt.codes.shape[0]
    out = torch.empty((groups, m, n), dtype=dtype, device=at.codes.device)
    st = load_mx4().ou_mx4_grouped_outer(dt, *_ptrs(at), m, *_ptrs(bt), n, rows, offsets.data_ptr(), groups,
                                         out.data_ptr(), handle)
    if st:
        _fail(st)
    return out


def mx4_grouped_outer(at: Mx4, bt: Mx4, offsets: torch.Tensor, rows: int, dtype: torch.dtype = torch.bfloat16,
                      stream=None) -> torch.Tensor:
    """[E, M, N]: for every group the sum over its rows of a's row times b's,
    from the transposed forms [M, *] and [N, *] that ``mx4_quantize_grouped``
    made of matrices of ``rows`` rows with the same offsets."""
    index = _held_on(at, "at", 2)
    _same(index, _held_on(bt, "bt", 2), "bt")
    dt = _result_type(dtype)
    groups = _offsets(offsets, index)
    p = _grouped_columns(rows, groups)
    if at.k != p or bt.k != p:
        raise ValueError(f"{rows} rows in {groups} groups are held in {p} columns: got {at.k} and {bt.k}")
    return _run(index, stream, _do_outer, at, bt, offsets, groups, rows, dtype, dt)


# ------------------------------------------------------------------ layers

class Mx4Weight:
    """The 4-bit forms of a weight [N, K] or [E, N, K] for the layers below:
    ``q`` along K (forward) and ``qt`` along N (the input's gradient).
    ``refresh()`` quantises the weight's present values into them; an optimizer
    that it is given to (``attach_mx4``) does so after every step, so that the
    passes in between (micro-batches) read the 4-bit forms alone.  The layers
    use the forms as they are and warn where the weight was written since:
    by torch, by assigning another one, or by a step of a collection optimizer
    that the forms are not attached to.  (Single updates and plans, and writes
    through ``weight.data``, are not seen.)"""

    live = weakref.WeakSet()
    _made_of = None   # address and version of the weight that the forms are of

    def __init__(self, weight: torch.Tensor):
        if weight.dim() not in (2, 3):
            raise ValueError("weight must be [N, K] or [E, N, K]")
        if not weight.is_contiguous():
            raise ValueError("weight must be contiguous")
        self.weight = weight
        self.version = 0   # of the forms: a backward pass refuses later ones than its forward pass read
        self.q, self.qt = mx4_quantize_both(weight.detach())
        self._made_of = self._weight_state()
        Mx4Weight.live.add(self)

    def _weight_state(self) -> tuple[int, int]:
        w = self.weight
        return w.data_ptr(), 0 if w.is_inference() else w._version

    def _warn_if_stale(self) -> None:
        if self._made_of != self._weight_state():
            warnings.warn("the weight was written after its 4-bit forms were made, and the layer uses the forms: "
                          "refresh() brings them up to date", stacklevel=4)

    def _check_forms(self) -> None:
        """Raises if the weight has taken another shape or device than its
        forms (a new ``weight`` or ``weight.data``): the kernels take sizes
        from the one and addresses from the others."""
        *lead, r, c = shape = self.weight.shape
        q, qt, index = self.q, self.qt, self.weight.get_device()
        if q.k != c or q.codes.shape[:-1] != shape[:-1] or qt.k != r or qt.codes.shape[:-1] != (*lead, c):
            raise ValueError(f"the 4-bit forms are of a weight of shape {list(q.shape)}, the weight is now "
                             f"{list(shape)}: make a new Mx4Weight")
        if q.codes.get_device() != index or qt.codes.get_device() != index:
            raise ValueError("the 4-bit forms are on another device than the weight: make a new Mx4Weight")

    def refresh(self, stream=None) -> None:
        """Quantise the weight's present values into the same buffers."""
        self._check_forms()
        w = self.weight.detach()
        dt = _values(w, "weight")
        if not w.is_contiguous():
            raise ValueError("the weight changed its layout")
        _run(w.get_device(), stream, self._refresh, w, dt)
        self.version += 1
        self._made_of = self._weight_state()

    def _refresh(self, w, dt, handle):
        *lead, r, c = w.shape
        st = load_mx4().ou_mx4_quantize(dt, w.data_ptr(), math.prod(lead), r, c, c, r * c, *_ptrs(self.q),
                                        *_ptrs(self.qt), handle)
        if st:
            _fail(st)


class _Room:
    """Places of held matrices in one buffer: the layers' own forms, which
    nobody else sees, are spared a tensor for each of their parts."""

    __slots__ = ("bytes",)

    def __init__(self):
        self.bytes = 0

    def form(self, rows: int, columns: int) -> tuple[int, int]:
        """Offsets of codes and scales of `rows` rows of padded `columns`."""
        codes = self.bytes
        scales = codes + rows * columns // 2
        self.bytes = scales + -(-rows * columns // MX4_BLOCK // 16) * 16
        return codes, scales

    def make(self, device) -> tuple[torch.Tensor, int]:
        buf = torch.empty(self.bytes, dtype=torch.uint8, device=device)
        return buf, buf.data_ptr()


def _rows_apart(x: torch.Tensor) -> torch.Tensor:
    """x, or a copy whose columns are neighbours and whose rows do not overlap."""
    r, c = x.shape
    return x if x.is_contiguous() or (c <= 1 or x.stride(1) == 1) and (r <= 1 or x.stride(0) >= c) else x.contiguous()


def _place(base, offsets):
    return (None, None) if offsets is None else (base + offsets[0], base + offsets[1])


class _Layer(torch.autograd.Function):
    """Both layers; offsets: None for the plain one."""

    @staticmethod
    def forward(ctx, x, w, offsets, held):
        return _run(x.get_device(), None, _Layer._forward, ctx, _rows_apart(x), w, offsets, held)

    @staticmethod
    def _forward(ctx, x, w, offsets, held, handle):
        lib, device = load_mx4(), x.device
        need_x, need_w = ctx.needs_input_grad[:2]
        m, k = x.shape
        n, groups = w.shape[-2], w.shape[0] if offsets is not None else 1
        pk, rs = _columns(k), _row_stride(x, "x")
        xd, off = DTYPES[x.dtype], None if offsets is None else offsets.data_ptr()
        held_m = _columns(m) if offsets is None else _grouped_columns(m, groups)
        temp, kept = _Room(), _Room()
        wq = temp.form(groups * n, pk) if held is None else None
        wt = kept.form(groups * k, _columns(n)) if held is None and need_x else None
        xq = temp.form(m, pk) if need_w else None
        xt = kept.form(k, held_m) if need_w else None
        grow = 0
        if not need_w:   # x goes in as values
            grow = _matmul_workspace(m, n, k, True) if off is None else _grouped_workspace(m, n, k, groups, True)
        ws = temp.bytes
        temp.bytes += grow
        buf, at = temp.make(device)
        keep, kp = kept.make(device)
        st = 0
        if held is None:
            st = lib.ou_mx4_quantize(DTYPES[w.dtype], w.data_ptr(), groups, n, k, k, n * k, *_place(at, wq), *_place(kp, wt),
                                     handle)
            right = _place(at, wq)
        else:
            right = _ptrs(held.q)
        if st:
            _fail(st)
        y = torch.empty((m, n), dtype=x.dtype, device=device)
        if need_w:
            if off is None:
                st = lib.ou_mx4_quantize(xd, x.data_ptr(), 1, m, k, rs, 0, *_place(at, xq), *_place(kp, xt), handle)
            else:
                st = lib.ou_mx4_quantize_grouped(xd, x.data_ptr(), m, k, rs, off, groups, *_place(at, xq),
                                                 *_place(kp, xt), handle)
            if st:
                _fail(st)
        _multiply(lib, xd, None if need_w else x, rs, _place(at, xq), m, xd, right, n, k, off, groups, y, at + ws, grow,
                  handle)
        ctx.shape = (m, n, k, groups, held_m)
        ctx.types = (x.dtype, w.dtype)
        ctx.wt, ctx.xt = wt, xt
        ctx.held = held if need_x else None
        if ctx.held is not None:
            ctx.version, ctx.qt = held.version, held.qt   # the form that the shapes were checked against
        # as saved tensors: freed by the backward pass, seen by hooks and checkpoints
        ctx.save_for_backward(keep if kept.bytes else None, offsets)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        if ctx.held is not None and ctx.held.version != ctx.version:
            raise RuntimeError("the Mx4Weight was refreshed between the forward and the backward pass")
        return _run(dy.get_device(), None, _Layer._backward, ctx, _rows_apart(dy))

    @staticmethod
    def _backward(ctx, dy, handle):
        lib, device = load_mx4(), dy.device
        need_x, need_w = ctx.needs_input_grad[:2]
        m, n, k, groups, held_m = ctx.shape
        x_dtype, w_dtype = ctx.types
        keep, offsets = ctx.saved_tensors
        off = None if offsets is None else offsets.data_ptr()
        pn, rs, yd = _columns(n), _row_stride(dy, "the gradient"), DTYPES[dy.dtype]
        kp = 0 if keep is None else keep.data_ptr()
        temp = _Room()
        dq = temp.form(m, pn) if need_x and need_w else None
        dt = temp.form(n, held_m) if need_w else None
        ws = temp.bytes
        grow = 0
        if not need_w:
            grow = _matmul_workspace(m, k, n, True) if off is None else _grouped_workspace(m, k, n, groups, True)
            temp.bytes += grow
        buf, at = temp.make(device)
        dx = dw = None
        if need_w:
            if off is None:
                st = lib.ou_mx4_quantize(yd, dy.data_ptr(), 1, m, n, rs, 0, *_place(at, dq), *_place(at, dt), handle)
            else:
                st = lib.ou_mx4_quantize_grouped(yd, dy.data_ptr(), m, n, rs, off, groups, *_place(at, dq),
                                                 *_place(at, dt), handle)
            if st:
                _fail(st)
            if off is None:
                dw = torch.empty((n, k), dtype=w_dtype, device=device)
                _multiply(lib, 0, None, 0, _place(at, dt), n, DTYPES[w_dtype], _place(kp, ctx.xt), k, m, None, 0, dw, None,
                          0, handle)
            else:
                dw = torch.empty((groups, n, k), dtype=w_dtype, device=device)
                st = lib.ou_mx4_grouped_outer(DTYPES[w_dtype], *_place(at, dt), n, *_place(kp, ctx.xt), k, m, off, groups,
                                              dw.data_ptr(), handle)
                if st:
                    _fail(st)
        if need_x:
            dx = torch.empty((m, k), dtype=x_dtype, device=device)
            right = _ptrs(ctx.qt) if ctx.held is not None else _place(kp, ctx.wt)
            _multiply(lib, yd, None if need_w else dy, rs, _place(at, dq), m, DTYPES[x_dtype], right, k, n, off, groups, dx,
                      at + ws, grow, handle)
        return dx, dw, None, None


def _multiply(lib, xd, x, rs, left, m, od, right, n, k, off, groups, out, ws, need, handle):
    """A product of a layer: x as values, or the held matrix `left`."""
    ws = ws if need else None
    tail = (out.data_ptr(), n)
    if off is None:
        if x is None:
            st = lib.ou_mx4_matmul(od, *left, m, *right, n, k, *tail, None, 0, handle)
        else:
            st = lib.ou_mx4_matmul_values(xd, x.data_ptr(), m, rs, od, *right, n, k, *tail, ws, need, handle)
    elif x is None:
        st = lib.ou_mx4_grouped_matmul(od, *left, m, *right, n, k, off, groups, *tail, 1, None, 0, handle)
    else:
        st = lib.ou_mx4_grouped_matmul_values(xd, x.data_ptr(), m, rs, od, *right, n, k, off, groups, *tail, 1, ws, need,
                                              handle)
    if st:
        _fail(st)


def _layer_operands(x, w, dims: int):
    held = w if isinstance(w, Mx4Weight) else None
    weight = held.weight if held is not None else w
    if held is not None:
        held._check_forms()
    _values(x, "x")
    _values(weight, "w", dims)
    _same(x.get_device(), weight.get_device(), "w")
    if not weight.is_contiguous():
        raise ValueError("w must be contiguous")
    if x.dim() < 2 or x.shape[-1] != weight.shape[-1]:
        raise ValueError(f"x must be [..., {weight.shape[-1]}], got {list(x.shape)}")
    if held is not None:
        held._warn_if_stale()
    return held, weight


def _apply(x, weight, offsets, held):
    if not torch.is_grad_enabled():
        # the forward pass sees what requires gradients, not whether any are
        # recorded: without, x goes in as values and no transposed form is made
        x, weight = x.detach(), weight.detach()
    return _Layer.apply(x, weight, offsets, held)


def mx4_linear(x: torch.Tensor, w) -> torch.Tensor:
    """x w^T with its gradients, the three products in 4 bits: with Q the
    rounding along the contracted axis (in blocks of 32),
        y = Q(x) Q(w)^T,  dx = Q(dy) Q(w^T)^T,  dw = Q(dy^T) Q(x^T)^T,
    each summed in binary32 and rounded once to the dtype of x (y, dx) or w
    (dw).  x is [..., K], w [N, K] or an ``Mx4Weight`` (its 4-bit forms are
    used as they are, with a warning if the weight was written since; its
    ``weight`` gets the gradient; it must not be refreshed before the backward
    pass).  For the backward pass 4-bit forms
    are kept, not x."""
    held, weight = _layer_operands(x, w, 2)
    if x.dim() == 2:
        return _apply(x, weight, None, held)
    y = _apply(x.reshape(math.prod(x.shape[:-1]), x.shape[-1]), weight, None, held)
    return y.view(*x.shape[:-1], weight.shape[0])


def mx4_grouped_linear(x: torch.Tensor, w, offsets: torch.Tensor) -> torch.Tensor:
    """``mx4_linear`` by groups: rows offsets[e]:offsets[e + 1] of x [T, K]
    with expert e of w [E, N, K] (or an ``Mx4Weight``).  Rows of no group give
    0 and get 0; an expert without rows gets a gradient of 0."""
    held, weight = _layer_operands(x, w, 3)
    if x.dim() != 2:
        raise ValueError("x must be [T, K]")
    if _offsets(offsets, x.get_device()) != weight.shape[0]:
        raise ValueError(f"offsets name {offsets.shape[0] - 1} groups, w holds {weight.shape[0]}")
    return _apply(x, weight, offsets, held)
