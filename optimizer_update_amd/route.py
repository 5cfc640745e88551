"""Routing to experts: which experts a token's rows go to and with what
weights, the order of the rows by expert, their dispatch and their weighted
combination, with the gradients (binding of ``liboptimizer_experts.so``,
``include/optimizer_experts.h``).

    w, ids = route_topk(logits, k)            weights [T, k] and experts [T, k]
    order = route_order(ids, experts)         RouteOrder: offsets, slots, places
    rows = route_dispatch(x, order)           the rows of x [T, H], by expert: [T k, H]
    y = mx4_grouped_linear(rows, we, order.offsets)
    out = route_combine(y, w, order, add=x)   [T, H]: add + the weighted sums
    bias = route_balance(bias, order, rate)   the bias of the choice, towards equal loads

Nothing is read back to the host: the products by expert
(``mx4_grouped_linear``, ``mx4_grouped_matmul``, ``int4_grouped_matmul``) take
``order.offsets`` on the device.  ``route_topk``, ``route_dispatch`` and
``route_combine`` record gradients (of the logits; of x; of y, the weights and
what is added); experts are constants of them.  Functions check and marshal
arguments; all arithmetic runs in the HIP kernels.  Every call goes to the
current stream of the operands' device, or to ``stream`` where there is one (a
stream of that device or its handle, 0 being the default stream); results and
workspaces are allocated on that stream.  An operand of another stream must
stay until the call's work is done (``record_stream``).  A result that is given
(``out``) counts as written for autograd, as one of torch's own in-place
operations does.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

from . import DTYPES, _lib
from .mx4 import _row_stride, _rows_apart, _run, _same, _values

HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(HERE, "liboptimizer_experts.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "optimizer_experts.h")

SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_SCORES = {"best": 0, "best two": 1}
_experts = None
_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8


def load_experts(path: str = LIBRARY) -> ctypes.CDLL:
    """Load the library of the operators around experts (raises if it is missing)."""
    global _experts
    if _experts is not None and path == LIBRARY:
        return _experts
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built; run __graft_entry__.build() "
                          "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    i32, i64, f32, vp = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
    for name, res, args in (
            ("ou_route_topk", i32, [i32, vp, i64, i32, i64, i32, vp, i32, i32, i32, i32, f32, vp, i32, vp, vp, vp]),
            ("ou_route_topk_backward", i32, [i32, vp, i64, i32, i64, i32, i32, f32, vp, vp, i32, vp, vp]),
            ("ou_route_order_workspace_bytes", i64, [i64, i32]),
            ("ou_route_order", i32, [vp, i64, i32, vp, vp, vp, vp, i64, vp]),
            ("ou_route_dispatch", i32, [i32, vp, i64, i64, i64, i32, vp, vp, vp, i64, i32, vp]),
            ("ou_route_combine", i32, [i32, vp, i64, i64, i64, i32, vp, vp, vp, i64, vp, i64, vp]),
            ("ou_route_combine_backward", i32, [i32, vp, i64, i64, i64, i32, vp, i64, vp, vp, vp, vp, vp, vp]),
            ("ou_route_balance", i32, [vp, vp, i32, f32, vp, vp]),
            ("ou_int4_quantize", i32, [i32, vp, i64, i64, i64, i32, i32, vp, vp, vp, vp]),
            ("ou_int4_dequantize", i32, [i32, vp, i32, vp, vp, i64, i64, i32, vp, i64, vp]),
            ("ou_int4_matmul", i32, [i32, vp, i64, i64, i32, vp, i32, vp, vp, i64, i64, i32, vp, i64, vp]),
            ("ou_int4_grouped_matmul", i32, [i32, vp, i64, i64, i32, vp, i32, vp, vp, i64, i64, i32, vp, i32, vp, i64, i32,
                                             vp]),
            ("ou_experts_last_error", ctypes.c_char_p, [])):
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    if path == LIBRARY:
        _install_fast(lib)
        _experts = lib
    return lib


# Entry points that the CPython module _fast_experts also exposes.
FAST_ENTRY_POINTS = ("ou_route_topk", "ou_route_topk_backward", "ou_route_order", "ou_route_dispatch", "ou_route_combine",
                     "ou_route_combine_backward", "ou_route_balance", "ou_int4_matmul", "ou_int4_grouped_matmul")


def _install_fast(lib: ctypes.CDLL) -> None:
    """Route the calls of the in-tree library through _fast_experts when it is
    built: the same functions and positional arguments, converted in C."""
    try:
        from . import _fast_experts
    except ImportError:
        return
    for name in FAST_ENTRY_POINTS:
        setattr(lib, name, getattr(_fast_experts, name))


def _fail(status: int) -> None:
    raise _lib.OptimizerUpdateError(status, load_experts().ou_experts_last_error().decode(errors="replace"))


def _written(out: torch.Tensor) -> torch.Tensor:
    """``out``, for torch's check of saved tensors a written one."""
    torch.autograd.graph.increment_version(out)
    return out


def _whole(x, name: str, dims: int) -> None:
    if not isinstance(x, torch.Tensor) or x.dtype != torch.int32 or x.dim() != dims or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {dims} axes")


# ------------------------------------------------------------------ the choice

class _Topk(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, bias, mask, k, call):
        w, ids = _run(logits.get_device(), None, _Topk._forward, logits, bias, mask, k, call)
        ctx.k, ctx.call = k, call
        ctx.save_for_backward(logits, ids)
        ctx.mark_non_differentiable(ids)
        ctx.set_materialize_grads(False)
        return w, ids

    @staticmethod
    def _forward(logits, bias, mask, k, call, handle):
        t, e = logits.shape
        scores, groups, top_groups, group_score, renorm, scale = call
        w = logits.new_empty((t, k), dtype=_F32)
        ids = logits.new_empty((t, k), dtype=_I32)
        st = load_experts().ou_route_topk(
            DTYPES[logits.dtype], logits.data_ptr(), t, e, _row_stride(logits, "logits"), scores,
            None if bias is None else bias.data_ptr(), groups, top_groups, group_score, renorm, scale,
            None if mask is None else mask.data_ptr(), k, w.data_ptr(), ids.data_ptr(), handle)
        if st:
            _fail(st)
        return w, ids

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dw, _):
        if dw is None:
            return None, None, None, None, None
        logits, ids = ctx.saved_tensors
        return (_run(dw.get_device(), None, _Topk._backward, ctx, logits, ids, dw.contiguous()), None, None, None, None)

    @staticmethod
    def _backward(ctx, logits, ids, dw, handle):
        t, e = logits.shape
        scores, _, _, _, renorm, scale = ctx.call
        dx = logits.new_empty((t, e))
        st = load_experts().ou_route_topk_backward(
            DTYPES[logits.dtype], logits.data_ptr(), t, e, _row_stride(logits, "logits"), scores, renorm, scale,
            ids.data_ptr(), dw.data_ptr(), ctx.k, dx.data_ptr(), handle)
        if st:
            _fail(st)
        return dx


def route_topk(logits: torch.Tensor, k: int, *, scores: str = "softmax", bias: torch.Tensor | None = None,
               groups: int = 1, top_groups: int = 1, group_score: str = "best two", renormalize: bool = True,
               scale: float = 1.0, mask: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(weights, ids): the k experts of each token and their weights, float32
    and int32 [T, k], in falling order of the choice.  ``logits`` [T, E] has
    any row stride.  Scores s are the softmax of a token's logits or their
    logistic function (``scores="sigmoid"``); the choice goes by s + ``bias``
    (float32 [E], a constant), ties to the lower expert.  With ``groups``, the experts are as many equal parts; a
    part counts by its largest choice or the sum of its two largest
    (``group_score``: "best", "best two"), and experts come from the
    ``top_groups`` that count most.  Weights are ``scale`` times the s of the
    chosen, with ``renormalize`` divided by their sum.  An expert whose logit
    is -inf is absent; a token has ids of -1 with weights of 0 where experts
    run out, or everywhere with a False in ``mask`` (bool [T], a padded
    batch).  Gradients: of the logits, by the weights.  The backward pass
    reads the logits again."""
    _values(logits, "logits", 2)
    t, e = logits.shape
    if scores not in SCORES or group_score not in GROUP_SCORES:
        raise ValueError(f"scores is one of {list(SCORES)}, group_score one of {list(GROUP_SCORES)}")
    index = logits.get_device()
    if bias is not None:
        if not isinstance(bias, torch.Tensor) or bias.dtype != torch.float32 or tuple(bias.shape) != (e,) or not bias.is_contiguous():
            raise ValueError(f"bias must be a contiguous float32 tensor of {e} values")
        _same(index, bias.get_device(), "bias")
        if bias.requires_grad:
            bias = bias.detach()
    if mask is not None:
        if not isinstance(mask, torch.Tensor) or mask.dtype != torch.bool or tuple(mask.shape) != (t,) or not mask.is_contiguous():
            raise ValueError(f"mask must be a contiguous bool tensor of {t} values")
        _same(index, mask.get_device(), "mask")
    call = (SCORES[scores], int(groups), int(top_groups), GROUP_SCORES[group_score], int(bool(renormalize)), float(scale))
    logits = _rows_apart(logits)
    if logits.requires_grad and torch.is_grad_enabled():
        return _Topk.apply(logits, bias, mask, int(k), call)
    return _run(index, None, _Topk._forward, logits, bias, mask, int(k), call)


# ------------------------------------------------------------------ the order

class RouteOrder:
    """The rows of a batch's slots by expert.  Slot t * k + j is token t's
    j-th choice; ``offsets`` [E + 1]: expert e has rows
    offsets[e]:offsets[e + 1]; ``slots`` [T k]: the slot of each row, -1
    behind the last expert's; ``places`` [T, k]: the row of each slot, -1 for
    those of no expert.  All int32, contiguous, on one device."""

    __slots__ = ("offsets", "slots", "places")

    def __init__(self, offsets: torch.Tensor, slots: torch.Tensor, places: torch.Tensor):
        _whole(offsets, "offsets", 1)
        _whole(slots, "slots", 1)
        _whole(places, "places", 2)
        if offsets.shape[0] < 2 or slots.shape[0] != places.numel():
            raise ValueError(f"offsets hold experts + 1 values, slots as many as places: got {list(offsets.shape)}, "
                             f"{list(slots.shape)} and {list(places.shape)}")
        if not offsets.get_device() == slots.get_device() == places.get_device():
            raise ValueError("offsets, slots and places must be on one device")
        self.offsets, self.slots, self.places = offsets, slots, places

    @property
    def experts(self) -> int:
        return self.offsets.shape[0] - 1

    @property
    def tokens(self) -> int:
        return self.places.shape[0]

    @property
    def choices(self) -> int:
        return self.places.shape[1]

    @property
    def device(self) -> torch.device:
        return self.offsets.device

    def __repr__(self) -> str:
        return f"RouteOrder(tokens={self.tokens}, choices={self.choices}, experts={self.experts}, device={self.device})"


def _held_order(offsets, slots, places) -> RouteOrder:
    """A RouteOrder of tensors made here."""
    order = RouteOrder.__new__(RouteOrder)
    order.offsets, order.slots, order.places = offsets, slots, places
    return order


@functools.lru_cache(maxsize=4096)
def _order_workspace(slots: int, experts: int) -> int:
    return int(load_experts().ou_route_order_workspace_bytes(slots, experts))


def _do_order(ids, experts, handle):
    n = ids.numel()
    need = _order_workspace(n, experts)
    new = ids.new_empty
    offsets, slots, places = new(experts + 1), new(n), new(ids.shape)
    ws = new(need, dtype=_U8) if need > 0 else None
    st = load_experts().ou_route_order(ids.data_ptr(), n, experts, offsets.data_ptr(), slots.data_ptr(), places.data_ptr(),
                                       None if ws is None else ws.data_ptr(), need, handle)
    if st:
        _fail(st)
    return _held_order(offsets, slots, places)


def route_order(ids: torch.Tensor, experts: int, stream=None) -> RouteOrder:
    """The slots of ids [T, k] (int32) sorted by expert, stable.  Ids outside
    [0, experts) are of no expert."""
    _whole(ids, "ids", 2)
    index = ids.get_device()
    if index < 0:
        raise ValueError("ids must be on a HIP device")
    return _run(index, stream, _do_order, ids, int(experts))


def _ordered(order, index: int) -> None:
    if not isinstance(order, RouteOrder):
        raise ValueError("order must be a RouteOrder")
    _same(index, order.offsets.get_device(), "order")


def _do_balance(bias, order, rate, out, handle):
    made = torch.empty_like(bias) if out is None else out
    st = load_experts().ou_route_balance(bias.data_ptr(), order.offsets.data_ptr(), order.experts, rate, made.data_ptr(),
                                         handle)
    if st:
        _fail(st)
    return made if out is None else _written(out)


def route_balance(bias: torch.Tensor, order: RouteOrder, rate: float, out: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """bias + rate * sign(mean load - load): the bias (float32 [E]) of the
    next step's choice, ``rate`` nearer to equal loads of the experts.  ``out``
    may be ``bias`` itself."""
    for x, name in ((bias, "bias"), (out, "out")):
        if x is not None and (not isinstance(x, torch.Tensor) or x.dtype != torch.float32 or x.dim() != 1
                              or not x.is_contiguous() or x.get_device() < 0):
            raise ValueError(f"{name} must be a contiguous float32 tensor of one axis on a HIP device")
    index = bias.get_device()
    _ordered(order, index)
    if out is not None:
        _same(index, out.get_device(), "out")
    if bias.shape[0] != order.experts or out is not None and out.shape != bias.shape:
        raise ValueError(f"bias and out must hold {order.experts} values")
    return _run(index, stream, _do_balance, bias.detach(), order, float(rate), out)


# ------------------------------------------------------------------ rows

def _do_dispatch(x, order, out, handle):
    (t, h), k = x.shape, order.places.shape[1]
    given = out is not None
    if given:
        stride, rest = _row_stride(out, "out"), 0
    else:
        out, stride, rest = x.new_empty((t * k, h)), h, 1
    st = load_experts().ou_route_dispatch(DTYPES[x.dtype], x.data_ptr(), t, h, _row_stride(x, "x"), k,
                                          order.slots.data_ptr(), order.places.data_ptr(), out.data_ptr(), stride, rest,
                                          handle)
    if st:
        _fail(st)
    return _written(out) if given else out


def _do_combine(y, w, order, add, out, handle):
    (t, k), h = order.places.shape, y.shape[1]
    given = out is not None
    if given:
        stride = _row_stride(out, "out")
    else:
        out, stride = y.new_empty((t, h)), h
    st = load_experts().ou_route_combine(
        DTYPES[y.dtype], y.data_ptr(), t, h, _row_stride(y, "y"), k, None if w is None else w.data_ptr(),
        order.places.data_ptr(), None if add is None else add.data_ptr(), 0 if add is None else _row_stride(add, "add"),
        out.data_ptr(), stride, handle)
    if st:
        _fail(st)
    return _written(out) if given else out


def _do_combine_backward(dout, y, w, order, need_y, need_w, handle):
    t, h = dout.shape
    k = order.places.shape[1]
    dy = dout.new_empty((t * k, h)) if need_y else None
    dw = dout.new_empty((t, k), dtype=_F32) if need_w else None
    st = load_experts().ou_route_combine_backward(
        DTYPES[dout.dtype], dout.data_ptr(), t, h, _row_stride(dout, "the gradient"), k,
        y.data_ptr() if need_w else None, _row_stride(y, "y") if need_w else 0, w.data_ptr() if need_y else None,
        order.slots.data_ptr(), order.places.data_ptr(), dy.data_ptr() if need_y else None,
        dw.data_ptr() if need_w else None, handle)
    if st:
        _fail(st)
    return dy, dw


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, order):
        ctx.save_for_backward(order.offsets, order.slots, order.places)
        return _run(x.get_device(), None, _do_dispatch, x, order, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        order = _held_order(*ctx.saved_tensors)
        return _run(dy.get_device(), None, _do_combine, _rows_apart(dy), None, order, None, None), None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, w, add, order):
        need_y, need_w, _ = ctx.needs_input_grad[:3]
        ctx.save_for_backward(y if need_w else None, w if need_y else None, order.offsets, order.slots, order.places)
        return _run(y.get_device(), None, _do_combine, y, w, order, add, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        y, w, *order = ctx.saved_tensors
        need_y, need_w, need_add = ctx.needs_input_grad[:3]
        dy = dw = None
        if need_y or need_w:
            dy, dw = _run(dout.get_device(), None, _do_combine_backward, _rows_apart(dout), y, w, _held_order(*order),
                          need_y, need_w)
        return dy, dw, dout if need_add else None, None


def _output_like(out, rows: int, x: torch.Tensor, inputs) -> None:
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (*inputs, out)):
        raise ValueError("gradients are not recorded into out")
    if not isinstance(out, torch.Tensor) or out.dtype != x.dtype or tuple(out.shape) != (rows, x.shape[1]):
        raise ValueError(f"out must be {x.dtype} of shape [{rows}, {x.shape[1]}]")
    _same(x.get_device(), out.get_device(), "out")
    _row_stride(out, "out")


def route_dispatch(x: torch.Tensor, order: RouteOrder, out: torch.Tensor | None = None) -> torch.Tensor:
    """The rows of x [T, H] by expert, [T k, H]: row p is that of token
    ``order.slots[p] // k``.  Rows of no slot are 0 in a new result and left as
    they were in ``out`` (any row stride; no gradients are recorded then)."""
    _values(x, "x", 2)
    index = x.get_device()
    _ordered(order, index)
    if x.shape[0] != order.places.shape[0]:
        raise ValueError(f"x has {x.shape[0]} rows, the order {order.tokens} tokens")
    if out is not None:
        _output_like(out, order.slots.shape[0], x, (x,))
    x = _rows_apart(x)
    if x.requires_grad and torch.is_grad_enabled():
        return _Dispatch.apply(x, order)
    return _run(index, None, _do_dispatch, x, order, out)


def route_combine(y: torch.Tensor, weights: torch.Tensor, order: RouteOrder, add: torch.Tensor | None = None,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """add + the rows of y [T k, H] (by expert) summed for each token with
    ``weights`` (float32 [T, k]), [T, H]: in binary32, rounded once.  ``add``
    has y's dtype.  Rows of no slot are not read.  With ``out`` (any row
    stride) no gradients are recorded."""
    _values(y, "y", 2)
    index = y.get_device()
    _ordered(order, index)
    t, k = order.places.shape
    if y.shape[0] != t * k:
        raise ValueError(f"y has {y.shape[0]} rows, the order {t * k} slots")
    if not isinstance(weights, torch.Tensor) or weights.dtype != torch.float32 or weights.shape != order.places.shape:
        raise ValueError(f"weights must be float32 of shape [{t}, {k}]")
    _same(index, weights.get_device(), "weights")
    if add is not None:
        if not isinstance(add, torch.Tensor) or add.dtype != y.dtype or tuple(add.shape) != (t, y.shape[1]):
            raise ValueError(f"add must be {y.dtype} of shape [{t}, {y.shape[1]}]")
        _same(index, add.get_device(), "add")
    if out is not None:
        _output_like(out, t, y, (y, weights, add))
    y, weights = _rows_apart(y), weights.contiguous()
    if add is not None:
        add = _rows_apart(add)
    if (y.requires_grad or weights.requires_grad or add is not None and add.requires_grad) and torch.is_grad_enabled():
        return _Combine.apply(y, weights, add, order)
    return _run(index, None, _do_combine, y, weights, order, add, out)
