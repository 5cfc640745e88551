"""GPU: routing to experts against its definition in 64 bits
(tests/experts_reference.py).  Experts, orders and copies are compared for
equality, sums within the bounds derived there."""
import numpy as np
import pytest
import torch

import optimizer_update_amd as ou
from tests import experts_reference as R

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
DTYPES = [F32, F16, BF16]
INF, NAN = float("inf"), float("nan")


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _near(got, want, bound, dtype=F32):
    got = R.host(got)
    ok = np.abs(got - want) <= bound + np.abs(want) * (R.step(dtype) if dtype != F32 else 0) + R.TINY[dtype]
    ok |= np.isnan(got) & np.isnan(want)
    assert got.shape == want.shape and ok.all(), (np.abs(got - want)[~ok][:5], np.argwhere(~ok)[:5])


def _check(x, k, g=None, **kw):
    """route_topk of x (host) and its gradient against the definition."""
    print("topk", tuple(x.shape), x.dtype, k, {n: v if not torch.is_tensor(v) else tuple(v.shape) for n, v in kw.items()},
          flush=True)
    dev = {n: v.cuda() if torch.is_tensor(v) else v for n, v in kw.items()}
    xd = x.cuda().requires_grad_(True)
    w, ids = ou.route_topk(xd, k, **dev)
    assert w.dtype == F32 and ids.dtype == torch.int32 and not ids.requires_grad
    host = {n: R.host(v) if torch.is_tensor(v) and v.dtype != torch.bool else v.numpy() if torch.is_tensor(v) else v
            for n, v in kw.items()}
    want, at, r, s = R.topk(R.host(x), k, **host)
    assert np.array_equal(ids.cpu().numpy(), at)
    bound = R.weights_bound(R.host(x), at)
    _near(w, want, np.abs(want) * bound)
    g = torch.randn(w.shape, generator=_gen(3)) if g is None else g
    w.backward(g.cuda())
    scores, renorm, scale = host.get("scores", "softmax"), host.get("renormalize", True), host.get("scale", 1.0)
    dx, size = R.topk_backward(R.host(x), at, R.host(g), scores, renorm, scale)
    # the products of a score (its bound) and a difference of two (its and the sum's bounds), and 64 more half steps
    # for the sum over the choices
    _near(xd.grad, dx, size * (3 * bound + 64 * R.U), x.dtype)
    return ids


KINDS = [dict(scores=s, renormalize=r) for s in ("softmax", "sigmoid") for r in (True, False)]


@pytest.mark.parametrize("kw", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 64, 6), (5, 7, 7), (33, 60, 4), (130, 128, 8), (67, 256, 8), (9, 300, 16),
                                   (19, 512, 3), (3, 1024, 64), (6, 65, 64), (1000, 16, 2)])
def test_topk(t, e, k, dtype, kw):
    x = (torch.randn((t, e), generator=_gen(t + e)) * 2).to(dtype)
    _check(x, k, scale=2.5, **kw)


@pytest.mark.parametrize("kw", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("e,k,groups,top,score", [(256, 8, 8, 4, "best two"), (64, 6, 8, 3, "best"), (96, 5, 3, 2, "best two"),
                                                  (160, 6, 8, 3, "best"), (70, 4, 7, 2, "best two"), (64, 4, 64, 9, "best"),
                                                  (1024, 32, 64, 3, "best two"), (24, 8, 1, 1, "best"), (40, 4, 2, 1, "best two"),
                                                  (512, 12, 4, 4, "best two"), (36, 3, 12, 5, "best two")])
@pytest.mark.parametrize("biased", [True, False])
def test_topk_groups_and_bias(e, k, groups, top, score, dtype, biased, kw):
    x = (torch.randn((41, e), generator=_gen(e)) * 1.5).to(dtype)
    bias = torch.randn(e, generator=_gen(k)) * 0.1 if biased else None
    _check(x, k, bias=bias, groups=groups, top_groups=top, group_score=score, **kw)


@pytest.mark.parametrize("e", [60, 256, 700])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [True, False])
def test_topk_neighbours_that_32_bits_do_not_tell_apart(e, scores, biased):
    g = _gen(e)
    x = torch.stack([1 + torch.randperm(e, generator=g) * 2.0 ** -23 for _ in range(40)])
    x[20:] = 3 + torch.randint(0, 9, (20, e), generator=g) * 2.0 ** -22   # and equal ones among them
    bias = torch.randint(0, 2, (e,), generator=g) * 2.0 ** -60 if biased else None
    _check(x, 8, scores=scores, bias=bias)
    _check(x, 3, scores=scores, bias=bias, groups=2, top_groups=1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("e,k", [(8, 4), (64, 8), (256, 8), (1000, 40)])
def test_topk_ties_go_to_the_lower_expert(e, k, dtype):
    x = torch.randint(-2, 3, (50, e), generator=_gen(e)).to(dtype)
    x[0] = 0
    x[1, ::2], x[1, 1::2] = -0.0, 0.0
    for bias in (None, torch.zeros(e), torch.randint(0, 2, (e,), generator=_gen(5)).float()):
        ids = _check(x, k, scores="sigmoid", bias=bias)
        if bias is None:
            assert ids[0].tolist() == list(range(k)) and ids[1].tolist() == list(range(k))
    _check(x, k, scores="softmax", bias=torch.zeros(e))
    _check(x, k, scores="sigmoid", groups=4, top_groups=2) if e // 2 >= k else None


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("e", [32, 200])
def test_topk_absent_experts_and_tokens(scores, renormalize, biased, e):
    x = torch.randn((12, e), generator=_gen(1))
    x[0] = -INF                       # nobody
    x[1, 3:] = -INF                   # three
    x[2, : e // 2] = -INF             # whole groups
    x[3] = torch.finfo(F32).min       # the lowest number is there
    x[4, 5:] = torch.finfo(F32).min
    x[5] = torch.where(torch.rand(e, generator=_gen(2)) < 0.5, -INF, x[5])
    x[6] *= 30                        # scores that underflow
    x[7] = -200 - x[7]
    mask = torch.ones(12, dtype=torch.bool)
    mask[9:11] = False
    bias = torch.randn(e, generator=_gen(4)) * 0.1 if biased else None
    ids = _check(x, 6, scores=scores, renormalize=renormalize, bias=bias, mask=mask)
    assert (ids[0] == -1).all() and (ids[9:11] == -1).all() and (ids[1, 3:] == -1).all() and (ids[1, :3] >= 0).all()
    _check(x, 6, scores=scores, renormalize=renormalize, bias=bias, mask=mask, groups=4, top_groups=2)


def test_topk_nan_and_infinities():
    x = torch.randn((4, 40), generator=_gen(1))
    x[0, 7], x[1, 9], x[2, 3] = NAN, INF, NAN
    for scores in ("softmax", "sigmoid"):
        for kw in (dict(), dict(bias=torch.randn(40, generator=_gen(2)).cuda()), dict(groups=4, top_groups=2)):
            w, ids = ou.route_topk(x.cuda(), 4, scores=scores, **kw)
            w, ids = w.cpu(), ids.cpu()
            assert ((ids >= 0) & (ids < 40)).all() and all(len(set(row)) == 4 for row in ids.tolist())
            assert torch.isfinite(w[3]).all() and torch.isnan(w[0]).any() and torch.isnan(w[2]).any()
            if scores == "softmax":
                assert torch.isnan(w[:3]).all()
            elif not kw:
                assert ids[0, 0] == 7 and ids[1, 0] == 9 and torch.isfinite(w[1]).all()
    # a NaN or infinite bias
    b = torch.zeros(40)
    b[5], b[6], b[8] = NAN, INF, -INF
    w, ids = ou.route_topk(x[3:].cuda(), 40, scores="sigmoid", bias=b.cuda())
    assert ids[0, 0] == 5 and ids[0, 1] == 6 and ids[0, 39] == 8 and torch.isfinite(w).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_topk_strides(dtype):
    base = torch.randn((40, 300), generator=_gen(2)).to(dtype).cuda()
    for view in (base[:, 3:131], base[::3, 1:65], base.t()[:70], base[:1].expand(9, 300), base[:, ::4]):
        w, ids = ou.route_topk(view, 5, scores="sigmoid")
        want = ou.route_topk(view.contiguous().clone(), 5, scores="sigmoid")
        assert torch.equal(w, want[0]) and torch.equal(ids, want[1])
    # gradients reach a broadcast row as the sum of its copies'
    row = base[:1].float().requires_grad_(True)
    w, ids = ou.route_topk(row.expand(9, 300), 5)
    g = torch.randn(9, 5, generator=_gen(1)).cuda()
    w.backward(g)
    dx, _ = R.topk_backward(np.repeat(R.host(row), 9, 0), ids.cpu().numpy(), R.host(g), "softmax", True, 1.0)
    np.testing.assert_allclose(R.host(row.grad)[0], dx.sum(0), atol=1e-5)


@pytest.mark.parametrize("kw", KINDS)
def test_topk_gradient_against_differences(kw):
    x = torch.randn((6, 24), generator=_gen(9)).double().numpy()
    w, ids = ou.route_topk(torch.tensor(x, dtype=F32).cuda().requires_grad_(True), 4, scale=1.5, **kw)
    g = torch.randn(6, 4, generator=_gen(8))
    dx, _ = R.topk_backward(np.float32(x).astype(np.float64), ids.cpu().numpy(), g.double().numpy(), kw["scores"],
                            kw["renormalize"], 1.5)
    xd = torch.tensor(x, dtype=F32).cuda().requires_grad_(True)
    ou.route_topk(xd, 4, scale=1.5, **kw)[0].backward(g.cuda())
    h, x32 = 1e-6, np.float32(x).astype(np.float64)
    for e in range(24):
        for sign, store in ((1, "up"), (-1, "down")):
            y = x32.copy()
            y[:, e] += sign * h
            v = (R.topk(y, 4, scale=1.5, **kw)[0] * g.double().numpy()).sum(-1)
            up, down = (v, None) if store == "up" else (up, v)
        # differences of order h^2 and of rounding 2^-53 / h
        np.testing.assert_allclose(dx[:, e], (up - down) / (2 * h), atol=1e-8)
        np.testing.assert_allclose(R.host(xd.grad)[:, e], (up - down) / (2 * h), atol=2e-6)


def test_topk_of_no_tokens_and_no_gradient():
    x = torch.zeros((0, 16), device="cuda", requires_grad=True)
    w, ids = ou.route_topk(x, 2)
    assert w.shape == ids.shape == (0, 2)
    w.sum().backward()
    assert x.grad.shape == (0, 16)
    x = torch.randn((3, 16), device="cuda", requires_grad=True)
    with torch.no_grad():
        assert not ou.route_topk(x, 2)[0].requires_grad
    w, ids = ou.route_topk(x, 2)
    x.data.add_(0)
    with torch.no_grad():
        x.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        w.sum().backward()


# ------------------------------------------------------------------ the order

def _ids(t, k, e, seed, none=0.1):
    g = _gen(seed)
    share = torch.rand(e, generator=g) ** 3 + 1e-3
    ids = torch.multinomial(share, t * k, replacement=True, generator=g).view(t, k).int() if t else torch.zeros((0, k)).int()
    drop = torch.rand((t, k), generator=g)
    ids[drop < none] = -1
    ids[drop > 1 - none / 4] = e + 3
    return ids


@pytest.mark.parametrize("t,k,e", [(0, 2, 5), (1, 1, 1), (1, 8, 256), (13, 2, 16), (64, 1, 3), (511, 8, 64), (512, 8, 1024), (513, 8, 7),
                                   (5000, 3, 100), (20000, 8, 256), (70001, 1, 2), (200000, 8, 31)])
@pytest.mark.parametrize("none", [0.0, 0.2, 1.0])
def test_order(t, k, e, none):
    print("order", t, k, e, none, flush=True)
    ids = _ids(t, k, e, t + e, none)
    if none == 1.0:
        ids[:] = -5
    o = ou.route_order(ids.cuda(), e)
    offsets, slots, places = R.order(ids.numpy(), e)
    assert np.array_equal(o.offsets.cpu().numpy(), offsets)
    assert np.array_equal(o.slots.cpu().numpy(), slots)
    assert np.array_equal(o.places.cpu().numpy(), places)
    assert (o.experts, o.tokens, o.choices) == (e, t, k)


def test_order_of_one_expert_only():
    ids = torch.full((4097, 3), 77, dtype=torch.int32, device="cuda")
    o = ou.route_order(ids, 200)
    assert o.offsets.cpu().tolist() == [0] * 78 + [4097 * 3] * 123
    assert torch.equal(o.slots.cpu(), torch.arange(4097 * 3).int()) and torch.equal(o.places.flatten(), o.slots)


def test_balance():
    ids = _ids(1000, 4, 37, 3)
    o = ou.route_order(ids.cuda(), 37)
    count = np.diff(R.order(ids.numpy(), 37)[0].astype(np.int64))
    bias = torch.randn(37, generator=_gen(2))
    want = bias.numpy() + np.float32(0.01) * np.sign(count.sum() - 37 * count).astype(np.float32)
    got = ou.route_balance(bias.cuda(), o, 0.01)
    assert np.array_equal(got.cpu().numpy(), want)
    b = bias.cuda()
    assert ou.route_balance(b, o, 0.01, out=b) is b and torch.equal(b, got)
    even = ou.route_order(torch.arange(37, dtype=torch.int32).view(37, 1).cuda(), 37)
    assert torch.equal(ou.route_balance(bias.cuda(), even, 1.0).cpu(), bias)


# ------------------------------------------------------------------ rows

ROWS = [(1, 1, 1, 1), (5, 2, 4, 3), (13, 6, 64, 1000), (8, 2, 16, 1001), (40, 8, 30, 2048), (7, 64, 90, 72), (300, 3, 5, 136),
        (17, 9, 12, 5000), (3, 33, 40, 16392)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,k,e,h", ROWS)
def test_dispatch(t, k, e, h, dtype):
    print("dispatch", t, k, e, h, dtype, flush=True)
    ids = _ids(t, k, e, t + h)
    o = ou.route_order(ids.cuda(), e)
    offsets, slots, places = R.order(ids.numpy(), e)
    x = torch.randn((t, h), generator=_gen(1)).to(dtype)
    x.view(-1)[0] = NAN     # copied like anything else
    xd = x.cuda().requires_grad_(True)
    rows = ou.route_dispatch(xd, o)
    want = torch.where(torch.tensor(slots < 0)[:, None], torch.zeros((), dtype=dtype), x[torch.tensor(np.maximum(slots, 0) // k).long()])
    kind = torch.int32 if dtype == F32 else torch.int16
    assert torch.equal(rows.detach().cpu().view(kind), want.view(kind))
    g = torch.randn((t * k, h), generator=_gen(2)).to(dtype)
    rows.backward(g.cuda())
    parts = np.where((places < 0)[..., None], 0, R.host(g)[np.maximum(places, 0)])
    _near(xd.grad, parts.sum(1), np.abs(parts).sum(1) * k * R.U, dtype)
    # rows of no slot stay as they were in a result that is given, between its rows too
    room = torch.full((t * k, h + 5), 7.0, dtype=dtype, device="cuda")
    with torch.no_grad():
        assert ou.route_dispatch(xd, o, out=room[:, 2:2 + h]).data_ptr() == room[:, 2:].data_ptr()
    room = room.cpu()
    assert (room[:, :2] == 7).all() and (room[:, 2 + h:] == 7).all() and (room[offsets[-1]:] == 7).all()
    assert torch.equal(room[:offsets[-1], 2:2 + h].contiguous().view(kind), want[:offsets[-1]].view(kind))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,k,e,h", ROWS)
@pytest.mark.parametrize("added", [True, False])
def test_combine(t, k, e, h, dtype, added):
    print("combine", t, k, e, h, dtype, added, flush=True)
    ids = _ids(t, k, e, t + h)
    o = ou.route_order(ids.cuda(), e)
    offsets, slots, places = R.order(ids.numpy(), e)
    y = torch.randn((t * k, h), generator=_gen(1)).to(dtype)
    y[offsets[-1]:] = NAN    # never read
    w = torch.rand((t, k), generator=_gen(2))
    add = torch.randn((t, h), generator=_gen(3)).to(dtype) if added else None
    yd, wd = y.cuda().requires_grad_(True), w.cuda().requires_grad_(True)
    ad = add.cuda().requires_grad_(True) if added else None
    out = ou.route_combine(yd, wd, o, add=ad)
    rows = np.where((places < 0)[..., None], 0, R.host(y)[np.maximum(places, 0)])
    parts = rows * R.host(w)[..., None]
    want, size = parts.sum(1), np.abs(parts).sum(1)
    if added:
        want, size = want + R.host(add), size + np.abs(R.host(add))
    _near(out, want, size * (k + 1) * R.U, dtype)
    g = torch.randn((t, h), generator=_gen(4)).to(dtype)
    out.backward(g.cuda())
    g64 = R.host(g)
    dots = rows * g64[:, None]
    _near(wd.grad, np.where(places < 0, 0, dots.sum(-1)), np.abs(dots).sum(-1) * h * R.U)
    dy = np.where((slots < 0)[:, None], 0, R.host(w).reshape(-1)[np.maximum(slots, 0), None] * g64[np.maximum(slots, 0) // k])
    _near(yd.grad, dy, np.abs(dy) * R.U, dtype)
    if added:
        assert torch.equal(ad.grad.cpu(), g)
    # one gradient alone, strided operands, a result that is given
    only, = torch.autograd.grad(ou.route_combine(y.cuda(), wd, o), wd, g.cuda())
    assert torch.equal(only, wd.grad)
    only, = torch.autograd.grad(ou.route_combine(yd, w.cuda(), o), yd, g.cuda())
    assert torch.equal(only, yd.grad)
    room = torch.full((t, h + 3), 5.0, dtype=dtype, device="cuda")
    wide = torch.zeros((t * k, h + 8), dtype=dtype, device="cuda")
    wide[:, :h] = y.cuda()
    ou.route_combine(wide[:, :h], w.cuda(), o, add=None if add is None else add.cuda(), out=room[:, 1:1 + h])
    assert torch.equal(room[:, 1:1 + h], out.detach()) and (room[:, 0] == 5).all() and (room[:, 1 + h:] == 5).all()


def test_combine_keeps_what_it_should_not_read():
    """An infinite gradient times a slot without a row is 0; and results of a
    size that goes past the caches."""
    places = torch.tensor([[0, -1]], dtype=torch.int32, device="cuda")
    o = ou.RouteOrder(torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([0, -1], dtype=torch.int32, device="cuda"), places)
    y = torch.ones((2, 64), device="cuda").requires_grad_(True)
    w = torch.ones((1, 2), device="cuda").requires_grad_(True)
    out = ou.route_combine(y, w, o)
    out.backward(torch.full((1, 64), INF, device="cuda"))
    assert w.grad[0, 0] == INF and w.grad[0, 1] == 0 and (y.grad[1] == 0).all() and (y.grad[0] == INF).all()
    t, k, h = 4096, 4, 8192   # 256 MiB in bfloat16
    ids = _ids(t, k, 16, 5)
    o = ou.route_order(ids.cuda(), 16)
    x = torch.randn((t, h), device="cuda", dtype=BF16).requires_grad_(True)
    w = torch.rand((t, k), device="cuda").requires_grad_(True)
    rows = ou.route_dispatch(x, o)
    out = ou.route_combine(rows, w, o)
    g = torch.randn((t, h), device="cuda", dtype=BF16)
    dx, dw = torch.autograd.grad(out, (x, w), g)
    live = (o.places >= 0).float()
    total = (w.detach() * live).sum(1, keepdim=True)
    # each product and partial sum to half a step of the type at most, and the last rounding
    torch.testing.assert_close(out.float(), x.detach().float() * total, rtol=2.0 ** -8, atol=1e-5)
    torch.testing.assert_close(dx.float(), g.float() * total, rtol=3 * 2.0 ** -8, atol=2.0 ** -7)
    ref = (x.detach().float() * g.float()).sum(1, keepdim=True) * live
    torch.testing.assert_close(dw, ref, rtol=1e-4, atol=2e-2)


def test_rows_without_columns():
    o = ou.route_order(torch.zeros((3, 2), dtype=torch.int32, device="cuda"), 4)
    x = torch.zeros((3, 0), device="cuda", requires_grad=True)
    w = torch.ones((3, 2), device="cuda", requires_grad=True)
    rows = ou.route_dispatch(x, o)
    out = ou.route_combine(rows, w, o)
    assert rows.shape == (6, 0) and out.shape == (3, 0)
    dx, dw = torch.autograd.grad(out, (x, w), torch.zeros((3, 0), device="cuda"))
    assert dx.shape == (3, 0) and torch.equal(dw, torch.zeros((3, 2), device="cuda"))


def test_orders_with_bad_rows_stay_inside():
    """Places that a program made itself: what points nowhere is as -1."""
    places = torch.tensor([[5, -7], [1 << 30, 0]], dtype=torch.int32, device="cuda")
    o = ou.RouteOrder(torch.zeros(3, dtype=torch.int32, device="cuda"), torch.full((4,), -1, dtype=torch.int32, device="cuda"), places)
    x = torch.randn((2, 64), device="cuda")
    rows = ou.route_dispatch(x, o)
    assert rows.shape == (4, 64)
    y = torch.randn((4, 64), device="cuda").requires_grad_(True)
    out = ou.route_combine(y, torch.ones((2, 2), device="cuda"), o)
    assert torch.equal(out[0], torch.zeros(64, device="cuda")) and torch.equal(out[1], y[0])
    out.sum().backward()


# ------------------------------------------------------------------ together

def _layer(x, wr, bias, we, mask=None):
    """A layer of experts as a program writes it."""
    w, ids = ou.route_topk(x @ wr.t(), 2, scores="sigmoid", bias=bias, groups=2, top_groups=1, mask=mask)
    order = ou.route_order(ids, wr.shape[0])
    y = ou.mx4_grouped_linear(ou.route_dispatch(x, order), we, order.offsets)
    return ou.route_combine(y, w, order, add=x), order


def test_a_layer_of_experts_trains():
    """Router, order, dispatch, the experts' products in 4 bits and the
    combination, with a collection optimizer's step and the balance bias:
    gradients reach all of it and equal those of the parts in torch."""
    g = _gen(5)
    x = torch.randn((96, 64), generator=g).cuda().requires_grad_(True)
    wr = torch.nn.Parameter((torch.randn((8, 64), generator=g) / 8).cuda())
    we = torch.nn.Parameter((torch.randn((8, 64, 64), generator=g) / 8).cuda())
    bias = torch.zeros(8, device="cuda")
    mask = torch.arange(96, device="cuda") < 90
    opt = ou.AdamW32([wr, we], lr=1e-3)
    for _ in range(3):
        out, order = _layer(x, wr, bias, we, mask)
        target = torch.randn(out.shape, generator=g).cuda()
        (out * target).sum().backward()
        # the same sums in torch over the same rows; the experts' products through the same 4-bit layer
        xs, ws, es = (v.detach().clone().requires_grad_(True) for v in (x, wr, we))
        s = torch.sigmoid(xs @ ws.t())
        w, ids = ou.route_topk((x @ wr.t()).detach(), 2, scores="sigmoid", bias=bias, groups=2, top_groups=1, mask=mask)
        live = ids >= 0
        c = s.gather(1, ids.clamp(min=0).long()) * live
        wt = torch.where(live, c / c.sum(-1, keepdim=True).clamp(min=1e-20), 0.0)
        n = int(order.offsets[-1])
        slot = order.slots[:n].long()
        rows = torch.cat([xs[slot // 2], torch.zeros((192 - n, 64), device="cuda")])
        y = ou.mx4_grouped_linear(rows, es, order.offsets)[:n]
        ref = xs.index_add(0, slot // 2, y * wt.flatten()[slot, None])
        torch.testing.assert_close(out, ref, rtol=1e-5, atol=1e-5)
        assert torch.equal(out[90:], x[90:])
        (ref * target).sum().backward()
        for a, b in ((x, xs), (wr, ws), (we, es)):
            torch.testing.assert_close(a.grad, b.grad, rtol=1e-4, atol=1e-4 * float(b.grad.abs().max()))
        x.grad = None
        opt.step()
        opt.zero_grad()
        ou.route_balance(bias, order, 1e-2, out=bias)
    assert bias.abs().max() > 0


@pytest.mark.parametrize("grad", [False, True])
def test_captured_and_replayed(grad):
    """A whole pass in a graph, replayed on other inputs with eager work and
    synchronizations between."""
    t, e, k, h = 300, 64, 4, 64
    x = torch.randn((t, h), generator=_gen(1)).cuda()
    logits = torch.randn((t, e), generator=_gen(2)).cuda()
    wx = (torch.randn((h, h), generator=_gen(3)) / 8).cuda()
    xs, ls, g = torch.zeros_like(x), torch.zeros_like(logits), torch.randn((t, h), generator=_gen(4)).cuda()

    def run(x, logits):
        if grad:
            x, logits = x.detach().requires_grad_(True), logits.detach().requires_grad_(True)
        w, ids = ou.route_topk(logits, k, renormalize=False)
        o = ou.route_order(ids, e)
        out = ou.route_combine(ou.route_dispatch(x, o) * 2, w, o, add=x)
        got = [out.detach(), ids, o.offsets, o.slots, o.places]
        return got + list(torch.autograd.grad(out, (x, logits), g)) if grad else got

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(xs, ls)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(xs, ls)
    for i in range(4):
        xs.copy_(x * (i + 1))
        ls.copy_(logits.roll(i, 0) * (1 + i))
        graph.replay()
        want = run(x * (i + 1), logits.roll(i, 0) * (1 + i))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        (wx @ wx).sum()
        torch.cuda.synchronize()


def test_streams():
    ids = _ids(5000, 8, 64, 1).cuda()
    bias = torch.zeros(64, device="cuda")
    want = ou.route_order(ids, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        o = ou.route_order(ids, 64, stream=stream)
        b = ou.route_balance(bias, o, 0.5, stream=stream)
        s.synchronize()
        assert torch.equal(o.slots, want.slots) and torch.equal(o.places, want.places) and b.abs().max() == 0.5
    o = ou.route_order(ids, 64, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(o.slots, want.slots)
    # two passes at once, each on a stream of its own
    x = torch.randn((5000, 256), generator=_gen(2)).cuda()
    logits = torch.randn((5000, 64), generator=_gen(3)).cuda()
    torch.cuda.synchronize()

    def run(f):
        w, i = ou.route_topk(logits * f, 4)
        o = ou.route_order(i, 64)
        return ou.route_combine(ou.route_dispatch(x * f, o), w, o)

    ref = [run(1.0), run(2.0)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = run(1.0 + i)
        torch.cuda.synchronize()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_large_offsets():
    """Rows past 2^31 elements and 2^32 bytes."""
    t, k, h = 70000, 4, 8192
    x = torch.randn((t, h), device="cuda", dtype=BF16)
    ids = torch.randint(0, 4, (t, k), device="cuda", dtype=torch.int32)
    o = ou.route_order(ids, 4)
    rows = ou.route_dispatch(x, o)
    for p in (0, 1, 131071, 200000, t * k - 1):
        assert torch.equal(rows[p], x[int(o.slots[p]) // k])
    w = torch.full((t, k), 0.25, device="cuda")
    out = ou.route_combine(rows, w, o)
    assert torch.equal(out, x)
