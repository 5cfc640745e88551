"""GPU: 4-bit whole-number weights with group scales against their definition
in 64 bits (tests/experts_reference.py)."""
import numpy as np
import pytest
import torch

import optimizer_update_amd as ou
from tests import experts_reference as R

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
DTYPES = [F32, F16, BF16]


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _weights(lead, k, group, dtype, zeros, seed=0):
    g = _gen(seed)
    codes = torch.randint(0, 256, (*lead, k // 2), generator=g, dtype=torch.uint8)
    scales = ((torch.rand((*lead, k // group), generator=g) - 0.3) / 8).to(dtype)
    # whole and other zeros, also outside of the codes
    z = (torch.rand((*lead, k // group), generator=g) * 20 - 2).to(dtype) if zeros else None
    if zeros and z.numel() > 2:
        z.view(-1)[::2] = z.view(-1)[::2].round()
    return ou.Int4(codes.cuda(), scales.cuda(), None if z is None else z.cuda(), group)


def _bound(size, k, dtype, want):
    """Sums of k exact products in binary32 in any order, group by group, then
    the group's two terms times its scale (five more half steps), one rounding."""
    return size * (k + 8) * R.U + np.abs(want) * (R.step(dtype) if dtype != F32 else 0) + R.TINY[dtype]


def _check(got, want, size, k, dtype):
    got = R.host(got)
    ok = np.abs(got - want) <= _bound(size, k, dtype, want)
    assert got.shape == want.shape and ok.all(), (got[~ok][:4], want[~ok][:4], np.argwhere(~ok)[:4])


SHAPES = [(1, 1, 32, 32), (1, 5, 64, 32), (2, 16, 128, 128), (3, 17, 160, 32), (4, 33, 192, 64), (13, 70, 384, 96), (16, 64, 256, 256),
          (17, 129, 1024, 128), (33, 31, 512, 64), (64, 100, 2048, 128), (70, 16, 4096, 128), (1, 300, 5120, 640), (5, 48, 8224, 32)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("m,n,k,group", SHAPES)
def test_matmul(m, n, k, group, dtype, zeros):
    print("int4 matmul", m, n, k, group, dtype, zeros, flush=True)
    q = _weights((n,), k, group, DTYPES[(m + n) % 3], zeros)
    x = (torch.randn((m, k), generator=_gen(1)) * torch.exp2(torch.randn(k, generator=_gen(2)) * 3)).to(dtype)
    want, size = R.int4_product(R.host(x), q)
    xd = x.cuda()
    y = ou.int4_matmul(xd, q)
    assert y.dtype == dtype
    _check(y, want, size, k, dtype)
    for od in DTYPES:
        _check(ou.int4_matmul(xd, q, dtype=od), want, size, k, od) if od != F16 or np.abs(want).max() < 6e4 else None
    # strided operands, a result that is given
    wide = torch.zeros((m, k + 8), dtype=dtype, device="cuda")
    wide[:, 8:] = xd
    room = torch.full((m, n + 3), 9.0, dtype=dtype, device="cuda")
    assert ou.int4_matmul(wide[:, 8:], q, out=room[:, 1:1 + n]) is not None
    assert torch.equal(room[:, 1:1 + n], y) and (room[:, 0] == 9).all() and (room[:, 1 + n:] == 9).all()
    odd = torch.zeros((m, k + 3), dtype=dtype, device="cuda")
    odd[:, 1:1 + k] = xd
    assert torch.equal(ou.int4_matmul(odd[:, 1:1 + k], q), y)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("counts,n,k,group", [([1], 16, 64, 64), ([0, 3, 0, 16, 17, 1], 33, 256, 128), ([5] * 70, 8, 96, 32),
                                              ([0, 0], 5, 64, 32), ([100, 0, 1, 33], 100, 512, 64), ([2] * 130, 40, 128, 128)])
def test_grouped_matmul(counts, n, k, group, dtype, zeros):
    print("int4 grouped", len(counts), n, k, group, dtype, zeros, flush=True)
    e, front, behind = len(counts), 3, 18
    m = front + sum(counts) + behind
    q = _weights((e, n), k, group, BF16, zeros)
    x = torch.randn((m, k), generator=_gen(1)).to(dtype)
    at = front + np.concatenate([[0], np.cumsum(counts)])
    offsets = torch.tensor(at, dtype=torch.int32).cuda()
    y = ou.int4_grouped_matmul(x.cuda(), q, offsets)
    room = torch.full((m, n + 1), 3.0, dtype=dtype, device="cuda")
    ou.int4_grouped_matmul(x.cuda(), q, offsets, out=room[:, :n])
    assert (y[:front] == 0).all() and (y[at[-1]:] == 0).all()
    assert (room[:front] == 3).all() and (room[at[-1]:] == 3).all() and (room[:, n] == 3).all()
    assert torch.equal(room[front:at[-1], :n], y[front:at[-1]])
    for i in range(e):
        want, size = R.int4_product(R.host(x[at[i]:at[i + 1]]), q[i])
        _check(y[at[i]:at[i + 1]], want, size, k, dtype)


# many tiles: more than one slab of columns, an odd edge, experts without rows and with more than a unit's
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("counts,n,k,group", [([3, 0, 17, 1] * 20, 2100, 512, 128), ([1] * 65, 2063, 2560, 64), ([9, 8, 7, 2] * 16, 2085, 2432, 32),
                                              ([1, 2] * 36, 2051, 4608, 128)])
def test_grouped_matmul_of_many_tiles(counts, n, k, group, dtype, zeros):
    print("int4 many tiles", len(counts), n, k, group, dtype, zeros, flush=True)
    e, front, behind = len(counts), 2, 19
    m = front + sum(counts) + behind
    q = _weights((e, n), k, group, DTYPES[(n + k // 128) % 3], zeros)
    x = (torch.randn((m, k), generator=_gen(1)) * torch.exp2(torch.randn(k, generator=_gen(2)))).to(dtype)
    at = front + np.concatenate([[0], np.cumsum(counts)])
    y = ou.int4_grouped_matmul(x.cuda(), q, torch.tensor(at, dtype=torch.int32).cuda())
    assert (y[:front] == 0).all() and (y[at[-1]:] == 0).all()
    for i in (*range(0, e, 7), e - 1):
        want, size = R.int4_product(R.host(x[at[i]:at[i + 1]]), q[i])
        _check(y[at[i]:at[i + 1]], want, size, k, dtype)
        one = ou.int4_matmul(x[at[i]:at[i + 1]].cuda(), q[i])
        _check(one, want, size, k, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_matmul_of_many_tiles(dtype):
    q = _weights((131077,), 512, 64, F16, True)
    x = torch.randn((5, 512), generator=_gen(1)).to(dtype)
    want, size = R.int4_product(R.host(x), q)
    _check(ou.int4_matmul(x.cuda(), q), want, size, 512, dtype)


def _some_rows(q, rows):
    return ou.Int4(q.codes[rows].clone(), q.scales[rows].clone(), None if q.zeros is None else q.zeros[rows].clone(), q.group)


# two and four tiles of weights a block, runs of columns that end inside a turn or a step, edges inside a block
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scales", [F32, BF16])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("m,n,k,group", [(1, 8200, 6304, 32), (17, 4117, 6400, 64), (20, 8200, 6528, 128), (3, 16400, 4192, 32),
                                         (5, 16390, 1600, 64), (40, 6007, 1344, 96)])
def test_matmul_of_wide_blocks(m, n, k, group, zeros, scales, dtype):
    print("int4 wide blocks", m, n, k, group, zeros, scales, dtype, flush=True)
    q = _weights((n,), k, group, scales, zeros)
    x = (torch.randn((m, k), generator=_gen(1)) * torch.exp2(torch.randn(k, generator=_gen(2)))).to(dtype)
    xd = x.cuda()
    y = ou.int4_matmul(xd, q)
    at = [*range(0, 70), *range(90, n - 80, 271), *range(n - 80, n)]
    want, size = R.int4_product(R.host(x), _some_rows(q, at))
    _check(y[:, at], want, size, k, dtype)
    odd = torch.zeros((m, k + 3), dtype=dtype, device="cuda")
    odd[:, 1:1 + k] = xd
    room = torch.full((m, n + 3), 9.0, dtype=dtype, device="cuda")
    ou.int4_matmul(odd[:, 1:1 + k], q, out=room[:, 1:1 + n])
    assert torch.equal(room[:, 1:1 + n], y) and (room[:, 0] == 9).all() and (room[:, 1 + n:] == 9).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scales", [F32, F16])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("counts,n,k,group", [([3, 0, 17, 1] * 8, 520, 4224, 128), ([2] * 16, 515, 4160, 64), ([2, 18] * 9, 907, 3232, 32),
                                              ([1, 0, 30] * 6, 1000, 2112, 64)])
def test_grouped_matmul_of_wide_blocks(counts, n, k, group, zeros, scales, dtype):
    print("int4 grouped wide blocks", len(counts), n, k, group, zeros, scales, dtype, flush=True)
    e, front, behind = len(counts), 2, 19
    m = front + sum(counts) + behind
    q = _weights((e, n), k, group, scales, zeros)
    x = torch.randn((m, k), generator=_gen(1)).to(dtype)
    at = front + np.concatenate([[0], np.cumsum(counts)])
    offsets = torch.tensor(at, dtype=torch.int32).cuda()
    y = ou.int4_grouped_matmul(x.cuda(), q, offsets)
    room = torch.full((m, n + 1), 3.0, dtype=dtype, device="cuda")
    ou.int4_grouped_matmul(x.cuda(), q, offsets, out=room[:, :n])
    assert (y[:front] == 0).all() and (y[at[-1]:] == 0).all()
    assert (room[:front] == 3).all() and (room[at[-1]:] == 3).all() and (room[:, n] == 3).all()
    assert torch.equal(room[front:at[-1], :n], y[front:at[-1]])
    for i in (0, 2, e - 1):
        want, size = R.int4_product(R.host(x[at[i]:at[i + 1]]), q[i])
        _check(y[at[i]:at[i + 1]], want, size, k, dtype)


# 16-bit scales, tiles enough for x to be held: 7 to 8 and 13 to 16 steps, all or some of the waves' registers filled
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scales", [F16, BF16])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("m,n,k,group", [(3, 24593, 1024, 32), (17, 12300, 928, 32), (2, 25000, 896, 128), (1, 24600, 960, 64),
                                         (16, 98320, 2048, 128), (40, 32790, 1632, 96)])
def test_matmul_with_rows_held(m, n, k, group, zeros, scales, dtype):
    print("int4 held", m, n, k, group, zeros, scales, dtype, flush=True)
    q = _weights((n,), k, group, scales, zeros)
    x = (torch.randn((m, k), generator=_gen(1)) * torch.exp2(torch.randn(k, generator=_gen(2)))).to(dtype)
    xd = x.cuda()
    y = ou.int4_matmul(xd, q)
    at = [*range(0, 70), *range(90, n - 300, 271), *range(n - 300, n)]
    want, size = R.int4_product(R.host(x), _some_rows(q, at))
    _check(y[:, at], want, size, k, dtype)
    odd = torch.zeros((m, k + 3), dtype=dtype, device="cuda")
    odd[:, 1:1 + k] = xd
    assert torch.equal(ou.int4_matmul(odd[:, 1:1 + k], q), y)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scales", [F16, BF16])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("counts,n,k,group", [([3, 0, 17, 1] * 12, 2100, 2048, 128), ([2] * 48, 2063, 1632, 32), ([18, 1] * 24, 2085, 1984, 64),
                                              ([1, 0, 30] * 8, 1100, 1024, 64)])
def test_grouped_matmul_with_rows_held(counts, n, k, group, zeros, scales, dtype):
    print("int4 grouped held", len(counts), n, k, group, zeros, scales, dtype, flush=True)
    e, front, behind = len(counts), 2, 19
    m = front + sum(counts) + behind
    q = _weights((e, n), k, group, scales, zeros)
    x = torch.randn((m, k), generator=_gen(1)).to(dtype)
    at = front + np.concatenate([[0], np.cumsum(counts)])
    y = ou.int4_grouped_matmul(x.cuda(), q, torch.tensor(at, dtype=torch.int32).cuda())
    assert (y[:front] == 0).all() and (y[at[-1]:] == 0).all()
    for i in (0, 2, e - 1):
        want, size = R.int4_product(R.host(x[at[i]:at[i + 1]]), q[i])
        _check(y[at[i]:at[i + 1]], want, size, k, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scales", [F32, BF16])
@pytest.mark.parametrize("n", [8192, 16384])
def test_rows_do_not_mix_in_wide_blocks(n, scales, dtype):
    q = _weights((n,), 1056, 32, scales, True)
    x = torch.randn((5, 1056), generator=_gen(3)).to(dtype).cuda()
    y = ou.int4_matmul(x, q)
    # the first row stands in for those that are not there, the last columns for those behind them
    x[0, 3], x[3, 1055] = float("nan"), float("inf")
    z = ou.int4_matmul(x, q)
    assert not torch.isfinite(z[[0, 3]]).any() and torch.equal(y[[1, 2, 4]], z[[1, 2, 4]])


def test_grouped_matmul_with_offsets_that_fall_or_leave():
    q = _weights((4, 24), 64, 64, F32, True)
    x = torch.randn((40, 64), generator=_gen(1)).cuda()
    y = ou.int4_grouped_matmul(x, q, torch.tensor([-5, 10, 4, 90, 90], dtype=torch.int32).cuda())
    same = ou.int4_grouped_matmul(x, q, torch.tensor([0, 10, 10, 40, 40], dtype=torch.int32).cuda())
    assert torch.equal(y, same)


def test_no_rows_no_columns():
    q = _weights((8,), 64, 32, F32, True)
    assert ou.int4_matmul(torch.zeros((0, 64), device="cuda"), q).shape == (0, 8)
    empty = ou.Int4(torch.zeros((8, 0), dtype=torch.uint8, device="cuda"), torch.zeros((8, 0), device="cuda"), None, 32)
    assert torch.equal(ou.int4_matmul(torch.zeros((3, 0), device="cuda"), empty), torch.zeros((3, 8), device="cuda"))
    none = ou.Int4(torch.zeros((0, 32), dtype=torch.uint8, device="cuda"), torch.zeros((0, 2), device="cuda"), None, 32)
    assert ou.int4_matmul(torch.zeros((3, 64), device="cuda"), none).shape == (3, 0)


def test_rows_do_not_mix():
    """A row with an infinity or a NaN spoils itself alone."""
    q = _weights((40,), 256, 64, BF16, True)
    for dtype in DTYPES:
        x = torch.randn((20, 256), generator=_gen(3)).to(dtype).cuda()
        y = ou.int4_matmul(x, q)
        x[4, 9], x[17, 200] = float("nan"), float("inf")
        z = ou.int4_matmul(x, q)
        assert not torch.isfinite(z[4]).any() and not torch.isfinite(z[17]).any()
        keep = [i for i in range(20) if i not in (4, 17)]
        assert torch.equal(y[keep], z[keep])


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_do_not_mix_where_tiles_are_many(dtype):
    e, n, k = 70, 600, 512
    q = _weights((e, n), k, 128, BF16, True)
    off = torch.arange(0, 3 * e + 1, 3, dtype=torch.int32, device="cuda")
    x = torch.randn((3 * e, k), generator=_gen(3)).to(dtype).cuda()
    y = ou.int4_grouped_matmul(x, q, off)
    bad = [4, 17, 100, 3 * e - 1]
    for i, r in enumerate(bad):
        x[r, 100 * i + 9] = float("nan") if i % 2 else float("inf")
    z = ou.int4_grouped_matmul(x, q, off)
    keep = [i for i in range(3 * e) if i not in bad]
    assert not torch.isfinite(z[bad]).any() and torch.equal(y[keep], z[keep])


def test_small_and_large_values():
    """x over the range of its type, with scales that bring the sums back."""
    for dtype, top, low in ((F32, 1e30, 1e-30), (BF16, 1e30, 1e-30), (F16, 6e4, 1e-6)):
        for f in (top, low):
            q = _weights((32,), 128, 32, F32, True)
            q.scales.mul_(1e-4 / f if f == top else 1.0)
            x = ((torch.rand((5, 128), generator=_gen(1)) - 0.5) * f).to(dtype)
            want, size = R.int4_product(R.host(x), q)
            _check(ou.int4_matmul(x.cuda(), q, dtype=F32), want, size, 128, F32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale_dtype", DTYPES)
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("lead,k,group", [((1,), 32, 32), ((7,), 192, 96), ((33,), 1024, 128), ((3, 5), 256, 64)])
def test_quantize_and_back(lead, k, group, dtype, scale_dtype, zeros):
    x = (torch.randn((*lead, k), generator=_gen(k)) * 0.3).to(dtype)
    x.view(-1, group)[0] = 0
    if x.numel() > 2 * group:
        x.view(-1, group)[1].abs_()
        x.view(-1, group)[2] = -x.view(-1, group)[2].abs()
    q = ou.int4_quantize(x.cuda(), group, zeros, scale_dtype)
    assert q.shape == x.shape and q.scales.dtype == scale_dtype and (q.zeros is None) == (not zeros)
    v = R.host(x).reshape(*lead, k // group, group)
    s = R.host(q.scales)
    lo, hi = np.minimum(v.min(-1), 0), np.maximum(v.max(-1), 0)
    best = (hi - lo) / 15 if zeros else np.maximum(hi / 7, lo / -8)
    # one rounding to the type and three in binary32
    assert (np.abs(s - best) <= best * (R.step(scale_dtype) + 3 * R.U) + R.TINY[scale_dtype]).all()
    values, codes = R.int4_values(q.codes.cpu().numpy(), q.scales, q.zeros, group)
    got = values.reshape(v.shape)
    # within half a step of the scale, and where a rounded scale fell short of the ends (by 15 times its error)
    room = s * (0.5 + (0.5 if zeros else 0)) + 15 * np.abs(s - best) + np.abs(v).max(-1) * 8 * R.U
    assert (np.abs(got - v) <= room[..., None]).all()
    if zeros:
        z = R.host(q.zeros)
        assert (z == np.round(z)).all() and (z >= 0).all() and (z <= 15).all()
    for od in DTYPES:
        back = ou.int4_dequantize(q, od)
        # (code - zero) is exact, the product rounded once in binary32 and once to the type
        assert (np.abs(R.host(back) - values) <= np.abs(values) * (R.U + R.step(od)) + R.TINY[od]).all()
    out = torch.empty(q.shape, dtype=BF16, device="cuda")
    assert torch.equal(ou.int4_dequantize(q, out=out), ou.int4_dequantize(q, BF16))


def test_quantize_strides_and_views():
    base = torch.randn((40, 200), generator=_gen(1)).cuda()
    for view in (base[:, 4:132], base[::2, :64], base.t()[:64, :32]):
        a, b = ou.int4_quantize(view, 32), ou.int4_quantize(view.contiguous().clone(), 32)
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales) and torch.equal(a.zeros, b.zeros)


def test_serving_a_layer_of_experts():
    """Router, order, dispatch, 4-bit experts, combination: one call after
    another as in serving, against 64 bits on the host."""
    t, e, k, h, n = 9, 12, 3, 128, 48
    x = torch.randn((t, h), generator=_gen(1))
    logits = torch.randn((t, e), generator=_gen(2))
    q = ou.int4_quantize((torch.randn((e, n, h), generator=_gen(3)) / 10).cuda(), 32)
    w, ids = ou.route_topk(logits.cuda(), k)
    order = ou.route_order(ids, e)
    y = ou.int4_grouped_matmul(ou.route_dispatch(x.cuda(), order), q, order.offsets)
    out = R.host(ou.route_combine(y, w, order))
    want, at, _, _ = R.topk(R.host(logits), k)
    for i in range(t):
        ref = np.zeros(n)
        size = np.zeros(n)
        for j in range(k):
            y64, s64 = R.int4_product(R.host(x[i:i + 1]), q[int(at[i, j])])
            ref += want[i, j] * y64[0]
            size += want[i, j] * s64[0]
        assert (np.abs(out[i] - ref) <= size * (h + 100) * R.U).all()


def test_captured_and_streams():
    q = _weights((64,), 512, 128, BF16, True)
    x = torch.randn((3, 512), generator=_gen(1)).to(BF16).cuda()
    xs = torch.zeros_like(x)
    want = ou.int4_matmul(x, q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ou.int4_matmul(xs, q)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ou.int4_matmul(xs, q)
    for i in range(3):
        xs.copy_(x * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ou.int4_matmul(x * (i + 1), q))
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        y = ou.int4_matmul(x, q, stream=stream)
        s.synchronize()   # what is compared on the current stream is done on the other one
        assert torch.equal(y, want)


# codes in one kernel's steps and in the other's runs of tiles
@pytest.mark.parametrize("e,n,k", [(136, 8192, 8192), (540, 8192, 2048)])
def test_many_experts_past_32_bits(e, n, k):
    """Weights whose last matrices lie past 2^32 bytes."""
    q = ou.Int4(torch.randint(0, 256, (e, n, k // 2), dtype=torch.uint8, device="cuda"),
                torch.full((e, n, k // 128), 2.0 ** -6, dtype=BF16, device="cuda"), None, 128)
    x = torch.randn((4, k), device="cuda").to(BF16)
    off = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    off[e] = 4
    y = ou.int4_grouped_matmul(x, q, off)
    last = ou.Int4(q.codes[e - 1].clone(), q.scales[e - 1].clone(), None, 128)
    want, size = R.int4_product(R.host(x), last)
    _check(y, want, size, k, BF16)


def test_held_rows_past_32_bits():
    """As above, by the kernel that holds x over many tiles."""
    e, n, k = 540, 8192, 2048
    q = ou.Int4(torch.randint(0, 256, (e, n, k // 2), dtype=torch.uint8, device="cuda"),
                torch.full((e, n, k // 128), 2.0 ** -6, dtype=BF16, device="cuda"), None, 128)
    x = torch.randn((16, k), device="cuda").to(BF16)
    off = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    off[e] = 16
    y = ou.int4_grouped_matmul(x, q, off)
    last = ou.Int4(q.codes[e - 1].clone(), q.scales[e - 1].clone(), None, 128)
    want, size = R.int4_product(R.host(x), last)
    _check(y, want, size, k, BF16)
