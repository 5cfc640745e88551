"""GPU: the microscaled 4-bit operators against their definition in 64 bits
(tests/mx4_reference.py).  Quantisation and dequantisation are exact: codes,
scales and values are compared for equality.  Products are held to the
tolerance derived there."""
import warnings

import numpy as np
import pytest
import torch

import optimizer_update_amd as ou
from optimizer_update_amd import _lib
from tests import mx4_reference as R

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
DTYPES = [F32, F16, BF16]


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _values(shape, dtype, seed, spread=8.0, special=True):
    """Values whose blocks differ in scale; some blocks are zero, subnormal or
    hold ties; the first element of a tensor is a negative zero."""
    g = _gen(seed)
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randn(shape[-1:], generator=g) * spread / 4)
    if special and x.numel():
        flat = x.view(-1)
        pick = torch.rand(flat.shape, generator=g)
        ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0])[torch.randint(0, 8, flat.shape, generator=g)]
        flat[pick < 0.3] = ties[pick < 0.3]
        flat[pick > 0.95] = 0
        flat[0] = -0.0
    return x.to(dtype)


def _check_form(q, x64):
    code, scale = R.quantize(x64)
    assert tuple(q.shape) == x64.shape
    got = R.unpack(q.codes.cpu().numpy())
    assert np.array_equal(q.scales.cpu().numpy(), scale)
    assert np.array_equal(got, code)


SHAPES = [(1, 1), (1, 32), (3, 31), (2, 33), (5, 127), (4, 128), (33, 1000), (129, 257), (128, 128), (300, 64), (1, 5000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_is_the_definition(shape, dtype):
    print("quantize", shape, dtype, flush=True)
    x = _values(shape, dtype, 1)
    xd = x.cuda()
    _check_form(ou.mx4_quantize(xd), R.host(x))
    q, qt = ou.mx4_quantize_both(xd)
    _check_form(q, R.host(x))
    _check_form(qt, R.host(x).T)
    _check_form(ou.mx4_quantize(xd.t()), R.host(x).T)       # a transposed view


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_extreme_blocks(dtype):
    """Blocks of the type's smallest and largest magnitudes, of one value
    beside zeros, of infinities and of NaN (also a NaN beside an infinity)."""
    f = torch.finfo(dtype)
    tiny = f.smallest_normal * f.eps
    rows = []
    for top in (tiny, 2 * tiny, 3 * tiny, f.smallest_normal, 2 * f.smallest_normal, f.max, 1.0, float("inf"),
                -float("inf"), float("nan"), 0.0, -0.0):
        for rest in (0.0, -0.0, tiny, f.max):
            r = [top] + [rest] * 31
            rows += [r, r[::-1]]
    rows.append([float("nan"), float("inf")] * 16)
    x = torch.tensor(rows, dtype=torch.float64).to(dtype)
    xd = x.cuda()
    q, qt = ou.mx4_quantize_both(xd)
    _check_form(q, R.host(x))
    _check_form(qt, R.host(x).T)
    _check_form(ou.mx4_quantize(xd), R.host(x))
    want = R.rounded(R.host(x))
    got = R.host(ou.mx4_dequantize(q, F32))
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_quantize_every_16_bit_value(dtype):
    """Every finite value of the type beside every power of two that can be
    its block's largest magnitude (the scale)."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    x = bits.view(dtype)
    x = x[torch.isfinite(x.float())]
    lo, hi = (-24, 15) if dtype == F16 else (-133, 127)
    for e in range(lo, hi + 1, 3):
        top = 2.0 ** e
        v = x[x.double().abs() < 2 * top]
        v = torch.cat((v, v.new_zeros(-v.numel() % 31))).view(-1, 31)
        v = torch.cat((torch.full((v.shape[0], 1), top, dtype=torch.float64).to(dtype), v), 1)
        _check_form(ou.mx4_quantize(v.cuda()), R.host(v))


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_strides_alignment_and_batches(dtype):
    big = _values((70, 301), dtype, 2).cuda()
    for view in (big[:, 1:], big[:, 3:67], big[::2, 8:200], big[5:6, 7:], big[:, :1], big[3:, 16:272]):
        q, qt = ou.mx4_quantize_both(view)
        _check_form(q, R.host(view))
        _check_form(qt, R.host(view).T)
        _check_form(ou.mx4_quantize(view), R.host(view))
    x = _values((3, 40, 200), dtype, 3).cuda()
    q, qt = ou.mx4_quantize_both(x)
    one = ou.mx4_quantize(x)
    for i in range(3):
        _check_form(q[i], R.host(x[i]))
        _check_form(qt[i], R.host(x[i]).T)
        _check_form(one[i], R.host(x[i]))
    for bad in (big[:, ::2], big.expand(2, 70, 301), x.transpose(1, 2)):
        with pytest.raises(ValueError):
            ou.mx4_quantize(bad)


def test_quantize_empty():
    for shape in ((0, 64), (5, 0), (0, 5, 64), (2, 0, 64)):
        q, qt = ou.mx4_quantize_both(torch.empty(shape, device="cuda"))
        assert tuple(q.shape) == shape and tuple(qt.shape) == (*shape[:-2], shape[-1], shape[-2])
        assert ou.mx4_dequantize(q).shape == q.shape


def _offsets(counts, front=0):
    return torch.tensor(np.concatenate([[front], front + np.cumsum(counts)]), dtype=torch.int32)


COUNTS = [[5], [0, 3, 0], [128, 1, 127, 0, 129], [33, 0, 64, 200], [1] * 70, [0] * 3, [300, 31]]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts", COUNTS)
def test_quantize_grouped(counts, dtype):
    t, c = sum(counts) + 3, 150
    x = _values((t, c), dtype, 4)
    off = _offsets(counts, 1)
    q, qt = ou.mx4_quantize_grouped(x.cuda(), off.cuda())
    x64 = R.host(x)
    code, scale = R.unpack(qt.codes.cpu().numpy()), qt.scales.cpu().numpy()
    held = R.held(q)
    at = 0
    for a, b in zip(off[:-1].tolist(), off[1:].tolist()):
        wc, ws = R.quantize(x64[a:b].T)
        w = R.columns(b - a)
        assert np.array_equal(code[:, at:at + w], wc) and np.array_equal(scale[:, at // 32:(at + w) // 32], ws)
        assert np.array_equal(held[a:b], R.rounded(x64[a:b]), equal_nan=True)
        at += w
    only = ou.mx4_quantize_grouped(x.cuda(), off.cuda(), rows=False)
    assert only[0] is None
    assert torch.equal(only[1].codes[:, :at // 2], qt.codes[:, :at // 2])


@pytest.mark.parametrize("dtype", DTYPES)
def test_dequantize_every_code_and_scale(dtype):
    scale = torch.arange(256, dtype=torch.uint8).repeat_interleave(4).view(256, 4)
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)[:, torch.randperm(256, generator=_gen(5))[:64]]
    codes[:, :8] = torch.tensor([0x10, 0x32, 0x54, 0x76, 0x98, 0xba, 0xdc, 0xfe], dtype=torch.uint8)
    for k in (128, 121, 1):
        q = ou.Mx4(codes.cuda(), scale.cuda(), k)
        want = torch.from_numpy(R.held(q)).to(dtype)         # rounded once, to nearest even
        got = ou.mx4_dequantize(q, dtype).cpu()
        assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0)) and torch.equal(got.isnan(), want.isnan())
        out = torch.full((256, k), 3.0, dtype=dtype, device="cuda")
        assert ou.mx4_dequantize(q, out=out) is out and torch.equal(out.cpu().nan_to_num(7.0), want.nan_to_num(7.0))


def _random_held(rows, k, seed, lo=119, hi=135, lead=()):
    """Any codes and scales, zeros behind k."""
    g = _gen(seed)
    p = R.columns(k)
    code = torch.randint(0, 16, (*lead, rows, p), generator=g, dtype=torch.uint8)
    code[..., k:] = 0
    scales = torch.randint(lo, hi, (*lead, rows, p // 32), generator=g, dtype=torch.uint8)
    codes = torch.from_numpy(R.pack(code.numpy())) if p else torch.zeros((*lead, rows, 0), dtype=torch.uint8)
    return ou.Mx4(codes.cuda().contiguous(), scales.cuda().contiguous(), k)


# rows, columns and depths around every border of the kernels' tiles
PRODUCTS = [(13, 70, 4100), (16, 33, 3000), (5, 16500, 300), (2, 20000, 140), (1, 1, 1), (1, 64, 128), (1, 4096, 1024), (2, 33, 33), (3, 300, 4000), (15, 17, 500), (16, 16, 129),
            (16, 512, 384), (17, 65, 256), (31, 127, 640), (32, 128, 100), (33, 129, 1100), (63, 40, 2048), (64, 64, 64),
            (65, 200, 900), (100, 1000, 257), (128, 256, 512), (129, 255, 511), (130, 2000, 700), (255, 129, 383),
            (256, 256, 256), (257, 257, 1025), (300, 70, 5000), (512, 512, 4096), (700, 900, 1300), (1030, 1100, 640), (40, 90, 1930), (40, 90, 2060),
            (500, 2100, 600), (500, 2100, 4100)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_matmul(m, n, k, dtype):
    print("matmul", m, n, k, dtype, flush=True)
    b = _random_held(n, k, 7)
    a = _random_held(m, k, 6)
    want, mag = R.product(R.held(a), R.held(b))
    R.check_product(ou.mx4_matmul(a, b, dtype), want, mag, k)
    # values on the left: bitwise the product of their 4-bit form
    x = _values((m, k), dtype, 8).cuda()
    got = ou.mx4_matmul(x, b)
    assert got.dtype == dtype
    xq = ou.mx4_quantize(x)
    want, mag = R.product(R.held(xq), R.held(b))
    R.check_product(got, want, mag, k)
    assert torch.equal(got, ou.mx4_matmul(xq, b, dtype))


# many tiles of 128 and of 256, ragged edges, odd and even numbers of k-steps
@pytest.mark.parametrize("m,n,k,dtype", [(1500, 1490, 129, F32), (1411, 1537, 1200, BF16), (2500, 700, 2200, F16),
                                         (4099, 4100, 100, BF16), (4200, 4001, 257, F32), (4097, 3905, 640, F16),
                                         (3841, 4100, 1300, F32), (200, 70000, 500, BF16)])
def test_matmul_many_tiles(m, n, k, dtype):
    print("many tiles", m, n, k, dtype, flush=True)
    a, b = _random_held(m, k, 28), _random_held(n, k, 29)
    a.scales[m // 2, 0] = 255                      # one NaN block: its row alone
    got = ou.mx4_matmul(a, b, dtype)
    want, mag = R.product(R.held(a), R.held(b))
    R.check_product(got, want, mag, k)
    buf = torch.full((m, n + 5), 3.0, dtype=dtype, device="cuda")
    ou.mx4_matmul(a, b, out=buf[:, 1:n + 1])       # no 16 bytes aligned
    assert torch.equal(buf[:, 1:n + 1].nan_to_num(7.0), got.nan_to_num(7.0))
    assert (buf[:, 0] == 3).all() and (buf[:, n + 1:] == 3).all()


@pytest.mark.parametrize("counts,front,back,n,k", [([700, 0, 1300, 129, 1], 0, 0, 1100, 300),
                                                   ([2100, 900, 0, 2000, 300], 3, 5, 4100, 200)])
def test_grouped_products_of_many_tiles(counts, front, back, n, k):
    t, e = front + sum(counts) + back, len(counts)
    off = _offsets(counts, front).cuda()
    x, b = _values((t, k), BF16, 34).cuda(), _random_held(n, k, 35, lead=(e,))
    dy = _values((t, n), BF16, 36).cuda()
    got = ou.mx4_grouped_matmul(x, b, off)
    xq, xt = ou.mx4_quantize_grouped(x, off)
    _, dt = ou.mx4_quantize_grouped(dy, off, rows=False)
    dw = ou.mx4_grouped_outer(dt, xt, off, t, F32)
    x64, d64 = R.host(x), R.host(dy)
    out = torch.full((t, n), 5.0, dtype=BF16, device="cuda")
    ou.mx4_grouped_matmul(x, b, off, out=out)
    for i, (lo, hi) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())):
        R.check_product(got[lo:hi], *R.product(R.rounded(x64[lo:hi]), R.held(b[i])), k)
        R.check_product(dw[i], *R.product(R.rounded(d64[lo:hi].T), R.rounded(x64[lo:hi].T)), max(1, hi - lo))
        assert torch.equal(out[lo:hi], got[lo:hi])
    for rest in (slice(0, front), slice(t - back, t)):
        assert (got[rest] == 0).all() and (out[rest] == 5).all()


@pytest.mark.parametrize("m,n", [(3, 40), (70, 65)])
@pytest.mark.parametrize("k", [(1 << 24) - 200, (1 << 25) - 5])
def test_matmul_of_the_greatest_depths(m, n, k):
    """Operands that are zero but for a few k-steps at the start, between and
    at the end: the product of those steps alone."""
    p = R.columns(k)
    steps = [0, 1, p // 256 - 1, p // 256, p // 128 - 3, p // 128 - 2, p // 128 - 1]
    forms = []
    for rows, seed in ((m, 90), (n, 91)):
        part = _random_held(rows, 128 * len(steps), seed)
        part.codes.view(rows, len(steps), 64)[:, -1, (k - p + 128) // 2:] = 0
        codes = torch.zeros(rows, p // 128, 64, dtype=torch.uint8, device="cuda")
        scales = torch.full((rows, p // 128, 4), 127, dtype=torch.uint8, device="cuda")
        codes[:, steps] = part.codes.view(rows, len(steps), 64)
        scales[:, steps] = part.scales.view(rows, len(steps), 4)
        forms.append((part, ou.Mx4(codes.view(rows, p // 2), scales.view(rows, p // 32), k)))
    (a, far_a), (b, far_b) = forms
    want, mag = R.product(R.held(a), R.held(b))
    R.check_product(ou.mx4_matmul(far_a, far_b, F32), want, mag, 128 * len(steps))


@pytest.mark.parametrize("m", [1, 16, 40, 200])
def test_matmul_scales_of_every_size(m):
    """Scales over the whole range of binary32, results up to infinity."""
    for seed, lo, hi in ((1, 60, 195), (2, 0, 66), (3, 180, 254)):
        a, b = _random_held(m, 512, seed, lo, hi), _random_held(70, 512, seed + 9, 127, 128)
        want, mag = R.product(R.held(a), R.held(b))
        R.check_product(ou.mx4_matmul(a, b, F32), want, mag, 512)


@pytest.mark.parametrize("m", [1, 9, 40, 300])
def test_matmul_nan_and_infinity_stay_in_their_rows(m):
    x = torch.ones(m, 200, device="cuda", dtype=BF16)
    w = torch.ones(150, 200, device="cuda", dtype=BF16)
    x[0, 3], w[7, 190] = float("nan"), float("inf")
    y = ou.mx4_matmul(x, ou.mx4_quantize(w))
    bad = torch.zeros(m, 150, dtype=torch.bool)
    bad[0], bad[:, 7] = True, True
    assert torch.equal(y.isnan().cpu(), bad) and (y.cpu()[~bad] == 200).all()


def test_matmul_depth_zero_and_empty_sides():
    z = ou.mx4_quantize(torch.empty(70, 0, device="cuda"))
    for m in (1, 5, 40, 300):
        assert torch.equal(ou.mx4_matmul(torch.empty(m, 0, device="cuda"), z), torch.zeros(m, 70, device="cuda"))
        assert torch.equal(ou.mx4_matmul(ou.mx4_quantize(torch.empty(m, 0, device="cuda")), z, F16),
                           torch.zeros(m, 70, device="cuda", dtype=F16))
    b = _random_held(70, 64, 1)
    assert ou.mx4_matmul(torch.empty(0, 64, device="cuda"), b).shape == (0, 70)
    none = ou.mx4_quantize(torch.empty(0, 64, device="cuda"))
    assert ou.mx4_matmul(torch.ones(3, 64, device="cuda"), none).shape == (3, 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n", [(1, 77), (12, 130), (50, 70), (200, 300), (260, 513)])
def test_matmul_into_part_of_a_matrix(m, n, dtype):
    """Strided results, also where no 4 of them are aligned: the rest of the
    buffer keeps its values.  x with strides and without alignment."""
    k = 200
    b = _random_held(n, k, 11)
    wide = _values((m, k + 9), dtype, 12).cuda()
    for shift in (0, 1, 8):
        x = wide[:, shift:shift + k]
        buf = torch.full((m + 2, n + 13), 3.0, dtype=dtype, device="cuda")
        out = buf[1:m + 1, shift:shift + n]
        assert ou.mx4_matmul(x, b, out=out) is out
        want = ou.mx4_matmul(x.contiguous(), b)
        keep = torch.full_like(buf, 3.0)
        keep[1:m + 1, shift:shift + n] = want
        assert torch.equal(buf, keep)


GROUPS = [([5], 0, 0), ([0, 3, 0, 1], 0, 0), ([1] * 16, 0, 0), ([2, 0, 1, 9, 4], 3, 2), ([128, 1, 127, 0, 129], 0, 1),
          ([33, 0, 64, 200], 2, 0), ([1] * 70, 0, 5), ([0] * 3, 0, 4), ([300, 31, 257], 0, 0), ([17] * 90, 1, 1)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,front,back", GROUPS)
@pytest.mark.parametrize("n,k", [(150, 200), (257, 640)])
def test_grouped_matmul(counts, front, back, n, k, dtype):
    print("grouped", counts[:8], front, back, n, k, dtype, flush=True)
    t, e = front + sum(counts) + back, len(counts)
    off = _offsets(counts, front)
    b = _random_held(n, k, 13, lead=(e,))
    x = _values((t, k), dtype, 14).cuda()
    xq = ou.mx4_quantize(x)
    got = ou.mx4_grouped_matmul(x, b, off.cuda())
    assert torch.equal(got, ou.mx4_grouped_matmul(xq, b, off.cuda(), dtype))
    a64, b64 = R.held(xq), R.held(b)
    want, mag = np.zeros((t, n)), np.zeros((t, n))
    for i, (lo, hi) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())):
        want[lo:hi], mag[lo:hi] = R.product(a64[lo:hi], b64[i])
    R.check_product(got, want, mag, k)
    # rows of no group stay as they were in a given result
    out = torch.full((t, n + 3), 5.0, dtype=dtype, device="cuda")
    ou.mx4_grouped_matmul(x, b, off.cuda(), out=out[:, :n])
    keep = torch.full_like(out, 5.0)
    keep[front:t - back, :n] = got[front:t - back]
    assert torch.equal(out, keep)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,front,back", GROUPS)
def test_grouped_outer(counts, front, back, dtype):
    m, n = 140, 270
    t, e = front + sum(counts) + back, len(counts)
    off = _offsets(counts, front)
    a, b = _values((t, m), dtype, 15), _values((t, n), dtype, 16)
    _, at = ou.mx4_quantize_grouped(a.cuda(), off.cuda(), rows=False)
    _, bt = ou.mx4_quantize_grouped(b.cuda(), off.cuda(), rows=False)
    got = ou.mx4_grouped_outer(at, bt, off.cuda(), t, dtype)
    a64, b64 = R.host(a), R.host(b)
    for i, (lo, hi) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())):
        want, mag = R.product(R.rounded(a64[lo:hi].T), R.rounded(b64[lo:hi].T))
        R.check_product(got[i], want, mag, max(1, hi - lo))


@pytest.mark.parametrize("bad", [[0, 50, 20, 90], [-5, 10, 60, 80], [0, 10, 500, 80], [90, 60, 30, 0],
                                 [2**31 - 1, -2**31, 2**31 - 1, -2**31]])
def test_offsets_that_point_nowhere_stay_inside(bad):
    """Offsets out of range or falling are clamped: nothing outside the
    result is written, and a group that is in order gets its rows."""
    t, n, k, e = 80, 70, 130, 3
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    x, b = _values((t, k), BF16, 17).cuda(), _random_held(n, k, 18, lead=(3,))
    buf = torch.full((t + 40, n), 5.0, dtype=BF16, device="cuda")
    ou.mx4_grouped_matmul(x, b, off, out=buf[20:20 + t])
    assert (buf[:20] == 5).all() and (buf[20 + t:] == 5).all()
    _, xt = ou.mx4_quantize_grouped(x, off)
    dw = ou.mx4_grouped_outer(xt, xt, off, t)
    assert dw.shape == (3, k, k)
    if bad == [0, 50, 20, 90]:
        want = ou.mx4_matmul(x[:50], b[0])
        assert torch.equal(buf[20:30], want[:10])


def _representable(shape, seed):
    """Whole numbers that every block holds exactly (a 4 in each fixes the
    scale at 1), along either axis."""
    g = _gen(seed)
    x = torch.tensor([0.0, 1, 2, 3, 4, 6])[torch.randint(0, 6, shape, generator=g)] * torch.where(
        torch.rand(shape, generator=g) < 0.5, -1.0, 1.0)
    r, c = shape[-2:]
    i, j = torch.arange(r).view(-1, 1), torch.arange(c).view(1, -1)
    return torch.where((i + j) % 32 == 0, torch.tensor(4.0), x)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(1, 40, 70), (33, 130, 200), (200, 256, 320)])
def test_linear_forward_and_gradients(m, n, k, dtype):
    x, w, dy = _values((m, k), dtype, 20), _values((n, k), dtype, 21), _values((m, n), dtype, 22)
    xd, wd = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    y = ou.mx4_linear(xd, wd)
    y.backward(dy.cuda())
    x64, w64, d64 = R.host(x), R.host(w), R.host(dy)
    R.check_product(y, *R.product(R.rounded(x64), R.rounded(w64)), k)
    R.check_product(xd.grad, *R.product(R.rounded(d64), R.rounded(w64.T)), n)
    R.check_product(wd.grad, *R.product(R.rounded(d64.T), R.rounded(x64.T)), m)
    # one gradient alone, and through kept 4-bit forms, gives the same bits
    held = ou.Mx4Weight(wd.detach().requires_grad_())
    for weight in (wd.detach(), held):
        x2 = x.cuda().requires_grad_()
        y2 = ou.mx4_linear(x2, weight)
        assert torch.equal(y2, y)
        y2.backward(dy.cuda())
        assert torch.equal(x2.grad, xd.grad)
    assert torch.equal(held.weight.grad, wd.grad)
    w2 = w.cuda().requires_grad_()
    ou.mx4_linear(x.cuda(), w2).backward(dy.cuda())
    assert torch.equal(w2.grad, wd.grad)
    # more axes in front, an expanded gradient
    w3, x3 = w.cuda().requires_grad_(), x.cuda().view(1, m, k).requires_grad_()
    y3 = ou.mx4_linear(x3, w3)
    assert y3.shape == (1, m, n) and torch.equal(y3[0], y)
    y3.sum().backward()
    one = np.ones((m, n))
    R.check_product(w3.grad, *R.product(R.rounded(one.T), R.rounded(x64.T)), m)


def test_linear_gradients_against_differences():
    """Where every value is held exactly the layer is bilinear, and its
    central differences along directions that keep it so are exact."""
    m, n, k = 64, 96, 128
    x, w, c = (_representable(s, i).cuda() for i, s in enumerate(((m, k), (n, k), (m, n))))
    xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
    loss = (ou.mx4_linear(xg, wg) * c).sum()
    loss.backward()

    def value(a, b):
        return (ou.mx4_linear(a, b).double() * c.double()).sum().item()

    g = _gen(3)
    for _ in range(6):
        # move a value between -1 and 1: both are held exactly
        i, j = int(torch.randint(0, m, (1,), generator=g)), int(torch.randint(0, k, (1,), generator=g))
        if (i + j) % 32:
            up, down = x.clone(), x.clone()
            up[i, j], down[i, j] = 1.0, -1.0
            assert (value(up, w) - value(down, w)) / 2 == xg.grad[i, j].item()
        i = int(torch.randint(0, n, (1,), generator=g))
        if (i + j) % 32:
            up, down = w.clone(), w.clone()
            up[i, j], down[i, j] = 1.0, -1.0
            assert (value(x, up) - value(x, down)) / 2 == wg.grad[i, j].item()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,front,back", [([33, 0, 64, 5], 0, 0), ([2, 1, 0], 3, 4), ([300, 31], 0, 1)])
def test_grouped_linear_forward_and_gradients(counts, front, back, dtype):
    t, n, k, e = front + sum(counts) + back, 130, 190, len(counts)
    x, w, dy = _values((t, k), dtype, 23), _values((e, n, k), dtype, 24), _values((t, n), dtype, 25)
    off = _offsets(counts, front)
    xd, wd = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    y = ou.mx4_grouped_linear(xd, wd, off.cuda())
    y.backward(dy.cuda())
    x64, w64, d64 = R.host(x), R.host(w), R.host(dy)
    inside = np.zeros(t, bool)
    for i, (a, b) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())):
        inside[a:b] = True
        R.check_product(y[a:b], *R.product(R.rounded(x64[a:b]), R.rounded(w64[i])), k)
        R.check_product(xd.grad[a:b], *R.product(R.rounded(d64[a:b]), R.rounded(w64[i].T)), n)
        R.check_product(wd.grad[i], *R.product(R.rounded(d64[a:b].T), R.rounded(x64[a:b].T)), max(1, b - a))
    assert (R.host(y)[~inside] == 0).all() and (R.host(xd.grad)[~inside] == 0).all()
    held = ou.Mx4Weight(wd.detach().requires_grad_())
    x2 = x.cuda().requires_grad_()
    y2 = ou.mx4_grouped_linear(x2, held, off.cuda())
    y2.backward(dy.cuda())
    assert torch.equal(y2, y) and torch.equal(x2.grad, xd.grad) and torch.equal(held.weight.grad, wd.grad)


@pytest.mark.parametrize("make", [lambda p: ou.AdamW32(p, lr=1e-2), lambda p: ou.AdamW8bit(p, lr=1e-2),
                                  lambda p: ou.Lion32(p, lr=1e-3), lambda p: ou.AdamW32(p, lr=1e-2, max_unorm=1.0)])
@pytest.mark.parametrize("how", ["step", "graph", "per tensor"])
def test_training_with_kept_forms(make, how):
    """Two layers and an expert layer trained through kept 4-bit forms, two
    micro-batches a step: every step's products are those of the weights that
    the optimizer has just updated, bit for bit."""
    m, k, h, n = 60, 96, 128, 64
    off = _offsets([20, 0, 40]).cuda()
    w1, w2 = (torch.nn.Parameter(_values(s, BF16, i, special=False).cuda() * 0.1) for i, s in ((80, (h, k)), (81, (n, h))))
    we = torch.nn.Parameter(_values((3, n, n), BF16, 82, special=False).cuda() * 0.1)
    params = [w1, w2, we]
    for p in params:
        p.grad = torch.zeros_like(p)
    opt = make(params)
    held = [ou.Mx4Weight(p) for p in params]
    opt.attach_mx4(held)
    for step in range(3):
        opt.zero_grad()
        want = [torch.zeros_like(p) for p in params]
        for micro in range(2):
            x = _values((m, k), BF16, 90 + 2 * step + micro, special=False).cuda()
            outs = []
            for a, b, c in (held, params):
                y = ou.mx4_grouped_linear(ou.mx4_linear(ou.mx4_linear(x, a).relu(), b), c, off)
                outs.append(y)
            assert torch.equal(outs[0], outs[1])
            dy = _values((m, n), BF16, 70 + micro, special=False).cuda()
            grads = torch.autograd.grad(outs[1], params, dy)
            outs[0].backward(dy)                      # adds to .grad in place
            for t, g in zip(want, grads):
                t += g
        for p, t in zip(params, want):
            assert torch.equal(p.grad, t)
        before = [p.detach().clone() for p in params]
        opt.step_per_tensor() if how == "per tensor" else opt.step(graph=how == "graph")
        for p, b, q in zip(params, before, held):
            assert not torch.equal(p, b)
            fresh = ou.mx4_quantize_both(p.detach())
            for got, new in zip((q.q, q.qt), fresh):
                assert torch.equal(got.codes, new.codes) and torch.equal(got.scales, new.scales)
    with pytest.raises(ValueError):
        opt.attach_mx4([ou.Mx4Weight(torch.ones(4, 4, device="cuda"))])
    with pytest.raises(ValueError):
        opt.attach_mx4([w1])
    opt.close()


def test_results_do_not_change_from_call_to_call():
    x, w = _values((500, 900), BF16, 26).cuda(), _values((700, 900), BF16, 27).cuda()
    first = ou.mx4_matmul(x, ou.mx4_quantize(w))
    for _ in range(5):
        assert torch.equal(ou.mx4_matmul(x, ou.mx4_quantize(w)), first)


@pytest.mark.parametrize("m", [1, 48, 600])
def test_captured_and_replayed(m):
    """A whole training step of the layer in a graph, replayed on new inputs
    with eager work between the replays."""
    k, n, counts = 256, 384, [m // 3, 0, m - m // 3]
    off = _offsets(counts).cuda()
    x, w = _values((m, k), BF16, 30).cuda().requires_grad_(), _values((n, k), BF16, 31).cuda().requires_grad_()
    we = _values((3, n, k), BF16, 32).cuda().requires_grad_()
    dy = _values((m, n), BF16, 33).cuda()

    def step():
        y = ou.mx4_linear(x, w)
        z = ou.mx4_grouped_linear(x, we, off)
        return [y.detach(), z.detach(), *torch.autograd.grad(y, (x, w), dy), *torch.autograd.grad(z, (x, we), dy),
                ou.mx4_matmul(x.detach(), ou.mx4_quantize(w.detach()))]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in range(4):
        with torch.no_grad():
            x.copy_(_values((m, k), BF16, 40 + seed))
            w.copy_(_values((n, k), BF16, 50 + seed))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, step()):
            assert torch.equal(got, want)


def test_streams():
    """Calls on a stream of their own, as an object and as a handle, one of
    them current; the two at once do not meet."""
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    x, w = _values((300, 512), BF16, 60).cuda(), _values((256, 512), BF16, 61).cuda()
    q = ou.mx4_quantize(w)
    want = ou.mx4_matmul(x, q)
    torch.cuda.synchronize()
    outs = []
    for i in range(8):
        outs.append(ou.mx4_matmul(x, q, stream=a))
        outs.append(ou.mx4_matmul(x, q, stream=b.cuda_stream))
        with torch.cuda.stream(a):
            outs.append(ou.mx4_matmul(x, ou.mx4_quantize(w)))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_rows_far_behind_4_gib():
    """A matrix whose codes and whose results pass 32-bit offsets."""
    n, k = (1 << 20) + 5, 8192 + 128
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.randint(120, 130, (n, k // 32), dtype=torch.uint8, device="cuda")
    b = ou.Mx4(codes, scales, k)
    assert codes.numel() > 1 << 32
    a = _random_held(2, k, 70)
    got = ou.mx4_matmul(a, b, F32)
    tail = ou.Mx4(codes[-300:].clone(), scales[-300:].clone(), k)
    R.check_product(got[:, -300:], *R.product(R.held(a), R.held(tail)), k)
    # as the left operand: results of 2^20 rows, and the 4-bit form's values
    c = _random_held(1030, k, 71)
    out = ou.mx4_matmul(b, c, F32)
    assert out.numel() * 4 > 1 << 32
    R.check_product(out[-300:], *R.product(R.held(tail), R.held(c)), k)
    back = ou.mx4_dequantize(tail, BF16)
    again = ou.mx4_quantize(back)
    assert np.array_equal(R.held(again), R.held(tail))


@pytest.mark.parametrize("grouped", [False, True])
def test_layers_without_gradients(grouped):
    """Where no gradients are recorded the layers are the products alone, also
    of leaves that require gradients: no form of x that outlives the call and
    none along the rows (x [4096, 1024]: 2.1 MiB each, of it the values' form
    passes through the workspace)."""
    m, n, k = 4096, 64, 1024
    x = _values((m, k), BF16, 87).cuda().requires_grad_()
    w = _values((2, n, k) if grouped else (n, k), BF16, 88).cuda().requires_grad_()
    off = torch.tensor([0, 1000, m], dtype=torch.int32, device="cuda")
    held = ou.Mx4Weight(w)

    def layer():
        return ou.mx4_grouped_linear(x, held, off) if grouped else ou.mx4_linear(x, held)

    xs = x.detach()
    want = ou.mx4_grouped_matmul(xs, held.q, off) if grouped else ou.mx4_matmul(xs, held.q)
    assert torch.equal(layer(), want)
    form = m * k // 2 + m * k // 32
    for mode in (torch.no_grad, torch.inference_mode):
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        with mode():
            y = layer()
        assert torch.equal(y, want) and not y.requires_grad
        del y
        # the result, the form, the comparison's flags and roundings of sizes
        assert torch.cuda.max_memory_allocated() - before < 1.5 * form + m * n * 3


def test_no_rows_no_groups():
    """No rows at all, or no groups: empty results, zero gradients."""
    w = _values((64, 96), BF16, 85).cuda().requires_grad_()
    x = torch.empty(0, 96, device="cuda", dtype=BF16, requires_grad=True)
    ou.mx4_linear(x, w).backward(torch.empty(0, 64, device="cuda", dtype=BF16))
    assert x.grad.shape == (0, 96) and (w.grad == 0).all()
    we = _values((3, 64, 96), BF16, 86).cuda().requires_grad_()
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 96, device="cuda", dtype=BF16, requires_grad=True)
    ou.mx4_grouped_linear(x, we, off).backward(torch.empty(0, 64, device="cuda", dtype=BF16))
    assert (we.grad == 0).all()
    none = ou.mx4_quantize(torch.empty(0, 64, 96, device="cuda"))
    for t in (1, 5, 300):
        y = ou.mx4_grouped_matmul(torch.ones(t, 96, device="cuda"), none, off[:1])
        assert torch.equal(y, torch.zeros(t, 64, device="cuda"))


def test_layers_take_any_strides():
    """An input and a gradient whose rows overlap or whose columns are apart
    are copied; the 4-bit forms must stay until the backward pass."""
    x, w = _values((40, 96), BF16, 83).cuda(), _values((64, 96), BF16, 84).cuda()
    for view in (x.t().contiguous().t(), x[:1].expand(40, 96), torch.cat((x, x), 1)[:, 3:99], x[::2]):
        v = view.detach().requires_grad_()
        d = v.detach().contiguous().requires_grad_()
        for dy in (torch.ones(view.shape[0], 64, device="cuda", dtype=BF16).t().contiguous().t(),
                   torch.ones((), device="cuda", dtype=BF16).expand(view.shape[0], 64)):
            got = torch.autograd.grad(ou.mx4_linear(v, w), v, dy)[0]
            want = torch.autograd.grad(ou.mx4_linear(d, w), d, dy.contiguous())[0]
            assert torch.equal(got, want)
    held = ou.Mx4Weight(w.clone().requires_grad_())
    y = ou.mx4_linear(x.clone().requires_grad_(), held)
    held.refresh()
    with pytest.raises(RuntimeError):
        y.sum().backward()


def test_refusals_on_the_device():
    x = torch.ones(4, 64, device="cuda")
    q = ou.mx4_quantize(x)
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    e = ou.mx4_quantize(x[None])
    for call in (lambda: ou.mx4_quantize(x.int()), lambda: ou.mx4_quantize(x[0]), lambda: ou.mx4_matmul(x[:, :32], q),
                 lambda: ou.mx4_matmul(x, e), lambda: ou.mx4_matmul(x, q, torch.float64),
                 lambda: ou.mx4_matmul(x, q, out=torch.empty(4, 5, device="cuda")),
                 lambda: ou.mx4_matmul(x, q, out=torch.empty(4, 8, device="cuda")[:, ::2]),
                 lambda: ou.mx4_matmul(x, q, out=torch.empty(4, 4)),
                 lambda: ou.mx4_grouped_matmul(x, e, off.long()), lambda: ou.mx4_grouped_matmul(x, e, off.cpu()),
                 lambda: ou.mx4_grouped_matmul(x, e, off[:1]), lambda: ou.mx4_grouped_matmul(x, q, off),
                 lambda: ou.mx4_grouped_outer(q, q, off, 4), lambda: ou.mx4_dequantize(q, torch.int32),
                 lambda: ou.mx4_dequantize(q, out=torch.empty(4, 63, device="cuda")),
                 lambda: ou.mx4_linear(x, x.t()), lambda: ou.mx4_linear(x[:, :32], x),
                 lambda: ou.mx4_grouped_linear(x, x[None], off[:1])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(_lib.OptimizerUpdateError) as err:       # the result over the operand
        ou.mx4_matmul(x, q, out=x[:, :4])
    assert err.value.status == -4


def test_replaced_weights_are_refused():
    """Kept forms whose weight was replaced by one of another shape, or that
    are on another device than it: refused before anything is launched."""
    x = torch.ones(5, 96, device="cuda")
    for now in ((65, 96), (640, 96), (32, 96)):
        held = ou.Mx4Weight(torch.ones(64, 96, device="cuda"))
        assert ou.mx4_linear(x, held).shape == (5, 64)
        held.weight.data = torch.ones(now, device="cuda")
        for call in (lambda: ou.mx4_linear(x, held), held.refresh):
            with pytest.raises(ValueError, match="forms are of a weight of shape"):
                call()
    off = torch.tensor([0, 2, 5, 5], dtype=torch.int32, device="cuda")
    held = ou.Mx4Weight(torch.ones(2, 64, 96, device="cuda"))
    held.weight = torch.ones(3, 64, 96, device="cuda")
    with pytest.raises(ValueError, match="forms are of a weight of shape"):
        ou.mx4_grouped_linear(x, held, off)
    held = ou.Mx4Weight(torch.ones(64, 96, device="cuda"))
    held.q = ou.Mx4(held.q.codes.cpu(), held.q.scales.cpu(), 96)
    with pytest.raises(ValueError, match="forms are on another device"):
        ou.mx4_linear(x, held)


@pytest.mark.parametrize("grouped", [False, True])
def test_forms_for_the_backward_pass_are_saved_tensors(grouped):
    """What a layer keeps is freed by the backward pass although the result
    lives, passes through hooks on saved tensors, and is dropped and made again
    under a checkpoint."""
    from torch.utils.checkpoint import checkpoint
    m, n, k = 2048, 128, 1024
    x = _values((m, k), BF16, 93).cuda().requires_grad_()
    w = _values((2, n, k) if grouped else (n, k), BF16, 94).cuda().requires_grad_()
    dy = _values((m, n), BF16, 95).cuda()
    off = torch.tensor([0, 900, m], dtype=torch.int32, device="cuda")

    def layer(x, w):
        return ou.mx4_grouped_linear(x, w, off) if grouped else ou.mx4_linear(x, w)

    form = m * k // 2 + m * k // 32                    # x along its rows, without padding
    y = layer(x, w)
    before = torch.cuda.memory_allocated()
    want = torch.autograd.grad(y, (x, w), dy)
    made = sum(t.numel() * 2 for t in want)
    assert torch.cuda.memory_allocated() <= before + made - form
    with pytest.raises(RuntimeError):                  # once, like torch's own layers
        torch.autograd.grad(y, (x, w), dy)
    packed = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: packed.append(t) or t.cpu(), lambda t: t.cuda()):
        y2 = layer(x, w)
    assert sum(t.numel() * t.element_size() for t in packed) >= form
    del packed
    for got, ref in zip(torch.autograd.grad(y2, (x, w), dy), want):
        assert torch.equal(got, ref)
    before = torch.cuda.memory_allocated()
    y3 = checkpoint(layer, x, w, use_reentrant=False)
    assert torch.cuda.memory_allocated() < before + m * n * 2 + form // 2
    for got, ref in zip(torch.autograd.grad(y3, (x, w), dy), want):
        assert torch.equal(got, ref)


def _falling(t):
    return [[0, t, t // 2, 4 * t // 5], [3, t // 2, t // 4, t - 2], [t + 5, -3, t // 2, 2], [-7, 2**31 - 1, 0, 5],
            [t // 3, t // 5, t // 2, t // 2 - 1]]


# few rows; tiles of 64, with the k-steps shared, of 128, of 256
@pytest.mark.parametrize("t,n,k", [(10, 40, 130), (100, 70, 300), (100, 70, 4100), (2500, 1200, 130), (4100, 2100, 130)])
def test_offsets_that_fall_make_no_row_of_two_groups(t, n, k):
    """An offset below an earlier one counts as that one: every row of a new
    result is of one group, or 0; each group's part of the contraction is of
    its own rows."""
    x, b = _values((t, k), BF16, 97).cuda(), _random_held(n, k, 98, lead=(3,))
    x64 = R.host(x)
    for bad in _falling(t):
        print("falling", t, n, k, bad, flush=True)
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        rising = np.maximum.accumulate(np.clip(bad, 0, t))
        rest = torch.full((t, n), float("nan"), dtype=BF16, device="cuda")
        del rest                                       # what a new result is made of
        got = ou.mx4_grouped_matmul(x, b, off)
        into = torch.full((t, n), 5.0, dtype=BF16, device="cuda")
        ou.mx4_grouped_matmul(x, b, off, out=into)
        q, xt = ou.mx4_quantize_grouped(x, off)
        assert torch.equal(got, ou.mx4_grouped_matmul(q, b, off))
        dw = ou.mx4_grouped_outer(xt, xt, off, t, F32) if k < 1000 else None
        inside = np.zeros(t, bool)
        for e, (lo, hi) in enumerate(zip(rising[:-1], rising[1:])):
            inside[lo:hi] = True
            R.check_product(got[lo:hi], *R.product(R.rounded(x64[lo:hi]), R.held(b[e])), k)
            if dw is not None:
                R.check_product(dw[e], *R.product(R.rounded(x64[lo:hi].T), R.rounded(x64[lo:hi].T)), max(1, hi - lo))
        inside = torch.from_numpy(inside).cuda()
        assert (got[~inside] == 0).all() and (into[~inside] == 5).all() and torch.equal(into[inside], got[inside])


@pytest.mark.parametrize("groups", [63, 64, 65, 150, 200])
def test_offsets_of_many_groups_that_fall(groups):
    """More groups than lanes: what an earlier chunk of groups has reached
    counts for the later ones."""
    t, n, k = 1000, 40, 130
    g = _gen(groups)
    bad = torch.sort(torch.randint(-20, t + 20, (groups + 1,), generator=g)).values
    bad += torch.randint(-60, 60, (groups + 1,), generator=g)
    bad[groups // 2] = t - 300                          # behind it most fall
    rising = np.maximum.accumulate(np.clip(bad.numpy(), 0, t))
    off = bad.to(torch.int32).cuda()
    x, b = _values((t, k), BF16, 99).cuda(), _random_held(n, k, 100, lead=(groups,))
    x64 = R.host(x)
    for rows in (t, 37):                                # few rows a group, and hardly any
        ends = np.minimum(rising, rows)
        got = ou.mx4_grouped_matmul(x[:rows], b, off)
        _, xt = ou.mx4_quantize_grouped(x[:rows], off)
        dw = ou.mx4_grouped_outer(xt, xt, off, rows, F32)
        inside = torch.zeros(rows, dtype=torch.bool, device="cuda")
        for e, (lo, hi) in enumerate(zip(ends[:-1], ends[1:])):
            inside[lo:hi] = True
            R.check_product(got[lo:hi], *R.product(R.rounded(x64[lo:hi]), R.held(b[e])), k)
            R.check_product(dw[e], *R.product(R.rounded(x64[lo:hi].T), R.rounded(x64[lo:hi].T)), max(1, hi - lo))
        assert (got[~inside] == 0).all()


def test_forms_older_than_their_weight_are_used_with_a_warning():
    """The layers use kept forms as they are; a weight that torch, a new
    tensor or an optimizer without these forms has written since is warned of,
    until the forms are refreshed."""
    x = _values((9, 96), BF16, 101).cuda()
    w = torch.nn.Parameter(_values((64, 96), BF16, 102, special=False).cuda())
    w.grad = torch.ones_like(w)
    held, other = ou.Mx4Weight(w), ou.Mx4Weight(torch.ones(64, 96, device="cuda", dtype=BF16))
    opt = ou.AdamW32([w], lr=1e-2)

    def quiet(form=held):
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            return ou.mx4_linear(x, form)

    def stepped(attached):
        opt.attach_mx4(attached)
        opt.step()

    def assigned():
        held.weight = torch.nn.Parameter(w.detach() + 1)

    quiet()
    for write in (lambda: w.detach().copy_(_values((64, 96), BF16, 103)), lambda: stepped([]), assigned):
        old = quiet()
        write()
        with pytest.warns(UserWarning, match="refresh"):
            assert torch.equal(ou.mx4_linear(x, held), old)
        held.refresh()
        assert torch.equal(quiet(), ou.mx4_linear(x, held.weight))
    held.weight = w
    stepped([held])
    assert torch.equal(quiet(), ou.mx4_linear(x, w))
    quiet(other)
    with torch.inference_mode():
        form = ou.Mx4Weight(torch.ones(64, 96, device="cuda", dtype=BF16))
        quiet(form)
    opt.close()


def _check_by_rows(counts, front, back, n, k, dtype, seed):
    t, e = front + sum(counts) + back, len(counts)
    off = _offsets(counts, front).cuda()
    x, b = _values((t, k), dtype, seed).cuda(), _random_held(n, k, seed + 1, lead=(e,))
    q = ou.mx4_quantize(x)
    got = ou.mx4_grouped_matmul(q, b, off, dtype)
    assert torch.equal(got, ou.mx4_grouped_matmul(x, b, off))
    buf = torch.full((t, n + 3), 5.0, dtype=dtype, device="cuda")
    ou.mx4_grouped_matmul(q, b, off, out=buf[:, :n])
    held = R.held(q)
    for i, (lo, hi) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())):
        R.check_product(got[lo:hi], *R.product(held[lo:hi], R.held(b[i])), k)
    for rest in (slice(0, front), slice(t - back, t)):
        assert (got[rest] == 0).all() and (buf[rest] == 5).all()
    assert torch.equal(buf[front:t - back, :n], got[front:t - back]) and (buf[:, n:] == 5).all()


# By rows, 64-tiles whose k-steps two groups of waves share (17, 33 and 16
# steps, the last two groups' parts of even and odd numbers); then 256-tiles of
# 3 and 8 steps with ragged edges and rows of no group.
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,front,back,n,k", [([33, 0, 64, 200], 2, 5, 150, 2060), ([70, 1, 129], 0, 1, 65, 4100),
                                                   ([20, 31, 17], 1, 0, 257, 2048), ([2400, 0, 1500, 1893], 3, 4, 2100, 300),
                                                   ([1900, 1301, 1107], 3, 4, 2101, 900)])
def test_grouped_matmul_of_every_tile(counts, front, back, n, k, dtype):
    print("by rows", counts, n, k, dtype, flush=True)
    _check_by_rows(counts, front, back, n, k, dtype, 110)


# By contraction: 64-tiles with shared k-steps, groups of 11, 0, 2, 6, 3 and 1
# steps (a group's steps start anywhere, its second half is odd, or nothing);
# of 21, 1 and 12; then tiles of 128 and of 256 with odd numbers of steps.
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,m,n", [([1400, 0, 129, 700, 300, 1], 140, 270), ([2600, 100, 1500], 20, 33),
                                        ([300, 0, 700], 1200, 1100), ([300, 650, 130], 2100, 2101)])
def test_grouped_outer_of_every_tile(counts, m, n, dtype):
    print("by contraction", counts, m, n, dtype, flush=True)
    front, back = 1, 2
    t = front + sum(counts) + back
    off = _offsets(counts, front)
    a, b = _values((t, m), dtype, 112), _values((t, n), dtype, 113)
    at, bt = (ou.mx4_quantize_grouped(v.cuda(), off.cuda(), rows=False)[1] for v in (a, b))
    got = ou.mx4_grouped_outer(at, bt, off.cuda(), t, dtype)
    a64, b64 = R.host(a), R.host(b)
    for i, (lo, hi) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())):
        R.check_product(got[i], *R.product(R.rounded(a64[lo:hi].T), R.rounded(b64[lo:hi].T)), max(1, hi - lo))


def test_every_unattached_form_of_a_stepped_weight_is_stale():
    """Also where one form is attached twice, or a copy of a form is."""
    import copy
    x = torch.ones(3, 64, device="cuda", dtype=BF16)
    for attach in (lambda a: [a, a], lambda a: [copy.copy(a)]):
        w = torch.nn.Parameter(_values((32, 64), BF16, 104, special=False).cuda())
        w.grad = torch.ones_like(w)
        held, other = ou.Mx4Weight(w), ou.Mx4Weight(w)
        opt = ou.AdamW32([w], lr=1e-2)
        opt.attach_mx4(attach(held))
        opt.step()
        with pytest.warns(UserWarning, match="refresh"):
            ou.mx4_linear(x, other)
        opt.close()


def test_handle_of_the_default_stream():
    """A call on the handle of the default stream is ordered with that stream's
    work, also while another one is current."""
    from optimizer_update_amd import mx4
    handle = torch.cuda.default_stream().cuda_stream
    with mx4._Call(torch.cuda.current_device(), handle) as got:
        assert got == handle and torch.cuda.current_stream() == torch.cuda.default_stream()
    w = torch.nn.Parameter(_values((512, 1024), BF16, 105, special=False).cuda())
    w.grad = torch.ones_like(w)
    x, held = _values((64, 1024), BF16, 106).cuda(), ou.Mx4Weight(w)
    opt = ou.AdamW32([w], lr=1e-2)
    opt.attach_mx4([held])
    for _ in range(4):
        opt.step(stream=handle)
        got = ou.mx4_matmul(x, held.q, stream=handle)
        assert torch.equal(got, ou.mx4_matmul(x, ou.mx4_quantize(w.detach())))
    opt.close()
