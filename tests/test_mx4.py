"""CPU: the library of the 4-bit operators: its exports, its refusals (no
device is touched before the arguments are checked) and the binding's."""
import contextlib
import ctypes
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import optimizer_update_amd as ou
from optimizer_update_amd import _lib, mx4
from tests import mx4_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, EUNSUPPORTED, EALIGN, EOVERLAP = 0, -1, -2, -3, -4
X, C, S, CT, ST, O, W = (0x100000000 * i for i in range(1, 8))


@pytest.fixture(scope="module")
def L():
    return ou.load_mx4()


@pytest.fixture
def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("calls that pass the checks would launch on these addresses")


def test_exports_every_header_function(L):
    names = _lib.header_functions(mx4.HEADER)
    assert len(names) == 13 and len(set(names)) == 13
    out = subprocess.run(["nm", "-D", "--defined-only", mx4.LIBRARY], capture_output=True, text=True, check=True).stdout
    assert set(re.findall(r" T (\w+)$", out, flags=re.M)) == set(names)


def test_header_is_plain_c(tmp_path):
    c = tmp_path / "t.c"
    c.write_text('#include "optimizer_mx4.h"\nint main(void) { return ou_mx4_columns(1) == 128 ? 0 : 1; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-c", str(c), "-o",
                    str(tmp_path / "t.o")], check=True)


def _registers(operand):
    m = re.match(r"([va])\[(\d+):(\d+)\]$", operand)
    if m:
        return {(m[1], i) for i in range(int(m[2]), int(m[3]) + 1)}
    m = re.match(r"([va])(\d+)$", operand)
    return {(m[1], int(m[2]))} if m else set()


def _wait_state_faults(instructions):
    """Places where a matrix instruction stands within two wait states of the
    vector instruction that makes one of its operands, or where a vector
    instruction touches an accumulator within 18 of the matrix instruction
    that makes it."""
    faults, made, summed, now = [], {}, {}, 0
    for op, operands in instructions:
        now += 1 + (int(operands[0]) if op == "s_nop" else 0)
        if op.startswith("v_mfma"):
            for r in set().union(*map(_registers, operands[1:6])):
                if now - made.get(r, -9) <= 2:
                    faults.append((now, op, r))
            summed |= dict.fromkeys(_registers(operands[0]), now)
        elif op.startswith("v_"):
            for r in set().union(*map(_registers, operands)) if operands else ():
                if now - summed.get(r, -99) <= 18:
                    faults.append((now, op, r))
            made |= dict.fromkeys(_registers(operands[0]) if operands else (), now)
    return faults


def test_matrix_instructions_keep_their_wait_states(tmp_path):
    """The tiled products write their matrix instruction as assembly, for which
    the compiler inserts no wait states: in what it makes of the kernels here,
    none is missing (checked in the order of the text, in which a loop's end is
    followed by more than that, and its barrier by an s_nop)."""
    made = [("v_bfe_u32", ["v1", "v2", "s0", "8"]), ("v_mfma_x", ["a[0:3]", "v[4:7]", "v[8:11]", "a[0:3]", "v1", "v3"])]
    assert _wait_state_faults(made) and not _wait_state_faults([made[0], ("s_nop", ["1"]), made[1]])
    assert _wait_state_faults([made[1], ("v_accvgpr_read_b32", ["v9", "a2"])])
    from optimizer_update_amd import build
    out = tmp_path / "k.s"
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-shared", "-fPIC", "-Wall")]
    subprocess.run(["/opt/rocm/bin/hipcc", *flags, "-S", "--cuda-device-only", build.MX4_SOURCES[0], "-o", str(out)],
                   check=True, capture_output=True)
    kernels = re.findall(r"^(_ZN3mx4\S*k_matmul_tile\S*):[^\n]*\n(.*?)^\.Lfunc_end", out.read_text(), flags=re.M | re.S)
    assert len(kernels) == 36
    for name, body in kernels:
        instructions = []
        for line in body.split("\n"):
            words = line.split(";")[0].replace(",", " ").split()
            if words and not words[0].startswith(".") and not words[0].endswith(":"):
                instructions.append((words[0], words[1:]))
        assert sum(op.startswith("v_mfma") for op, _ in instructions) in (8, 32, 128), name
        assert not _wait_state_faults(instructions), name


def test_missing_library_fails_loudly(tmp_path):
    with pytest.raises(ImportError):
        ou.load_mx4(str(tmp_path / "liboptimizer_mx4.so"))


@pytest.mark.parametrize("k,p", [(0, 0), (1, 128), (127, 128), (128, 128), (129, 256), (1 << 31, 1 << 31), (-1, -1)])
def test_columns(L, k, p):
    assert L.ou_mx4_columns(k) == p


@pytest.mark.parametrize("counts", [[], [0], [1], [128], [129, 0, 1], [127, 128, 129], [1] * 50])
def test_grouped_columns_hold_any_split(L, counts):
    rows = sum(counts)
    have = L.ou_mx4_grouped_columns(rows, len(counts))
    assert have % 128 == 0 and have >= sum(R.columns(c) for c in counts)
    assert L.ou_mx4_grouped_columns(-1, 1) == -1 and L.ou_mx4_grouped_columns(1, -1) == -1


def _quantize(L, dtype=0, x=X, batch=1, rows=64, cols=256, rs=256, bs=0, c=C, s=S, ct=None, st=None):
    return L.ou_mx4_quantize(dtype, x, batch, rows, cols, rs, bs, c, s, ct, st, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), EINVAL), (dict(dtype=-1), EINVAL), (dict(x=None), EINVAL), (dict(rows=-1), EINVAL),
    (dict(cols=-1), EINVAL), (dict(rows=(1 << 31) + 1), EINVAL), (dict(rs=255), EINVAL), (dict(batch=-1), EINVAL),
    (dict(batch=65536), EINVAL), (dict(batch=2, bs=255), EINVAL), (dict(bs=-1), EINVAL), (dict(c=None), EINVAL),
    (dict(s=None), EINVAL), (dict(c=None, s=None), EINVAL), (dict(ct=CT), EINVAL), (dict(st=ST), EINVAL),
    (dict(x=X + 2), EALIGN), (dict(dtype=1, x=X + 1), EALIGN), (dict(c=C + 8), EALIGN), (dict(s=S + 2), EALIGN),
    (dict(ct=CT + 4, st=ST), EALIGN), (dict(c=X), EOVERLAP), (dict(c=X + 64 * 256 * 4 - 16), EOVERLAP),
    (dict(s=C + 64), EOVERLAP), (dict(ct=CT, st=C), EOVERLAP), (dict(ct=C, st=ST), EOVERLAP),
    (dict(rows=1 << 31, cols=1 << 31, rs=1 << 31), EINVAL),
])
def test_quantize_refusals(L, kw, code):
    assert _quantize(L, **kw) == code
    assert L.ou_mx4_last_error()


def test_quantize_passes_its_checks(L, no_gpu):
    assert _quantize(L) == EUNSUPPORTED
    assert _quantize(L, c=X + 64 * 256 * 4) == EUNSUPPORTED      # right behind x
    assert _quantize(L, c=None, s=None, ct=CT, st=ST) == EUNSUPPORTED
    assert _quantize(L, batch=3, bs=64 * 256, ct=CT, st=ST) == EUNSUPPORTED


def test_nothing_to_do_is_no_error(L):
    assert _quantize(L, rows=0, x=None) == OK and _quantize(L, cols=0, x=None) == OK
    assert _quantize(L, batch=0, x=None) == OK
    assert L.ou_mx4_dequantize(0, None, None, 0, 5, None, 5, None) == OK
    assert L.ou_mx4_matmul(0, None, None, 0, None, None, 4, 4, None, 4, None, 0, None) == OK
    assert L.ou_mx4_matmul(0, None, None, 4, None, None, 0, 4, None, 4, None, 0, None) == OK
    assert L.ou_mx4_grouped_outer(0, C, S, 8, CT, ST, 8, 0, X, 0, None, None) == OK


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), EINVAL), (dict(rows=-1), EINVAL), (dict(cols=-2), EINVAL), (dict(rs=99), EINVAL),
    (dict(off=None), EINVAL), (dict(off=O + 2), EALIGN), (dict(groups=-1), EINVAL), (dict(groups=65536), EINVAL),
    (dict(c=None), EINVAL), (dict(ct=None), EINVAL), (dict(st=None), EINVAL), (dict(ct=CT + 1), EALIGN),
    (dict(ct=X), EOVERLAP), (dict(st=O), EOVERLAP), (dict(x=None), EINVAL),
])
def test_quantize_grouped_refusals(L, kw, code):
    a = dict(dtype=2, x=X, rows=200, cols=100, rs=100, off=O, groups=4, c=C, s=S, ct=CT, st=ST) | kw
    assert L.ou_mx4_quantize_grouped(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), EINVAL), (dict(rows=-1), EINVAL), (dict(cols=-1), EINVAL), (dict(rs=63), EINVAL),
    (dict(c=None), EINVAL), (dict(out=None), EINVAL), (dict(out=O + 1), EALIGN), (dict(out=C), EOVERLAP),
    (dict(c=C + 4), EALIGN), (dict(s=S + 1), EALIGN),
])
def test_dequantize_refusals(L, kw, code):
    a = dict(dtype=0, c=C, s=S, rows=16, cols=64, out=O, rs=64) | kw
    assert L.ou_mx4_dequantize(*a.values(), None) == code


MATMUL = dict(dt=2, a=X, as_=X + (1 << 24), m=40, b=C, bs=S, n=72, k=300, out=O, os=72, ws=W, wb=1 << 24)
BAD_PRODUCTS = [
    (dict(dt=9), EINVAL), (dict(m=-1), EINVAL), (dict(n=-1), EINVAL), (dict(k=-1), EINVAL), (dict(b=None), EINVAL),
    (dict(bs=None), EINVAL), (dict(os=71), EINVAL), (dict(out=None), EINVAL), (dict(out=O + 1), EALIGN),
    (dict(b=C + 8), EALIGN), (dict(bs=S + 2), EALIGN), (dict(out=C), EOVERLAP), (dict(out=X), EOVERLAP),
    (dict(m=1 << 31, n=1 << 31, os=1 << 31), EINVAL), (dict(k=(1 << 25) + 1), EINVAL),
]


@pytest.mark.parametrize("kw,code", BAD_PRODUCTS + [
    (dict(a=None), EINVAL), (dict(as_=None), EINVAL), (dict(a=X + 4), EALIGN)])
def test_matmul_refusals(L, kw, code):
    assert L.ou_mx4_matmul(*(MATMUL | kw).values(), None) == code


def _matmul_values(L, xd=0, xs=300, **kw):
    a = MATMUL | kw
    return L.ou_mx4_matmul_values(xd, a["a"], a["m"], xs, a["dt"], a["b"], a["bs"], a["n"], a["k"], a["out"], a["os"],
                                  a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,code", BAD_PRODUCTS + [
    (dict(xd=4), EINVAL), (dict(xs=299), EINVAL), (dict(a=None), EINVAL), (dict(a=X + 2), EALIGN),
    (dict(ws=None), EINVAL), (dict(wb=10), EINVAL), (dict(ws=W + 8), EALIGN), (dict(ws=X), EOVERLAP),
    (dict(ws=O), EOVERLAP)])
def test_matmul_values_refusals(L, kw, code):
    assert _matmul_values(L, **kw) == code


def _grouped(L, values, off=0x900000000, groups=3, **kw):
    a = MATMUL | kw
    tail = (a["b"], a["bs"], a["n"], a["k"], off, groups, a["out"], a["os"], 1, a["ws"], a["wb"], None)
    if values:
        return L.ou_mx4_grouped_matmul_values(0, a["a"], a["m"], 300, a["dt"], *tail)
    return L.ou_mx4_grouped_matmul(a["dt"], a["a"], a["as_"], a["m"], *tail)


@pytest.mark.parametrize("values", [False, True])
@pytest.mark.parametrize("kw,code", BAD_PRODUCTS + [
    (dict(m=(1 << 28) + 1), EINVAL),
    (dict(off=None), EINVAL), (dict(off=0x900000001), EALIGN), (dict(groups=-1), EINVAL),
    (dict(groups=65536), EINVAL), (dict(out=0x900000000), EOVERLAP)])
def test_grouped_matmul_refusals(L, values, kw, code):
    assert _grouped(L, values, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), EINVAL), (dict(m=-1), EINVAL), (dict(n=-1), EINVAL), (dict(rows=-1), EINVAL), (dict(off=None), EINVAL),
    (dict(groups=-2), EINVAL), (dict(rows=(1 << 25) + 1), EINVAL), (dict(rows=(1 << 28) + 1), EINVAL), (dict(a=None), EINVAL), (dict(bs=None), EINVAL), (dict(out=None), EINVAL),
    (dict(out=O + 1), EALIGN), (dict(a=C + 8), EALIGN), (dict(out=C), EOVERLAP), (dict(out=X), EOVERLAP)])
def test_grouped_outer_refusals(L, kw, code):
    a = dict(dt=1, a=C, as_=S, m=48, b=CT, bs=ST, n=80, rows=500, off=X, groups=5, out=O) | kw
    assert L.ou_mx4_grouped_outer(*a.values(), None) == code


def test_products_pass_their_checks(L, no_gpu):
    assert L.ou_mx4_matmul(*MATMUL.values(), None) == EUNSUPPORTED
    assert _matmul_values(L) == EUNSUPPORTED
    assert _grouped(L, False) == EUNSUPPORTED and _grouped(L, True) == EUNSUPPORTED


def test_binding_refuses_host_tensors_and_bad_forms():
    x = torch.zeros(4, 64)
    q = ou.Mx4(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8), 64)
    assert list(q.shape) == [4, 64]
    off = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: ou.mx4_quantize(x), lambda: ou.mx4_quantize_both(x), lambda: ou.mx4_dequantize(q),
                 lambda: ou.mx4_matmul(x, q), lambda: ou.mx4_matmul(q, q), lambda: ou.mx4_matmul(x, x),
                 lambda: ou.mx4_quantize_grouped(x, off), lambda: ou.mx4_linear(x, x), lambda: ou.Mx4Weight(x),
                 lambda: ou.mx4_grouped_linear(x, x[None], off), lambda: ou.mx4_grouped_matmul(x, q, off)):
        with pytest.raises(ValueError):
            call()
    for codes, scales, k in (((4, 32), (4, 4), 64), ((4, 64), (4, 2), 64), ((4, 64), (3, 4), 64), ((64,), (4,), 64),
                             ((4, 64), (4, 4), 129), ((4, 64), (4, 4), -1)):
        with pytest.raises(ValueError):
            ou.Mx4(torch.zeros(codes, dtype=torch.uint8), torch.zeros(scales, dtype=torch.uint8), k)
    with pytest.raises(ValueError):
        ou.Mx4(torch.zeros(4, 64), torch.zeros(4, 4, dtype=torch.uint8), 64)
    with pytest.raises(ValueError):
        ou.Mx4(torch.zeros(64, 4, dtype=torch.uint8).t(), torch.zeros(4, 4, dtype=torch.uint8), 64)


def test_reference_rounds_to_the_nearest_level():
    """The reference's codes are the nearest of the 15 values, ties to the
    even code, by brute force over the distances."""
    m = np.concatenate([np.arange(0, 8.001, 1 / 64), R.BORDERS])
    x = np.zeros((m.size, 32))
    x[:, 0], x[:, 1] = 4.0, m                       # 4 fixes the scale at 1 for what is below 8
    x = x[m < 8]
    code, s = R.quantize(x)
    assert (s[:, 0] == 127).all()
    for v, c in zip(x[:, 1], code[:, 1]):
        d = np.abs(np.minimum(v, 6.0) - R.LEVELS)
        near = np.flatnonzero(d == d.min())
        assert c == (near[0] if near.size == 1 else near[near % 2 == 0][0]), v


def _kept(weight, of=None):
    """An Mx4Weight whose forms are those of a matrix of shape `of`, without a device."""
    def form(*shape):
        p = R.columns(shape[-1])
        return ou.Mx4(torch.zeros(*shape[:-1], p // 2, dtype=torch.uint8),
                      torch.zeros(*shape[:-1], p // 32, dtype=torch.uint8), shape[-1])

    *lead, r, c = of or weight.shape
    held = object.__new__(ou.Mx4Weight)
    held.weight, held.version, held.q, held.qt = weight, 0, form(*lead, r, c), form(*lead, c, r)
    return held


@pytest.mark.parametrize("now", [(65, 96), (63, 96), (64, 97), (64, 224), (96, 64)])
def test_kept_forms_of_another_shape_are_refused(now):
    """A weight that grew or shrank since its forms were made: the layers and
    the refresh refuse it before they touch an address of the forms."""
    held = _kept(torch.zeros(64, 96))
    held._check_forms()
    held.weight.data = torch.zeros(now)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (held._check_forms, held.refresh, lambda: ou.mx4_linear(torch.zeros(5, now[1]), held)):
        with pytest.raises(ValueError, match="forms are of a weight of shape"):
            call()
    for of in ((1, *now), (3, *now)):
        held = _kept(torch.zeros(2, *now), of)
        with pytest.raises(ValueError, match="forms are of a weight of shape"):
            ou.mx4_grouped_linear(torch.zeros(5, now[1]), held, off)


def test_kept_forms_on_another_device_are_refused():
    held = _kept(torch.zeros(64, 96))
    held.weight = type("Elsewhere", (), {"shape": torch.Size((64, 96)), "get_device": lambda self: 1})()
    for call in (held._check_forms, held.refresh, lambda: ou.mx4_linear(torch.zeros(5, 96), held)):
        with pytest.raises(ValueError, match="forms are on another device"):
            call()


FAR = [1 << 43, 2 << 43, 3 << 43, 4 << 43, 5 << 43, 6 << 43, 7 << 43]


def test_more_tiles_than_a_launch_holds_are_refused(L):
    """Grids of 2^32 threads and more: refused with the other checks, before
    a device is looked for or anything (a left matrix's 4-bit form) is made."""
    x, c, s, ct, st, w, o = FAR
    big = 1 << 30
    quantize = lambda rows, *to: L.ou_mx4_quantize(2, x, 1, rows, 1, 1, 0, *to, None)  # noqa: E731
    need = L.ou_mx4_matmul_workspace_bytes(4096, 1 << 31, 1, 1)
    calls = [lambda: quantize(big, c, s, None, None), lambda: quantize(1 << 31, None, None, ct, st),
             lambda: L.ou_mx4_dequantize(0, c, s, big, 1, o, 1, None),
             lambda: L.ou_mx4_matmul(2, x, s, 1, c, st, big, 1, o, big, None, 0, None),
             lambda: L.ou_mx4_matmul_values(2, x, 4096, 1, 2, c, s, 1 << 31, 1, o, 1 << 31, w, need, None),
             lambda: L.ou_mx4_grouped_matmul(2, x, s, 65535, c, st, 1 << 20, 1, ct, 65535, o, 1 << 20, 0, None, 0, None),
             lambda: L.ou_mx4_grouped_outer(2, x, s, 1 << 20, c, st, 1 << 20, 1, ct, 2, o, None)]
    for i, call in enumerate(calls):
        assert call() == EINVAL, i
        assert "too many tiles" in L.ou_mx4_last_error().decode() or "too large" in L.ou_mx4_last_error().decode(), i


def test_the_largest_grids_pass_the_checks(L, no_gpu):
    x, c, s, ct, st, w, o = FAR
    n = (1 << 30) - 64
    assert L.ou_mx4_quantize(2, x, 1, n, 1, 1, 0, c, s, None, None, None) == EUNSUPPORTED
    assert L.ou_mx4_quantize(2, x, 1, (1 << 31) - 128, 1, 1, 0, None, None, ct, st, None) == EUNSUPPORTED
    assert L.ou_mx4_matmul(2, x, s, 1, c, st, n, 1, o, n, None, 0, None) == EUNSUPPORTED


def test_a_build_elsewhere_leaves_the_library_alone(monkeypatch, tmp_path):
    """A build of the update library to another path, with other flags,
    compiles nothing over this library."""
    from optimizer_update_amd import build
    made = []
    monkeypatch.setattr(build, "_compile", lambda sources, out, flags, quiet: made.append((out, flags)))
    monkeypatch.setattr(build, "build_fast", lambda: None)
    other = str(tmp_path / "variant.so")
    assert build.build(other, ["-g"]) == other and made == [(other, ["-g"])]
    made.clear()
    build.build()
    assert made == [(build.LIBRARY, None), (mx4.LIBRARY, None)] and build.MX4_LIBRARY == mx4.LIBRARY


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """A stream object names its device: the kernels would run there on
    addresses of the operands' device."""
    class Stream:
        def __init__(self, index):
            self.device_index, self.cuda_stream = index, 7

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    assert mx4._run(1, Stream(1), lambda a, handle: (a, handle), 5) == (5, 7)
    with pytest.raises(ValueError, match="device 0"):
        mx4._run(1, Stream(0), lambda a, handle: pytest.fail("called"), 5)


def test_parts_of_a_batch_are_held_matrices_or_refused():
    """The kernels read codes and scales without strides: what an index leaves
    apart in memory is refused."""
    q = ou.Mx4(torch.arange(4 * 6 * 64).view(4, 6, 64).to(torch.uint8), torch.arange(4 * 6 * 4).view(4, 6, 4).to(torch.uint8), 100)
    assert list(q[2].shape) == [6, 100] and torch.equal(q[-1].codes, q.codes[3]) and list(q[1:3].shape) == [2, 6, 100]
    assert len(list(q)) == 4
    assert torch.equal(q[0, :, 0:64].codes, q.codes[0])          # all of a row's bytes
    for index in (slice(None, None, 2), (slice(None), slice(0, 3)), (0, 0), (0, slice(None), slice(0, 32))):
        with pytest.raises(ValueError):
            q[index]


def test_handle_0_is_the_default_stream(monkeypatch):
    """As in the update's calls.  A stream made of the handle 0 is another one,
    which nothing orders behind the default stream's work."""
    class Stream:
        def __init__(self, handle, device):
            self.device_index, self.cuda_stream = device.index, handle or 99

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda i: type("Default", (), dict(device_index=i, cuda_stream=0))())
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    assert mx4._run(2, 0, lambda handle: handle) == 0
    assert mx4._run(2, 55, lambda handle: handle) == 55
