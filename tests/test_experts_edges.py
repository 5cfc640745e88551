"""CPU: calls of the operators around experts that their documentation allows
and the other tests do not make, as far as they can be seen without a device."""
import os
import subprocess

import pytest
import torch

import optimizer_update_amd as ou
from optimizer_update_amd import int4, route


@pytest.mark.parametrize("make", [lambda: torch.randn(64, 40).t(), lambda: torch.randn(64, 4, 64).transpose(0, 1),
                                  lambda: torch.randn(4, 64).t().contiguous().t()[:, ::2], lambda: torch.randn(1, 64).expand(5, 64)])
def test_quantize_copies_on_the_calls_stream(make, monkeypatch):
    """Views that take a copy are given to the call as they are: a copy made in
    front of it would be on the current stream, which `stream` does not wait for."""
    x, seen = make(), {}
    monkeypatch.setattr(int4, "_values", lambda *a: 0)
    monkeypatch.setattr(int4, "_run", lambda index, stream, fn, operand, *rest: seen.update(stream=stream, operand=operand))
    ou.int4_quantize(x, 32, stream=7)
    got = seen["operand"]
    assert seen["stream"] == 7 and got.data_ptr() == x.data_ptr() and got.shape == x.shape and got.stride() == x.stride()


# ------------------------------------------------------------------ numbers

A, B, C, D, E, F, G = (0x100000000 * i for i in range(1, 8))
CALLS = {
    # name: arguments (a stream behind them), and which of them are 32-bit numbers
    "ou_route_topk": ([0, A, 10, 64, 64, 0, None, 8, 2, 1, 1, 1.0, None, 4, B, C], (0, 3, 5, 7, 8, 9, 10, 13)),
    "ou_route_topk_backward": ([2, A, 10, 64, 64, 1, 0, 1.0, B, C, 4, D], (0, 3, 5, 6, 10)),
    "ou_route_order": ([A, 100, 16, B, C, D, None, 0], (2,)),
    "ou_route_dispatch": ([1, A, 10, 64, 64, 2, B, C, D, 64, 1], (0, 5, 10)),
    "ou_route_combine": ([1, A, 10, 64, 64, 2, B, C, E, 64, F, 64], (0, 5)),
    "ou_route_combine_backward": ([1, A, 10, 64, 64, 2, B, 64, C, D, E, F, G], (0, 5)),
    "ou_route_balance": ([A, B, 8, 0.1, C], (2,)),
    "ou_int4_matmul": ([2, A, 3, 256, 2, B, 2, C, D, 40, 256, 64, E, 40], (0, 4, 6, 11)),
    "ou_int4_grouped_matmul": ([2, A, 3, 256, 2, B, 2, C, D, 40, 256, 64, F, 4, E, 40, 1], (0, 4, 6, 11, 13, 16)),
}


@pytest.mark.parametrize("name", CALLS)
def test_numbers_that_pass_32_bits_are_refused(name):
    """2^32 more than a number that is allowed is not that number."""
    f = getattr(ou.load_experts(), name)
    args, small = CALLS[name]
    assert set(CALLS) == set(route.FAST_ENTRY_POINTS)
    for i in small:
        for more in (1 << 32, -(1 << 32), 1 << 40):
            bad = list(args)
            bad[i] += more
            with pytest.raises(OverflowError):
                f(*bad, None)


# ------------------------------------------------------------------ gradients

@pytest.mark.parametrize("grouped", [False, True])
def test_products_refuse_to_drop_gradients(grouped, monkeypatch):
    for name, to in (("_weights", lambda *a: -1), ("_values", lambda *a: 0), ("_output", lambda *a: (0, 3)), ("_run", lambda *a: "called")):
        monkeypatch.setattr(int4, name, to)
    lead = (2,) if grouped else ()
    q = ou.Int4(torch.zeros((*lead, 3, 32), dtype=torch.uint8), torch.zeros((*lead, 3, 2)), None, 32)
    offsets = (torch.tensor([0, 1, 2], dtype=torch.int32),) if grouped else ()
    f = ou.int4_grouped_matmul if grouped else ou.int4_matmul
    x, leaf = torch.zeros((2, 64)), torch.zeros((2, 64), requires_grad=True)
    assert f(x, q, *offsets) == "called"
    for operand in (leaf, leaf * 2):
        with pytest.raises(ValueError, match="gradients"):
            f(operand, q, *offsets)
        with torch.no_grad():
            assert f(operand, q, *offsets) == "called"
        assert f(operand.detach(), q, *offsets) == "called"
    with pytest.raises(ValueError, match="gradients"):
        f(x, q, *offsets, out=torch.zeros((2, 3), requires_grad=True))


class _Library:
    """Answers every call with OK."""

    def __getattr__(self, name):
        return lambda *args: 0


def test_results_that_are_given_count_as_written(monkeypatch):
    """A graph that saved `out` earlier must not go on with what is written into it now."""
    for m in (route, int4):
        monkeypatch.setattr(m, "load_experts", _Library)
    order = ou.RouteOrder(torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), torch.zeros((2, 2), dtype=torch.int32))
    q = ou.Int4(torch.zeros((3, 32), dtype=torch.uint8), torch.zeros((3, 2)), None, 32)
    x, y, w = torch.zeros((2, 64)), torch.zeros((4, 64)), torch.zeros((2, 2))
    offsets = torch.zeros(2, dtype=torch.int32)
    for shape, call in (((4, 64), lambda out: route._do_dispatch(x, order, out, None)),
                        ((2, 64), lambda out: route._do_combine(y, w, order, None, out, None)),
                        ((2,), lambda out: route._do_balance(torch.zeros(2), order, 0.1, out, None)),
                        ((3, 64), lambda out: int4._do_dequantize(q, torch.float32, out, None)),
                        ((2, 3), lambda out: int4._do_matmul(x, 0, 64, q, 2, 3, 64, torch.float32, 0, out, 3, None, 0, None)),
                        ((2, 3), lambda out: int4._do_matmul(x, 0, 64, q, 2, 3, 64, torch.float32, 0, out, 3, offsets, 1, None))):
        assert call(None).shape == shape and call(None)._version == 0
        out = torch.zeros(shape)
        saved = (torch.ones(shape, requires_grad=True) * out).sum()
        assert call(out) is out and out._version == 1
        with pytest.raises(RuntimeError, match="modified by an inplace"):
            saved.backward()
        with torch.inference_mode():
            call(torch.zeros(shape))


# ------------------------------------------------------------------ which kernel

MAIN = """
#include <cstdio>
#include "int4_choice.hpp"
int main()
{
    long long m, n, k, group, f32, half, experts;
    while (std::scanf("%lld %lld %lld %lld %lld %lld %lld", &m, &n, &k, &group, &f32, &half, &experts) == 7) {
        const experts::Int4Choice c = experts::int4_choice(f32, experts::int4_scales(static_cast<int32_t>(group)), half, (k + 127) / 128,
                                                           experts::int4_tiles(m, n, experts >= 0, experts));
        std::printf("%d %d %d %d\\n", c.held, c.tiles, c.waves, c.steps);
    }
}
"""
# m, n, k, group (of products by group: rows, and matrices behind them), and what is chosen for x of 16 bits, of
# binary32 with 16-bit scales, and with binary32 scales: the sizes that the tests on the device take for these kernels
ONE, TWO, FOUR, TWO_SMALL, HELD8, HELD16, HELD32 = ((0, 1, 8, 0), (0, 2, 8, 0), (0, 4, 4, 0), (0, 2, 4, 0), (1, 2, 8, 1), (1, 1, 4, 4),
                                                    (1, 1, 8, 2))
CHOICES = [
    ((1, 4096, 4096, 128, -1), ONE, ONE, ONE), ((64, 100, 2048, 128, -1), ONE, ONE, ONE), ((16, 40, 4096, 96, 16), ONE, ONE, ONE),
    # blocks of two and four tiles
    ((1, 8200, 6304, 32, -1), TWO_SMALL, TWO_SMALL, TWO_SMALL), ((17, 4117, 6400, 64, -1), TWO_SMALL, TWO_SMALL, TWO_SMALL),
    ((20, 8200, 6528, 128, -1), FOUR, FOUR, FOUR), ((3, 16400, 4192, 32, -1), FOUR, TWO_SMALL, TWO_SMALL),
    ((5, 16390, 1600, 64, -1), FOUR, TWO_SMALL, TWO_SMALL), ((40, 6007, 1344, 96, -1), FOUR, TWO_SMALL, TWO_SMALL),
    ((9, 8300, 4096, 128, -1), TWO, TWO, TWO), ((189, 520, 4224, 128, 32), FOUR, FOUR, FOUR), ((53, 515, 4160, 64, 16), TWO_SMALL, TWO_SMALL, TWO_SMALL),
    ((201, 907, 3232, 32, 18), FOUR, TWO_SMALL, TWO_SMALL), ((207, 1000, 2112, 64, 18), FOUR, TWO_SMALL, TWO_SMALL),
    # x held: 7 to 8 and 13 to 16 steps, up to 16 for binary32 with small groups
    ((3, 24593, 1024, 32, -1), HELD8, HELD8, TWO_SMALL), ((17, 12300, 928, 32, -1), HELD8, HELD8, TWO_SMALL),
    ((2, 25000, 896, 128, -1), HELD8, HELD8, FOUR), ((1, 24600, 960, 64, -1), HELD8, HELD8, TWO_SMALL),
    ((16, 98320, 2048, 128, -1), HELD16, FOUR, FOUR), ((40, 32790, 1632, 96, -1), HELD16, HELD32, TWO_SMALL),
    ((273, 2100, 2048, 128, 48), HELD16, FOUR, FOUR), ((117, 2063, 1632, 32, 48), HELD16, HELD32, TWO_SMALL),
    ((477, 2085, 1984, 64, 48), HELD16, HELD32, TWO_SMALL), ((269, 1100, 1024, 64, 24), HELD8, HELD8, TWO_SMALL),
    # past 32 bits of codes: 4 rows stream, 16 rows are held
    ((4, 8192, 8192, 128, 136), FOUR, FOUR, FOUR), ((4, 8192, 2048, 128, 540), FOUR, FOUR, FOUR), ((16, 8192, 2048, 128, 540), HELD16, FOUR, FOUR),
    ((0, 64, 1024, 128, 0), ONE, ONE, ONE),
]


def test_sizes_choose_the_kernels_they_are_tested_for(tmp_path):
    src = tmp_path / "t.cpp"
    src.write_text(MAIN)
    csrc = os.path.join(os.path.dirname(int4.__file__), "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", csrc, str(src), "-o", str(tmp_path / "t")], check=True)
    lines = [f"{m} {n} {k} {group} {f32} {half} {e}" for (m, n, k, group, e), *_ in CHOICES for f32, half in ((0, 1), (1, 1), (1, 0))]
    out = subprocess.run([str(tmp_path / "t")], input="\n".join(lines), capture_output=True, text=True, check=True).stdout.split("\n")
    got = [tuple(map(int, line.split())) for line in out if line]
    for i, (sizes, *want) in enumerate(CHOICES):
        assert got[3 * i:3 * i + 3] == want, sizes
    # binary32 scales are never held, whatever x is
    lines = [line.rsplit(" ", 2)[0] + " 0 " + line.split()[-1] for line in lines]
    out = subprocess.run([str(tmp_path / "t")], input="\n".join(lines), capture_output=True, text=True, check=True).stdout.split("\n")
    assert not any(int(line.split()[0]) for line in out if line)
