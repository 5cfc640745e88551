"""CPU: calls of the operators around experts that their documentation allows
and the other tests do not make, as far as they can be seen without a device."""
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
