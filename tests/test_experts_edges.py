"""CPU: calls of the operators around experts that their documentation allows
and the other tests do not make, as far as they can be seen without a device."""
import pytest
import torch

import optimizer_update_amd as ou
from optimizer_update_amd import int4


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
