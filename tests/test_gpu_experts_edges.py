"""GPU: calls of the operators around experts that their documentation allows
and the other tests do not make."""
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


@pytest.mark.parametrize("handle", [False, True])
def test_quantize_views_on_a_stream(handle):
    """Transposed, strided, broadcast and batched views on a stream that waits
    for what made them alone."""
    base = torch.randn((2048, 1024), generator=_gen(1)).cuda()
    s = torch.cuda.Stream()
    for view in (lambda b: b.t(), lambda b: b[:, ::2], lambda b: b[:1].expand(700, 1024), lambda b: b.view(2048, 8, 128).transpose(0, 1)):
        want = ou.int4_quantize(view(base).contiguous(), 64)
        torch.cuda.synchronize()
        for i in range(5):
            x = base * 1.0      # on the current stream
            s.wait_stream(torch.cuda.current_stream())
            got = ou.int4_quantize(view(x), 64, stream=s.cuda_stream if handle else s)
            s.synchronize()
            assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales) and torch.equal(got.zeros, want.zeros)
