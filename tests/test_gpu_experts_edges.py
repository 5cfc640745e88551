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


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("e,k,groups", [(2, 2, 1), (8, 2, 1), (8, 8, 1), (15, 7, 1), (16, 4, 1), (60, 5, 1), (64, 6, 8), (64, 6, 1), (96, 4, 6),
                                        (256, 8, 8), (300, 20, 1), (320, 17, 32), (700, 3, 4), (1024, 64, 1)])
def test_topk_of_rows_with_nan_alone(e, k, groups, biased, renormalize, scores, dtype):
    """A NaN counts as the largest, whatever else the token has: rows of NaN,
    rows where all else is absent, parts of NaN beside parts that are absent, +inf."""
    print("topk nan", e, k, groups, biased, renormalize, scores, dtype, flush=True)
    x = torch.randn((13, e), generator=_gen(e)).to(dtype)
    size = e // groups
    x[0] = NAN
    x[1] = -INF
    x[1, e // 2:] = NAN
    x[2, 1] = NAN
    x[3] = -INF                        # nobody
    x[4] = -INF
    x[4, e - 1] = NAN                  # one, and it is NaN
    x[5, ::2] = NAN
    x[6, -size:] = NAN                 # the last part
    x[7, : e - size] = -INF
    x[7, -size:] = NAN                 # and all others absent
    x[8] = torch.where(torch.arange(e) % 3 == 0, -INF, NAN).to(dtype)
    if scores == "softmax":            # all of a row's scores are NaN
        x[9, e // 2] = INF
    bias = None
    if biased:
        bias = torch.randn(e, generator=_gen(k)) * 0.1
        bias[0] = -INF
    top = 2 if groups > 1 else 1
    if top * size < k:
        top = -(-k // size)
    kw = dict(scores=scores, renormalize=renormalize, groups=groups, top_groups=top, group_score="best" if biased else "best two")
    w, ids = ou.route_topk(x.cuda(), k, bias=None if bias is None else bias.cuda(), **kw)
    with np.errstate(all="ignore"):
        want, at, _, _ = R.topk(R.host(x), k, bias=None if bias is None else R.host(bias), **kw)
    assert np.array_equal(ids.cpu().numpy(), at)
    w = w.cpu().numpy()
    assert np.array_equal(np.isnan(w), np.isnan(want)) and (w[at < 0] == 0).all()
    live = (at >= 0).sum(1)
    assert live[0] == k and live[3] == 0 and live[4] == 1 and live[9] == k and np.isfinite(w[10:]).all()
