"""The microscaled 4-bit format from its definition, in 64 bits on the CPU:
what the tests of the 4-bit operators compare with."""
from __future__ import annotations

import numpy as np
import torch

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# where the rounding passes from one code to the next; a tie goes to the even code
BORDERS = (LEVELS[1:] + LEVELS[:-1]) / 2


def columns(k: int) -> int:
    return -(-k // 128) * 128


def host(t: torch.Tensor) -> np.ndarray:
    """Values of a tensor, exactly, as float64."""
    return t.detach().double().cpu().numpy()


def quantize(x: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """x [..., K] (binary32 values in float64) to codes [..., P] (one a byte)
    and scale codes [..., P / 32]."""
    k = x.shape[-1]
    v = np.zeros((*x.shape[:-1], columns(k)))
    v[..., :k] = x
    v = v.reshape(*x.shape[:-1], columns(k) // 32, 32)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        top = np.abs(v).max(-1)
        bad = ~np.isfinite(top)
        safe = np.where(bad, 1.0, top)
        e = np.where(safe < 2.0 ** -126, 0, np.frexp(np.maximum(safe, 2.0 ** -126))[1] - 1 + 127)
        s = np.where(bad, 255, np.maximum(e - 2, 0)).astype(np.int64)
        m = np.abs(v) / np.exp2(s - 127.0)[..., None]
        code = np.zeros(v.shape, np.int64)
        for i, b in enumerate(BORDERS):   # code i | i + 1; a tie passes if i + 1 is even
            code += (m >= b) if i % 2 else (m > b)
        code += 8 * np.signbit(v)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(*x.shape[:-1], columns(k)).astype(np.uint8), s.astype(np.uint8)


def pack(code: np.ndarray) -> np.ndarray:
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(codes: np.ndarray) -> np.ndarray:
    return np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])


def values(code: np.ndarray, scale: np.ndarray, k: int) -> np.ndarray:
    """The float64 values of codes (one a byte) and scale codes, k columns."""
    c = code.astype(np.int64)
    mag = LEVELS[c & 7] * np.where(c & 8, -1.0, 1.0)
    unit = np.where(scale == 255, np.nan, np.exp2(scale.astype(np.float64) - 127.0))
    return (mag * np.repeat(unit, 32, axis=-1))[..., :k]


def rounded(x: np.ndarray) -> np.ndarray:
    """x with its values replaced by those of its 4-bit form (last axis)."""
    return values(*quantize(x), x.shape[-1])


def held(q) -> np.ndarray:
    """The values of an Mx4, in float64."""
    return values(unpack(q.codes.cpu().numpy()), q.scales.cpu().numpy(), q.k)


def product(a: np.ndarray, b: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """a b^T and the sums of the terms' magnitudes."""
    return a @ b.T, np.abs(a) @ np.abs(b).T


def tolerance(want: np.ndarray, magnitude: np.ndarray, k: int, dtype: torch.dtype) -> np.ndarray:
    """How far a product may be off.  Every term is exact in binary32 (two
    significands of two bits); a sum over k runs through k / 64 instructions
    at most, each adding to the accumulator once and summing 128 products at
    most inside (7 levels).  Each of these roundings is off by at most one
    step, 2^-23 of the magnitudes summed so far.  The result is rounded once
    to dtype: half a step, finfo.eps / 2 of it (or of the smallest normal
    number)."""
    roundings = k / 64 + 7 + 1
    f = torch.finfo(dtype)
    slack = roundings * 2.0 ** -23 * magnitude
    if dtype == torch.float32:
        return slack + 2.0 ** -126   # results below the smallest normal number may be flushed
    return slack + f.eps / 2 * np.maximum(np.abs(want) + slack, f.tiny)


def check_product(got: torch.Tensor, want: np.ndarray, magnitude: np.ndarray, k: int) -> None:
    g = host(got)
    assert g.shape == want.shape, (g.shape, want.shape)
    nan = np.isnan(want)
    # Where the terms' magnitudes sum to more than binary32 holds, a partial
    # sum may leave its range, whatever the whole sum is: a + b - b with
    # a, b near the largest number is infinite or NaN in some order of its
    # sums.  There nothing is asked; elsewhere no partial sum can exceed the
    # magnitudes' sum, so the results are finite up to the rounding of out.
    open_ = ~nan & (magnitude >= np.finfo(np.float32).max)
    assert np.array_equal(np.isnan(g) & ~open_, nan), "NaN in other places"
    # what the result's type cannot hold is infinite, or its largest number
    # where the sum is within its error of that
    f = torch.finfo(got.dtype)
    tol = tolerance(np.where(nan, 0, want), np.where(nan, 0, magnitude), k, got.dtype)
    big = ~nan & ~open_ & (np.abs(want) + tol >= f.max)
    assert (np.abs(g[big]) >= f.max * (1 - f.eps) - tol[big]).all() and (g[big] * want[big] > 0).all()
    skip = nan | open_ | big
    off = np.abs(np.where(skip, 0, g) - np.where(skip, 0, want))
    worst = np.unravel_index(np.argmax(off - tol), off.shape) if off.size else None
    assert (off <= tol).all(), f"at {worst}: {g[worst]} for {want[worst]}, off {off[worst]:.3g}, allowed {tol[worst]:.3g}"
