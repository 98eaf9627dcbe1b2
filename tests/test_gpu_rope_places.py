"""The last places of fp32 norms and rotations, where spec_qk_rope's bounds come from: angles next to whole quarter turns, whose
small sines and cosines have no more than their own roundings, and the norm's reciprocal root by itself.

Angle. The plan's turns are right to 2^-32 of a turn (2 pi 2^-32 radians). Less its nearest quarter turn, in whole numbers, the
angle is at most 1/4 half turn and rounded to fp32 relative to itself (2^-24); the sine and cosine of that add two places (2^-22 of
a value). An angle that were rounded before the quarter turns leave it, as half turns of up to 1, would be off by pi 2^-25
radians: 60 times the bound of a sine of 2^-12.

Root. v = mean + eps is rounded once (2^-24, of which the root takes half). The reciprocal root after Newton's step
f + f / 2 (1 - v f f): the product v f rounded (2^-24, of which the step takes half), the step's sum rounded (2^-24); together
2^-23. Elements are powers of two, so that their squares' sums and the last products are exact."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from speculative_decoding_token_temp_gb300 import api

from test_gpu_attention import dev, i32  # noqa: F401 (dev: the fixture)

pytestmark = pytest.mark.gpu

TWO_PI = Fraction(6283185307179586476925286766559005768394, 10 ** 39)


def turn(position, freq):
    """(cosine, sine) of position * freq and what the angle is as a share of a turn, from exact arithmetic."""
    x = Fraction(freq) * position / TWO_PI
    x -= math.floor(x)
    quarter = round(x * 4)
    rest = float((x - Fraction(quarter, 4)) * TWO_PI)
    c, s = math.cos(rest), math.sin(rest)
    return [(c, s), (-s, c), (-c, -s), (s, -c)][quarter % 4], float(x)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("start", [0, 1_000_001, 2 ** 31 - 400])
def test_angles_next_to_quarter_turns(dev, dim, interleaved, start):  # noqa: F811
    half = dim // 2
    freq = [math.pi / 2 * (1 + (j + 0.1) * (1e-7 if start == 0 else 1e-14)) for j in range(half)]
    positions = np.arange(start, start + 397)
    rope = api.Rope(dim, dev, inv_freq=freq, interleaved=interleaved)
    q = torch.zeros(len(positions), 1, dim, device=dev)
    first = torch.arange(0, dim, 2) if interleaved else torch.arange(half)
    q[:, :, first] = 1.0  # pairs (1, 0): they turn to (cosine, sine)
    got = api.spec_qk_rope(q, q, rope, i32(positions, dev))["q"].double().cpu().numpy()[:, 0]
    other = (first + (1 if interleaved else half)).numpy()
    turns = [[turn(int(p), f) for f in freq] for p in positions]
    want = np.array([[t[0] for t in row] for row in turns])
    off = np.abs(np.stack([got[:, first.numpy()], got[:, other]], -1) - want)
    lim = np.abs(want) * (2.0 ** -22 + 2.0 ** -24) * 1.01 + 2 * math.pi * 2.0 ** -32
    assert (off <= lim).all(), f"{(off / lim).max():.3g} of the bound"
    # what half turns rounded to fp32 at once would give does not pass
    at = np.array([[t[1] for t in row] for row in turns])
    at = 2 * np.where(at >= 0.5, at - 1, at)
    coarse = np.pi * (at.astype(np.float32).astype(np.float64))
    worse = np.abs(np.stack([np.cos(coarse), np.sin(coarse)], -1) - want)
    assert (worse > lim).any()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 0.37])
def test_reciprocal_roots(dev, dim, eps):  # noqa: F811
    """n of a head's elements are 2^a, the others 2^b: 12 pairs of exponents, every n."""
    pairs = [(a, b) for a in (-7, 0, 3) for b in (a - 5, a - 3, a - 1, a)]
    x = np.empty((len(pairs) * (dim + 1), dim))
    for i, (a, b) in enumerate(pairs):
        for n in range(dim + 1):
            x[i * (dim + 1) + n] = np.where(np.arange(dim) < n, 2.0 ** a, 2.0 ** b)
    q = torch.from_numpy(x).float().view(-1, 1, dim).to(dev)
    rope = api.Rope(dim, dev, rot_dim=0)
    got = api.spec_qk_rope(q, q, rope, torch.zeros(q.shape[0], dtype=torch.int32, device=dev), eps=eps)["k"].double().cpu().numpy()[:, 0]
    want = x / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps)))
    off = np.abs(got / want - 1)
    assert (off <= 2.0 ** -23 * 1.001).all(), f"{off.max() * 2 ** 23:.3g} of 2^-23"
