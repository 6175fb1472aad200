"""Rotary angles at far positions and of slow pairs, against angles reduced in big integers."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from invariant_gemm_bi_gb300 import binding as bi
from tests import serving_reference as ref
from tests import serving_tight as tight
from tests.gpu_helpers import bits_equal

pytestmark = pytest.mark.gpu

F32 = torch.float32


def _normal(shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=F32)


def _rotated(x, angle, interleaved):
    """(result, |x1| + |x2|) in 64 bits, the whole head rotated by angle [T, pairs]."""
    x = ref.f64(x)
    half = angle.shape[1]
    i1 = np.arange(half) * 2 if interleaved else np.arange(half)
    i2 = i1 + (1 if interleaved else half)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    y, size = np.zeros_like(x), np.zeros_like(x)
    y[..., i1], y[..., i2] = x[..., i1] * c - x[..., i2] * s, x[..., i1] * s + x[..., i2] * c
    size[..., i1] = size[..., i2] = np.abs(x[..., i1]) + np.abs(x[..., i2])
    return y, size


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("base,R", [(10000.0, 128), (500000.0, 64), (10000.0, 256)])
def test_far_positions(base, R, interleaved):
    pos = [1 << 24, (1 << 31) - 1, -(1 << 31), 1 << 33, (1 << 36) + 17, -(1 << 38) + 5, (1 << 40) + 12345, -(1 << 40)]
    freq = [base ** (-2.0 * i / R) for i in range(R // 2)]
    x = _normal((len(pos), 3, R), 1)
    y = bi.bi_rope(x, torch.tensor(pos, device="cuda"), bi.bi_rope_config(R, frequencies=freq, interleaved=interleaved))
    want, size = _rotated(x, tight.angles(freq, pos), interleaved)
    # beside the fp32 arithmetic the phase's own rounding, 2^-65 of a turn a position
    far = 2 * math.pi * 2.0 ** -65 * np.abs(np.array(pos, np.float64))[:, None, None] * size
    ref.assert_within(y, want, ref.rope_bound(want, size, F32) + far)


@pytest.mark.parametrize("base,R", [(10000.0, 128), (500000.0, 256), (1e8, 64)])
def test_small_angles_keep_their_digits(base, R):
    # x = (1, 0) in every pair: the second result is the angle's sine alone
    pos = [1, 2, 3, 7, 100, 1021]
    freq = [base ** (-2.0 * i / R) for i in range(R // 2)]
    x = torch.zeros(len(pos), 1, R, device="cuda")
    x[..., :R // 2] = 1.0
    y = bi.bi_rope(x, torch.tensor(pos, device="cuda"), bi.bi_rope_config(R, frequencies=freq))
    angle = tight.angles(freq, pos)
    want = np.sin(angle)
    # the half-turn argument's rounding is 2^-24 of the angle, which moves the sine by
    # 2^-24 |angle|; sincospif is good to 2 ulp, 2^-22 of the sine; the product with the
    # magnitude 2^-24; and the phase's own rounding, 2^-65 of a turn a position
    far = 2 * math.pi * 2.0 ** -65 * np.array(pos, np.float64)[:, None]
    bound = 2.0 ** -24 * np.abs(angle) + (2.0 ** -22 + 2.0 ** -24) * np.abs(want) + far
    ref.assert_within(y[:, 0, R // 2:], want, bound)


@pytest.mark.parametrize("dt", [F32, torch.bfloat16])
@pytest.mark.parametrize("D,interleaved", [(128, False), (128, True), (36, False)])
def test_opposite_positions_are_mirror_images(D, interleaved, dt):
    # the map at -n is the transposed map at n, bit for bit
    pos = torch.tensor([0, 1, 5, 1000, 131071, (1 << 31) - 1, 1 << 40], device="cuda")
    x = _normal((7, 4, D), 2).to(dt)
    cfg = bi.bi_rope_config(D, interleaved=interleaved)
    assert bits_equal(bi.bi_rope(x, -pos, cfg), bi.bi_rope(x, pos, cfg, backward=True))
