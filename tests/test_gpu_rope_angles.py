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
