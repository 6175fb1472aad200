"""Extents at which the reading back of a cache in 8 bits would leave its 32-bit counts:
refused before any launch (the descriptors point at fake addresses that are never touched)."""
from __future__ import annotations

import pytest

from tests.test_quantized_cpu import BF16, E4M3, F32, INVALID, I64, REACHED, _load, lib, no_gpu  # noqa: F401


def _heads(H, D, T=2):
    cache = lambda a, o: a.t([2, 1, H, D], E4M3)  # noqa: E731
    scale = lambda a, o: a.t([2, 1, H], F32)  # noqa: E731
    rows = lambda a, o: a.t([T, H, D], BF16)  # noqa: E731
    return dict(kc=cache, vc=cache, ks=scale, vs=scale, k=rows, v=rows, slots=lambda a, o: a.t([T], I64))


@pytest.mark.parametrize("H,D", [(1 << 30, 1), ((1 << 29) + 1, 1), (1 << 29, 80), (1 << 25, 1024), ((1 << 28) + 1, 128)])
def test_load_quantized_refuses_heads_past_its_counts(lib, H, D):  # noqa: F811
    assert _load(lib, **_heads(H, D)) == INVALID


@pytest.mark.skipif(not no_gpu, reason="fake addresses")
@pytest.mark.parametrize("H,D", [(1 << 29, 1), ((1 << 25) - 1, 1024), ((1 << 28) - 1, 128)])
def test_load_quantized_takes_heads_up_to_them(lib, H, D):  # noqa: F811
    assert _load(lib, **_heads(H, D)) == REACHED
