"""Sines and cosines of the cache write in 8 bits, read off its turned queries: a pair (1, 0)
is turned to the cosine and the sine."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from invariant_gemm_bi_gb300 import binding as bi
from tests.gpu_helpers import bits_equal
from tests.test_gpu_quantized import BF16, F32, _cache, _clean_status, _gen, _normal  # noqa: F401

pytestmark = pytest.mark.gpu


def _turned(q, pos, cfg):
    T, D = q.shape[0], q.shape[2]
    kc, ks = _cache(2, 8, 1, D, 1)
    vc, vs = _cache(2, 8, 1, D, 2)
    k = _normal((T, 1, D), q.dtype, 3)
    return bi.bi_paged_store_quantized(k, k, torch.full((T,), -1, device="cuda"), kc, ks, vc, vs, q=q, positions=pos, config=cfg)


@pytest.mark.parametrize("D", [128, 96, 1024])  # 16-byte units, one pair at a time
def test_sines_and_cosines_to_less_than_a_last_place(D):
    R = min(D, 256)
    cfg = bi.bi_rope_config(R)
    far = torch.randint(-2 ** 40, 2 ** 40, (4000,), generator=_gen(1), device="cuda")
    pos = torch.cat([torch.arange(-2000, 20000, device="cuda"), far])
    q = torch.zeros((pos.shape[0], 1, D), dtype=F32, device="cuda")
    q[..., :R // 2] = 1.0
    y = _turned(q, pos, cfg)[:, 0].cpu().numpy()
    # the angles in 2^-64 turns, exactly, then in 64 bits
    phase = np.array(list(cfg.desc.phase)[:R // 2], dtype=np.uint64)
    turns = (pos.cpu().numpy().astype(np.uint64)[:, None] * phase[None, :]).view(np.int64)
    quarters = ((turns.view(np.uint64) + np.uint64(1 << 61)) >> np.uint64(62)).astype(np.int64)
    angle = (turns.view(np.uint64) - (quarters.view(np.uint64) << np.uint64(62))).view(np.int64) * (np.pi / 2 ** 63)
    sine, cosine = np.sin(angle), np.cos(angle)
    s = np.choose(quarters & 3, [sine, cosine, -sine, -cosine])
    c = np.choose(quarters & 3, [cosine, -sine, -cosine, sine])
    for got, want in ((y[:, :R // 2], c), (y[:, R // 2:R], s)):
        # Half a last place by the final rounding.  What it adds to theta, at most 0.12 of
        # it, comes of five roundings, each of at most half a last place of that, and ends
        # at 2^-28: in all 0.12 * 2.5 + 0.06 of a place; 1 - theta^2 / 2 has less.
        place = np.spacing(np.abs(want).astype(np.float32)).astype(np.float64)
        err = np.abs(got.astype(np.float64) - want) / place
        assert err.max() <= 0.86
    assert (y[:, R:] == 0).all()


def test_turned_queries_beside_bi_rope():
    # the same angles, sines rounded otherwise: within two last places of the pair's size,
    # and where no angle has to be rounded the same bits
    D, T = 128, 300
    cfg = bi.bi_rope_config(D)
    q = _normal((T, 4, D), F32, 5)
    pos = torch.randint(0, 2 ** 20, (T,), generator=_gen(2), device="cuda")
    a, b = _turned(q, pos, cfg), bi.bi_rope(q, pos, cfg)
    size = torch.hypot(q[..., :64], q[..., 64:]).repeat(1, 1, 2)
    # sines of either: under 2^-22 off (bi_rope's angle 2^-24 of pi, sincospif two last
    # places), times |x1| + |x2|, at most sqrt(2) of the size; products and sums 2^-24 each
    assert ((a - b).abs() <= 2.0 ** -20 * size).all()
    zero = torch.zeros_like(pos)
    assert bits_equal(_turned(q, zero, cfg), bi.bi_rope(q, zero, cfg))
    quarter = bi.bi_rope_config(2, frequencies=[np.pi / 2])  # whole quarter turns
    at = torch.arange(T, device="cuda")
    assert torch.equal(_turned(q, at, quarter), bi.bi_rope(q, at, quarter))
