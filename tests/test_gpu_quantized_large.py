"""Results of the 8-bit operations with more than 2^31 elements: their last rows are those of
small calls, bit for bit."""
from __future__ import annotations

import pytest
import torch

from invariant_gemm_bi_gb300 import binding as bi
from tests.gpu_helpers import bits_equal
from tests.test_gpu_quantized import BF16, E4M3, F16, F32, _cache, _clean_status, _gen, _operands  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,out", [(8200, BF16), (8201, F16), (8204, F32)])  # stores by tile, by row, by 16 bytes
def test_mm_blockscaled_many_rows(N, out):
    M, K = 262149, 130
    a, sa, b, sb = _operands(M, N, K, 3)
    sa = sa * 2.0 ** -8
    c = bi.bi_mm_blockscaled(a, sa, b, sb, out_dtype=out)
    assert c.numel() > 2 ** 31
    for rows in (slice(0, 300), slice(M // 2, M // 2 + 129), slice(M - 261, M)):
        assert bits_equal(c[rows].contiguous(), bi.bi_mm_blockscaled(a[rows], sa[rows], b, sb, out_dtype=out))


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("K", [4096, 4100])
def test_quantize_many_rows(block_rows, K):
    M = 128 * 4200
    x = torch.empty((M, K), dtype=F16, device="cuda")
    x.view(-1, 64 * K)[:] = torch.randn((64 * K,), generator=_gen(1), device="cuda").to(F16)
    x *= torch.exp2(torch.randint(-6, 7, (M, 1), generator=_gen(2), device="cuda").to(F16))
    assert x.numel() > 2 ** 31
    q = bi.bi_quantize_blocks(x, block_rows)
    for rows in (slice(0, 256), slice(M - 256, M)):
        want = bi.bi_quantize_blocks(x[rows], block_rows)
        assert bits_equal(q.values[rows].contiguous(), want.values.contiguous())
        s = slice(rows.start // block_rows, rows.stop // block_rows)
        assert torch.equal(q.scales[s], want.scales)


@pytest.mark.parametrize("H,D", [(2, 1024), (3, 683)])  # 16-byte units, an element a lane
def test_load_quantized_many_rows(H, D):
    T, pages, page = 1050000, 700, 16
    kc, ks = _cache(pages, page, H, D, 3)
    vc, vs = _cache(pages, page, H, D, 5)
    slots = torch.randint(0, pages * page, (T,), generator=_gen(1), device="cuda")
    got = bi.bi_paged_load_quantized(slots, kc, ks, vc, vs)
    assert got.k.numel() > 2 ** 31
    for rows in (slice(0, 100), slice(T - 100, T)):
        want = bi.bi_paged_load_quantized(slots[rows].contiguous(), kc, ks, vc, vs)
        assert bits_equal(got.k[rows].contiguous(), want.k) and bits_equal(got.v[rows].contiguous(), want.v)


def test_store_quantized_many_rows():
    # q of 2^31 elements and more, turned in place; half of the tokens are not stored
    T, Hq, H, D = 270000, 64, 1, 128
    q = torch.empty((T, Hq, D), dtype=BF16, device="cuda")
    q[:] = torch.randn((Hq, D), generator=_gen(1), device="cuda").to(BF16)
    assert q.numel() > 2 ** 31
    k = torch.randn((T, H, D), generator=_gen(2), device="cuda").to(BF16)
    pos = torch.arange(T, device="cuda")
    page, pages = 16, T // 32 + 1
    slots = torch.where(pos % 2 == 0, pos // 2, -1)
    kc, ks = _cache(pages, page, H, D, 3)
    vc, vs = _cache(pages, page, H, D, 5)
    cfg = bi.bi_rope_config(D)
    first = q[:1].clone()
    bi.bi_paged_store_quantized(k, k, slots, kc, ks, vc, vs, q=q, positions=pos, config=cfg, q_out=q)
    for rows in (slice(0, 50), slice(T - 50, T)):
        n = rows.stop - rows.start
        c8, s8 = _cache(pages, page, H, D, 3)
        d8, t8 = _cache(pages, page, H, D, 5)
        want = bi.bi_paged_store_quantized(k[rows], k[rows], slots[rows].contiguous(), c8, s8, d8, t8,
                                           q=first.expand(n, Hq, D).contiguous(), positions=pos[rows].contiguous(), config=cfg)
        assert bits_equal(q[rows].contiguous(), want)
        at = slots[rows][slots[rows] >= 0]
        for x, y in ((kc, c8), (vc, d8)):
            assert torch.equal(x.view(torch.uint8).view(-1, H, D)[at], y.view(torch.uint8).view(-1, H, D)[at])
        for x, y in ((ks, s8), (vs, t8)):
            assert torch.equal(x.view(-1, H)[at], y.view(-1, H)[at])
