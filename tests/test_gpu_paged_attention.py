"""Attention over the paged cache where a slip would be small: repeated calls, the
mass of every piece of a long cache, and results of 16 bits beside those of 32."""
from __future__ import annotations

import pytest
import torch

from invariant_gemm_bi_gb300 import binding as bi
from tests.gpu_helpers import bits_equal

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, dtype, seed, std=1.0):
    return (torch.randn(shape, generator=_gen(seed), device="cuda", dtype=F32) * std).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.fixture(autouse=True)
def _clean_status():
    bi.load()
    assert bi.bi_device_status() == bi.BI_OK
    yield
    assert bi.bi_device_status() == bi.BI_OK


def _tables(lens, page, seed, width=0):
    """(pages of the cache, table) with every request's pages at random places."""
    need = [-(-n // page) for n in lens]
    ids = torch.randperm(sum(need) + 2, generator=_gen(seed), device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max([width, 1] + need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return sum(need) + 2, table


# Warps join through shared memory, a slot of which the lanes of one warp read and
# then replace: four and eight warps a block, one and more warps that do so, heads
# that some lanes have and others have not, one launch and two.
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 32, 8), (64, 3, 1), (128, 24, 2), (256, 5, 1), (64, 32, 2)])
@pytest.mark.parametrize("lens,width", [([1021], 0), ([1021], 400), ([700, 3, 0, 2048], 0), ([9000, 250, 4097], 0)])
def test_repeated_calls_give_the_same_bits(D, Hq, Hkv, lens, width):
    P, table = _tables(lens, 16, 1, width)
    kc, vc = _normal((P, 16, Hkv, D), BF16, 2), _normal((P, 16, Hkv, D), BF16, 3)
    q, ln = _normal((len(lens), Hq, D), BF16, 4), _i32(lens)
    for out in (F32, BF16):
        first = bi.bi_paged_attention(q, kc, vc, table, ln, D ** -0.5, out_dtype=out)
        differ = torch.zeros((), dtype=torch.int64, device="cuda")
        for _ in range(150):
            again = bi.bi_paged_attention(q, kc, vc, table, ln, D ** -0.5, out_dtype=out)
            differ += (again != first).sum()
        assert differ.item() == 0 and bits_equal(again, first)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 32, 8), (64, 3, 1), (128, 24, 2), (256, 5, 1), (64, 32, 2)])
@pytest.mark.parametrize("lens,width", [([1021], 0), ([255, 3, 0, 2048], 400), ([9000, 250, 4097], 0)])
def test_results_of_16_bits_are_those_of_32_rounded(dt, D, Hq, Hkv, lens, width):
    P, table = _tables(lens, 16, 5, width)
    kc, vc = _normal((P, 16, Hkv, D), dt, 6), _normal((P, 16, Hkv, D), dt, 7)
    q, ln = _normal((len(lens), Hq, D), dt, 8), _i32(lens)
    o = bi.bi_paged_attention(q, kc, vc, table, ln, D ** -0.5)
    for out in (BF16, F16):
        assert bits_equal(bi.bi_paged_attention(q, kc, vc, table, ln, D ** -0.5, out_dtype=out), o.to(out))
