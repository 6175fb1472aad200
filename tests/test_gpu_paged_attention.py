"""Attention over the paged cache where a slip would be small: repeated calls, the
mass of every piece of a long cache, and results of 16 bits beside those of 32."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from invariant_gemm_bi_gb300 import binding as bi
from tests import serving_reference as ref
from tests import serving_tight as tight
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


# Every sixteenth key, so some of every warp, stands above all others by x bits and has
# no value: the result is the others' weights alone, which are small beside those they
# are computed next to.
@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("D,Hq", [(64, 4), (64, 12), (128, 4), (128, 12), (256, 3)])
@pytest.mark.parametrize("n", [256, 700, 5000])
@pytest.mark.parametrize("x", [12.0, 20.5, 25.5, 28.3, 33.0])
def test_small_weights_beside_large_ones_keep_their_share(dt, D, Hq, n, x):
    P, table = _tables([n], 16, 9)
    j = torch.arange(n, device="cuda")
    k, v = torch.zeros(n, 1, D, device="cuda"), torch.full((n, 1, D), 1024.0, device="cuda")
    k[::16, 0, 0], v[::16] = x * 0.6931471805599453, 0.0
    k, v = k.to(dt), v.to(dt)
    kc, vc = torch.zeros(P, 16, 1, D, dtype=dt, device="cuda"), torch.zeros(P, 16, 1, D, dtype=dt, device="cuda")
    page = table[0, j // 16].long()
    kc[page, j % 16], vc[page, j % 16] = k, v
    q = torch.zeros(1, Hq, D, dtype=dt, device="cuda")
    q[..., 0] = 1.0
    o = bi.bi_paged_attention(q, kc, vc, table, _i32([n]), 1.0)
    want, bound = tight.attention(q[0], k, v, 1.0, dt, F32)
    assert np.all(want > 0) and np.all(bound < 0.02 * want)  # a bound that a lost weight would break
    ref.assert_within(o[0], want, bound)


# Long caches whose values mark their keys (tests/serving_tight.py): a piece, a group of
# pieces or a tile that is left out or taken twice moves some results by their own size.
@pytest.mark.parametrize("D,Hq", [(64, 2), (64, 12), (128, 2), (128, 12), (256, 2)])
@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("n,page", [(700, 16), (2048, 24), (2049, 16), (32769, 128), (65536, 16), (65537, 64), (70001, 24),
                                    (131071, 64), (131072, 16), (200001, 128)])
def test_every_key_of_a_long_cache_counts_once(D, Hq, dt, n, page):
    P, table = _tables([n, 40], page, 10)
    q = _normal((2, Hq, D), dt, 11)
    k = _normal((n, 1, D), dt, 12)
    j = torch.arange(n, device="cuda")
    at = table[0, j // page].long(), j % page
    kc = torch.full((P, page, 1, D), float("nan"), dtype=dt, device="cuda")
    vc = kc.clone()
    kc[at] = k
    kc[table[1, :-(-40 // page)].long()] = 1.0
    vc[table[1, :-(-40 // page)].long()] = 1.0
    for every in (256, 16):
        v = tight.marked_values(n, 1, D, every)
        vc[at] = torch.from_numpy(v).to(dt).cuda()
        o = bi.bi_paged_attention(q, kc, vc, table, _i32([n, 40]), D ** -0.5)
        want, bound = tight.attention(q[0], k, v, D ** -0.5, dt, F32)
        ref.assert_within(o[0], want, bound, f"every {every}")


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 2), (128, 8, 2), (256, 2, 1)])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_ragged_batches_of_marked_values(D, Hq, Hkv, dt):
    # units of many requests on few blocks: the pieces of all lengths at once
    lens = [5, 9000, 0, 257, 2048, 2049, 40000, 1, 511, 6000, 12345]
    P, table = _tables(lens, 32, 13)
    q = _normal((len(lens), Hq, D), dt, 14)
    kc, vc = _normal((P, 32, Hkv, D), dt, 15), torch.full((P, 32, Hkv, D), float("inf"), dtype=dt, device="cuda")
    values = []
    for b, n in enumerate(lens):
        j = torch.arange(n, device="cuda")
        values.append(tight.marked_values(n, Hkv, D, 64))
        vc[table[b, j // 32].long(), j % 32] = torch.from_numpy(values[b]).to(dt).cuda()
    o = bi.bi_paged_attention(q, kc, vc, table, _i32(lens), D ** -0.5)
    for b, n in enumerate(lens):
        if n:
            j = torch.arange(n, device="cuda")
            want, bound = tight.attention(q[b], kc[table[b, j // 32].long(), j % 32], values[b], D ** -0.5, dt, F32)
            ref.assert_within(o[b], want, bound, f"request {b}")


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("D,n", [(64, 200), (128, 3000), (256, 700)])
def test_infinities_in_live_rows(dt, D, n):
    P, table = _tables([n], 16, 16)
    kc, vc = _normal((P, 16, 2, D), dt, 17), _normal((P, 16, 2, D), dt, 18)
    q = _normal((1, 6, D), dt, 19)
    q[..., 7] = 1.0
    j = torch.arange(n, device="cuda")
    pages = table[0, j // 16].long(), j % 16

    def call():
        return bi.bi_paged_attention(q, kc, vc, table, _i32([n]), D ** -0.5)

    whole = call()
    # an infinite value: not finite in its dimension for the heads that read it, the rest as it
    # was.  (Its weight is a sum of 16-bit numbers p = hi + lo ...: hi is rounded to nearest, so lo
    # may be positive, which gives an infinity, or negative or zero, inf - inf and 0 inf.)
    kept = vc.clone()
    vc[table[0, n // 32].long(), 5, 1, 9] = float("inf")
    o = call()
    assert not o[0, 3:, 9].isfinite().any() and bits_equal(o[0, :3], whole[0, :3])
    other = torch.arange(D, device="cuda") != 9
    assert bits_equal(o[0, 3:][:, other].contiguous(), whole[0, 3:][:, other].contiguous())
    vc[table[0, n // 32].long(), 5, 1, 9] = float("nan")
    o = call()
    assert o[0, 3:, 9].isnan().all() and bits_equal(o[0, 3:][:, other].contiguous(), whole[0, 3:][:, other].contiguous())
    vc.copy_(kept)
    # keys whose score is -inf weigh nothing
    out = torch.zeros(n, dtype=torch.bool, device="cuda")
    out[::3] = True
    kc[pages[0][out], pages[1][out], :, 7] = float("-inf")
    want, bound = tight.attention(q[0], kc[pages][~out], vc[pages][~out], D ** -0.5, dt, F32)
    _, more = tight.attention(q[0], _normal((n, 2, D), dt, 17), vc[pages], D ** -0.5, dt, F32)  # n keys' roundings
    ref.assert_within(call()[0], want, bound + more)
    kc[pages[0], pages[1], :, 7] = float("-inf")
    assert not call().any()  # all of them: as without keys
    # a score of +inf: NaN for the head it belongs to
    kc.copy_(_normal((P, 16, 2, D), dt, 17))
    kc[table[0, 0].long(), 3, 0, 7] = float("inf")
    o = call()
    assert o[0, :3].isnan().all() and bits_equal(o[0, 3:], whole[0, 3:])
