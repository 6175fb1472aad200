"""The 8-bit operations on the GPU -- quantisation in blocks, the block-scaled
product, the paged cache in 8 bits -- against plain 64-bit implementations
(tests/quantized_reference.py holds the bounds and where they come from), and
their invariances bit for bit."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from invariant_gemm_bi_gb300 import binding as bi
from tests import quantized_reference as ref
from tests import serving_reference as sref
from tests.gpu_helpers import bits_equal

pytestmark = pytest.mark.gpu

BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, dtype, seed, std=1.0):
    return (torch.randn(shape, generator=_gen(seed), device="cuda", dtype=F32) * std).to(dtype)


def _uniform(shape, seed):
    return torch.rand(shape, generator=_gen(seed), device="cuda", dtype=F32)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _i64(v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


def _e4m3(shape, seed):
    """Any finite e4m3 number, subnormals and zeros of both signs among them."""
    b = torch.randint(0, 254, shape, generator=_gen(seed), device="cuda")
    return torch.where(b < 127, b, b + 1).to(torch.uint8).view(E4M3)


@pytest.fixture(autouse=True)
def _clean_status():
    bi.load()
    assert bi.bi_device_status() == bi.BI_OK
    yield
    assert bi.bi_device_status() == bi.BI_OK


# -- quantisation in blocks ---------------------------------------------------------------

def _same(got, want, what=""):
    g = ref.from_e4m3(got) if got.dtype == E4M3 else sref.f64(got)
    assert g.shape == want.shape and np.array_equal(g, want, equal_nan=True), what


@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (3, 129), (5, 7), (16, 4096), (130, 300), (257, 1000), (128, 128)])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_quantize_matches_the_definition(M, K, block_rows, dt):
    # sizes from the type's smallest numbers to its largest
    top = 60000.0 if dt == F16 else 3e38
    x = (_normal((M, K), F32, M + K) * torch.exp2(_uniform((M, 1), 1) * 200 - 120)).clamp(-top, top).to(dt)
    r = bi.bi_quantize_blocks(x, block_rows)
    q, s = ref.quantize_blocks(x, block_rows)
    _same(r.scales, s, "scales")
    _same(r.values, q, "values")


def test_quantize_borders_and_values_that_are_not_finite():
    rows = torch.zeros((12, 128), device="cuda")
    rows[0, 5] = 448.0  # exactly the largest number at scale 1
    rows[1, 5] = float(np.nextafter(np.float32(448), np.float32(1e9)))  # just past it: scale 2
    rows[2, 5] = -448.0 * 2.0 ** 100
    rows[3] = torch.arange(128) * 1.0  # ties between neighbours
    rows[4, 127] = 1e-45
    rows[5, 0] = float("nan")
    rows[6, 9] = float("inf")
    rows[7, 9] = -float("inf")
    rows[8, :] = 2.0 ** -126 * 447
    rows[9, 3] = 3.4028234663852886e38
    rows[10] = -0.0
    for br in (1, 128):
        for lo, hi in ((0, 5), (5, 12), (8, 12)):
            r = bi.bi_quantize_blocks(rows[lo:hi], br)
            q, s = ref.quantize_blocks(rows[lo:hi], br)
            _same(r.scales, s)
            _same(r.values, q)
    assert bi.bi_quantize_blocks(rows).scales[:2, 0].tolist() == [1.0, 2.0]


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_layouts_give_the_same_bits(dt, block_rows):
    M, K = 150, 517
    wide = _normal((M, K + 11), dt, 5)
    x = wide[:, 3:3 + K]  # rows off 16 bytes
    want = bi.bi_quantize_blocks(x.contiguous().clone(), block_rows)
    store = torch.full((M, K + 5), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((8, 400), -1.0, device="cuda")
    mb = want.scales.shape[0]
    out = bi.QuantizedBlocks(store.view(E4M3)[:, 2:2 + K], scales.t()[:mb, :5] if block_rows == 1 else scales[:mb, :10:2])
    bi.bi_quantize_blocks(x, block_rows, out=out)
    assert bits_equal(out.values.contiguous(), want.values.contiguous()) and torch.equal(out.scales, want.scales)
    assert (store[:, :2] == 0x55).all() and (store[:, 2 + K:] == 0x55).all()
    # a row's blocks are its own
    if block_rows == 1:
        one = bi.bi_quantize_blocks(x[77:78])
        assert bits_equal(one.values.contiguous(), want.values[77:78].contiguous())
        assert torch.equal(one.scales, want.scales[77:78])


def test_quantize_empty():
    assert bi.bi_quantize_blocks(torch.empty((0, 300), device="cuda")).scales.shape == (0, 3)
    assert bi.bi_quantize_blocks(torch.empty((4, 0), device="cuda"), 128).values.shape == (4, 0)


# -- the block-scaled product ---------------------------------------------------------------

def _operands(M, N, K, seed, fill=0x7F):
    """e4m3 operands with powers of two for scales, in rows padded with NaNs."""
    Kp = (K + 15) // 16 * 16 + 16
    a = torch.full((M, Kp), fill, dtype=torch.uint8, device="cuda")
    b = torch.full((N, Kp), fill, dtype=torch.uint8, device="cuda")
    a[:, :K], b[:, :K] = _e4m3((M, K), seed).view(torch.uint8), _e4m3((N, K), seed + 1).view(torch.uint8)
    kb = -(-K // 128)
    sa = torch.exp2(torch.floor(6 * _uniform((M, kb), seed + 2)) - 8)
    sb = torch.exp2(torch.floor(6 * _uniform((-(-N // 128), kb), seed + 3)) - 8)
    return a.view(E4M3)[:, :K], sa, b.view(E4M3)[:, :K].t(), sb.t()


MM = [(1, 1, 1), (1, 64, 128), (2, 65, 129), (16, 200, 300), (32, 256, 256), (33, 129, 257), (128, 64, 384),
      (130, 392, 512), (257, 500, 128), (300, 1000, 1111), (5, 128, 14336), (700, 513, 640)]


@pytest.mark.parametrize("M,N,K", MM)
@pytest.mark.parametrize("out,bias", [(F32, None), (BF16, BF16), (F16, F32)])
def test_mm_blockscaled_matches_reference(M, N, K, out, bias):
    a, sa, b, sb = _operands(M, N, K, M + N + K)
    if out == F16:
        sa = sa * 2.0 ** -10  # results that fp16 holds
    bv = _normal((N,), bias, 9) if bias is not None else None
    c = bi.bi_mm_blockscaled(a, sa, b, sb, bias=bv, out_dtype=out)
    want, bound = ref.mm(a, sa, b, sb, bv, out)
    sref.assert_within(c, want, bound, f"{M}x{N}x{K}")


def test_mm_blockscaled_of_the_quantiser():
    x, w = _normal((45, 777), BF16, 1), _normal((333, 777), BF16, 2, 0.05)
    xq, wq = bi.bi_quantize_blocks(x), bi.bi_quantize_blocks(w, 128)
    c = bi.bi_mm_blockscaled(xq.values, xq.scales, wq.values.t(), wq.scales.t(), out_dtype=F32)
    want, bound = ref.mm(xq.values, xq.scales, wq.values.t(), wq.scales.t(), None, F32)
    sref.assert_within(c, want, bound)
    # and near the unquantised product: two roundings of 2^-4 of an element at most, and the
    # subnormals' 2^-10 of a scale that is at most 2^-7 of a block's largest (2^-17 of it)
    x64, w64 = sref.f64(x), sref.f64(w)
    far = (2.0 ** -3 + 2.0 ** -8) * (np.abs(x64) @ np.abs(w64).T)
    far = far + 2.0 ** -16 * 777 * np.abs(x64).max() * np.abs(w64).max()
    assert np.all(np.abs(sref.f64(c) - x64 @ w64.T) <= far)


def test_mm_blockscaled_rows_do_not_depend_on_the_batch():
    # over the tile widths and both layouts of A, and columns over the number of columns
    N, K = 20000, 400
    a, sa, b, sb = _operands(1000, N, K, 4)
    full = bi.bi_mm_blockscaled(a, sa, b, sb, out_dtype=F32)
    for M in (1, 16, 32, 33, 128, 129, 256, 257, 600):
        c = bi.bi_mm_blockscaled(a[:M], sa[:M], b, sb, out_dtype=F32)
        assert bits_equal(c, full[:M].contiguous()), M
    for n in (1, 64, 65, 300, 5000):
        for M in (1, 40, 1000):
            c = bi.bi_mm_blockscaled(a[:M], sa[:M], b[:, :n], sb, out_dtype=F32) if n > 19900 else \
                bi.bi_mm_blockscaled(a[:M], sa[:M], b[:, :n], sb[:, :-(-n // 128)], out_dtype=F32)
            assert bits_equal(c, full[:M, :n].contiguous()), (M, n)
    # any row, anywhere
    c = bi.bi_mm_blockscaled(a[517:518], sa[517:518], b, sb, out_dtype=F32)
    assert bits_equal(c, full[517:518].contiguous())


def test_mm_blockscaled_layouts():
    M, N, K = 150, 300, 260
    a, sa, b, sb = _operands(M, N, K, 8)
    want = bi.bi_mm_blockscaled(a, sa, b, sb, out_dtype=BF16)
    # scales of other strides, an output inside a wider one, bias with a stride
    sa2 = torch.zeros((3, M * 2), device="cuda").t()[::2]
    sa2.copy_(sa)
    sb2 = torch.zeros((3 * 2, 3), device="cuda")[::2]
    sb2.copy_(sb)
    store = torch.full((M, N + 7), 3.0, dtype=BF16, device="cuda")
    bi.bi_mm_blockscaled(a, sa2, b, sb2, out=store[:, 1:1 + N])
    assert bits_equal(store[:, 1:1 + N].contiguous(), want)
    assert (store[:, 0] == 3).all() and (store[:, 1 + N:] == 3).all()
    bias = _normal((2 * N,), F32, 3)[::2]
    x = bi.bi_mm_blockscaled(a, sa, b, sb, bias=bias, out_dtype=F32)
    y = bi.bi_mm_blockscaled(a, sa, b, sb, bias=bias.contiguous(), out_dtype=F32)
    assert bits_equal(x, y)


def test_mm_blockscaled_nan_stays_in_its_rows_and_empty_sums():
    M, N, K = 40, 200, 300
    a, sa, b, sb = _operands(M, N, K, 6)
    clean = bi.bi_mm_blockscaled(a, sa, b, sb, out_dtype=F32)
    bad = a.clone()
    bad.view(torch.uint8)[7, 299] = 0x7F
    sc = sa.clone()
    sc[9, 1], sc[11, 2], sc[12, 0], sc[13, 0] = float("nan"), 0.75, 0.0, -1.0  # none of them a power of two
    store = torch.zeros((M, 304), dtype=torch.uint8, device="cuda").view(E4M3)[:, :K]
    store.view(torch.uint8).copy_(bad.view(torch.uint8))
    c = bi.bi_mm_blockscaled(store, sc, b, sb, out_dtype=F32)
    gone = [7, 9, 11, 12, 13]
    keep = [m for m in range(M) if m not in gone]
    assert torch.isnan(c[gone]).all() and bits_equal(c[keep], clean[keep])
    wide = sa.clone()
    wide[3], wide[4] = 2.0 ** 100, 2.0 ** -126  # the whole range
    c = bi.bi_mm_blockscaled(a, wide, b, sb, out_dtype=F32)
    want, bound = ref.mm(a, wide, b, sb, None, F32)
    sref.assert_within(c[[3, 5]], want[[3, 5]], bound[[3, 5]])
    assert (c[4].abs() < 2.0 ** -90).all()
    bias = _normal((N,), BF16, 1)
    e = bi.bi_mm_blockscaled(torch.empty((M, 0), device="cuda").to(E4M3), sa[:, :0],
                             torch.empty((N, 0), device="cuda").to(E4M3).t(), sb[:0], bias=bias, out_dtype=F32)
    assert torch.equal(e, bias.float().expand(M, N))
    assert bi.bi_mm_blockscaled(a[:0], sa[:0], b, sb).shape == (0, N)


# -- the cache in 8 bits ------------------------------------------------------------------------

def _cache(pages, page, hkv, d, seed):
    """Values and scales of any size: what is not written stays."""
    return (_e4m3((pages, page, hkv, d), seed), torch.exp2(4 * _uniform((pages, page, hkv), seed + 1) - 3))


STORES = [  # T, Hq, Hkv, D, rotary, interleaved, page, type of q, k and v, of q's result
    (1, 4, 1, 64, 64, False, 16, BF16, BF16), (7, 8, 2, 128, 128, False, 16, BF16, BF16),
    (9, 8, 2, 128, 64, True, 24, F16, F16), (33, 2, 1, 256, 256, True, 64, BF16, BF16),
    (5, 2, 2, 256, 128, False, 8, F32, F32), (700, 4, 2, 128, 128, False, 16, BF16, F32),
    (11, 3, 3, 80, 40, False, 16, BF16, BF16), (6, 2, 1, 66, 2, True, 16, F16, F16), (4, 1, 1, 7, 6, False, 8, F32, BF16),
    (3, 1, 1, 512, 32, False, 8, BF16, BF16), (3, 1, 2, 1024, 64, True, 8, BF16, BF16), (13, 1, 1, 96, 96, False, 8, F16, F16),
    (20, 5, 5, 16, 16, False, 16, BF16, BF16)]


def _stored(T, Hq, Hkv, D, R, inter, page, dt, qdt, shift=0, seed=0):
    """Arguments of a call over a projection's output, `shift` elements into its storage."""
    n = T * (Hq + 2 * Hkv) * D
    flat = _normal((n + shift,), dt, seed)[shift:]
    x = flat.view(T, Hq + 2 * Hkv, D)
    pages = 2 * (-(-T // page)) + 1
    slots = torch.randperm(pages * page, generator=_gen(seed + 1), device="cuda")[:T].contiguous()
    if T > 2:
        slots[T // 2] = -1
    pos = torch.randint(0, 100000, (T,), generator=_gen(seed + 2), device="cuda", dtype=torch.int32)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], slots, pos, pages


@pytest.mark.parametrize("case", STORES)
def test_store_quantized_matches_reference(case):
    T, Hq, Hkv, D, R, inter, page, dt, qdt = case
    q, k, v, slots, pos, pages = _stored(*case)
    kc, ks = _cache(pages, page, Hkv, D, 3)
    vc, vs = _cache(pages, page, Hkv, D, 5)
    before = [t.clone() for t in (kc, ks, vc, vs)]
    mag = 1.25
    cfg = bi.bi_rope_config(R, interleaved=inter, magnitude=mag)
    qo = bi.bi_paged_store_quantized(k, v, slots, kc, ks, vc, vs, q=q, positions=pos, config=cfg, q_dtype=qdt)
    freq = sref.frequencies(R)
    want, size = sref.rope(q, pos.tolist(), freq, inter, magnitude=mag)
    sref.assert_within(qo, want, sref.rope_bound(want, size, qdt), "q")
    # scales, exactly: sums of two fp32 numbers, rounded, times the magnitude, rounded
    k32 = k.float().cpu().numpy()
    i1 = np.arange(R // 2) * 2 if inter else np.arange(R // 2)
    i2 = i1 + (1 if inter else R // 2)
    sizes = ((np.abs(k32[..., i1]) + np.abs(k32[..., i2])) * np.float32(mag)).max(-1)
    sizes = np.maximum(sizes, np.abs(k32[..., R:]).max(-1, initial=0))
    want_ks, want_vs = ref.scale_of(sizes.astype(np.float64)), ref.scale_of(np.abs(sref.f64(v)).max(-1))
    want_k, size = sref.rope(k, pos.tolist(), freq, inter, magnitude=mag)
    ref_v = ref.round_e4m3(sref.f64(v) / want_vs[..., None])
    flat = [t.view(torch.uint8).view(-1, Hkv, D) if t.dtype == E4M3 else t.view(-1, Hkv) for t in (kc, ks, vc, vs)]
    old = [t.view(torch.uint8).view(-1, Hkv, D) if t.dtype == E4M3 else t.view(-1, Hkv) for t in before]
    live = slots >= 0
    at, tok = slots[live], live.nonzero()[:, 0].cpu().numpy()
    _same(flat[1][at], want_ks[tok], "key scales")
    _same(flat[3][at], want_vs[tok], "value scales")
    _same(flat[2][at].view(E4M3), ref_v[tok], "values")
    got = ref.from_e4m3(flat[0][at].view(E4M3)) * want_ks[tok][..., None]
    # half a step of e4m3: 2^-4 of the element, or half the subnormals' 2^-9 times the
    # scale; and before it the turn in fp32 (the bound of bi_rope without its rounding)
    e = 2.0 ** -21 * size[tok]
    bound = e + np.maximum((np.abs(want_k[tok]) + e) * 2.0 ** -4, want_ks[tok][..., None] * 2.0 ** -10)
    sref.assert_within(torch.from_numpy(got), want_k[tok], bound, "keys")
    # everything else as it was
    other = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    other[at] = False
    for new, was in zip(flat, old):
        assert torch.equal(new[other], was[other])


@pytest.mark.parametrize("case", [c for c in STORES if c[3] in (64, 128, 256) and c[7] != F32])
def test_store_quantized_is_the_same_off_16_bytes(case):
    T, Hq, Hkv, D, R, inter, page, dt, qdt = case
    cfg = bi.bi_rope_config(R, interleaved=inter)
    got = []
    for shift in (0, 1):
        q, k, v, slots, pos, pages = _stored(*case, seed=4)
        if shift:  # the same numbers, a row of everything one element into its storage
            q, k, v = (torch.cat([t.reshape(-1)[:1], t.reshape(-1)])[1:].view(t.shape) for t in (q, k, v))
        kc, ks = _cache(pages, page, Hkv, D, 3)
        vc, vs = _cache(pages, page, Hkv, D, 5)
        qo = bi.bi_paged_store_quantized(k, v, slots, kc, ks, vc, vs, q=q, positions=pos, config=cfg)
        got.append((qo, kc, ks, vc, vs))
    for a, b in zip(*got):
        assert bits_equal(a, b)


def test_store_quantized_scales_do_not_depend_on_positions():
    k, v = _normal((1, 2, 128), BF16, 1).expand(50, 2, 128).contiguous(), _normal((50, 2, 128), BF16, 2)
    kc, ks = _cache(4, 16, 2, 128, 3)
    vc, vs = _cache(4, 16, 2, 128, 5)
    pos = torch.randint(-10 ** 6, 10 ** 6, (50,), generator=_gen(3), device="cuda")
    bi.bi_paged_store_quantized(k, v, torch.arange(50, device="cuda"), kc, ks, vc, vs, positions=pos,
                                config=bi.bi_rope_config(128))
    s = ks.view(-1, 2)[:50]
    assert torch.equal(s, s[:1].expand(50, 2))


def test_store_quantized_without_rotation_bad_slots_and_values_that_are_not_finite():
    T, H, D, page = 6, 2, 64, 8
    k, v = _normal((T, H, D), BF16, 1), _normal((T, H, D), BF16, 2)
    k[1, 0, 5] = float("nan")
    v[2, 1, 7] = float("inf")
    k[3] = 0
    kc, ks = _cache(2, page, H, D, 3)
    vc, vs = _cache(2, page, H, D, 5)
    old = [t.clone() for t in (kc, ks, vc, vs)]
    assert bi.bi_paged_store_quantized(k, v, _i64([0, 3, 5, 9, 16, -7]), kc, ks, vc, vs) is None
    assert bi.bi_device_status() == bi.BI_ERR_INVALID_ARG and "bad index" in bi.last_error_message()
    for name, x, c, s in (("k", k, kc, ks), ("v", v, vc, vs)):
        for t, slot in enumerate([0, 3, 5, 9]):
            for h in range(H):
                q, sc = ref.quantize_blocks(x[t, h][None], 1)
                _same(s.view(-1, H)[slot, h][None, None], sc, name)
                _same(c.view(torch.uint8).view(-1, H, D)[slot, h][None].view(E4M3), q, name)
    rest = [i for i in range(16) if i not in (0, 3, 5, 9)]
    for new, was in zip((kc, ks, vc, vs), old):
        n, w = ((t.view(torch.uint8).view(16, -1) if t.dtype == E4M3 else t.view(16, -1)) for t in (new, was))
        assert torch.equal(n[rest], w[rest])


def test_store_quantized_strided_caches_and_in_place_queries():
    # keys and values of one cache tensor, scales of another, q turned where it lies
    T, Hq, Hkv, D, page = 40, 4, 2, 128, 16
    q, k, v, slots, pos, pages = _stored(T, Hq, Hkv, D, D, False, page, BF16, BF16)
    kv = _e4m3((pages, 2, page, Hkv, D), 1)
    sc = torch.ones((pages, page, Hkv, 2), device="cuda")
    cfg = bi.bi_rope_config(D)
    kc, ks = _cache(pages, page, Hkv, D, 3)
    vc, vs = _cache(pages, page, Hkv, D, 5)
    want = bi.bi_paged_store_quantized(k, v, slots, kc, ks, vc, vs, q=q, positions=pos, config=cfg)
    got = bi.bi_paged_store_quantized(k, v, slots, kv[:, 0], sc[..., 0], kv[:, 1], sc[..., 1], q=q, positions=pos,
                                      config=cfg, q_out=q)
    assert got.data_ptr() == q.data_ptr() and bits_equal(got.contiguous(), want)
    at = slots[slots >= 0]
    pg, row = at // page, at % page
    for a, b in ((kv[:, 0], kc), (kv[:, 1], vc)):
        assert torch.equal(a.view(torch.uint8)[pg, row], b.view(torch.uint8)[pg, row])
    for a, b in ((sc[..., 0], ks), (sc[..., 1], vs)):
        assert torch.equal(a[pg, row], b[pg, row])


@pytest.mark.parametrize("H,D,page,dt", [(8, 128, 16, BF16), (1, 64, 24, F16), (2, 256, 64, F32), (3, 80, 8, BF16),
                                         (2, 7, 8, F32), (1, 1024, 3, F16)])
def test_load_quantized_matches_reference(H, D, page, dt):
    pages, T = 9, 131
    kc, ks = _cache(pages, page, H, D, 3)
    vc, vs = _cache(pages, page, H, D, 5)
    slots = torch.randint(0, pages * page, (T,), generator=_gen(1), device="cuda")  # some of them twice
    slots[5], slots[77] = -1, -1000
    got = bi.bi_paged_load_quantized(slots, kc, ks, vc, vs, out_dtype=dt)
    keep = slots.clamp(min=0)
    for g, c, s in ((got.k, kc, ks), (got.v, vc, vs)):
        x = c.view(torch.uint8).view(-1, H, D)[keep].view(E4M3).double() * s.view(-1, H)[keep][..., None].double()
        x[slots < 0] = 0
        # the product of 4 bits and 24 fits fp64: one rounding to fp32, as the kernel's, then one
        assert torch.equal(g, x.float().to(dt))
    assert bi.bi_paged_load_quantized(slots[:0], kc, ks, vc, vs).k.shape == (0, H, D)


def test_load_quantized_strided_and_past_the_cache():
    H, D, page = 2, 64, 16
    kv = _e4m3((3, 2, page, H, D), 1)
    sc = torch.exp2(_uniform((3, page, H, 2), 2))
    slots = _i64([0, 47, 48, 13, 2 ** 40, 13])
    store = torch.full((6, 2, H, D + 3), 9.0, dtype=BF16, device="cuda")
    out = bi.CacheRows(store[:, 0, :, 1:1 + D], store[:, 1, :, 1:1 + D])
    bi.bi_paged_load_quantized(slots, kv[:, 0], sc[..., 0], kv[:, 1], sc[..., 1], out=out)
    assert bi.bi_device_status() == bi.BI_ERR_INVALID_ARG and "slot" in bi.last_error_message()
    want = bi.bi_paged_load_quantized(_i64([0, 47, -1, 13, -1, 13]), kv[:, 0].contiguous(), sc[..., 0].contiguous(),
                                      kv[:, 1].contiguous(), sc[..., 1].contiguous())
    assert torch.equal(out.k, want.k) and torch.equal(out.v, want.v)
    assert (store[..., 0] == 9).all() and (store[..., 1 + D:] == 9).all()


# -- attention over the cache in 8 bits ------------------------------------------------------------

def _problem(lens, Hq, Hkv, D, page, dt, seed=0, width=None, spread=2.0):
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    ids = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(lens), width or max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    q = _normal((len(lens), Hq, D), dt, seed + 1)
    x = _normal((2, pages, page, Hkv, D), F32, seed + 2)
    s = torch.exp2(spread * (_uniform((2, pages, page, Hkv), seed + 3) - 0.5)) / 100
    kv = (x / s[..., None] / 30).clamp(-448, 448).to(E4M3)
    # what no request holds is NaN: it must not be read
    held = torch.zeros(pages * page, dtype=torch.bool)
    for b, n in enumerate(lens):
        j = torch.arange(n)
        held[table[b, j // page].long() * page + j % page] = True
    free = ~held.view(pages, page).cuda()
    kv.view(torch.uint8)[:, free] = 0x7F
    s[:, free] = float("nan")
    return q, kv[0], s[0] * 30, kv[1], s[1] * 30, table.cuda(), _i32(lens)


ATTEND = [  # lens, Hq, Hkv, D, page, type
    ([1], 1, 1, 64, 16, BF16), ([0, 1, 2, 15, 16, 17], 4, 2, 128, 16, BF16), ([31, 32, 33, 255, 256, 257], 8, 1, 64, 24, F16),
    ([1021], 32, 8, 128, 16, BF16), ([2047, 2048, 2049, 5], 5, 1, 256, 64, F16), ([4096, 700, 0, 4097], 16, 1, 128, 8, F16),
    ([300] * 40, 16, 16, 64, 32, BF16), ([9000, 3], 20, 2, 128, 128, BF16), ([17000], 8, 8, 256, 16, BF16),
    ([70001], 2, 1, 64, 64, F16), ([777, 12], 16, 1, 256, 16, BF16), ([600] * 3, 24, 2, 64, 16, BF16)]


@pytest.mark.parametrize("case", ATTEND)
@pytest.mark.parametrize("out", [F32, None])
def test_attention_quantized_matches_reference(case, out):
    lens, Hq, Hkv, D, page, dt = case
    q, kc, ks, vc, vs, table, n = _problem(*case)
    o = bi.bi_paged_attention_quantized(q, kc, ks, vc, vs, table, n, D ** -0.5, out_dtype=out or dt)
    want, bound = ref.attention(q, kc, ks, vc, vs, table, n, D ** -0.5, out or dt)
    sref.assert_within(o, want, bound, str(case))


@pytest.mark.parametrize("D,group", [(64, 4), (128, 4), (128, 12), (256, 3)])
def test_attention_quantized_scales_far_apart(D, group):
    # values whose scales span 2^40, largest where the weights are least, and scales that
    # are no powers of two, negative, and zero
    q, kc, ks, vc, vs, table, n = _problem([1500, 40], group, 1, D, 16, BF16, seed=5)
    live = ~torch.isnan(vs)
    vs[live] = (torch.exp2(40 * _uniform(vs.shape, 8) - 20) * torch.where(_uniform(vs.shape, 9) < 0.5, -1.3, 1.1))[live]
    vs[live & (_uniform(vs.shape, 10) < 0.1)] = 0.0
    ks[live & (_uniform(vs.shape, 11) < 0.1)] = 0.0
    o = bi.bi_paged_attention_quantized(q, kc, ks, vc, vs, table, n, D ** -0.5)
    want, bound = ref.attention(q, kc, ks, vc, vs, table, n, D ** -0.5, F32)
    sref.assert_within(o, want, bound)
    # a value's scale so large beside the others that its own weight is all that is left of it
    vs[live] = 1.0
    page = int(table[0, 0])
    ks[page, 3], vs[page, 3], ks[page, 4] = -ks[page, 4].abs() * 50, 2.0 ** 30, ks[page, 4].abs()
    kc.view(torch.uint8)[page, 3] = kc.view(torch.uint8)[page, 4]
    o = bi.bi_paged_attention_quantized(q, kc, ks, vc, vs, table, n, D ** -0.5)
    want, bound = ref.attention(q, kc, ks, vc, vs, table, n, D ** -0.5, F32)
    sref.assert_within(o, want, bound)


@pytest.mark.parametrize("dt,tiny", [(BF16, 1e-30), (BF16, 1e30), (F16, 6e-8), (F16, 60000.0)])
def test_attention_quantized_queries_of_any_size(dt, tiny):
    q, kc, ks, vc, vs, table, n = _problem([500], 4, 1, 128, 16, dt, seed=6)
    q = (q.float() * tiny).clamp(-65504, 65504).to(dt) if dt == F16 else (q.float() * tiny).to(dt)
    scale = 0.1 / tiny if tiny != 6e-8 else 1e6
    o = bi.bi_paged_attention_quantized(q, kc, ks, vc, vs, table, n, scale)
    want, bound = ref.attention(q, kc, ks, vc, vs, table, n, float(np.float32(scale)), F32)
    sref.assert_within(o, want, bound)


def test_attention_quantized_invariances():
    # alone, in a batch, over other pages, another page size, a wider table: the same bits
    lens, Hq, Hkv, D, page = [0, 1, 300, 2048, 3000, 5000, 33], 8, 2, 128, 16
    q, kc, ks, vc, vs, table, n = _problem(lens, Hq, Hkv, D, page, BF16)
    full = bi.bi_paged_attention_quantized(q, kc, ks, vc, vs, table, n, 0.1)
    assert (full[0] == 0).all()
    for b in range(len(lens)):
        w = max(1, -(-lens[b] // page))
        for width in (w, table.shape[1]):
            o = bi.bi_paged_attention_quantized(q[b:b + 1], kc, ks, vc, vs, table[b:b + 1, :width], n[b:b + 1], 0.1)
            assert bits_equal(o, full[b:b + 1].contiguous()), (b, width)
    wide = torch.full((len(lens), 9000), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    assert bits_equal(bi.bi_paged_attention_quantized(q, kc, ks, vc, vs, wide, n, 0.1), full)
    j = torch.arange(table.shape[1] * page, device="cuda")
    slot = table.long()[:, j // page] * page + j % page  # pages of one token
    slot = torch.where(j[None, :] < n[:, None], slot, -1).to(torch.int32)
    one = [t.reshape(-1, 1, *t.shape[2:]) for t in (kc, ks, vc, vs)]
    assert bits_equal(bi.bi_paged_attention_quantized(q, *one, slot, n, 0.1), full)
    big = q.repeat(60, 1, 1), table.repeat(60, 1), n.repeat(60)
    o = bi.bi_paged_attention_quantized(big[0], kc, ks, vc, vs, big[1], big[2], 0.1)
    assert bits_equal(o, full.repeat(60, 1, 1))


def test_attention_quantized_values_that_are_not_finite_and_bad_pages():
    q, kc, ks, vc, vs, table, n = _problem([200, 50, 40, 9], 4, 2, 64, 16, BF16, seed=3)
    clean = bi.bi_paged_attention_quantized(q, kc, ks, vc, vs, table, n, 0.125)
    q2 = q.clone()
    q2[0, 1, 3], q2[1, 2, 9] = float("nan"), float("inf")
    o = bi.bi_paged_attention_quantized(q2, kc, ks, vc, vs, table, n, 0.125)
    hit = torch.zeros((4, 4), dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[1, 2] = True
    assert torch.isnan(o[hit]).all() and bits_equal(o[~hit], clean[~hit])
    page = int(table[2, 0])
    for t, value in ((ks, float("nan")), (vs, float("nan"))):  # a key's, a value's scale of one head
        keep = t[page, 2, 1].clone()
        t[page, 2, 1] = value
        o = bi.bi_paged_attention_quantized(q, kc, ks, vc, vs, table, n, 0.125)
        assert torch.isnan(o[2, 2:]).all()
        assert bits_equal(o[[0, 1, 3]], clean[[0, 1, 3]]) and bits_equal(o[2, :2], clean[2, :2])
        t[page, 2, 1] = keep
    vc.view(torch.uint8)[page, 2, 1, 7] = 0x7F  # a NaN among the values: its dimension
    o = bi.bi_paged_attention_quantized(q, kc, ks, vc, vs, table, n, 0.125)
    assert torch.isnan(o[2, 2:, 7]).all() and not torch.isnan(o[2, :, :7]).any()
    bad = table.clone()
    bad[1, 2], bad[3, 0] = 10 ** 6, -5
    o = bi.bi_paged_attention_quantized(q, kc, ks, vc, vs, bad, n, 0.125)
    assert bi.bi_device_status() == bi.BI_ERR_INVALID_ARG and "page" in bi.last_error_message()
    want, bound = ref.attention(q, kc, ks, vc, vs, bad, n, 0.125, F32)
    sref.assert_within(o[[0, 1, 3]], want[[0, 1, 3]], bound[[0, 1, 3]])
    assert (o[3] == 0).all()
    o = bi.bi_paged_attention_quantized(q, kc, ks, vc, vs, table, _i32([500, 50, 40, 9]), 0.125)  # past the table
    assert bi.bi_device_status() == bi.BI_ERR_INVALID_ARG


def test_attention_quantized_strided_operands():
    q, kc, ks, vc, vs, table, n = _problem([700, 33], 8, 2, 128, 16, BF16, seed=2)
    want = bi.bi_paged_attention_quantized(q, kc, ks, vc, vs, table, n, 0.1, out_dtype=BF16)
    P = kc.shape[0]
    kv = torch.zeros((P, 2, 2, 16, 128), dtype=torch.uint8, device="cuda")  # [page, k or v, head, row, D]
    kv[:, 0], kv[:, 1] = kc.view(torch.uint8).transpose(1, 2), vc.view(torch.uint8).transpose(1, 2)
    sc = torch.stack([ks, vs], -1)
    qs = torch.zeros((2, 12, 128), dtype=BF16, device="cuda")
    qs[:, 2:10] = q
    store = torch.full((2, 8, 136), 7.0, dtype=BF16, device="cuda")
    k, v = (kv[:, i].view(E4M3).transpose(1, 2) for i in range(2))
    bi.bi_paged_attention_quantized(qs[:, 2:10], k, sc[..., 0], v, sc[..., 1], table, n, 0.1, out=store[..., :128])
    assert bits_equal(store[..., :128].contiguous(), want) and (store[..., 128:] == 7).all()
