"""The serving operations on the GPU: page planning, rotary positions, cache
writes, paged attention and token log probabilities against plain 64-bit
implementations (tests/serving_reference.py holds the bounds and where they come
from), their invariances bit for bit, and a decode step of all of them."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from invariant_gemm_bi_gb300 import binding as bi
from tests import serving_reference as ref
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


def _bad_index():
    assert bi.bi_device_status() == bi.BI_ERR_INVALID_ARG
    assert "bad index" in bi.last_error_message()


# -- page planning -----------------------------------------------------------------------

def _check_plan(ctx, new, page, W, F, T, seed=0, ld=None):
    rng = np.random.default_rng(seed)
    B = len(ctx)
    store = rng.integers(0, 1 << 20, (B, ld or W)).astype(np.int32)
    pool = (1 << 20) + rng.permutation(F).astype(np.int32)
    table = torch.from_numpy(store).cuda()
    got = bi.bi_paged_plan(_i32(ctx), _i32(new), table[:, :W], torch.from_numpy(pool).cuda(), page, T)
    want = ref.plan(ctx, new, store[:, :W], pool, page, T)
    full = store.copy()
    full[:, :W] = want[0]
    assert np.array_equal(table.cpu().numpy(), full)  # columns past W and rows' other entries as they were
    for g, w, name in zip(got, want[1:], ("seq_lens", "token_offsets", "positions", "slots", "totals")):
        assert np.array_equal(g.cpu().numpy(), w), name


@pytest.mark.parametrize("B,page,ctx_to,new_to", [(1, 16, 0, 1), (1, 1, 5, 3), (5, 16, 100, 1), (33, 24, 500, 40),
                                                  (256, 16, 4000, 3), (257, 64, 4000, 5), (1025, 8, 60, 4),
                                                  (2500, 128, 1000, 2)])
def test_plan_matches_reference(B, page, ctx_to, new_to):
    rng = np.random.default_rng(B)
    ctx = rng.integers(0, ctx_to + 1, B)
    new = rng.integers(0, new_to + 1, B)
    W = (ctx_to + new_to + page - 1) // page + 1
    _check_plan(ctx, new, page, W, B * (new_to + 1), int(new.sum()) + 7, ld=W + 3)


def test_plan_long_prefill_and_many_blocks():
    _check_plan([0, 100000, 7], [70001, 13, 0], 16, 7000, 5000, 70014 + 1000)


def test_plan_short_pool_narrow_table_short_outputs():
    _check_plan([10, 30, 0, 64], [40, 40, 100, 0], 16, 8, 5, 200)   # pool runs out
    _check_plan([10, 30, 0, 64], [40, 40, 100, 0], 16, 4, 50, 200)  # tables too narrow
    _check_plan([10, 30, 0, 64], [40, 40, 100, 0], 16, 8, 50, 77)   # fewer token outputs than tokens
    _check_plan([10, 30], [40, 40], 16, 8, 0, 100)                  # an empty pool
    _check_plan([10, 30], [40, 40], 16, 8, 50, 0)                   # no token outputs
    _check_plan([-5, 3, -1], [2, -7, -1], 16, 2, 9, 5)              # negative lengths count as 0


def test_plan_saturates_and_empty_batch():
    p = bi.bi_paged_plan(_i32([2 ** 31 - 1] * 3), _i32([2 ** 31 - 1] * 3), torch.zeros(3, 1, dtype=torch.int32).cuda(),
                         _i32([5]), 1 << 20, 4)
    assert p.seq_lens.tolist() == [2 ** 31 - 1] * 3
    assert p.token_offsets.tolist() == [0, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]
    assert p.totals.tolist() == [3 * 2048, 2 ** 31 - 1] and p.slots.tolist() == [-1] * 4
    e = bi.bi_paged_plan(_i32([]), _i32([]), torch.zeros(0, 4, dtype=torch.int32).cuda(), _i32([1]), 16, 3)
    assert e.token_offsets.tolist() == [0] and e.slots.tolist() == [-1] * 3 and e.totals.tolist() == [0, 0]


def test_plan_lengths_that_no_table_can_hold():
    # 2^31 - 1 pages for each of 300 requests, three columns a row: every row's own
    # columns are written, the first ones from the pool
    B, most = 300, 2 ** 31 - 1
    table = torch.full((B, 3), 7, dtype=torch.int32, device="cuda")
    p = bi.bi_paged_plan(_i32([1] + [0] * (B - 1)), _i32([most] * B), table, _i32([5, 6]), 1, 4)
    want = torch.full((B, 3), -1, dtype=torch.int32)
    want[0] = torch.tensor([7, 5, 6])
    assert torch.equal(table.cpu(), want)
    assert p.totals.tolist() == [most, most] and p.slots.tolist() == [5, 6, -1, -1]
    assert p.positions.tolist() == [1, 2, 3, 4] and p.seq_lens.tolist() == [most] * B


# -- rotary positions ------------------------------------------------------------------------

ROPES = [  # heads, D, rotary, interleaved
    (8, 256, 256, False), (4, 128, 64, True), (3, 64, 64, False), (5, 128, 128, True), (2, 80, 40, False),
    (2, 96, 96, True), (1, 7, 6, False), (3, 66, 2, True), (1, 1024, 32, False), (6, 64, 16, False)]


@pytest.mark.parametrize("H,D,R,inter", ROPES)
@pytest.mark.parametrize("dt,out", [(BF16, BF16), (F16, F16), (F32, BF16), (F32, F32), (BF16, F16)])
@pytest.mark.parametrize("backward", [False, True])
def test_rope_matches_reference(H, D, R, inter, dt, out, backward):
    T = 13
    x = _normal((T, H, D), dt, 1)
    pos = torch.tensor([0, 1, -1, 2, 816, 4095, 32768, 131071, 1 << 20, (1 << 31) - 1, -(1 << 31), 77, 5],
                       dtype=torch.int32, device="cuda")
    cfg = bi.bi_rope_config(R, interleaved=inter, magnitude=1.25)
    y = bi.bi_rope(x, pos, cfg, backward=backward, out_dtype=out)
    assert y.dtype == out
    want, size = ref.rope(x, pos.tolist(), ref.frequencies(R), inter, backward, 1.25)
    ref.assert_within(y, want, ref.rope_bound(want, size, out), "rope")
    assert bits_equal(y, bi.bi_rope(x, pos.long(), cfg, backward=backward, out_dtype=out))


@pytest.mark.parametrize("kw", [("linear", 4.0), ("base", 8.0), ("ramp_turns", 8.0, 8192.0, 1.0, 4.0),
                                ("ramp_index", 16.0, 4096.0, 1.0, 32.0)])
def test_rope_scaled_frequencies(kw):
    x = _normal((9, 4, 128), F32, 2)
    pos = torch.arange(9, device="cuda", dtype=torch.int64) * 15999
    y = bi.bi_rope(x, pos, bi.bi_rope_config(128, base=500000.0, scaling=bi.RopeScaling(*kw)))
    want, size = ref.rope(x, pos.tolist(), ref.frequencies(128, 500000.0, *kw), False)
    ref.assert_within(y, want, ref.rope_bound(want, size, F32))


def test_rope_very_far_positions_int64():
    # 2^40 * 2^-65 turns of the phase's own rounding are nothing beside fp32
    x = _normal((4, 2, 64), F32, 3)
    pos = [1 << 40, -(1 << 40) + 3, (1 << 40) + 12345, 1 << 33]
    f = [2.0 ** -20 * (1 + i / 32) * 6.283185307179586 for i in range(32)]  # turns are exact binary fractions
    y = bi.bi_rope(x, torch.tensor(pos, device="cuda"), bi.bi_rope_config(64, frequencies=f))
    want, size = ref.rope(x, pos, np.array(f), False)
    ref.assert_within(y, want, ref.rope_bound(want, size, F32))


@pytest.mark.parametrize("T", [1, 7, 3000])
def test_rope_layouts_give_the_same_bits(T):
    # strided views, misaligned rows (the one-pair kernel) and in place: all the same bits;
    # 3000 tokens run four heads a thread
    H, D = 32, 128
    cfg = bi.bi_rope_config(64, interleaved=False)
    pos = torch.randint(0, 100000, (T,), generator=_gen(4), device="cuda", dtype=torch.int32)
    wide = _normal((T, H + 5, D + 8), BF16, 5)
    x = wide[:, 2:2 + H, 8:]
    y = bi.bi_rope(x.contiguous(), pos, cfg)
    assert bits_equal(bi.bi_rope(x, pos, cfg), y)
    off = torch.empty(T * H * (D + 1) + 1, dtype=BF16, device="cuda")[1:].view(T, H, D + 1)[..., :D]
    off.copy_(x)
    assert bits_equal(bi.bi_rope(off, pos, cfg), y)
    keep = wide.clone()
    assert bi.bi_rope(x, pos, cfg, out=x) is x and bits_equal(x, y)
    wide[:, 2:2 + H, 8:] = keep[:, 2:2 + H, 8:]
    assert bits_equal(wide, keep)  # nothing around it was written
    bi.bi_rope(off, pos, cfg, out=off)
    assert bits_equal(off, y)
    assert bits_equal(bi.bi_rope(keep[T // 2:T // 2 + 1, 2:2 + H, 8:], pos[T // 2:T // 2 + 1], cfg), y[T // 2:T // 2 + 1])
    # expanded heads are read through a zero stride
    one = keep[:, 2:3, 8:]
    assert bits_equal(bi.bi_rope(one.expand(T, H, D), pos, cfg),
                      bi.bi_rope(one.expand(T, H, D).contiguous(), pos, cfg))


@pytest.mark.parametrize("inter", [False, True])
def test_rope_backward_is_the_gradient(inter):
    T, H, D, R = 6, 3, 64, 48
    cfg = bi.bi_rope_config(R, interleaved=inter, magnitude=0.75)
    pos = torch.arange(T, device="cuda", dtype=torch.int32) * 999
    x, dy = _normal((T, H, D), F32, 6), _normal((T, H, D), F32, 7)
    dx = bi.bi_rope(dy, pos, cfg, backward=True)
    # the formula's: the transposed map in 64 bits
    want, size = ref.rope(dy, pos.tolist(), ref.frequencies(R), inter, True, 0.75)
    ref.assert_within(dx, want, ref.rope_bound(want, size, F32))
    # against differences: the map is linear, so (f(x + h e) - f(x - h e)) / 2h is exact
    # for any h; here in 64 bits of the reference, along random directions
    for seed in (8, 9):
        e = _normal((T, H, D), F32, seed)
        up, _ = ref.rope(ref.f64(x) + 0.5 * ref.f64(e), pos.tolist(), ref.frequencies(R), inter, False, 0.75)
        dn, _ = ref.rope(ref.f64(x) - 0.5 * ref.f64(e), pos.tolist(), ref.frequencies(R), inter, False, 0.75)
        slope = float(((up - dn) * ref.f64(dy)).sum())
        b = float((ref.rope_bound(want, size, F32) * np.abs(ref.f64(e))).sum())
        assert abs(float((ref.f64(dx) * ref.f64(e)).sum()) - slope) <= b + 1e-9 * abs(slope)


# -- cache writes ---------------------------------------------------------------------------------

@pytest.mark.parametrize("Hq,Hkv,D,R,inter", [(8, 2, 128, 128, False), (4, 4, 64, 32, True), (5, 1, 256, 256, False),
                                              (3, 3, 80, 40, True)])
@pytest.mark.parametrize("dt,cdt", [(BF16, BF16), (F16, F16), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("page", [16, 7])
def test_store_matches_reference(Hq, Hkv, D, R, inter, dt, cdt, page):
    T, P = 37, 9
    qkv = _normal((T, Hq + 2 * Hkv, D), dt, 10)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    pos = torch.randint(0, 50000, (T,), generator=_gen(11), device="cuda", dtype=torch.int32)
    slots = torch.randperm(P * page, generator=_gen(12), device="cuda")[:T].contiguous()
    slots[5], slots[T - 1] = -1, -(1 << 40)
    kc, vc = _normal((P, page, Hkv, D), cdt, 13), _normal((P, page, Hkv, D), cdt, 14)
    kw, vw = ref.f64(kc).copy(), ref.f64(vc).copy()
    f = ref.frequencies(R)
    kr, size = ref.rope(k, pos.tolist(), f, inter)
    kb, vb = np.zeros_like(kw), np.zeros_like(vw)
    v64 = ref.f64(v)
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            kw[s // page, s % page], kb[s // page, s % page] = kr[t], ref.rope_bound(kr[t], size[t], cdt)
            vw[s // page, s % page] = v64[t]
            vb[s // page, s % page] = np.abs(v64[t]) * ref.HALF_STEP[cdt] + ref.SUBNORMAL[cdt]
    cfg = bi.bi_rope_config(R, interleaved=inter)
    qo = bi.bi_paged_store(k, v, slots, kc, vc, q=q, positions=pos, config=cfg)
    ref.assert_within(kc, kw, kb, "k_cache")  # rows that no token names: bound 0
    ref.assert_within(vc, vw, vb, "v_cache")
    assert qo.dtype == cdt and bits_equal(qo, bi.bi_rope(q, pos, cfg, out_dtype=cdt))
    # without q, the caches as two views of one tensor, the same bits
    both = torch.zeros(P, page, 2, Hkv, D, dtype=cdt, device="cuda")
    kc2, vc2 = both[:, :, 0], both[:, :, 1]
    assert bi.bi_paged_store(k, v, slots, kc2, vc2, positions=pos, config=cfg) is None
    s = slots[slots >= 0]
    assert bits_equal(kc2[s // page, s % page], kc[s // page, s % page])
    assert bits_equal(vc2[s // page, s % page], vc[s // page, s % page])
    # without rotation: k as it is
    bi.bi_paged_store(k, v, slots, kc2, vc2)
    assert bits_equal(kc2[s // page, s % page], k[slots >= 0].to(cdt))


def test_store_views_of_pages_and_heads():
    # views with each cache's pages apart, heads before rows
    T, P, page, H, D = 11, 4, 8, 3, 64
    k, v = _normal((T, H, D), BF16, 15), _normal((T, H, D), BF16, 16)
    slots = torch.randperm(P * page, generator=_gen(17), device="cuda")[:T].contiguous()
    kv = torch.zeros(P, 2, H, page, D, dtype=BF16, device="cuda")
    kc, vc = kv[:, 0].transpose(1, 2), kv[:, 1].transpose(1, 2)
    with pytest.raises(bi.BiError):  # their memory ranges interleave page by page
        bi.bi_paged_store(k, v, slots, kc, kc)
    bi.bi_paged_store(k, v, slots, kc, vc)
    assert bits_equal(kc[slots // page, slots % page], k) and bits_equal(vc[slots // page, slots % page], v)


def test_rope_and_store_with_nothing_to_do():
    cfg = bi.bi_rope_config(64)
    x = torch.empty(0, 4, 64, dtype=BF16, device="cuda")
    assert bi.bi_rope(x, _i32([]), cfg).shape == (0, 4, 64)
    y = torch.empty(3, 0, 64, dtype=BF16, device="cuda")
    assert bi.bi_rope(y, _i32([1, 2, 3]), cfg).shape == (3, 0, 64)
    none = torch.empty(0, 16, 2, 64, dtype=BF16, device="cuda")
    k = _normal((2, 2, 64), BF16, 20)
    bi.bi_paged_store(k, k.clone(), torch.tensor([-1, -1], device="cuda"), none, none.clone())
    bi.bi_paged_store(k, k.clone(), torch.tensor([0, -1], device="cuda"), none, none.clone())
    _bad_index()


def test_store_slot_past_the_cache_is_reported_and_skipped():
    T, P, page, H, D = 4, 2, 16, 2, 64
    k, v = _normal((T, H, D), BF16, 18), _normal((T, H, D), BF16, 19)
    kc, vc = torch.zeros(P, page, H, D, dtype=BF16, device="cuda"), torch.zeros(P, page, H, D, dtype=BF16, device="cuda")
    bi.bi_paged_store(k, v, torch.tensor([3, P * page, 1 << 40, 31], device="cuda"), kc, vc)
    _bad_index()
    assert bits_equal(kc[0, 3], k[0]) and bits_equal(vc[1, 15], v[3])
    kc[0, 3], kc[1, 15] = 0, 0
    assert not kc.any()


# -- attention over the paged cache -------------------------------------------------------------

def _cache(lens, page, Hkv, D, dtype, seed, W=None, extra=3):
    need = [-(-max(n, 0) // page) for n in lens]
    P = sum(need) + extra
    ids = torch.randperm(P, generator=_gen(seed), device="cuda").to(torch.int32).cpu()
    table = torch.full((len(lens), W or max(max(need), 1)), -7, dtype=torch.int32)  # entries past a length: never read
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    kc, vc = _normal((P, page, Hkv, D), dtype, seed + 1), _normal((P, page, Hkv, D), dtype, seed + 2)
    # rows that belong to no token hold what must not be read into a result
    used = torch.zeros(P * page, dtype=torch.bool)
    for b, n in enumerate(lens):
        j = torch.arange(max(n, 0))
        used[table[b, j // page].long() * page + j % page] = True
    kc.view(P * page, Hkv, D)[~used.cuda()] = float("nan")
    vc.view(P * page, Hkv, D)[~used.cuda()] = float("inf")
    return kc, vc, table.cuda(), _i32(lens)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (6, 2), (8, 1), (16, 1), (10, 2), (40, 2)])
@pytest.mark.parametrize("dt,out", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
@pytest.mark.parametrize("page", [16, 7])
def test_attention_matches_reference(D, Hq, Hkv, dt, out, page):
    lens = [0, 1, 2, 15, 16, 17, 128, 255, 256, 257, 700, -3]
    kc, vc, table, ln = _cache(lens, page, Hkv, D, dt, 20)
    q = _normal((len(lens), Hq, D), dt, 23)
    o = bi.bi_paged_attention(q, kc, vc, table, ln, D ** -0.5, out_dtype=out)
    want, bound = ref.attention(q, kc, vc, table, ln, D ** -0.5, out)
    ref.assert_within(o, want, bound, "paged attention")
    assert not o[0].any() and not o[-1].any()  # no key: zeros


@pytest.mark.parametrize("n,page,dt", [(32768, 16, BF16), (32769, 128, BF16), (70001, 24, F16), (131071, 64, BF16)])
def test_attention_long_caches(n, page, dt):
    lens = [n, 5]
    kc, vc, table, ln = _cache(lens, page, 1, 64, dt, 30)
    q = _normal((2, 4, 64), dt, 33, std=2.0)
    for out in (F32, dt):
        o = bi.bi_paged_attention(q, kc, vc, table, ln, 0.125, out_dtype=out)
        want, bound = ref.attention(q, kc, vc, table, ln, 0.125, out)
        ref.assert_within(o, want, bound)


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 16, 1), (256, 4, 1)])
def test_attention_rows_do_not_depend_on_batch_pages_or_workspace(D, Hq, Hkv):
    lens = [1300, 40, 0, 257, 5000, 256]
    kc, vc, table, ln = _cache(lens, 16, Hkv, D, BF16, 40)
    q = _normal((len(lens), Hq, D), BF16, 43)
    o = bi.bi_paged_attention(q, kc, vc, table, ln, 0.1)
    big = torch.full((bi.bi_paged_attention_workspace_bytes(6, Hq, D, table.shape[1] * 16) + 64,), 255,
                     dtype=torch.uint8, device="cuda")  # NaN patterns: contents on entry do not matter
    assert bits_equal(bi.bi_paged_attention(q, kc, vc, table, ln, 0.1, workspace=big), o)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        # alone, on other pages of another size
        j = torch.arange(n, device="cuda")
        rows = table[b, j // 16].long(), j % 16
        page = 24
        P = -(-n // page) + 2
        k2 = torch.full((P, page, Hkv, D), float("nan"), dtype=BF16, device="cuda")
        v2 = k2.clone()
        t2 = torch.randperm(P, generator=_gen(44), device="cuda")[:P - 2].to(torch.int32)[None]
        k2[t2[0, j // page].long(), j % page] = kc[rows]
        v2[t2[0, j // page].long(), j % page] = vc[rows]
        assert bits_equal(bi.bi_paged_attention(q[b:b + 1], k2, v2, t2, ln[b:b + 1], 0.1), o[b:b + 1]), n
        # one query head's group alone
        g = Hq // Hkv
        assert bits_equal(bi.bi_paged_attention(q[b:b + 1, :g], k2[:, :, :1], v2[:, :, :1], t2, ln[b:b + 1], 0.1),
                          o[b:b + 1, :g])


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 3, 1), (128, 32, 2), (256, 8, 2)])
@pytest.mark.parametrize("out", [F32, BF16])
def test_attention_bits_do_not_depend_on_the_table_width(D, Hq, Hkv, out):
    # a narrow table (its pieces joined by a cluster in one launch) and a wide one
    for lens in ([1], [256], [257, 0], [700, 40, 2048], [1500] * 3):
        kc, vc, table, ln = _cache(lens, 16, Hkv, D, BF16, 46)
        q = _normal((len(lens), Hq, D), BF16, 49)
        o = bi.bi_paged_attention(q, kc, vc, table, ln, 0.1, out_dtype=out)
        for width in (129, 300, 1000):
            wide = torch.zeros(len(lens), width, dtype=torch.int32, device="cuda")
            wide[:, :table.shape[1]] = table
            assert bits_equal(bi.bi_paged_attention(q, kc, vc, wide, ln, 0.1, out_dtype=out), o), (lens, width)
        want, bound = ref.attention(q, kc, vc, table, ln, 0.1, out)
        ref.assert_within(o, want, bound)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 3, 1), (128, 8, 2), (256, 4, 1)])
def test_attention_bits_where_pieces_grow(D, Hq, Hkv):
    # 256 keys a piece up to 2048, 512 from there on: alone in narrow tables and
    # together in wide ones
    lens = [2047, 2048, 2049, 2560, 4095, 4096, 4097, 1, 65536, 65537]
    kc, vc, table, ln = _cache(lens, 16, Hkv, D, BF16, 47)
    q = _normal((len(lens), Hq, D), BF16, 48)
    o = bi.bi_paged_attention(q, kc, vc, table, ln, 0.1, out_dtype=F32)
    for i, n in enumerate(lens):
        own = table[i:i + 1, :(n + 15) // 16].contiguous()
        assert bits_equal(bi.bi_paged_attention(q[i:i + 1], kc, vc, own, ln[i:i + 1], 0.1, out_dtype=F32), o[i:i + 1]), n
    want, bound = ref.attention(q, kc, vc, table, ln, 0.1, F32)
    ref.assert_within(o, want, bound)


def test_attention_strided_operands():
    lens, page, Hkv, D, Hq = [300, 33], 16, 2, 64, 4
    kc, vc, table, ln = _cache(lens, page, Hkv, D, F16, 50)
    P = kc.shape[0]
    q = _normal((2, Hq, D), F16, 53)
    o = bi.bi_paged_attention(q, kc, vc, table, ln, 0.125)
    kv = torch.empty(P, 2, Hkv, page, D + 8, dtype=F16, device="cuda")
    k2, v2 = kv[:, 0, ..., :D].transpose(1, 2), kv[:, 1, ..., 8:].transpose(1, 2)
    k2.copy_(kc), v2.copy_(vc)
    qw = torch.empty(2, Hq + 3, D + 8, dtype=F16, device="cuda")
    qw[:, 1:1 + Hq, :D] = q
    tw = torch.full((2, table.shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    tw[:, :table.shape[1]] = table
    out = torch.full((2, Hq + 1, D + 4), 3.0, dtype=F32, device="cuda")
    bi.bi_paged_attention(qw[:, 1:1 + Hq, :D], k2, v2, tw[:, :table.shape[1]], ln, 0.125, out=out[:, 1:, :D])
    assert bits_equal(out[:, 1:, :D], o)
    assert bool((out[:, :1] == 3.0).all()) and bool((out[..., D:] == 3.0).all())


def test_attention_offsets_past_32_bits():
    # the last pages of a cache of 2^32 elements and more, by page and by slot
    page, Hkv, D = 16, 8, 128
    P = (1 << 32) // (page * Hkv * D) + 8
    kc = torch.empty(P, page, Hkv, D, dtype=BF16, device="cuda")
    vc = torch.empty(P, page, Hkv, D, dtype=BF16, device="cuda")
    n = 100
    table = torch.arange(P - 7, P, dtype=torch.int32, device="cuda")[None].contiguous()
    slots = table[0].long().repeat_interleave(page)[:n] * page + torch.arange(n, device="cuda") % page
    k, v = _normal((n, Hkv, D), BF16, 60), _normal((n, Hkv, D), BF16, 61)
    bi.bi_paged_store(k, v, slots, kc, vc)
    q = _normal((1, 32, D), BF16, 62)
    o = bi.bi_paged_attention(q, kc, vc, table, _i32([n]), D ** -0.5)
    want, bound = ref.attention(q, kc, vc, table, _i32([n]), D ** -0.5, F32)
    ref.assert_within(o, want, bound)
    assert bits_equal(kc[P - 7], k[:page])


def test_attention_absent_pages_and_overlong_lengths_are_reported():
    lens, page, Hkv, D = [100, 64], 16, 1, 64
    kc, vc, table, ln = _cache(lens, page, Hkv, D, BF16, 70)
    kc.nan_to_num_(0.0), vc.nan_to_num_(0.0, 0.0, 0.0)
    q = _normal((2, 2, D), BF16, 73)
    bad = table.clone()
    bad[0, 2], bad[0, 4], bad[1, :4] = -1, kc.shape[0], 1 << 30
    o = bi.bi_paged_attention(q, kc, vc, bad, ln, 0.125)
    _bad_index()
    want, bound = ref.attention(q, kc, vc, bad, ln, 0.125, F32)
    ref.assert_within(o, want, bound)
    assert not o[1].any()
    long = _i32([10 ** 9, 64])
    o = bi.bi_paged_attention(q[1:], kc, vc, table[1:, :4], long[:1], 0.125)
    _bad_index()
    assert bits_equal(o, bi.bi_paged_attention(q[1:], kc, vc, table[1:, :4], ln[1:], 0.125))


def test_attention_extreme_scores():
    # scores far apart: one key takes all; and NaN and infinity inside a request's own rows
    lens, page, Hkv, D = [600], 16, 1, 64
    kc, vc, table, ln = _cache(lens, page, Hkv, D, BF16, 80)
    q = torch.full((1, 1, D), 16.0, dtype=BF16, device="cuda")
    j = 437
    row = (table[0, j // page].long(), j % page)
    kc[row] = 64.0
    o = bi.bi_paged_attention(q, kc, vc, table, ln, 1.0)
    want, bound = ref.attention(q, kc, vc, table, ln, 1.0, F32)
    ref.assert_within(o, want, bound)
    # every other weight is 2^-huge = 0 and the row's own 1: the value itself, by one rounding of 1 / 1
    assert np.array_equal(ref.f64(o[0, 0]), ref.f64(vc[row][0]))
    kc[row] = float("nan")
    assert bi.bi_paged_attention(q, kc, vc, table, ln, 1.0).isnan().all()


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_attention_zero_and_negative_scale(scale):
    kc, vc, table, ln = _cache([300, 3], 16, 2, 64, BF16, 85)
    q = _normal((2, 4, 64), BF16, 88)
    o = bi.bi_paged_attention(q, kc, vc, table, ln, scale)
    want, bound = ref.attention(q, kc, vc, table, ln, scale, F32)
    ref.assert_within(o, want, bound)


def test_attention_empty_cache_and_empty_tables():
    q = _normal((2, 4, 64), BF16, 89)
    none = torch.empty(0, 16, 2, 64, dtype=BF16, device="cuda")
    t = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    assert not bi.bi_paged_attention(q, none, none, t, _i32([0, 0]), 0.1).any()
    assert not bi.bi_paged_attention(q, none, none, t, _i32([5, 40]), 0.1).any()
    _bad_index()  # pages of a cache that has none
    kc = _normal((2, 16, 2, 64), BF16, 90)
    assert not bi.bi_paged_attention(q, kc, kc, t[:, :0], _i32([0, 7]), 0.1).any()
    _bad_index()  # a length past an empty table


def test_attention_a_nan_head_stays_alone():
    kc, vc, table, ln = _cache([700], 16, 1, 128, F16, 91)
    q = _normal((1, 12, 128), F16, 94)
    o = bi.bi_paged_attention(q, kc, vc, table, ln, 0.09)
    q[0, 5] = float("nan")
    p = bi.bi_paged_attention(q, kc, vc, table, ln, 0.09)
    assert p[0, 5].isnan().all()
    keep = [h for h in range(12) if h != 5]
    assert bits_equal(p[:, keep], o[:, keep])


def test_attention_many_requests():
    # more requests than a block has threads: pieces are found by a walk
    lens = [(i * 37) % 300 for i in range(700)]
    kc, vc, table, ln = _cache(lens, 32, 1, 64, BF16, 95)
    q = _normal((700, 2, 64), BF16, 98)
    o = bi.bi_paged_attention(q, kc, vc, table, ln, 0.125)
    want, bound = ref.attention(q, kc, vc, table, ln, 0.125, F32)
    ref.assert_within(o, want, bound)


def test_attention_graph_replay_follows_lengths_and_tables():
    page, Hkv, D, Hq, B = 16, 2, 128, 8, 3
    kc, vc = _normal((64, page, Hkv, D), BF16, 90), _normal((64, page, Hkv, D), BF16, 91)
    table = torch.zeros(B, 32, dtype=torch.int32, device="cuda")
    lens = _i32([1, 1, 1])
    q = _normal((B, Hq, D), BF16, 92)
    out = torch.empty(B, Hq, D, dtype=BF16, device="cuda")
    ws = torch.empty(bi.bi_paged_attention_workspace_bytes(B, Hq, D, 32 * page), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bi.bi_paged_attention(q, kc, vc, table, lens, 0.1, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bi.bi_paged_attention(q, kc, vc, table, lens, 0.1, out=out, workspace=ws)
    for seed, now in enumerate(([512, 0, 300], [5, 257, 256], [511, 512, 1])):
        table.copy_(torch.stack([torch.randperm(64, generator=_gen(seed), device="cuda")[:32] for _ in range(B)]))
        lens.copy_(_i32(now))
        q.copy_(_normal((B, Hq, D), BF16, 93 + seed))
        graph.replay()
        assert bits_equal(out, bi.bi_paged_attention(q, kc, vc, table, lens, 0.1, out_dtype=BF16))


# -- token log probabilities ---------------------------------------------------------------------------

def _check_logprobs(x, tokens, top):
    r = bi.bi_token_logprobs(x, tokens, top=top)
    lp, ent, tlp, ids, blp, bent, btlp = ref.logprobs(x, tokens.tolist(), top)
    ref.assert_same_nonfinite(r.logprobs, lp, blp, "logprobs")
    ref.assert_same_nonfinite(r.entropy, ent, bent, "entropy")
    if top:
        assert np.array_equal(r.top_ids.cpu().numpy(), ids), "ids"
        ref.assert_same_nonfinite(r.top_logprobs, tlp, btlp, "top_logprobs")
        # an alternative's log probability is the one it has as the given token
        for k in {0, top - 1}:
            again = bi.bi_token_logprobs(x, r.top_ids[:, k].contiguous())
            assert bits_equal(again.logprobs, r.top_logprobs[:, k].contiguous())
            assert bits_equal(again.entropy, r.entropy)
    return r


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("N,top", [(1, 1), (2, 0), (7, 7), (33, 5), (64, 64), (1000, 20), (1024, 64), (2048, 1),
                                   (2049, 64), (4096, 20), (4097, 64), (8192, 5), (8193, 64), (16384, 64), (16385, 20),
                                   (40003, 64), (65537, 20), (128256, 20), (300001, 64)])
def test_logprobs_match_reference(dt, N, top):
    R = 5 if N < 50000 else 3
    x = _normal((R, N), dt, 100 + N, std=3.0)
    tokens = torch.randint(0, N, (R,), generator=_gen(101), device="cuda")
    tokens[0] = N - 1
    _check_logprobs(x, tokens, top)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("N", [50, 3000, 12000, 40000, 200000])
def test_logprobs_ties_masks_and_nonfinite_rows(dt, N):
    ninf = float("-inf")
    rows = [torch.zeros(N),                                   # every token the same: the lowest indices
            torch.where(torch.arange(N) % 7 == 3, 2.0, -1.0),  # one in seven
            torch.full((N,), ninf).index_fill(0, torch.tensor([3, N - 1]), 1.5),  # two tokens allowed
            torch.full((N,), ninf),                           # none allowed: NaN
            torch.linspace(-50, 50, N),                       # ascending
            torch.linspace(50, -50, N),                       # descending
            torch.zeros(N).index_fill(0, torch.tensor([N // 2]), float("nan")),
            torch.zeros(N).index_fill(0, torch.tensor([1, N // 3]), float("inf")),
            torch.where(torch.arange(N) % 2 == 0, -0.0, 0.0),  # signed zeros are equal
            torch.arange(N) % 61 * 1.0]
    x = torch.stack(rows).to(dt).cuda()
    tokens = torch.tensor([0, 3, N - 1, 5, N - 1, 0, 2, 1, 7, -1], device="cuda")
    r = _check_logprobs(x, tokens, 20)
    assert r.top_ids[0].tolist() == list(range(20)) and r.top_ids[8].tolist() == list(range(20))
    assert r.top_ids[6, 0].item() == N // 2 and r.top_ids[2, :2].tolist() == [3, N - 1]
    assert r.logprobs[9].item() == ninf  # no such token
    assert r.logprobs.isnan().tolist() == [False] * 3 + [True] + [False] * 2 + [True] * 2 + [False] * 2
    assert bi.bi_token_logprobs(x[9:], torch.tensor([N], device="cuda")).logprobs.item() == ninf


@pytest.mark.parametrize("N", [1000, 9000, 70000])
def test_logprobs_rows_do_not_depend_on_batch_or_layout(N):
    x = _normal((6, N), BF16, 110, std=2.0)
    tokens = torch.randint(0, N, (6,), generator=_gen(111), device="cuda", dtype=torch.int32)
    r = bi.bi_token_logprobs(x, tokens, top=9)
    wide = torch.full((6, N + 13), float("nan"), dtype=BF16, device="cuda")
    wide[:, 5:5 + N] = x
    even = torch.full((6, N + 24), float("nan"), dtype=BF16, device="cuda")
    even = even[:, :(N + 24) // 8 * 8] if N % 8 else even
    even[:, 8:8 + N] = x
    for y, t in ((wide[:, 5:5 + N], tokens.long()), (wide[:, 5:5 + N], tokens), (even[:, 8:8 + N], tokens)):
        s = bi.bi_token_logprobs(y, t, top=9)
        assert all(bits_equal(a, b) for a, b in zip(r, s))
    for i in (0, 5):
        s = bi.bi_token_logprobs(x[i:i + 1], tokens[i:i + 1], top=9)
        assert all(bits_equal(a[i:i + 1], b) for a, b in zip(r, s))
    # a broadcast row, and outputs of the caller's own with parts left out
    s = bi.bi_token_logprobs(x[2:3].expand(3, N), tokens[2:3].expand(3).contiguous(), top=9)
    assert all(bits_equal(a[2:3].expand(b.shape), b) for a, b in zip(r, s))
    only = bi.TokenLogprobs(torch.empty(6, device="cuda"), None, None, None)
    bi.bi_token_logprobs(x, tokens, out=only)
    assert bits_equal(only.logprobs, r.logprobs)


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("R,N", [(3, 5), (3, 4099), (5, 20003), (400, 9001), (700, 37)])
def test_logprobs_rows_at_any_offset(dt, R, N):
    # rows of every alignment, among NaNs: the bits of rows on boundaries
    x = _normal((R, N), dt, 129, std=2.0)
    x[1, ::3] = float("-inf")
    tokens = torch.randint(0, N, (R,), generator=_gen(130), device="cuda")
    even = torch.full((R, (N + 15) // 8 * 8), float("nan"), dtype=dt, device="cuda")
    even[:, :N] = x
    r = bi.bi_token_logprobs(even[:, :N], tokens, top=min(N, 6))
    for at in range(8):
        for pad in (9, 16 - N % 8):  # another alignment every row, the same for all
            wide = torch.full((R, N + pad), float("nan"), dtype=dt, device="cuda")
            wide[:, at:at + N] = x
            s = bi.bi_token_logprobs(wide[:, at:at + N], tokens, top=min(N, 6))
            assert all(bits_equal(a, b) for a, b in zip(r, s)), (at, pad)


@pytest.mark.parametrize("dt,N,R", [(BF16, 128256, 330), (F32, 40001, 320), (F16, 16385, 310), (BF16, 70004, 310),
                                    (F32, 128256, 310), (F32, 9000, 310)])
def test_logprobs_many_long_rows(dt, N, R):
    # a CTA a row, and a cluster a row for a few rows: the same bits; rows on 16-byte
    # boundaries and others; a few unusual rows among them
    ninf = float("-inf")
    x = _normal((R, N), dt, 124, std=3.0)
    x[3] = ninf
    x[3, [7, 50]] = 1.0
    x[4] = ninf
    x[5, 11] = float("nan")
    x[6, N - 1] = float("inf")
    x[7] = torch.finfo(dt).min
    x[8] = 0.5
    x[9, ::2] = ninf
    tokens = torch.randint(0, N, (R,), generator=_gen(125), device="cuda")
    r = bi.bi_token_logprobs(x, tokens, top=20)
    for lo, hi in ((0, 12), (R - 3, R)):
        few = _check_logprobs(x[lo:hi], tokens[lo:hi], 20)
        assert all(bits_equal(a[lo:hi], b) for a, b in zip(r, few))
    order = torch.sort(x[12:].float(), dim=-1, descending=True, stable=True).indices[:, :20].int()
    assert torch.equal(r.top_ids[12:], order)
    s = bi.bi_token_logprobs(x, tokens, top=0, entropy=True)
    assert bits_equal(s.logprobs, r.logprobs) and bits_equal(s.entropy, r.entropy)


def test_logprobs_many_rows():
    x = _normal((700, 5000), F16, 120)
    tokens = torch.randint(0, 5000, (700,), generator=_gen(121), device="cuda")
    _check_logprobs(x, tokens, 3)
    x = _normal((200, 66000), BF16, 122)
    tokens = torch.randint(0, 66000, (200,), generator=_gen(123), device="cuda")
    _check_logprobs(x, tokens, 3)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_logprobs_rows_of_lowest_numbers_without_alternatives(dt):
    # many rows a CTA, all summed by the definition, nothing asked for but the
    # token's own: each row is as it is alone
    x = _normal((4000, 300), dt, 126)
    x[::2] = torch.finfo(dt).min
    x[::2, ::3] = float("-inf")
    x[::2, 5] = 0.75 * torch.finfo(dt).min
    x[6::8] = torch.finfo(dt).min
    tokens = torch.randint(0, 300, (4000,), generator=_gen(127), device="cuda")
    r = bi.bi_token_logprobs(x, tokens)
    few = _check_logprobs(x[:16], tokens[:16], 0)
    assert bits_equal(r.logprobs[:16], few.logprobs) and bits_equal(r.entropy[:16], few.entropy)
    # every eighth row holds one number: each of its 300 tokens has 1/300
    assert torch.equal(r.logprobs[6::8], r.logprobs[6:7].expand(500)) and torch.equal(r.entropy[6::8], r.entropy[6:7].expand(500))
    ref.assert_same_nonfinite(r.logprobs[6:7], *(np.full(1, v) for v in (-np.log(300.0), 2.0 ** -20)), "uniform")


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("N", [40, 9001, 40000])
def test_logprobs_logits_masked_by_low_numbers(dt, N):
    # rows whose maximum, or most of whose entries, are low numbers of any size up
    # to the type's lowest, with -inf, the lowest number and a NaN among the entries
    low = torch.finfo(dt).min
    tops = [low, 0.98 * low, 0.9 * low, 0.25 * low, 1e-3 * low, -3e30, -1e20, -1e12, -1e10, -1.1e9, -4e6, -2.2e6, -1.5e6,
            -1e6, -6e4, -5e3, -3.0, 8.0]
    tops = [t for t in tops if t >= low]
    x = torch.full((5 * len(tops), N), low, dtype=torch.float64)
    for i, t in enumerate(tops):
        x[5 * i:5 * i + 4, 2::5] = t
        x[5 * i + 1, ::3] = float("-inf")
        x[5 * i + 2] = float("-inf")
        x[5 * i + 2, [1, N - 2]] = t
        x[5 * i + 2, 7] = low
        x[5 * i + 3, N // 2] = float("nan")
        x[5 * i + 4] = t  # whole chunks of it in a row of others
        x[5 * i + 4, :min(N, 8192):3] = torch.linspace(-4, 4, len(range(0, min(N, 8192), 3)), dtype=torch.float64)
    tokens = torch.randint(0, N, (x.shape[0],), generator=_gen(128), device="cuda")
    _check_logprobs(x.to(dt).cuda(), tokens, 11)
    few = slice(-10, None)  # a cluster a row and a CTA a row: the same bits
    a, b = (bi.bi_token_logprobs(y.to(dt).cuda(), tokens[few].repeat(k)) for y, k in ((x[few], 1), (x[few].repeat(40, 1), 40)))
    assert bits_equal(a.logprobs, b.logprobs[:10]) and bits_equal(a.entropy, b.entropy[:10])


# -- streams and the whole step -------------------------------------------------------------------------

def test_calls_on_another_stream():
    s = torch.cuda.Stream()
    x = _normal((64, 8, 128), BF16, 130)
    pos = torch.arange(64, device="cuda", dtype=torch.int32)
    logits = _normal((4, 50000), F32, 131)
    tok = torch.zeros(4, dtype=torch.int64, device="cuda")
    kc, vc, table, ln = _cache([900], 16, 2, 128, BF16, 132)
    q = _normal((1, 8, 128), BF16, 135)
    cfg = bi.bi_rope_config(128)
    here = (bi.bi_rope(x, pos, cfg), bi.bi_paged_attention(q, kc, vc, table, ln, 0.1),
            bi.bi_token_logprobs(logits, tok, top=4).top_logprobs)
    s.wait_stream(torch.cuda.current_stream())
    there = (bi.bi_rope(x, pos, cfg, stream=s), bi.bi_paged_attention(q, kc, vc, table, ln, 0.1, stream=s),
             bi.bi_token_logprobs(logits, tok, top=4, stream=s).top_logprobs)
    torch.cuda.current_stream().wait_stream(s)
    assert all(bits_equal(a, b) for a, b in zip(here, there))


def test_decode_steps_captured_and_replayed():
    """Three requests and one padded row over six decode steps: plan, rotate and store,
    attend, project, log probabilities -- captured once, replayed a step at a time, each
    step against the reference run on the whole history."""
    B, page, W, Hq, Hkv, D, V = 4, 8, 6, 8, 2, 64, 1000
    cfg = bi.bi_rope_config(D, scaling=bi.RopeScaling("linear", 2.0))
    freq = ref.frequencies(D, 10000.0, "linear", 2.0)
    ctx, new = _i32([0, 7, 19, 0]), _i32([1, 1, 1, 0])
    table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
    table[1, 0], table[2, :3] = 20, _i32([21, 22, 23])
    pool = torch.arange(20, dtype=torch.int32, device="cuda").flip(0).contiguous()
    kc, vc = _normal((24, page, Hkv, D), BF16, 140), _normal((24, page, Hkv, D), BF16, 141)
    w_out = _normal((Hq * D, V), BF16, 142, std=0.05)
    qkv = torch.empty(B, Hq + 2 * Hkv, D, dtype=BF16, device="cuda")
    tok = torch.zeros(B, dtype=torch.int64, device="cuda")
    plan = bi.bi_paged_plan_buffers(B, B)
    ws = torch.empty(max(16, bi.bi_paged_attention_workspace_bytes(B, Hq, D, W * page)), dtype=torch.uint8, device="cuda")

    def step():
        bi.bi_paged_plan(ctx, new, table, pool, page, out=plan)
        q = bi.bi_paged_store(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], plan.slots, kc, vc, q=qkv[:, :Hq],
                              positions=plan.positions, config=cfg)
        o = bi.bi_paged_attention(q, kc, vc, table, plan.seq_lens, D ** -0.5, out_dtype=BF16, workspace=ws)
        logits = bi.bi_mm(o.view(B, Hq * D), w_out)
        return q, o, logits, bi.bi_token_logprobs(logits, tok, top=5)

    # the library's first calls on the device come before the capture, on scratch copies
    saved = [t.clone() for t in (table, kc, vc)]
    qkv.copy_(_normal(qkv.shape, BF16, 143))
    step()
    for t, s in zip((table, kc, vc), saved):
        t.copy_(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, o, logits, lp = step()
    for n in range(6):
        qkv.copy_(_normal(qkv.shape, BF16, 150 + n))
        tok.copy_(torch.randint(0, V, (B,), generator=_gen(160 + n), device="cuda"))
        before_k, before_v, before_table = kc.clone(), vc.clone(), table.clone()
        graph.replay()
        want = ref.plan(ctx.tolist(), new.tolist(), before_table.cpu().numpy(), pool.tolist(), page, B)
        assert np.array_equal(table.cpu().numpy(), want[0])
        for g, w in zip(plan, want[1:]):
            assert np.array_equal(g.cpu().numpy(), w)
        pos = plan.positions.tolist()
        qw, size = ref.rope(qkv[:, :Hq], pos, freq, False)
        ref.assert_within(q, qw, ref.rope_bound(qw, size, BF16))
        kw, size = ref.rope(qkv[:, Hq:Hq + Hkv], pos, freq, False)
        for t, s in enumerate(plan.slots.tolist()):
            if s < 0:
                continue
            ref.assert_within(kc[s // page, s % page], kw[t], ref.rope_bound(kw[t], size[t], BF16))
            assert bits_equal(vc[s // page, s % page], qkv[t, Hq + Hkv:])
            before_k[s // page, s % page], before_v[s // page, s % page] = kc[s // page, s % page], vc[s // page, s % page]
        assert bits_equal(kc, before_k) and bits_equal(vc, before_v)  # nothing else was written
        ow, bound = ref.attention(q, kc, vc, table, plan.seq_lens, D ** -0.5, BF16)
        ref.assert_within(o, ow, bound)
        assert not o[3].any()  # the padded row
        assert bits_equal(logits, bi.bi_mm(o.view(B, Hq * D), w_out))
        again = bi.bi_token_logprobs(logits, tok, top=5)
        assert all(bits_equal(a, b) for a, b in zip(lp, again))
        _check_logprobs(logits, tok, 5)
        taken = int(plan.totals[0].item())
        if taken:  # the host hands the rest of the pool to the next step
            pool.copy_(torch.cat([pool[taken:], pool[:taken]]))
        ctx.copy_(plan.seq_lens)
