"""The 8-bit operations and token sampling at the ends of what they take: many tiles a
CTA with odd numbers of segments, scales at the ends of fp32, piece borders, operands
more than 2^32 bytes apart, the longest rows, calls on two streams at once, captured
calls that share a workspace."""
from __future__ import annotations

import pytest
import torch

from invariant_gemm_bi_gb300 import binding as bi
from tests import quantized_reference as ref
from tests import serving_reference as sref
from tests.gpu_helpers import bits_equal
from tests.test_gpu_quantized import (BF16, E4M3, F16, F32, _clean_status, _i32, _i64, _normal, _operands,  # noqa: F401
                                      _problem, _uniform)
from tests.test_gpu_sample import _check, _f32

pytestmark = pytest.mark.gpu
FAR = 2 ** 32 + 2 ** 20  # elements


# -- the block-scaled product ---------------------------------------------------------------

@pytest.mark.parametrize("M,N,K", [(600, 20000, 2200), (20, 20000, 6500), (1500, 9000, 2048)])
def test_mm_many_tiles_and_odd_segments(M, N, K):
    # several tiles a pair of CTAs, with an odd number of groups of exponents or of segments each
    a, sa, b, sb = _operands(M, N, K, 3)
    c = bi.bi_mm_blockscaled(a, sa, b, sb, out_dtype=F32)
    rows = [0, M // 2, M - 1]
    want, bound = ref.mm(a[rows], sa[rows], b, sb, None, F32)
    sref.assert_within(c[rows], want, bound)
    alone = bi.bi_mm_blockscaled(a[M // 2:M // 2 + 1], sa[M // 2:M // 2 + 1], b, sb, out_dtype=F32)
    assert bits_equal(alone, c[M // 2:M // 2 + 1].contiguous())
    some = bi.bi_mm_blockscaled(a, sa, b[:, 4096:4500], sb[:, 32:36], out_dtype=F32)  # other tiles, other pairs
    assert bits_equal(some, c[:, 4096:4500].contiguous())


def test_mm_column_of_a_tall_matrix():
    a, sa, b, sb = _operands(30000, 1, 300, 5)
    c = bi.bi_mm_blockscaled(a, sa, b, sb, out_dtype=F32)
    want, bound = ref.mm(a, sa, b, sb, None, F32)
    sref.assert_within(c, want, bound)


def test_mm_streams_and_graph():
    ops = [_operands(M, 2000, 2500, M) for M in (7, 300)]
    want = [bi.bi_mm_blockscaled(*o) for o in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[bi.bi_mm_blockscaled(*ops[i], stream=streams[i]) for i in range(2)] for _ in range(8)]
    torch.cuda.synchronize()
    for pair in got:
        assert all(bits_equal(pair[i], want[i]) for i in range(2))
    out = torch.empty_like(want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bi.bi_mm_blockscaled(*ops[0], out=out)
    ops[0][1].mul_(2.0)  # a's scales: twice the result
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.float(), 2 * want[0].float())


def test_mm_beside_the_library_s_other_kernels():
    # kernels that take tensor memory too, on other streams at the same time
    ops = _operands(500, 3000, 2500, 1)
    x, w = _normal((400, 1024), BF16, 2), _normal((1024, 2048), BF16, 3)
    q, k, v = (_normal((16, 600, 64), BF16, i) for i in (4, 5, 6))
    calls = [lambda st: bi.bi_mm_blockscaled(*ops, stream=st), lambda st: bi.bi_mm(x, w, stream=st),
             lambda st: bi.bi_attention(q, k, v, 0.125, stream=st)]
    want = [c(None) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    outs = []
    for _ in range(10):
        for c, st in zip(calls, streams):
            with torch.cuda.stream(st):  # allocated for the stream that writes it
                outs.append(c(st))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert bits_equal(o, want[i % 3])


# -- attention over the cache in 8 bits ------------------------------------------------------

@pytest.mark.parametrize("shift", [-90, 60, 118])
def test_attention_value_scales_near_the_ends(shift):
    # (values of at most 32 times a scale of at most 2^120: results that fp32 holds)
    q, kc, ks, vc, vs, table, n = _problem([700, 9], 4, 2, 64, 16, BF16, seed=4)
    vc = vc.float().clamp(-32, 32).to(E4M3)
    vs = torch.exp2(torch.floor(torch.log2(vs))) * 2.0 ** shift
    o = bi.bi_paged_attention_quantized(q, kc, ks, vc, vs, table, n, 0.125)
    want, bound = ref.attention(q, kc, ks, vc, vs, table, n, 0.125, F32)
    sref.assert_within(o, want, bound)


def test_attention_piece_borders():
    # 512 keys a piece up to 8192, 1024 beyond; tables that end at either and far behind
    lens = [8191, 8192, 8193, 9216, 9217]
    q, kc, ks, vc, vs, table, n = _problem(lens, 2, 1, 64, 64, BF16, seed=8)
    full = bi.bi_paged_attention_quantized(q, kc, ks, vc, vs, table, n, 0.125)
    want, bound = ref.attention(q, kc, ks, vc, vs, table, n, 0.125, F32)
    sref.assert_within(full, want, bound)
    for b, length in enumerate(lens):
        for width in (-(-length // 64), 4096):
            t = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
            t[0, :min(width, table.shape[1])] = table[b, :min(width, table.shape[1])]
            o = bi.bi_paged_attention_quantized(q[b:b + 1], kc, ks, vc, vs, t, n[b:b + 1], 0.125)
            assert bits_equal(o, full[b:b + 1].contiguous()), (length, width)


def test_attention_nothing_to_read():
    q, kc, ks, vc, vs, table, n = _problem([0, 0], 4, 2, 64, 16, BF16)
    n[1] = -3
    assert (bi.bi_paged_attention_quantized(q, kc, ks, vc, vs, table, n, 0.125) == 0).all()
    none = [t[:0] for t in (kc, ks, vc, vs)]  # no page at all
    assert (bi.bi_paged_attention_quantized(q, *none, table, n, 0.125) == 0).all()
    assert (bi.bi_paged_attention_quantized(q, kc, ks, vc, vs, table[:, :0], n, 0.125) == 0).all()
    assert bi.bi_paged_attention_quantized(q[:0], kc, ks, vc, vs, table[:0], n[:0], 0.125).shape == (0, 4, 64)
    rows = bi.bi_paged_load_quantized(_i64([-1, -7]), *none)
    assert (rows.k == 0).all() and (rows.v == 0).all()


def test_attention_streams_and_graphs_that_share_a_workspace():
    a = _problem([5000, 1200, 40], 8, 2, 128, 16, BF16, seed=1)
    b = _problem([3000, 4000, 6000], 8, 2, 128, 16, F16, seed=2)
    want = [bi.bi_paged_attention_quantized(*x, 0.1) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[bi.bi_paged_attention_quantized(*x, 0.1, stream=s) for x, s in zip((a, b), streams)] for _ in range(8)]
    torch.cuda.synchronize()
    for pair in got:
        assert all(bits_equal(pair[i], want[i]) for i in range(2))
    # one workspace, two graphs, replayed one after the other in any order
    need = max(bi.bi_paged_attention_workspace_bytes(3, 8, 128, x[5].shape[1] * 16) for x in (a, b))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for x in (a, b):
        out, graph = torch.empty_like(want[0]), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            bi.bi_paged_attention_quantized(*x, 0.1, out=out, workspace=ws)
        outs.append(out), graphs.append(graph)
    for i in (0, 1, 1, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert bits_equal(outs[i], want[i])


# -- operands more than 2^32 bytes apart ---------------------------------------------------------

@pytest.fixture(scope="module")
def far():
    """A buffer of views whose rows or pages are 2^32 bytes and more apart (as_strided counts
    its offset from the buffer's start)."""
    return torch.empty(FAR + 2 ** 21, dtype=torch.uint8, device="cuda")


def test_far_pages(far):
    H, D, page = 2, 128, 16
    caches = [far.view(E4M3).as_strided((2, page, H, D), (FAR, H * D, D, 1), i * 2 ** 14) for i in range(2)]
    scales = [far.view(F32).as_strided((2, page, H), (FAR // 4, H, 1), 2 ** 15 + i * 2 ** 12) for i in range(2)]
    args = (caches[0], scales[0], caches[1], scales[1])
    near = (torch.zeros((2, page, H, D), dtype=torch.uint8, device="cuda").view(E4M3), torch.zeros((2, page, H), device="cuda"),
            torch.zeros((2, page, H, D), dtype=torch.uint8, device="cuda").view(E4M3), torch.zeros((2, page, H), device="cuda"))
    k, v = _normal((2 * page, H, D), BF16, 1), _normal((2 * page, H, D), BF16, 2)
    slots = torch.arange(2 * page, device="cuda")
    pos = torch.arange(2 * page, device="cuda", dtype=torch.int32)
    config = bi.bi_rope_config(D)
    q = _normal((2 * page, 4, D), BF16, 3)
    for cache in (args, near):
        bi.bi_paged_store_quantized(k, v, slots, *cache, q=q, positions=pos, config=config)
    for x, y in zip(args, near):
        x, y = x.contiguous(), y.contiguous()
        assert torch.equal(x.view(torch.uint8) if x.dtype == E4M3 else x, y.view(torch.uint8) if y.dtype == E4M3 else y)
    x, y = bi.bi_paged_load_quantized(slots, *args), bi.bi_paged_load_quantized(slots, *near)
    assert torch.equal(x.k, y.k) and torch.equal(x.v, y.v)
    table = _i32([[0, 1], [1, 0]])
    x, y = (bi.bi_paged_attention_quantized(q[:2], *c, table, _i32([31, 20]), 0.1) for c in (args, near))
    assert bits_equal(x, y)


def test_far_rows(far):
    x = far.view(BF16).as_strided((2, 300), (FAR // 2, 1), 0)
    x.copy_(_normal((2, 300), BF16, 4))
    q, want = bi.bi_quantize_blocks(x), bi.bi_quantize_blocks(x.contiguous())
    assert torch.equal(q.values.view(torch.uint8), want.values.view(torch.uint8)) and torch.equal(q.scales, want.scales)
    u = torch.tensor([0.3, 0.8], device="cuda")
    assert torch.equal(bi.bi_sample_tokens(x, u), bi.bi_sample_tokens(x.contiguous(), u))
    a, sa, b, sb = _operands(2, 70, 300, 6)
    c = bi.bi_mm_blockscaled(a, sa, b, sb)
    a2 = far.view(E4M3).as_strided((2, 300), (FAR, 1), 2 ** 16)
    a2.view(torch.uint8).copy_(a.view(torch.uint8))
    sa2 = far.view(F32).as_strided((2, 3), (FAR // 4, 1), 2 ** 15)
    sa2.copy_(sa)
    out = far.view(BF16).as_strided((2, 70), (FAR // 2, 1), 2 ** 17)
    bi.bi_mm_blockscaled(a2, sa2, b, sb, out=out)
    assert bits_equal(out.contiguous(), c)


# -- token sampling ------------------------------------------------------------------------------

@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("R", [2, 160])
def test_sample_longest_rows(dt, R):
    # 327680 tokens, a few rows and more than fill the GPU; rows of one value, whose bin holds all of them
    N = 327680
    x = _normal((2, N), dt, 7, 2.0)
    x[1] = 0.25
    x = x.repeat(R // 2, 1)
    u = _uniform((R,), 8)
    k = torch.tensor([0, 1000, 0, 5], dtype=torch.int32, device="cuda").repeat(R // 2)[:R].contiguous()
    p = torch.tensor([0.9, 1.0, 0.5, 0.3], device="cuda").repeat(R // 2)[:R].contiguous()
    got = bi.bi_sample_tokens(x, u, top_k=k, top_p=p).tolist()
    x64 = sref.f64(x[:2])
    for r in range(0, R, 1 if R == 2 else 37):
        want, near = ref.sample(x64[r % 2], float(u[r]), 1.0, int(k[r]), float(p[r]))
        assert near or got[r] == want, r


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("ties", [False, True])
def test_sample_lists_of_every_length(dt, ties):
    # top-k around the lengths of a warp's run and of the whole list, and past it; with few
    # values, many elements of which are alike, the limit falls among equals
    ks = (1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 400, 480, 500, 511, 512, 513, 600, 0)
    x = _normal((3 * len(ks), 5000), F32, 21, 1.5)
    if ties:
        x = torch.round(4 * x) / 4
    R = x.shape[0]
    k = _i32([v for v in ks for _ in range(3)])
    p = _f32([1.0, 0.9, 0.3] * len(ks))
    m = _f32([0.0, 0.0, 0.02, 0.0, 0.2] * R)[:R].contiguous()
    _check(x.to(dt), _uniform((R,), 22), temperature=_f32([0.8, 1.3] * R)[:R].contiguous(), top_k=k, top_p=p, min_p=m)


def test_sample_many_short_rows():
    R = 70000
    x, u = _normal((R, 3), F32, 9), _uniform((R,), 10)
    got = bi.bi_sample_tokens(x, u)
    w = torch.softmax(x.double(), 1).cumsum(1)
    gap = (w - u.double()[:, None]).abs().min(1).values > 1e-8
    want = (w <= u.double()[:, None]).sum(1).clamp(max=2)
    assert torch.equal(got[gap], want[gap]) and int((~gap).sum()) < 20


def test_sample_streams_and_in_one_graph_twice():
    x, u = _normal((9, 5000), BF16, 1, 3.0), _uniform((9,), 2)
    want = bi.bi_sample_tokens(x, u)
    outs = [torch.empty(9, dtype=torch.int64, device="cuda") for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for out in outs:
            bi.bi_sample_tokens(x, u, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
