"""Host-side checks of the 8-bit operations and of sampling that need no GPU:
refusals, all before any launch (the descriptors point at fake addresses that are
never touched), and the references themselves."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

from invariant_gemm_bi_gb300 import binding, build
from tests import quantized_reference as ref
from tests.test_serving_cpu import Arena, _r

BF16, F16, F32, I32, I64, E4M3 = range(6)
OK, INVALID, SHAPE, DTYPE, LAYOUT = (binding.BI_OK, binding.BI_ERR_INVALID_ARG, binding.BI_ERR_SHAPE_MISMATCH,
                                     binding.BI_ERR_UNSUPPORTED_DTYPE, binding.BI_ERR_UNSUPPORTED_LAYOUT)
REACHED = binding.BI_ERR_NO_DEVICE  # a valid call without a GPU
no_gpu = not torch.cuda.is_available()


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _with(o, a, change):
    o.update({k: (v(a, o) if callable(v) else v) for k, v in change.items()})
    return o


def _quantize(lib, **change):
    a = Arena()
    o = _with(dict(x=a.t([300, 400], BF16), br=128, q=a.t([300, 400], E4M3), s=a.t([3, 4], F32)), a, change)
    return lib.bi_quantize_blocks(_r(o["x"]), o["br"], _r(o["q"]), _r(o["s"]), None)


def test_quantize_refusals(lib):
    if no_gpu:
        assert _quantize(lib) == REACHED
        assert _quantize(lib, br=1, s=lambda a, o: a.t([300, 4], F32)) == REACHED
        assert _quantize(lib, x=lambda a, o: a.t([300, 400], F32, [401, 1])) == REACHED
        assert _quantize(lib, s=lambda a, o: a.t([3, 4], F32, [1, 3])) == REACHED
    assert _quantize(lib, x=None) == INVALID
    assert _quantize(lib, s=None) == INVALID
    assert _quantize(lib, br=64) == INVALID
    assert _quantize(lib, br=0) == INVALID
    assert _quantize(lib, s=lambda a, o: a.t([4, 4], F32)) == SHAPE
    assert _quantize(lib, br=1) == SHAPE
    assert _quantize(lib, q=lambda a, o: a.t([300, 401], E4M3)) == SHAPE
    assert _quantize(lib, q=lambda a, o: a.t([300, 400], BF16)) == DTYPE
    assert _quantize(lib, x=lambda a, o: a.t([300, 400], E4M3)) == DTYPE
    assert _quantize(lib, s=lambda a, o: a.t([3, 4], F16)) == DTYPE
    assert _quantize(lib, x=lambda a, o: a.t([300, 400], BF16, [1, 300])) == LAYOUT
    assert _quantize(lib, q=lambda a, o: a.t([300, 400], E4M3, [399, 1])) == LAYOUT  # rows on top of one another
    assert _quantize(lib, s=lambda a, o: a.t([3, 4], F32, [0, 1])) == LAYOUT
    assert _quantize(lib, q=lambda a, o: a.t([300, 400], E4M3, ptr=o["x"].ptr)) == INVALID
    assert _quantize(lib, s=lambda a, o: a.t([3, 4], F32, ptr=o["q"].ptr + 1000)) == INVALID
    assert _quantize(lib, br=1, x=lambda a, o: a.t([1 << 30, 400], BF16), q=lambda a, o: a.t([1 << 30, 400], E4M3),
                     s=lambda a, o: a.t([1 << 30, 4], F32)) == INVALID  # 2^32 blocks
    assert _quantize(lib, x=lambda a, o: a.t([0, 400], BF16), q=lambda a, o: a.t([0, 400], E4M3),
                     s=lambda a, o: a.t([0, 4], F32)) == OK


def _mm(lib, **change):
    a = Arena()
    o = _with(dict(a=a.t([20, 300], E4M3, [304, 1]), sa=a.t([20, 3], F32), b=a.t([300, 200], E4M3, [1, 304]),
                   sb=a.t([3, 2], F32, [1, 3]), bias=a.t([200], BF16), c=a.t([20, 200], BF16)), a, change)
    return lib.bi_mm_blockscaled(*(_r(o[k]) for k in ("a", "sa", "b", "sb", "bias", "c")), None)


def test_mm_blockscaled_refusals(lib):
    if no_gpu:
        assert _mm(lib) == REACHED
        assert _mm(lib, bias=None, c=lambda a, o: a.t([20, 200], F32, [333, 1])) == REACHED
        assert _mm(lib, bias=lambda a, o: a.t([200], F32, [7])) == REACHED
        assert _mm(lib, a=lambda a, o: a.t([1, 300], E4M3), sa=lambda a, o: a.t([1, 3], F32),
                   c=lambda a, o: a.t([1, 200], F16)) == REACHED  # one row: no stride to speak of
    assert _mm(lib, a=None) == INVALID
    assert _mm(lib, sb=None) == INVALID
    assert _mm(lib, a=lambda a, o: a.t([20, 300], BF16, [304, 1])) == DTYPE
    assert _mm(lib, b=lambda a, o: a.t([300, 200], F16, [1, 304])) == DTYPE
    assert _mm(lib, sa=lambda a, o: a.t([20, 3], BF16)) == DTYPE
    assert _mm(lib, c=lambda a, o: a.t([20, 200], E4M3)) == DTYPE
    assert _mm(lib, bias=lambda a, o: a.t([200], I32)) == DTYPE
    assert _mm(lib, sa=lambda a, o: a.t([20, 2], F32)) == SHAPE
    assert _mm(lib, sb=lambda a, o: a.t([2, 3], F32)) == SHAPE  # the weight's scales, not transposed
    assert _mm(lib, b=lambda a, o: a.t([299, 200], E4M3, [1, 304])) == SHAPE
    assert _mm(lib, c=lambda a, o: a.t([20, 201], BF16)) == SHAPE
    assert _mm(lib, bias=lambda a, o: a.t([199], BF16)) == SHAPE
    assert _mm(lib, b=lambda a, o: a.t([300, 200], E4M3, [208, 1])) == LAYOUT  # unit stride on N
    assert _mm(lib, a=lambda a, o: a.t([20, 300], E4M3, [300, 1])) == LAYOUT   # rows off 16 bytes
    assert _mm(lib, b=lambda a, o: a.t([300, 200], E4M3, [1, 300])) == LAYOUT
    assert _mm(lib, a=lambda a, o: a.t([20, 300], E4M3, [304, 1], ptr=0x7F1000000008)) == LAYOUT
    assert _mm(lib, a=lambda a, o: a.t([20, 300], E4M3, [0, 1])) == LAYOUT
    assert _mm(lib, c=lambda a, o: a.t([20, 200], BF16, [100, 1])) == LAYOUT
    assert _mm(lib, c=lambda a, o: a.t([20, 200], BF16, ptr=o["b"].ptr)) == INVALID
    assert "overlap" in binding.last_error_message()
    assert _mm(lib, c=lambda a, o: a.t([20, 200], BF16, ptr=o["sa"].ptr)) == INVALID


def _caches(a, P=10, ps=16, H=2, D=64):
    return dict(kc=a.t([P, ps, H, D], E4M3), ks=a.t([P, ps, H], F32), vc=a.t([P, ps, H, D], E4M3), vs=a.t([P, ps, H], F32))


def _store(lib, cfg, **change):
    a = Arena()
    o = _with(dict(pos=a.t([7], I32), slots=a.t([7], I64), q=a.t([7, 4, 64], BF16), qo=a.t([7, 4, 64], BF16),
                   k=a.t([7, 2, 64], BF16), v=a.t([7, 2, 64], BF16), **_caches(a)), a, change)
    return lib.bi_paged_store_quantized(ctypes.byref(cfg.desc) if cfg else None,
                                        *(_r(o[k]) for k in ("pos", "slots", "q", "qo", "k", "v", "kc", "ks", "vc", "vs")), None)


def test_store_quantized_refusals(lib):
    cfg = binding.bi_rope_config(64)
    if no_gpu:
        assert _store(lib, cfg) == REACHED
        assert _store(lib, cfg, qo=lambda a, o: o["q"]) == REACHED
        assert _store(lib, None, pos=None, q=None, qo=None) == REACHED
        assert _store(lib, cfg, ks=lambda a, o: a.t([10, 16, 2], F32, [64, 4, 2])) == REACHED
    assert _store(lib, None) == INVALID
    assert _store(lib, cfg, kc=lambda a, o: a.t([10, 16, 2, 64], BF16)) == DTYPE
    assert _store(lib, cfg, ks=lambda a, o: a.t([10, 16, 2], BF16)) == DTYPE
    assert _store(lib, cfg, vs=None) == INVALID
    assert _store(lib, cfg, vs=lambda a, o: a.t([10, 16, 3], F32)) == SHAPE
    assert _store(lib, cfg, vc=lambda a, o: a.t([10, 8, 2, 64], E4M3)) == SHAPE
    assert _store(lib, cfg, k=lambda a, o: a.t([7, 2, 64], E4M3), v=lambda a, o: a.t([7, 2, 64], E4M3)) == DTYPE
    assert _store(lib, cfg, qo=lambda a, o: a.t([7, 4, 64], E4M3)) == DTYPE
    assert _store(lib, cfg, ks=lambda a, o: a.t([10, 16, 2], F32, [32, 0, 1])) == LAYOUT
    assert _store(lib, cfg, vs=lambda a, o: a.t([10, 16, 2], F32, ptr=o["ks"].ptr)) == INVALID
    assert _store(lib, cfg, ks=lambda a, o: a.t([10, 16, 2], F32, ptr=o["kc"].ptr)) == INVALID
    assert _store(lib, cfg, vs=lambda a, o: a.t([10, 16, 2], F32, ptr=o["k"].ptr)) == INVALID
    assert _store(lib, cfg, slots=lambda a, o: a.t([7], I32)) == DTYPE
    # the 16-bit entry point takes no 8-bit caches
    a = Arena()
    assert lib.bi_paged_store(None, None, _r(a.t([7], I64)), None, None, _r(a.t([7, 2, 64], BF16)), _r(a.t([7, 2, 64], BF16)),
                              _r(a.t([10, 16, 2, 64], E4M3)), _r(a.t([10, 16, 2, 64], E4M3)), None) == DTYPE


def test_store_quantized_pages_that_hold_everything(lib):
    # a page's keys, values and scales side by side in one buffer, 4352 bytes a page
    def call(keys=0, values=2048, k_scales=4096, v_scales=4224, page=4352):
        at = 0x7E0000000000
        cache = lambda off: lambda a, o: a.t([10, 16, 2, 64], E4M3, [page, 128, 64, 1], ptr=at + off)  # noqa: E731
        scale = lambda off: lambda a, o: a.t([10, 16, 2], F32, [page // 4, 2, 1], ptr=at + off)  # noqa: E731
        return _store(lib, None, pos=None, q=None, qo=None, kc=cache(keys), vc=cache(values), ks=scale(k_scales), vs=scale(v_scales))
    if no_gpu:
        assert call() == REACHED
        assert call(keys=4352 * 3) == REACHED       # the views start in different pages
    assert call(k_scales=4092) == INVALID           # the last value's byte is the first scale's
    assert call(v_scales=4220) == INVALID
    assert call(v_scales=4352 - 124) == INVALID     # into the next page's keys
    assert call(values=2047) == INVALID
    assert "overlap" in binding.last_error_message()


def _load(lib, **change):
    a = Arena()
    o = _with(dict(slots=a.t([7], I64), **_caches(a), k=a.t([7, 2, 64], BF16), v=a.t([7, 2, 64], BF16)), a, change)
    return lib.bi_paged_load_quantized(*(_r(o[k]) for k in ("slots", "kc", "ks", "vc", "vs", "k", "v")), None)


def test_load_quantized_refusals(lib):
    if no_gpu:
        assert _load(lib) == REACHED
        assert _load(lib, k=lambda a, o: a.t([7, 2, 64], F32), v=lambda a, o: a.t([7, 2, 64], F32)) == REACHED
    assert _load(lib, v=lambda a, o: a.t([7, 2, 64], F32)) == DTYPE
    assert _load(lib, slots=lambda a, o: a.t([6], I64)) == SHAPE
    assert _load(lib, v=lambda a, o: a.t([7, 2, 63], BF16)) == SHAPE
    assert _load(lib, k=lambda a, o: a.t([7, 3, 64], BF16), v=lambda a, o: a.t([7, 3, 64], BF16)) == SHAPE
    assert _load(lib, vs=lambda a, o: a.t([10, 16], F32)) == INVALID
    assert _load(lib, k=lambda a, o: a.t([7, 2, 64], BF16, [0, 64, 1])) == LAYOUT
    assert _load(lib, v=lambda a, o: a.t([7, 2, 64], BF16, ptr=o["k"].ptr)) == INVALID
    assert _load(lib, k=lambda a, o: a.t([7, 2, 64], BF16, ptr=o["vc"].ptr)) == INVALID
    assert _load(lib, slots=lambda a, o: a.t([0], I64), k=lambda a, o: a.t([0, 2, 64], BF16),
                 v=lambda a, o: a.t([0, 2, 64], BF16)) == OK


def _attend(lib, **change):
    a = Arena()
    o = _with(dict(q=a.t([3, 4, 64], BF16), **_caches(a), table=a.t([3, 5], I32), lens=a.t([3], I32), scale=0.125,
                   o=a.t([3, 4, 64], F32), ws=a.t([1 << 20], F32), bytes=1 << 22), a, change)
    return lib.bi_paged_attention_quantized(*(_r(o[k]) for k in ("q", "kc", "ks", "vc", "vs", "table", "lens")), o["scale"],
                                            _r(o["o"]), o["ws"].ptr if o["ws"] is not None else None, o["bytes"], None)


def test_attention_quantized_refusals(lib):
    if no_gpu:
        assert _attend(lib) == REACHED
        assert _attend(lib, q=lambda a, o: a.t([3, 4, 64], F16), o=lambda a, o: a.t([3, 4, 64], BF16)) == REACHED
        assert _attend(lib, ws=None, bytes=0) == REACHED  # 80 keys: one piece
        assert _attend(lib, ks=lambda a, o: a.t([10, 16, 2], F32, [64, 2, 1])) == REACHED
    assert _attend(lib, q=lambda a, o: a.t([3, 4, 64], F32)) == DTYPE
    assert _attend(lib, kc=lambda a, o: a.t([10, 16, 2, 64], BF16), vc=lambda a, o: a.t([10, 16, 2, 64], BF16)) == DTYPE
    assert _attend(lib, ks=lambda a, o: a.t([10, 16, 2], F16)) == DTYPE
    assert _attend(lib, vs=lambda a, o: a.t([10, 15, 2], F32)) == SHAPE
    assert _attend(lib, kc=lambda a, o: a.t([10, 16, 2, 64], E4M3, [2060, 128, 64, 1])) == LAYOUT  # pages off 16 bytes
    assert _attend(lib, o=lambda a, o: a.t([3, 4, 64], F32, ptr=o["ks"].ptr)) == INVALID
    assert _attend(lib, table=lambda a, o: a.t([3, 50], I32), ws=None, bytes=0) == INVALID  # needs a workspace
    assert _attend(lib, table=lambda a, o: a.t([3, 50], I32), ws=lambda a, o: o["vs"]) == INVALID
    assert _attend(lib, scale=math.inf) == INVALID
    a = Arena()
    assert lib.bi_paged_attention(_r(a.t([3, 4, 64], BF16)), _r(a.t([10, 16, 2, 64], E4M3)), _r(a.t([10, 16, 2, 64], E4M3)),
                                  _r(a.t([3, 5], I32)), _r(a.t([3], I32)), 0.1, _r(a.t([3, 4, 64], F32)), None, 0, None) == DTYPE


def _sample(lib, **change):
    a = Arena()
    o = _with(dict(x=a.t([5, 1000], BF16), u=a.t([5], F32), t=a.t([5], F32), k=a.t([5], I32), p=a.t([5], F32),
                   m=a.t([5], F32), out=a.t([5], I64)), a, change)
    return lib.bi_sample_tokens(*(_r(o[k]) for k in ("x", "u", "t", "k", "p", "m", "out")), None)


def test_sample_refusals(lib):
    if no_gpu:
        assert _sample(lib) == REACHED
        assert _sample(lib, t=None, k=None, p=None, m=None, out=lambda a, o: a.t([5], I32)) == REACHED
        assert _sample(lib, x=lambda a, o: a.t([5, 327680], F32)) == REACHED
    assert _sample(lib, u=None) == INVALID
    assert _sample(lib, x=lambda a, o: a.t([5, 327681], F32)) == INVALID
    assert _sample(lib, x=lambda a, o: a.t([5, 0], F32)) == INVALID
    assert _sample(lib, x=lambda a, o: a.t([5, 1000], E4M3)) == DTYPE
    assert _sample(lib, u=lambda a, o: a.t([5], BF16)) == DTYPE
    assert _sample(lib, k=lambda a, o: a.t([5], I64)) == DTYPE
    assert _sample(lib, k=lambda a, o: a.t([5], F32)) == DTYPE
    assert _sample(lib, out=lambda a, o: a.t([5], F32)) == DTYPE
    for name in ("u", "t", "p", "m"):
        assert _sample(lib, **{name: lambda a, o: a.t([4], F32)}) == SHAPE
    assert _sample(lib, k=lambda a, o: a.t([6], I32)) == SHAPE
    assert _sample(lib, out=lambda a, o: a.t([6], I64)) == SHAPE
    assert _sample(lib, u=lambda a, o: a.t([5], F32, [2])) == LAYOUT
    assert _sample(lib, x=lambda a, o: a.t([5, 1000], BF16, [1, 5])) == LAYOUT
    assert _sample(lib, out=lambda a, o: a.t([5], I64, ptr=o["x"].ptr)) == INVALID
    assert _sample(lib, out=lambda a, o: a.t([5], I32, ptr=o["k"].ptr)) == INVALID
    assert _sample(lib, x=lambda a, o: a.t([0, 1000], BF16), **{n: (lambda a, o: a.t([0], F32)) for n in "utpm"},
                   k=lambda a, o: a.t([0], I32), out=lambda a, o: a.t([0], I64)) == OK


def test_bindings_refuse_what_the_library_cannot_be_told():
    x = torch.zeros((4, 128))
    for call in (lambda: binding.bi_quantize_blocks(x), lambda: binding.bi_mm_blockscaled(x, x, x, x),
                 lambda: binding.bi_sample_tokens(x, x[:, 0])):
        with pytest.raises(ValueError, match="expected a CUDA tensor"):
            call()


def test_reference_rounding_is_torch_s():
    # every pair of neighbours, their middle, and numbers beside it
    b = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    mid = (b[1:] + b[:-1]) / 2
    v = np.concatenate([b, mid, mid * (1 + 1e-6), mid * (1 - 1e-6)])
    v = np.concatenate([v, -v])
    assert np.array_equal(ref.round_e4m3(v), torch.from_numpy(v).float().to(torch.float8_e4m3fn).double().numpy())
    for size, scale in ((448.0, 1.0), (448.00003, 2.0), (1.0, 2.0 ** -8), (0.0, 1.0), (1e-45, 2.0 ** -126), (3.4e38, 2.0 ** 120)):
        assert ref.scale_of(np.array([size]))[0] == scale


def test_reference_sampling_by_hand():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    assert [ref.sample(x, u)[0] for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.71, 0.99)] == [0, 0, 1, 1, 2, 3, 3]
    assert [ref.sample(x, u, top_k=2)[0] for u in (0.0, 0.57, 0.58, 0.99)] == [1, 1, 3, 3]
    assert [ref.sample(x, u, top_p=0.75)[0] for u in (0.0, 0.43, 0.45, 0.66, 0.68)] == [1, 1, 2, 2, 3]
    assert [ref.sample(x, u, min_p=0.6)[0] for u in (0.0, 0.58)] == [1, 3]
    assert ref.sample(x, 0.99, t=0.0)[0] == 1 and ref.sample(np.full(4, -np.inf), 0.5)[0] == -1
    assert ref.sample(np.zeros(8), 0.99, top_k=3)[0] == 2  # the lower index among equals
