"""Host-side checks of the serving operations that need no GPU: refusals (all
before any launch; the descriptors point at fake addresses that are never
touched), workspace rules and the rotary configuration's frequencies."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

from invariant_gemm_bi_gb300 import binding, build
from tests import serving_reference as ref

BF16, F16, F32, I32, I64 = range(5)
INVALID, SHAPE, DTYPE, LAYOUT = (binding.BI_ERR_INVALID_ARG, binding.BI_ERR_SHAPE_MISMATCH,
                                 binding.BI_ERR_UNSUPPORTED_DTYPE, binding.BI_ERR_UNSUPPORTED_LAYOUT)
REACHED = binding.BI_ERR_NO_DEVICE  # a valid call without a GPU


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()



class Arena:
    """Descriptors at addresses of their own."""

    def __init__(self):
        self.at = 0x7F0000000000

    def t(self, shape, dtype, stride=None, ptr=None):
        if ptr is None:
            ptr = self.at
            self.at += 1 << 40
        d = binding.BiTensor()
        d.ptr, d.ndim, d.dtype = ptr, len(shape), dtype
        s = 1
        for i in reversed(range(len(shape))):
            d.shape[i] = shape[i]
            d.stride[i] = s if stride is None else stride[i]
            s *= max(shape[i], 1)
        return d


def _r(d):
    return ctypes.byref(d) if d is not None else None


def _plan(lib, **change):
    a = Arena()
    o = dict(ctx=a.t([3], I32), new=a.t([3], I32), table=a.t([3, 8], I32), pool=a.t([20], I32), page=16,
             lens=a.t([3], I32), offs=a.t([4], I32), pos=a.t([10], I32), slots=a.t([10], I64), totals=a.t([2], I32))
    o.update({k: (v(a, o) if callable(v) else v) for k, v in change.items()})
    return lib.bi_paged_plan(_r(o["ctx"]), _r(o["new"]), _r(o["table"]), _r(o["pool"]), o["page"], _r(o["lens"]),
                             _r(o["offs"]), _r(o["pos"]), _r(o["slots"]), _r(o["totals"]), None)


def test_plan_refusals(lib):
    if not torch.cuda.is_available():
        assert _plan(lib) == REACHED
    assert _plan(lib, ctx=lambda a, o: a.t([4], I32)) == SHAPE
    assert _plan(lib, offs=lambda a, o: a.t([3], I32)) == SHAPE
    assert _plan(lib, slots=lambda a, o: a.t([9], I64)) == SHAPE
    assert _plan(lib, totals=lambda a, o: a.t([1], I32)) == SHAPE
    assert _plan(lib, slots=lambda a, o: a.t([10], I32)) == DTYPE
    assert _plan(lib, ctx=lambda a, o: a.t([3], I64)) == DTYPE
    assert _plan(lib, table=lambda a, o: a.t([3, 8], F32)) == DTYPE
    assert _plan(lib, page=0) == INVALID
    assert _plan(lib, new=None) == INVALID
    assert _plan(lib, table=lambda a, o: a.t([3, 8], I32, [1, 3])) == LAYOUT
    assert _plan(lib, table=lambda a, o: a.t([3, 8], I32, [4, 1])) == LAYOUT  # rows on top of one another
    assert _plan(lib, pos=lambda a, o: a.t([10], I32, [2])) == LAYOUT
    # an output on top of an input or of another output
    assert _plan(lib, lens=lambda a, o: a.t([3], I32, ptr=o["ctx"].ptr)) == INVALID
    assert _plan(lib, offs=lambda a, o: a.t([4], I32, ptr=o["lens"].ptr + 8)) == INVALID
    assert "overlap" in binding.last_error_message()


def _rope(lib, cfg, **change):
    a = Arena()
    o = dict(x=a.t([5, 4, 128], BF16), pos=a.t([5], I32), y=a.t([5, 4, 128], BF16))
    o.update({k: (v(a, o) if callable(v) else v) for k, v in change.items()})
    return lib.bi_rope(ctypes.byref(cfg.desc) if cfg else None, _r(o["x"]), _r(o["pos"]), 0, _r(o["y"]), None)


def test_rope_refusals(lib):
    cfg = binding.bi_rope_config(64)
    if not torch.cuda.is_available():
        assert _rope(lib, cfg) == REACHED
        assert _rope(lib, cfg, y=lambda a, o: o["x"]) == REACHED  # in place
        assert _rope(lib, cfg, pos=lambda a, o: a.t([5], I64), y=lambda a, o: a.t([5, 4, 128], F32)) == REACHED
    assert _rope(lib, None) == INVALID
    assert _rope(lib, cfg, pos=None) == INVALID
    assert _rope(lib, cfg, pos=lambda a, o: a.t([4], I32)) == SHAPE
    assert _rope(lib, cfg, pos=lambda a, o: a.t([5], F32)) == DTYPE
    assert _rope(lib, cfg, x=lambda a, o: a.t([5, 4, 128], I32)) == DTYPE
    assert _rope(lib, cfg, y=lambda a, o: a.t([5, 4, 64], BF16)) == SHAPE
    assert _rope(lib, cfg, x=lambda a, o: a.t([5, 4, 128], BF16, [512, 1, 4])) == LAYOUT
    assert _rope(lib, cfg, y=lambda a, o: a.t([5, 4, 128], BF16, [0, 128, 1])) == LAYOUT  # tokens on one row
    # the head is narrower than the rotated part
    assert _rope(lib, cfg, x=lambda a, o: a.t([5, 4, 32], BF16), y=lambda a, o: a.t([5, 4, 32], BF16)) == INVALID
    # in place with another type, and shifted by one head
    assert _rope(lib, cfg, y=lambda a, o: a.t([5, 4, 128], F16, ptr=o["x"].ptr)) == INVALID
    assert _rope(lib, cfg, y=lambda a, o: a.t([5, 4, 128], BF16, ptr=o["x"].ptr + 256)) == INVALID
    assert _rope(lib, cfg, x=lambda a, o: a.t([0, 4, 128], BF16), y=lambda a, o: a.t([0, 4, 128], BF16),
                 pos=lambda a, o: a.t([0], I32)) == binding.BI_OK
    bad = binding.bi_rope_config(64)
    bad.desc.rotary_dim = 63
    assert _rope(lib, bad) == INVALID


@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=258), dict(base=1.0),
                                dict(base=float("nan")), dict(magnitude=float("inf")),
                                dict(scaling=("linear", 0.0)), dict(scaling=("ramp_turns", 8.0, 0.0, 1.0, 4.0)),
                                dict(scaling=("ramp_index", 8.0, 4096.0, 4.0, 4.0)),
                                dict(rotary_dim=2, scaling=("base", 2.0)),
                                dict(rotary_dim=4, frequencies=[1.0, float("nan")])])
def test_rope_config_refusals(lib, kw):
    kw = dict(kw)
    if "scaling" in kw:
        kw["scaling"] = binding.RopeScaling(*kw["scaling"])
    with pytest.raises(binding.BiError) as e:
        binding.bi_rope_config(kw.pop("rotary_dim", 64), **kw)
    assert e.value.status == INVALID
    with pytest.raises(ValueError):
        binding.bi_rope_config(64, frequencies=[1.0])


@pytest.mark.parametrize("rotary", [2, 64, 128, 256])
@pytest.mark.parametrize("scaling", [None, ("linear", 4.0), ("base", 8.0), ("ramp_turns", 8.0, 8192.0, 1.0, 4.0),
                                     ("ramp_index", 16.0, 4096.0, 1.0, 32.0)])
def test_rope_config_phases(lib, rotary, scaling):
    if scaling and scaling[0] == "base" and rotary == 2:
        pytest.skip("the base's exponent R / (R - 2) needs R > 2")
    cfg = binding.bi_rope_config(rotary, base=500000.0, scaling=binding.RopeScaling(*scaling) if scaling else None,
                                 interleaved=True, magnitude=1.25)
    kind, factor, orig, low, high = (list(scaling) + [0.0] * 3)[:5] if scaling else (None, 1.0, 0, 0, 0)
    f = ref.frequencies(rotary, 500000.0, kind, factor, orig, low, high)
    assert cfg.rotary_dim == rotary and cfg.interleaved and cfg.desc.magnitude == 1.25
    for i, x in enumerate(f):
        # a few roundings of 2^-53 in the frequency (power, ramp, division), and the phase
        # is a whole number of 2^-64 turns: half of one, 2^-65, whatever the frequency
        assert abs(cfg.desc.phase[i] / 2.0 ** 64 - x / (2 * math.pi)) <= 2.0 ** -48 * x + 2.0 ** -65, i
    again = binding.bi_rope_config(rotary, frequencies=[-x for x in f])
    for i in range(rotary // 2):  # a negative frequency is its complement of a turn
        assert abs((cfg.desc.phase[i] + again.desc.phase[i]) / 2.0 ** 64 - 1.0) < 1e-13


def _store(lib, cfg, **change):
    a = Arena()
    o = dict(pos=a.t([5], I64) if cfg else None, slots=a.t([5], I64), q=a.t([5, 8, 128], BF16) if cfg else None,
             q_out=a.t([5, 8, 128], BF16) if cfg else None, k=a.t([5, 2, 128], BF16), v=a.t([5, 2, 128], BF16),
             kc=a.t([9, 16, 2, 128], BF16), vc=a.t([9, 16, 2, 128], BF16))
    o.update({k: (v(a, o) if callable(v) else v) for k, v in change.items()})
    return lib.bi_paged_store(ctypes.byref(cfg.desc) if cfg else None, *(_r(o[n]) for n in (
        "pos", "slots", "q", "q_out", "k", "v", "kc", "vc")), None)


def test_store_refusals(lib):
    cfg = binding.bi_rope_config(128)
    if not torch.cuda.is_available():
        assert _store(lib, cfg) == REACHED
        assert _store(lib, None) == REACHED
        assert _store(lib, cfg, q=None, q_out=None) == REACHED
        assert _store(lib, cfg, q_out=lambda a, o: o["q"]) == REACHED
        # q, k, v as views of one [5, 12, 128] projection, q rotated in place
        base = 0x7E0000000000
        qkv = dict(q=lambda a, o: a.t([5, 8, 128], BF16, [1536, 128, 1], base),
                   k=lambda a, o: a.t([5, 2, 128], BF16, [1536, 128, 1], base + 2 * 1024),
                   v=lambda a, o: a.t([5, 2, 128], BF16, [1536, 128, 1], base + 2 * 1280))
        assert _store(lib, cfg, q_out=lambda a, o: a.t([5, 8, 128], BF16, [1536, 128, 1], base), **qkv) == REACHED
        # the same with q_out one head further: on top of k
        assert _store(lib, cfg, q_out=lambda a, o: a.t([5, 8, 128], BF16, [1536, 128, 1], base + 256), **qkv) == INVALID
    assert _store(lib, cfg, q_out=None) == INVALID
    assert _store(lib, cfg, pos=None) == INVALID
    assert _store(lib, None, pos=lambda a, o: a.t([5], I32)) == INVALID
    assert _store(lib, cfg, slots=lambda a, o: a.t([5], I32)) == DTYPE
    assert _store(lib, cfg, slots=lambda a, o: a.t([6], I64)) == SHAPE
    assert _store(lib, cfg, v=lambda a, o: a.t([5, 2, 128], F16)) == DTYPE
    assert _store(lib, cfg, vc=lambda a, o: a.t([9, 16, 2, 128], F16)) == DTYPE
    assert _store(lib, cfg, vc=lambda a, o: a.t([9, 8, 2, 128], BF16)) == SHAPE
    assert _store(lib, cfg, kc=lambda a, o: a.t([9, 16, 4, 128], BF16)) == SHAPE
    assert _store(lib, cfg, q=lambda a, o: a.t([4, 8, 128], BF16)) == SHAPE
    assert _store(lib, cfg, vc=lambda a, o: o["kc"]) == INVALID  # one cache for both
    assert _store(lib, cfg, kc=lambda a, o: a.t([9, 16, 2, 128], BF16, [0, 256, 128, 1])) == LAYOUT
    big = dict(kc=lambda a, o: a.t([1 << 20, 1 << 12, 2, 128], BF16, [1, 1, 1, 1]),
               vc=lambda a, o: a.t([1 << 20, 1 << 12, 2, 128], BF16, [1, 1, 1, 1]))
    assert _store(lib, cfg, **big) == INVALID
    narrow = binding.bi_rope_config(256)
    assert _store(lib, narrow) == INVALID


def _attend(lib, ws=0x7D0000000000, nbytes=1 << 40, scale=0.1, **change):
    a = Arena()
    o = dict(q=a.t([3, 8, 128], BF16), kc=a.t([9, 16, 2, 128], BF16), vc=a.t([9, 16, 2, 128], BF16),
             table=a.t([3, 40], I32), lens=a.t([3], I32), o=a.t([3, 8, 128], F32))
    o.update({k: (v(a, o) if callable(v) else v) for k, v in change.items()})
    return lib.bi_paged_attention(*(_r(o[n]) for n in ("q", "kc", "vc", "table", "lens")), ctypes.c_float(scale),
                                  _r(o["o"]), ws, nbytes, None)


def test_attention_refusals(lib):
    if not torch.cuda.is_available():
        assert _attend(lib) == REACHED
        assert _attend(lib, ws=None, nbytes=0, table=lambda a, o: a.t([3, 16], I32)) == REACHED  # 256 keys: one piece
    assert _attend(lib, scale=float("nan")) == INVALID
    assert _attend(lib, q=lambda a, o: a.t([3, 7, 128], BF16), o=lambda a, o: a.t([3, 7, 128], F32)) == SHAPE
    assert _attend(lib, q=lambda a, o: a.t([3, 8, 128], F16)) == DTYPE
    assert _attend(lib, q=lambda a, o: a.t([3, 8, 128], F32)) == DTYPE
    assert _attend(lib, table=lambda a, o: a.t([2, 40], I32)) == SHAPE
    assert _attend(lib, table=lambda a, o: a.t([3, 40], I64)) == DTYPE
    assert _attend(lib, lens=lambda a, o: a.t([3], I64)) == DTYPE
    assert _attend(lib, o=lambda a, o: a.t([3, 8, 64], F32)) == SHAPE
    assert _attend(lib, o=lambda a, o: a.t([3, 8, 128], BF16, ptr=o["q"].ptr)) == INVALID  # not in place
    assert _attend(lib, kc=lambda a, o: a.t([9, 16, 2, 128], BF16, [4200, 260, 130, 1])) == LAYOUT
    assert _attend(lib, kc=lambda a, o: a.t([9, 16, 2, 128], BF16, ptr=0x7C0000000008)) == LAYOUT
    for d in (32, 96, 512):
        assert _attend(lib, q=lambda a, o: a.t([3, 8, d], BF16), o=lambda a, o: a.t([3, 8, d], F32),
                       kc=lambda a, o: a.t([9, 16, 2, d], BF16), vc=lambda a, o: a.t([9, 16, 2, d], BF16)) == INVALID
    assert _attend(lib, table=lambda a, o: a.t([3, (1 << 26) + 1], I32)) == INVALID
    # workspace: absent, too small, misaligned, on top of the query
    need = lib.bi_paged_attention_workspace_bytes(3, 8, 128, 640)
    assert need == 3 * 8 * 3 * 130 * 4
    assert _attend(lib, ws=None, nbytes=0) == INVALID
    assert _attend(lib, nbytes=need - 1) == INVALID
    assert _attend(lib, nbytes=-1) == INVALID
    assert _attend(lib, ws=0x7D0000000008) == LAYOUT
    assert _attend(lib, ws=0x7F0000000000) == INVALID
    # nothing to do
    assert _attend(lib, q=lambda a, o: a.t([0, 8, 128], BF16), o=lambda a, o: a.t([0, 8, 128], F32),
                   table=lambda a, o: a.t([0, 40], I32), lens=lambda a, o: a.t([0], I32)) == binding.BI_OK


def test_attention_workspace_rule(lib):
    def n(max_len, B=2, Hq=4, D=64):
        return lib.bi_paged_attention_workspace_bytes(B, Hq, D, max_len)
    row = 2 * 4 * 66 * 4
    assert n(0) == n(1) == n(256) == 0
    assert n(257) == 2 * row and n(513) == 3 * row
    assert n(2048) == n(2049) == n(4096) == 8 * row and n(4097) == 9 * row  # longer requests have longer pieces
    assert n(128 * 512) == n(128 * 512 + 1) == n(1 << 30) == 128 * row  # never more than 128 pieces
    assert n(1000, D=96) == 0 and n(1000, B=0) == 0


def _lp(lib, **change):
    a = Arena()
    o = dict(x=a.t([3, 100], BF16), tok=a.t([3], I64), lp=a.t([3], F32), ent=a.t([3], F32), tlp=a.t([3, 5], F32),
             ids=a.t([3, 5], I32))
    o.update({k: (v(a, o) if callable(v) else v) for k, v in change.items()})
    return lib.bi_token_logprobs(*(_r(o[n]) for n in ("x", "tok", "lp", "ent", "tlp", "ids")), None)


def test_logprobs_refusals(lib):
    if not torch.cuda.is_available():
        assert _lp(lib) == REACHED
        assert _lp(lib, ent=None, tlp=None, ids=None) == REACHED
    assert _lp(lib, ids=None) == INVALID
    assert _lp(lib, tok=lambda a, o: a.t([4], I64)) == SHAPE
    assert _lp(lib, tok=lambda a, o: a.t([3], F32)) == DTYPE
    assert _lp(lib, lp=lambda a, o: a.t([3], BF16)) == DTYPE
    assert _lp(lib, ids=lambda a, o: a.t([3, 5], I64)) == DTYPE
    assert _lp(lib, tlp=lambda a, o: a.t([3, 6], F32)) == SHAPE
    assert _lp(lib, tlp=lambda a, o: a.t([3, 65], F32), ids=lambda a, o: a.t([3, 65], I32)) == INVALID
    assert _lp(lib, x=lambda a, o: a.t([3, 4], BF16)) == INVALID  # fewer logits than alternatives
    assert _lp(lib, x=lambda a, o: a.t([3, 0], BF16), tlp=None, ids=None) == INVALID
    assert _lp(lib, ids=lambda a, o: a.t([3, 5], I32, [8, 1])) == LAYOUT
    assert _lp(lib, x=lambda a, o: a.t([3, 100], BF16, [1, 3])) == LAYOUT
    assert _lp(lib, ent=lambda a, o: o["lp"]) == INVALID
    assert _lp(lib, x=lambda a, o: a.t([0, 100], BF16), tok=lambda a, o: a.t([0], I64), lp=lambda a, o: a.t([0], F32),
               ent=None, tlp=None, ids=None) == binding.BI_OK


def test_binding_refuses_what_it_cannot_describe(lib):
    x = torch.zeros(2, 4, 64)
    cfg = binding.bi_rope_config(64)
    with pytest.raises(ValueError, match="CUDA"):
        binding.bi_rope(x, torch.zeros(2, dtype=torch.int32), cfg)
    with pytest.raises(ValueError, match="CUDA"):
        binding.bi_token_logprobs(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        binding.bi_paged_attention(None, None, None, None, None, 1.0)


def test_descriptors_of_absurd_extent_are_refused(lib):
    big = (1 << 31) - 1
    assert _attend(lib, q=lambda a, o: a.t([3, 8, 128], BF16, [1 << 44, 1 << 44, 1]),
                   kc=lambda a, o: a.t([big, big, 2, 128], BF16, [1 << 43, 1 << 43, 128, 1])) == LAYOUT
    assert lib.bi_paged_attention_workspace_bytes(big, big, 256, 1 << 30) == (1 << 63) - 1
    cfg = binding.bi_rope_config(128)
    assert _store(lib, cfg, slots=lambda a, o: a.t([big], I64), pos=lambda a, o: a.t([big], I64), q=None, q_out=None,
                  k=lambda a, o: a.t([big, big, 128], BF16, [0, 0, 1]),
                  v=lambda a, o: a.t([big, big, 128], BF16, [0, 0, 1]),
                  kc=lambda a, o: a.t([1, 1, big, 128], BF16), vc=lambda a, o: a.t([1, 1, big, 128], BF16)) == INVALID
    assert _attend(lib, q=lambda a, o: a.t([big, 8, 128], BF16), table=lambda a, o: a.t([big, 40], I32),
                   lens=lambda a, o: a.t([big], I32), o=lambda a, o: a.t([big, 8, 128], F32)) == INVALID


def test_numbers_that_steps_would_carry_past_32_bits_are_refused(lib):
    big = (1 << 31) - 1
    cfg = binding.bi_rope_config(16)
    assert _rope(lib, cfg, x=lambda a, o: a.t([1, big, 16], BF16), pos=lambda a, o: a.t([1], I32),
                 y=lambda a, o: a.t([1, big, 16], BF16)) == INVALID
    assert _store(lib, cfg, slots=lambda a, o: a.t([1], I64), pos=lambda a, o: a.t([1], I64),
                  q=lambda a, o: a.t([1, big - 4, 16], BF16), q_out=lambda a, o: a.t([1, big - 4, 16], BF16),
                  k=lambda a, o: a.t([1, 2, 16], BF16), v=lambda a, o: a.t([1, 2, 16], BF16),
                  kc=lambda a, o: a.t([4, 16, 2, 16], BF16), vc=lambda a, o: a.t([4, 16, 2, 16], BF16)) == INVALID
    n = big - 1
    assert _plan(lib, ctx=lambda a, o: a.t([n], I32), new=lambda a, o: a.t([n], I32),
                 table=lambda a, o: a.t([n, 8], I32), lens=lambda a, o: a.t([n], I32),
                 offs=lambda a, o: a.t([n + 1], I32)) == INVALID


def test_scales_whose_base_2_form_overflows_are_refused(lib):
    assert _attend(lib, scale=3e38) == INVALID and _attend(lib, scale=-3e38) == INVALID


def test_integer_types_stay_refused_elsewhere(lib):
    a = Arena()
    assert lib.bi_mm(_r(a.t([4, 64], I32)), _r(a.t([64, 32], I32)), _r(a.t([4, 32], F32)), None) == DTYPE
    assert lib.bi_mean_lastdim(_r(a.t([4, 64], I64)), _r(a.t([4], F32)), None) == DTYPE


def test_reference_rope_of_far_positions():
    # the reference's two ways of taking off whole turns agree where both hold
    f = ref.frequencies(64)
    x = np.random.default_rng(0).standard_normal((3, 1, 64))
    pos = [2 ** 22 - 1, 2 ** 22, 2 ** 22 + 1]
    y, _ = ref.rope(x, pos, f, False)
    c = np.cos(np.array(pos)[:, None] * f) * x[:, 0, :32] - np.sin(np.array(pos)[:, None] * f) * x[:, 0, 32:]
    assert np.abs(y[:, 0, :32] - c).max() < 1e-8
