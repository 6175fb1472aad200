"""Numbers of the serving operations that the host computes, against big integers; and
that the bounds of tests/serving_tight.py reject what they are meant to."""
from __future__ import annotations

import math
import types

import numpy as np
import pytest
import torch

from invariant_gemm_bi_gb300 import binding, build
from tests import serving_tight as tight


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


def test_pi():
    assert tight.PI >> (tight.PI_BITS - 60) == 3622009729038561421  # 3.14159265358979323846... 2^60
    assert abs(tight.PI / 2 ** tight.PI_BITS - math.pi) <= 2.0 ** -52


def _phases(f):
    cfg = binding.bi_rope_config(2 * len(f), frequencies=f)
    return [int(p) for p in cfg.desc.phase[:len(f)]]


@pytest.mark.parametrize("base", [10000.0, 500000.0, 1e6])
@pytest.mark.parametrize("rotary", [64, 128, 256])
def test_phases_are_the_nearest_of_64_bits(base, rotary):
    f = [base ** (-2.0 * i / rotary) for i in range(rotary // 2)]
    for x, p in zip(f, _phases(f)):
        # 2^64 of a turn, off by half of one and 2^-10 for the division's own truncation
        exact = tight.turns(x, 1, 80)
        assert abs((p << 16) - exact) <= (1 << 15) + (1 << 6), x


def test_phases_of_any_frequency():
    rng = np.random.default_rng(7)
    f = [1.0, 0.75, 2 * math.pi, math.pi, 3.0, 1e-3, 1e-12, 2.0 ** -62, 2.0 ** -63, 2.0 ** -64, 1e-300, 5e-324, 0.0,
         1e9, 2.0 ** 40 + 1.0, 2.0 ** 52 + 1.0, 2.0 ** 53 - 1.0]
    f += [float(x) for x in np.exp(rng.uniform(math.log(2.0 ** -66), math.log(2.0 ** 53), 100))]
    got, mirrored = _phases(f), _phases([-x for x in f])
    for x, p, q in zip(f, got, mirrored):
        d = ((p << 16) - tight.turns(x, 1, 80)) % (1 << 80)
        assert min(d, (1 << 80) - d) <= (1 << 15) + (1 << 6), x
        assert (p + q) % (1 << 64) == 0, x  # a negative frequency is its complement of a turn
    assert got[12] == 0


@pytest.mark.parametrize("f", [2.0 ** 53, -2.0 ** 53, 1e300, float("inf"), float("nan")])
def test_frequencies_without_a_fraction_of_a_turn_are_refused(f):
    with pytest.raises(binding.BiError) as e:
        binding.bi_rope_config(4, frequencies=[1.0, f])
    assert e.value.status == binding.BI_ERR_INVALID_ARG


@pytest.mark.parametrize("more", [1 << 32, -(1 << 32), 1 << 40])
def test_numbers_past_32_bits_are_refused_and_not_cut(more):
    with pytest.raises(ValueError, match="rotary_dim"):
        binding.bi_rope_config(more + 64)

    class OnDevice(torch.Tensor):  # passes for a tensor on the current device
        def get_device(self):
            return 0

    t = torch.zeros(2, 4, dtype=torch.int32).as_subclass(OnDevice)
    with pytest.MonkeyPatch.context() as m:
        m.setattr(torch.cuda, "current_device", lambda: 0)
        m.setattr(binding, "_stream_ptr", lambda stream, device: 0)
        m.setattr(binding, "_lib", types.SimpleNamespace(bi_paged_plan=None))  # no entry point is reached
        i32 = [torch.zeros(n, dtype=torch.int32).as_subclass(OnDevice) for n in (2, 2, 9, 2, 3, 4, 2)]
        out = binding.PagedPlan(i32[3], i32[4], i32[5], torch.zeros(4, dtype=torch.int64).as_subclass(OnDevice), i32[6])
        with pytest.raises(ValueError, match="page_size"):
            binding.bi_paged_plan(i32[0], i32[1], t, i32[2], more + 16, out=out)


@pytest.mark.parametrize("D,group", [(64, 1), (128, 12), (256, 1)])
@pytest.mark.parametrize("n", [2049, 65537, 131071])
@pytest.mark.parametrize("dtype,every", [(torch.bfloat16, 256), (torch.float16, 256), (torch.bfloat16, 16)])
def test_the_attention_bound_rejects_work_left_out_or_done_twice(D, group, n, dtype, every):
    rng = np.random.default_rng(n + D)
    q, k = rng.standard_normal((1, D)), rng.standard_normal((n, 1, D))
    v = tight.marked_values(n, 1, D, every)
    ref, bound = tight.attention(np.repeat(q, group, 0), k, v, D ** -0.5, dtype, torch.float32)
    ref, bound = ref[0], bound[0]
    s = D ** -0.5 * (k[:, 0] @ q[0])
    p = np.exp(s - s.max())
    piece = tight.split_len(n)
    for at, size in ((0, piece), (n // piece // 2 * piece, piece), (n - n % piece, piece),  # first, middle and last piece
                     (0, min(16, n // piece // 2) * piece), (piece, 16), (n // 32 * 16, 16)):  # a join's group; a tile
        there = np.ones(n)
        for weight in (0.0, 2.0):
            there[at:at + size] = weight
            w = p * there
            for total in (w.sum(), p.sum()):  # left out of both sums, or of the values' alone
                off = np.abs((w @ v[:, 0]) / total - ref) > bound
                assert off.any(), (at, size, weight)
                if size == piece and every == 256:  # every dimension that the keys are marked in
                    assert off[np.unique(np.arange(at, min(n, at + size)) // every % D)].all(), (at, size, weight)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [50257, 128256, 128257, 300001])
def test_the_log_sum_bound_rejects_a_lost_unit(dtype, N):
    # 16 elements of an ordinary row, a 16-byte unit of a row without spread
    x = np.random.default_rng(N).standard_normal((4, N)) * np.array([[0.0], [0.1], [1.0], [3.0]])
    lp = x[:, :1] - np.log(np.exp(x).sum(-1, keepdims=True))
    bound = tight.logprobs_bounds(x, lp, dtype)[0][:, 0]
    for gone in (slice(N - 16, N), slice(0, 16), slice(4096, 4112)):
        rest = np.exp(x)
        rest[:, gone] = 0.0
        off = np.abs(np.log(rest.sum(-1)) - np.log(np.exp(x).sum(-1)))
        assert (off > bound)[:3].all() and (off > 0.3 * bound).all(), (off, bound)
