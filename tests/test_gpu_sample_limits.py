"""Rows with top-k and top-p both set: two searches for a limit in a row, one after the
other.  Every cluster size and both block sizes, many rows, again and again; every token
against a 64-bit evaluation, every repetition against the first."""
from __future__ import annotations

import pytest
import torch

from invariant_gemm_bi_gb300 import binding as bi
from tests.test_gpu_sample import BF16, F16, F32, _clean_status, _f32, _gen, _i32, _normal  # noqa: F401
from tests.test_gpu_sample_borders import kept, token

pytestmark = pytest.mark.gpu


def _again_and_again(x, u, t, k, p, times, most_near):
    w, near = kept(x, t, k, p)
    want, close = token(w, u)
    near = near | close
    assert int(near.sum()) <= most_near
    first = bi.bi_sample_tokens(x, u, temperature=t, top_k=k, top_p=p)
    wrong = (first != want) & ~near
    assert not wrong.any(), (wrong.nonzero()[:5, 0].tolist(), first[wrong][:5].tolist(), want[wrong][:5].tolist())
    for _ in range(times):
        assert torch.equal(bi.bi_sample_tokens(x, u, temperature=t, top_k=k, top_p=p), first)


def _rows(R, seed, ks, ps, ts=(1.0, 0.7, 1.3)):
    pick = lambda v: [v[(i * 7 + i // len(v)) % len(v)] for i in range(R)]  # noqa: E731
    return (torch.rand((R,), generator=_gen(seed), device="cuda"), _f32(pick(ts)), _i32(pick(ks)), _f32(pick(ps)))


# (a batch whose CTAs fill the GPU twice has slices of up to 32768 elements in 16 bits and
# 512 threads; one that an SM has a CTA of slices of 16384 and 1024 threads)
@pytest.mark.parametrize("R,N", [(2000, 20000), (1000, 40000), (500, 80000), (300, 200000),
                                 (120, 9000), (60, 30000), (30, 60000), (16, 128256), (100, 30000), (30, 128256)])
@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_both_limits_of_many_rows(R, N, dt):
    if dt != BF16 and R > 500:
        R = 300
    x = _normal((R, N), dt, R + N, 2.0)
    # limits among the most likely tokens and far down the row, close together and apart
    args = _rows(R, N, (2, 40, 50, 600, 1000, 5000, N // 2), (0.9, 0.5, 0.99, 0.2, 0.999))
    _again_and_again(x, *args, times=30, most_near=3)


@pytest.mark.parametrize("N", [12000, 30000, 50000, 128256])
@pytest.mark.parametrize("R", [12, 170])
@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_both_limits_among_thousands_of_equals(R, N, dt):
    # few values, thousands of elements each; in fp32 neighbours of a value too, so that the
    # bits of a bin's elements are searched down to the last one
    x = torch.round(_normal((R, N), F32, N, 1.5))
    if dt == F32:
        x = x * (1 + 2.0 ** -23 * torch.randint(0, 3, (R, N), generator=_gen(R), device="cuda"))
    args = _rows(R, N + 1, (600, 2000, N // 3, N // 2, N - 7), (0.9, 0.5, 0.97, 0.3))
    # (temperatures of 2 and 4 take the weights of bf16 rows out of their table)
    for ts in ((1.0, 0.7), (2.0, 4.0)):
        u, _, k, p = args
        t = _f32([ts[i % 2] for i in range(R)])
        _again_and_again(x.to(dt), u, t, k, p, times=20, most_near=3)
