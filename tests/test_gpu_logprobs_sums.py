"""Token log probabilities where an element lost or counted twice would be a small
error of a long sum: rows with all their weight on few elements, and ordinary rows
under bounds that count the kernel's roundings."""
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


def _wide(x, at, pad):
    """x as rows of a wider buffer, `at` elements into it, infinities around them."""
    R, N = x.shape
    wide = torch.full((R, N + pad), float("inf"), dtype=x.dtype, device=x.device)
    wide[:, at:at + N] = x
    return wide[:, at:at + N]


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("N", [17, 1001, 4096, 8191, 8193, 40003, 70000, 128257, 300001])
def test_every_element_counts_once(dt, N):
    sets = tight.marked_rows(N, dt)
    x = torch.full((len(sets), N), -40.0, dtype=dt, device="cuda")
    for r, s in enumerate(sets):
        x[r, s] = 0.0
    m = np.array([len(s) for s in sets], np.float64)
    total = m + (N - m) * np.exp(-40.0)
    lp = -np.log(total)
    entropy = np.log(total) + (N - m) * 40.0 * np.exp(-40.0) / total
    # the rest weighs N 40 e^-40 < 6e-11; the sum of equal terms, its logarithm, the differences
    err = tight.logprobs_sum_error(N, dt) + 2.0 ** -21 * np.log(total) + 2.0 ** -30
    assert np.all(err < 0.5 * np.log1p(1 / m))  # an element more or less would show
    for many in (1, 6):  # a cluster a row, a CTA a row
        for last in (False, True):
            tokens = torch.tensor([s[-1 if last else 0] for s in sets] * many, device="cuda")
            for y in [x.repeat(many, 1)] + [_wide(x.repeat(many, 1), at, pad) for at, pad in
                                            ((1, 9), (2, 16), (3, 8 + -N % 8), (7, 8 + -N % 8), (4, 8 + -N % 4))]:
                r = bi.bi_token_logprobs(y, tokens, top=1)
                ref.assert_within(r.logprobs, np.tile(lp, many), np.tile(err, many), "logprobs")
                ref.assert_within(r.entropy, np.tile(entropy, many), np.tile(2 * err + 2.0 ** -21, many), "entropy")
                assert r.top_ids[:, 0].tolist() == [s[0] for s in sets] * many
                ref.assert_within(r.top_logprobs[:, 0], np.tile(lp, many), np.tile(err, many), "alternative")


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("N", [33, 1000, 4099, 8192, 20003, 50257, 128256, 128257, 300001])
@pytest.mark.parametrize("std,shift", [(1.0, 0.0), (3.0, 0.0), (0.05, 11.0)])
def test_ordinary_rows_within_their_own_roundings(dt, N, std, shift):
    g = torch.Generator(device="cuda")
    g.manual_seed(N)
    x = (torch.randn((6, N), generator=g, device="cuda") * std + shift).to(dt)
    tokens = torch.randint(0, N, (6,), generator=g, device="cuda")
    tokens[0] = N - 1
    lp, entropy, top_lp, ids, *_ = ref.logprobs(x, tokens.tolist(), 5)
    x64 = ref.f64(x)
    first = bi.bi_token_logprobs(x, tokens, top=5)
    for y in (x, _wide(x, 3, 8 + -N % 8), _wide(x, 1, 10)):
        r = bi.bi_token_logprobs(y, tokens, top=5)
        assert all(bits_equal(a, b) for a, b in zip(r, first))
    lp_bound, entropy_bound = tight.logprobs_bounds(x64, lp, dt)
    ref.assert_within(first.logprobs, lp, lp_bound, "logprobs")
    ref.assert_within(first.entropy, entropy, entropy_bound, "entropy")
    ref.assert_within(first.top_logprobs, top_lp, tight.logprobs_bounds(x64, top_lp, dt)[0], "alternatives")
    assert np.array_equal(first.top_ids.cpu().numpy(), ids)
