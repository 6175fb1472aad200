"""Tokens drawn right at their borders: given numbers within a step of fp32 of a place where
one token's share ends and the next one's begins, so that one element more or less among
those that are kept, or a weight that is off, shows in the token."""
from __future__ import annotations

import pytest
import torch

from invariant_gemm_bi_gb300 import binding as bi
from tests.quantized_reference import MARGIN
from tests.test_gpu_sample import BF16, F16, F32, _clean_status, _f32, _gen, _normal  # noqa: F401

pytestmark = pytest.mark.gpu


def kept(x, t, k=None, p=None):
    """(weights in index order, zero where not kept; whether a limit's border is nearer than
    MARGIN) in 64 bits.  Where all that top-k keeps is alike, sums are whole numbers on both
    sides and a limit on a border is on it exactly."""
    z = x.double()
    s, order = torch.sort(z, dim=1, descending=True, stable=True)
    e = torch.exp((s - s[:, :1]) / t.double()[:, None])
    near = torch.zeros(x.shape[0], dtype=torch.bool, device=x.device)
    if k is not None:
        rank = torch.arange(x.shape[1], device=x.device)[None, :]
        e = torch.where(rank < k.long()[:, None], e, torch.zeros_like(e))
    if p is not None:
        mass = torch.cumsum(e, 1)
        limit = (p.double() * mass[:, -1])[:, None]
        exact = ((e == 0) | (e == 1)).all(1)
        near = ((mass - limit).abs() < MARGIN * mass[:, -1:]).any(1) & ~exact
        e = torch.where(mass - e < limit, e, torch.zeros_like(e))
    return torch.zeros_like(z).scatter_(1, order, e), near


def token(w, u):
    """(token, whether a border is nearer than MARGIN) of weights in index order."""
    mass = torch.cumsum(w, 1)
    limit = (u.double() * mass[:, -1])[:, None]
    exact = ((w == 0) | (w == 1)).all(1)
    return (mass <= limit).sum(1), ((mass - limit).abs() < MARGIN * mass[:, -1:]).any(1) & ~exact


def at_borders(w, seed):
    """A number for each row, at the end of some kept token's share: the nearest fp32 or one beside it."""
    R = w.shape[0]
    mass = torch.cumsum(w, 1)
    pick = (torch.rand((R,), generator=_gen(seed), device="cuda") * (w > 0).sum(1)).long() + 1
    i = ((w > 0).cumsum(1) < pick[:, None]).sum(1)
    u = (mass.gather(1, i[:, None])[:, 0] / mass[:, -1]).float()
    step = torch.randint(-1, 2, (R,), generator=_gen(seed + 1), device="cuda")
    return (u + step * 2.0 ** -24).clamp(0.0, 1 - 2.0 ** -24)


# Rows that MARGIN leaves out: a top-p put at a border is an fp32 number of [1/2, 1), off by up
# to 2^-25 evenly, so within 2^-30 of it one time in 32.  A given number at a border is one a third
# of the time; it is within 2^-30 one time in 32 in [1/2, 1), 16 in [1/4, 1/2) and so on: 1/64 for
# each of five binades, and 1/32 for all below.  1/32 + (5/64 + 1/32) / 3 = 0.068.
NEAR = 0.068


def check(x, t, k=None, p=None, seed=0):
    w, near = kept(x, t, k, p)
    u = at_borders(w, seed)
    want, close = token(w, u)
    skip = near | close
    expected = NEAR * x.shape[0]
    assert int(skip.sum()) <= expected + 4 * expected ** 0.5 + 3
    got = bi.bi_sample_tokens(x, u, temperature=t, top_k=k, top_p=p)
    wrong = (got != want) & ~skip
    assert not wrong.any(), (wrong.nonzero()[:5, 0].tolist(), got[wrong][:5].tolist(), want[wrong][:5].tolist())
    return u, got


# (a batch whose CTAs fill the GPU twice has slices of up to 32768 elements in 16 bits and 512
# threads, one that an SM has a CTA of slices of 16384 and 1024: clusters of 1, 2, 4 and 8)
SHAPES = [(400, 16000), (320, 40000), (310, 80000), (310, 200000), (120, 9000), (60, 30000), (30, 60000), (16, 128256),
          (100, 30000), (60, 60000), (30, 128256)]


@pytest.mark.parametrize("R,N", SHAPES)
@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_top_p_around_zero_and_over_all_magnitudes(R, N, dt):
    # the limit among logits near zero, which in bf16 are weighed one by one, and
    # temperatures at which all of a bf16 row is
    x = _normal((R, N), dt, R + N, 2.0)
    for t0, seed in ((1.0, 1), (0.75, 2), (2.0, 3), (4.0, 4)):
        t = torch.full((R,), t0, device="cuda")
        z, _ = torch.sort(x.double(), dim=1, descending=True)
        mass = torch.cumsum(torch.exp((z - z[:, :1]) / t0), 1)
        at = (z > 0).sum(1, keepdim=True) - 1
        check(x, t, p=(mass.gather(1, at) / mass[:, -1:])[:, 0].float(), seed=seed)
        check(x, t, p=_f32([(0.3, 0.5, 0.9, 0.99, 0.999)[i % 5] for i in range(R)]), seed=10 * seed)
        check(x, t, seed=100 * seed)


@pytest.mark.parametrize("R,N", SHAPES)
@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_top_k_at_borders(R, N, dt):
    x = _normal((R, N), dt, R + N + 1, 2.0)
    k = torch.tensor([(2, 40, 600, 5000, N // 2, N - 3)[i % 6] for i in range(R)], dtype=torch.int32, device="cuda")
    for t0 in (1.0, 4.0):
        check(x, torch.full((R,), t0, device="cuda"), k=k, seed=int(t0))


@pytest.mark.parametrize("R,N", [(400, 3000), (320, 40000), (310, 80000), (60, 30000), (16, 128256)])
@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_all_limits_together_at_borders(R, N, dt):
    # min-p keeps what is at least its share of the largest: by the value, below every other limit or above
    x = _normal((R, N), dt, R + N + 2, 2.0)
    k = torch.tensor([(3, 513, N // 3, N // 2, 0, N + 9)[i % 6] for i in range(R)], dtype=torch.int32, device="cuda")
    p = _f32([(0.4, 0.9, 0.999, 1.0)[i % 4] for i in range(R)])
    m = _f32([(0.0, 0.3, 0.01, -1.0, 0.0005)[i % 5] for i in range(R)])
    for t0 in (1.0, 4.0):
        t = torch.full((R,), t0, device="cuda")
        w, near = kept(x, t, torch.where(k <= 0, N, k), torch.where(p >= 1, 2.0, p))
        top = x.double().amax(1, keepdim=True)
        share = torch.exp((x.double() - top) / t0)
        least = m.double()[:, None]
        near |= ((share - least).abs() < MARGIN * least).any(1)
        w = torch.where(share >= least, w, torch.zeros_like(w))
        u = at_borders(w, int(t0))
        want, close = token(w, u)
        skip = near | close
        expected = NEAR * R
        assert int(skip.sum()) <= expected + 4 * expected ** 0.5 + 3
        got = bi.bi_sample_tokens(x, u, temperature=t, top_k=k, top_p=p, min_p=m)
        wrong = (got != want) & ~skip
        assert not wrong.any(), (wrong.nonzero()[:5, 0].tolist(), got[wrong][:5].tolist(), want[wrong][:5].tolist())
