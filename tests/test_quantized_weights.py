"""How finely attention over a cache in 8 bits carries its weights: queries so small that
scores add next to nothing to the error, where the bound is that of the weights themselves --
of 22 bits, in two fp16.  On the CPU it is shown that one fp16 would not do."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from invariant_gemm_bi_gb300 import binding as bi
from tests import quantized_reference as ref
from tests import serving_reference as sref

F32, BF16, F16, E4M3 = torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn

CASES = [  # lens, Hq, Hkv, D, type, size of q
    ([1, 2, 7], 2, 1, 64, BF16, 0.0), ([40, 16, 33], 4, 2, 128, F16, 0.0), ([300, 31], 12, 1, 64, BF16, 0.0),
    ([200], 16, 1, 128, BF16, 2.0 ** -9), ([90, 257, 15], 3, 1, 256, F16, 2.0 ** -9), ([256, 100], 2, 2, 128, F16, 2.0 ** -9)]


def _problem(lens, Hq, Hkv, D, dt, size, page=16):
    g = torch.Generator().manual_seed(len(lens) * 1000 + D)
    need = [-(-n // page) for n in lens]
    P = sum(need)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    q = (torch.randn((len(lens), Hq, D), generator=g) * size).to(dt)
    kv = torch.randn((2, P, page, Hkv, D), generator=g).to(E4M3)
    # scales with all the bits of an fp32, none a power of two
    s = torch.rand((2, P, page, Hkv), generator=g) + 0.5
    return q, kv[0], s[0], kv[1], s[1], table, torch.tensor(lens, dtype=torch.int32)


def _one_fp16(q, kc, ks, vc, vs, table, lens, scale):
    """Attention in 64 bits whose weights, times their values' scales, are rounded to one fp16."""
    B, Hq, D = q.shape
    page, G = kc.shape[1], Hq // kc.shape[2]
    out = np.zeros((B, Hq, D))
    for b in range(B):
        j = np.arange(int(lens[b]))
        at = torch.as_tensor(table[b].numpy()[j // page].astype(np.int64)), torch.as_tensor(j % page)
        k = ref.from_e4m3(kc.view(torch.uint8)[at].view(E4M3)) * sref.f64(ks[at])[..., None]
        v, sv = ref.from_e4m3(vc.view(torch.uint8)[at].view(E4M3)), sref.f64(vs[at])
        for h in range(Hq):
            t = scale * (k[:, h // G] @ sref.f64(q[b, h]))
            p = np.exp(t - t.max())
            w = (p * sv[:, h // G]).astype(np.float16).astype(np.float64)
            out[b, h] = w @ v[:, h // G] / p.sum()
    return out


@pytest.mark.parametrize("case", CASES)
def test_the_bound_tells_one_fp16_from_two(case):
    x = _problem(*case)
    want, bound = ref.attention(*x, 0.125, F32)
    # (one element past the bound fails the test below)
    assert (np.abs(_one_fp16(*x, 0.125) - want) > bound).sum() >= 10


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_attention_quantized_weights_of_22_bits(case):
    x = [t.cuda() for t in _problem(*case)]
    o = bi.bi_paged_attention_quantized(*x, 0.125)
    want, bound = ref.attention(*x, 0.125, F32)
    sref.assert_within(o, want, bound, str(case))
    assert bi.bi_device_status() == bi.BI_OK
