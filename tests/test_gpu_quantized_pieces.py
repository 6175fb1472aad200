"""Attention over a cache in 8 bits around the lengths at which the pieces of a request's
keys get longer: the 64-bit result, and the same bits whatever the table could hold and
whoever else is in the batch."""
from __future__ import annotations

import pytest
import torch

from invariant_gemm_bi_gb300 import binding as bi
from tests import quantized_reference as ref
from tests import serving_reference as sref
from tests.gpu_helpers import bits_equal
from tests.test_gpu_quantized import BF16, F16, F32, _clean_status, _problem  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[2047, 2048, 2049, 2561], [8192, 8193, 12289, 16383], [16384, 16385, 17409, 40000],
                                  [65535, 65536, 65537], [131071, 131072, 131073]])
@pytest.mark.parametrize("Hq,D,dt", [(2, 64, BF16), (1, 256, F16)])
def test_pieces_around_their_borders(lens, Hq, D, dt):
    q, kc, ks, vc, vs, table, n = _problem(lens, Hq, 1, D, 64, dt, seed=len(lens) + lens[0])
    full = bi.bi_paged_attention_quantized(q, kc, ks, vc, vs, table, n, D ** -0.5)
    want, bound = ref.attention(q, kc, ks, vc, vs, table, n, D ** -0.5, F32)
    sref.assert_within(full, want, bound)
    for b, length in enumerate(lens):
        for width in (-(-length // 64), 4096):
            t = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
            w = min(width, table.shape[1])
            t[0, :w] = table[b, :w]
            # a workspace of just the size that is asked for, with nothing past it written
            need = bi.bi_paged_attention_workspace_bytes(1, Hq, D, width * 64)
            store = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
            o = bi.bi_paged_attention_quantized(q[b:b + 1], kc, ks, vc, vs, t, n[b:b + 1], D ** -0.5,
                                                workspace=store[:need] if need else None)
            assert bits_equal(o, full[b:b + 1].contiguous()), (length, width)
            assert (store[need:] == 0x5A).all()
