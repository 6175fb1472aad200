"""Scales of the block-scaled product that change from block to block by far more than the
operands do: a scale of another block, row or turn in any one place is off by powers of two."""
from __future__ import annotations

import pytest
import torch

from invariant_gemm_bi_gb300 import binding as bi
from tests.gpu_helpers import bits_equal
from tests.test_gpu_quantized import BF16, F32, _clean_status, _gen, _operands  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(300, 200, 9000), (256, 14336, 4096), (1000, 5000, 2500), (4096, 4096, 1111),
                                   (130, 64, 20000), (20, 4096, 14336), (32, 200, 700)])
def test_opposite_scales_cancel(M, N, K):
    # 2^e of a's block and 2^-e of b's: each product is times 1, as with scales of 1, bit for
    # bit, whatever e is; e is drawn for each block, and for every column block in common
    a, _, b, _ = _operands(M, N, K, 7)
    kb, nb = -(-K // 128), -(-N // 128)
    one = bi.bi_mm_blockscaled(a, torch.ones((M, kb), device="cuda"), b, torch.ones((kb, nb), device="cuda"), out_dtype=F32)
    assert torch.isfinite(one).all()
    for seed in range(6):
        e = torch.randint(-60, 61, (kb,), generator=_gen(seed), device="cuda").float()
        sa, sb = torch.exp2(e).expand(M, kb).contiguous(), torch.exp2(-e)[:, None].expand(kb, nb).contiguous()
        for _ in range(8):
            assert bits_equal(bi.bi_mm_blockscaled(a, sa, b, sb, out_dtype=F32), one)
    # rows with exponents of their own: each row's result is times its power of two
    r = torch.randint(-20, 21, (M,), generator=_gen(99), device="cuda").float()
    sa = torch.exp2(e[None, :] + r[:, None])
    assert bits_equal(bi.bi_mm_blockscaled(a, sa, b, sb, out_dtype=F32), one * torch.exp2(r)[:, None])


def test_opposite_scales_cancel_on_two_streams():
    ops = []
    for M, N, K in ((512, 3000, 3000), (40, 6000, 5000)):
        a, _, b, _ = _operands(M, N, K, M)
        kb, nb = -(-K // 128), -(-N // 128)
        want = bi.bi_mm_blockscaled(a, torch.ones((M, kb), device="cuda"), b, torch.ones((kb, nb), device="cuda"), out_dtype=BF16)
        e = torch.randint(-60, 61, (kb,), generator=_gen(M), device="cuda").float()
        ops.append((a, torch.exp2(e).expand(M, kb).contiguous(), b, torch.exp2(-e)[:, None].expand(kb, nb).contiguous(), want))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in ops], []
    for _ in range(30):
        for (a, sa, b, sb, want), st in zip(ops, streams):
            got.append((bi.bi_mm_blockscaled(a, sa, b, sb, stream=st), want))
    torch.cuda.synchronize()
    for c, want in got:
        assert bits_equal(c, want)
