"""One workspace of the largest size serves products of every shape, in any order."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_05_gb300 import abi, build
from oracle import step as O

pytestmark = pytest.mark.gpu


def test_one_workspace_for_prefill_and_decode():
    build.build()
    N, K = 1024, 4096
    g = torch.Generator().manual_seed(0)
    code = lambda n: (torch.randn(n, K, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    b, sb = code(N), torch.rand(N // 128, K // 128, generator=g)
    bd, sbd = b.cuda(), sb.cuda()
    guard = 64
    ws = torch.full((abi.MATMUL_FP8_WORKSPACE_MAX + guard,), 0x5A, dtype=torch.uint8, device="cuda")
    for M in (1024, 32, 1, 128, 33, 300, 8):
        a, sa = code(M), torch.rand(M, K // 128, generator=g)
        C = torch.empty(M, N, device="cuda")
        abi.csa2_matmul_fp8(a.cuda(), sa.cuda(), bd, sbd, C, ws[:-guard])
        torch.cuda.synchronize()
        ref, mag = O.matmul_fp8(a.numpy(), sa.numpy(), b.numpy(), sb.numpy())
        # fp32 sums of 128 products, then of the blocks, each step off by at most 2^-23 of the magnitudes
        tol = (128 + K // 128 + 2) * 2.0 ** -23 * mag + np.abs(ref) * 2.0 ** -24
        assert np.all(np.abs(C.double().cpu().numpy() - ref) <= tol), M
        assert bool((ws[-guard:] == 0x5A).all())
    assert abi.csa2_get_status() == 0
