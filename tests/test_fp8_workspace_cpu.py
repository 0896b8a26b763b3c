"""Workspace sizes of the FP8 product: a size belongs to its very shape, and one constant covers every shape."""
import random

from compressed_sparse_attention_05_gb300 import abi, build


def size(M, N, K):
    return abi.csa2_matmul_fp8_workspace_size(M, N, K)


def test_the_constant_covers_every_shape():
    build.build()
    r = random.Random(0)
    log = lambda hi: int(round(2 ** r.uniform(0, hi)))  # noqa: E731
    largest = 0
    for _ in range(20000):
        largest = max(largest, size(log(14), log(17), 16 * log(11)))
    for M in range(1, 300):
        for N in (128, 1024, 4096, 7168, 19456):
            largest = max(largest, size(M, N, 7168))
    assert largest <= abi.MATMUL_FP8_WORKSPACE_MAX
    assert largest > abi.MATMUL_FP8_WORKSPACE_MAX // 2            # (not out of all proportion)
    # the shapes that show why a prefill's size does not serve a decode step
    assert size(4096, 4096, 7168) < size(32, 4096, 7168) < size(128, 4096, 7168) <= abi.MATMUL_FP8_WORKSPACE_MAX
    assert size(1 << 30, 1 << 30, 1 << 30) <= abi.MATMUL_FP8_WORKSPACE_MAX
