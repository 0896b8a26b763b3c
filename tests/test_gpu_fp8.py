"""FP8 rows and their product against oracle.step.

Packing is bit-exact (fp32 steps, each rounded as the reading says).  The product: code products are exact in fp32,
a block's 128 and then the blocks' sums are fp32 additions; an addition that truncates is off by at most 2^-23 of
the magnitudes added so far, scaling a block's sum by its two scales by 2 x 2^-24, so that C before its rounding is
within (128 + blocks + 2) 2^-23 of the sum of |a b|."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_05_gb300 import abi, build
from oracle import formats as F
from oracle import step as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    abi.lib()


def status():
    torch.cuda.synchronize()
    return abi.csa2_get_status()


def pack(x, guard=64):
    n, K = x.shape
    kb = -(-K // 128)
    codes = torch.full((n * K + guard,), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((n * kb + guard,), -5.0, device="cuda")
    abi.csa2_pack_fp8_blocks(x, codes[:n * K].view(n, K), scales[:n * kb].view(n, kb))
    assert bool((codes[n * K:] == 0xEE).all()) and bool((scales[n * kb:] == -5.0).all())
    return codes[:n * K].view(n, K), scales[:n * kb].view(n, kb)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,K,extra", [(1, 16, 0), (1, 128, 0), (3, 144, 16), (7, 1040, 0), (33, 4096, 48), (129, 272, 8),
                                       (1000, 2064, 0)])
def test_pack_bit_exact(n, K, extra, dtype):
    g = torch.Generator().manual_seed(n + K)
    x = torch.randn(n, K + extra, generator=g) * torch.exp(3 * torch.randn(n, 1, generator=g))
    x[torch.rand(x.shape, generator=g) < 0.3] = 0
    x[0, :K] = 0                                           # a row of zeros
    if n > 2:
        x[1, 0], x[2, :K] = 1e30, x[2, :K] * 1e-36         # an outlier; a row below the smallest scale
    x = x.to(dtype).cuda()[:, :K]
    codes, scales = pack(x)
    rc, rs = O.pack_fp8_blocks(x.float().cpu().numpy())
    np.testing.assert_array_equal(scales.cpu().numpy(), rs)
    np.testing.assert_array_equal(codes.cpu().numpy(), rc)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [16, 32, 48, 64, 80, 96, 112, 128, 208])
def test_pack_short_rows(K, dtype):
    """Rows of one short block (several share a warp's lanes), with infinities and NaN that stay in their rows."""
    for n in (1, 2, 37, 6001):
        g = torch.Generator().manual_seed(n + K)
        x = torch.randn(n, K + 16, generator=g) * torch.exp(3 * torch.randn(n, 1, generator=g))
        x[:, K:] = 1e20                                    # (not of the rows)
        nan = torch.rand(n, generator=g) < 0.2
        inf = (torch.rand(n, generator=g) < 0.2) & ~nan
        x = x.to(dtype).cuda()[:, :K]
        x[nan.cuda(), K // 3] = float("nan")
        clean = x.nan_to_num(nan=0.0).float().cpu().numpy()
        x[inf.cuda(), K - 1] = -float("inf")
        codes, scales = pack(x)
        rc, rs = O.pack_fp8_blocks(clean)
        codes, scales, nan, inf = codes.cpu().numpy(), scales.cpu().numpy(), nan.numpy(), inf.numpy()
        assert np.all(codes[nan, K // 3] & 0x7F == 0x7F)
        rc[nan, K // 3] = codes[nan, K // 3]
        last = (K - 1) // 128 * 128
        assert np.all(np.isinf(scales[inf, -1]))
        np.testing.assert_array_equal(scales[~inf], rs[~inf])
        np.testing.assert_array_equal(scales[:, :-1], rs[:, :-1])
        np.testing.assert_array_equal(codes[~inf], rc[~inf])
        np.testing.assert_array_equal(codes[:, :last], rc[:, :last])


def test_pack_every_bf16_value():
    """All finite bf16 patterns, each beside a maximum that puts it somewhere in the codes' range."""
    bits = np.arange(1 << 16, dtype=np.uint16)
    v = (bits.astype(np.uint32) << 16).view(np.float32)
    v = v[np.isfinite(v) & (np.abs(v) < 2.0 ** 100) & (np.abs(v) > 2.0 ** -90)]
    v = v[:len(v) // 127 * 127].reshape(-1, 127)
    x = np.concatenate([v, np.abs(v).max(axis=1, keepdims=True) * np.float32(1.25)], axis=1).astype(np.float32)
    t = torch.tensor(x).cuda()
    codes, scales = pack(t)
    rc, rs = O.pack_fp8_blocks(x)
    np.testing.assert_array_equal(scales.cpu().numpy(), rs)
    np.testing.assert_array_equal(codes.cpu().numpy(), rc)


def test_pack_infinities_and_nan():
    x = torch.ones(2, 256)
    x[0, 3], x[1, 200] = float("inf"), float("nan")
    codes, scales = pack(x.cuda())
    v = codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(128, dim=1)
    assert bool(v[0, :128].isnan().all()) and bool((v[0, 128:] == 1).all())
    assert bool(v[1, 200].isnan()) and int(v[1].isnan().sum()) == 1


def codes_of(n, K, g, wild=False):
    """E4M3 codes without NaN, spread over all exponents when wild."""
    c = torch.randint(0, 256, (n, K), dtype=torch.uint8, generator=g) if wild else (
        torch.randn(n, K, generator=g) * 60).to(torch.float8_e4m3fn).view(torch.uint8)
    c[(c & 0x7F) == 0x7F] = 0x35
    return c


def check_product(M, N, K, out=torch.bfloat16, seed=0, wild=False, ws_fill=0xFF):
    g = torch.Generator().manual_seed(seed + M + N + K)
    kb, nb = -(-K // 128), -(-N // 128)
    a, b = codes_of(M, K, g, wild), codes_of(N, K, g, wild)
    sa, sb = torch.rand(M, kb, generator=g) * 0.02 + 1e-4, torch.exp(torch.randn(nb, kb, generator=g)) * 1e-3
    ref, mag = O.matmul_fp8(a.numpy(), sa.numpy(), b.numpy(), sb.numpy())
    C = torch.full((M * N + 64,), 7.0, dtype=out, device="cuda")
    ws = torch.full((max(16, abi.csa2_matmul_fp8_workspace_size(M, N, K)),), ws_fill, dtype=torch.uint8, device="cuda")
    abi.csa2_matmul_fp8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), C[:M * N].view(M, N), ws)
    assert status() == 0
    assert bool((C[M * N:] == 7).all())
    got = C[:M * N].view(M, N).double().cpu().numpy()
    err = np.abs(got - ref)
    tol = (128 + kb + 2) * 2.0 ** -23 * mag
    tol += (np.abs(ref) + tol) * torch.finfo(out).eps / 2
    assert np.all(err <= tol), float((err / tol).max())
    return C[:M * N]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 128, 128), (1, 513, 4096), (3, 130, 144), (16, 1024, 512), (17, 1000, 1552), (32, 4096, 1024),
    (33, 257, 272), (64, 2048, 384), (65, 256, 128), (65, 1, 4096), (128, 300, 1040), (129, 257, 16), (161, 1001, 1552),
    (700, 515, 640), (2000, 4096, 256), (300, 20000, 384),
])
def test_product(M, N, K, out):
    check_product(M, N, K, out)


@pytest.mark.parametrize("M", [5, 50, 200])
def test_product_of_all_codes(M):
    check_product(M, 384, 640, torch.float32, wild=True)


@pytest.mark.parametrize("M,N", [(40, 30000), (4096, 10000)])
def test_product_many_tiles_per_sm(M, N):
    check_product(M, N, 768)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(100, 30001, 272), (128, 20480, 1024), (300, 9001, 528), (257, 12288, 640), (1500, 9547, 400), (2100, 58, 992)])
def test_product_of_wide_tiles(M, N, K, out):
    """One row of tiles, odd numbers of them, one wave and several, rows of C on 16 bytes and not."""
    check_product(M, N, K, out)


def test_scales_belong_to_their_rows_and_blocks():
    """Powers of two in every scale and ones in every code: C counts what each block contributes, exactly."""
    for M in (40, 130):
        N, K = 300, 400
        one = 0x38
        a = torch.full((M, K), one, dtype=torch.uint8).cuda()
        b = torch.full((N, K), one, dtype=torch.uint8).cuda()
        sa = 2.0 ** (torch.arange(M).unsqueeze(1) % 5 + torch.arange(4) * 3).float()
        sb = 2.0 ** (torch.arange(3).unsqueeze(1) * 2 - torch.arange(4)).float()
        C = torch.empty(M, N, device="cuda")
        ws = torch.empty(max(16, abi.csa2_matmul_fp8_workspace_size(M, N, K)), dtype=torch.uint8, device="cuda")
        abi.csa2_matmul_fp8(a, sa.cuda(), b, sb.cuda(), C, ws)
        n = torch.tensor([128.0, 128.0, 128.0, 16.0])
        ref = (sa * n) @ sb.t()
        assert torch.equal(C.cpu(), ref[:, torch.arange(N) // 128])


def test_nan_reaches_its_row_and_column_only():
    for M in (20, 200):
        N, K = 140, 256
        g = torch.Generator().manual_seed(M)
        a, b = codes_of(M, K, g), codes_of(N, K, g)
        a[7, 130] = 0x7F
        b[9, 5] = 0xFF
        C = torch.empty(M, N, device="cuda")
        ws = torch.empty(max(16, abi.csa2_matmul_fp8_workspace_size(M, N, K)), dtype=torch.uint8, device="cuda")
        abi.csa2_matmul_fp8(a.cuda(), torch.ones(M, 2, device="cuda"), b.cuda(), torch.ones(2, 2, device="cuda"), C, ws)
        bad = C.isnan().cpu()
        want = torch.zeros(M, N, dtype=torch.bool)
        want[7], want[:, 9] = True, True
        assert torch.equal(bad, want)


@pytest.mark.parametrize("M,N,K", [(24, 1024, 4096), (161, 1001, 1552), (400, 9000, 512)])
def test_same_bits_every_time(M, N, K):
    first = check_product(M, N, K, torch.float32)
    assert torch.equal(first, check_product(M, N, K, torch.float32, ws_fill=0x11))


def test_captured_streams_and_workspaces():
    """Two products with workspaces of their own in one graph, on two streams, replayed with other inputs."""
    g = torch.Generator().manual_seed(4)
    sets = []
    for M, N, K in ((12, 700, 2048), (130, 600, 1024)):
        x = torch.randn(M, K, generator=g).cuda()
        codes, scales = pack(x)
        b = codes_of(N, K, g).cuda()
        sb = torch.rand(-(-N // 128), K // 128, generator=g).cuda()
        C = torch.empty(M, N, device="cuda")
        ws = torch.empty(abi.csa2_matmul_fp8_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
        sets.append((x, codes, scales, b, sb, C, ws))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        for x, codes, scales, b, sb, C, ws in sets:
            s = torch.cuda.Stream()
            s.wait_stream(main)
            with torch.cuda.stream(s):
                abi.csa2_pack_fp8_blocks(x, codes, scales)
                abi.csa2_matmul_fp8(codes, scales, b, sb, C, ws)
            main.wait_stream(s)
    for _ in range(3):
        for s in sets:
            s[0].copy_(torch.randn(s[0].shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        for x, codes, scales, b, sb, C, ws in sets:
            rc, rs = O.pack_fp8_blocks(x.cpu().numpy())
            np.testing.assert_array_equal(codes.cpu().numpy(), rc)
            ref, mag = O.matmul_fp8(rc, rs, b.cpu().numpy(), sb.cpu().numpy())
            tol = (128 + rs.shape[1] + 2) * 2.0 ** -23 * mag + np.abs(ref) * 2.0 ** -24
            assert np.all(np.abs(C.double().cpu().numpy() - ref) <= tol)
    assert status() == 0


def test_operands_past_4_gb():
    """Rows of A and C whose byte offsets pass 2^32 (a scale per row tells them apart)."""
    M, N, K = 70000, 33000, 16
    one = 0x38
    a = torch.full((M, K), one, dtype=torch.uint8, device="cuda")
    b = torch.full((N, K), one, dtype=torch.uint8, device="cuda")
    sa = (torch.arange(M, device="cuda") % 251).float().unsqueeze(1)
    sb = (torch.arange(-(-N // 128), device="cuda") % 3 + 1).float().unsqueeze(1)
    C = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    abi.csa2_matmul_fp8(a, sa, b, sb, C)
    assert status() == 0
    cols = (torch.arange(N, device="cuda") // 128 % 3 + 1).float() * 16
    for m in (0, 1, 127, 128, 32767, 65100, 65300, 69999):
        assert torch.equal(C[m], (float(m % 251) * cols).bfloat16())
