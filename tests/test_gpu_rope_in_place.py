"""Rotation in place touches the rotated channels and no other: their bits stay, and neighbouring ranges of a head
can be rotated at the same time."""
import pytest
import torch

from compressed_sparse_attention_05_gb300 import abi, build

pytestmark = pytest.mark.gpu

RANGES = [(0, 62), (2, 4), (6, 2), (6, 4), (66, 62), (2, 126), (120, 6), (4, 8), (1, 62), (3, 6)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    abi.lib()


def table_of(r):
    t = torch.empty(r // 2, dtype=torch.int64, device="cuda")
    abi.csa2_rope_table(abi.RopeSpec(scaling=abi.ROPE_PLAIN, base=10000.0, factor=1.0), r, t)
    return t


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def with_nans(n, heads, d, dtype, seed):
    """NaN of every kind beside ordinary values: (x, where they are)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads, d, generator=g).to(dtype)
    nan = torch.rand(x.shape, generator=g) < 0.5
    if dtype == torch.bfloat16:
        b = torch.randint(0x7F81, 0x8000, x.shape, generator=g) - 0x8000 * torch.randint(0, 2, x.shape, generator=g)
        b = b.to(torch.int16)
    else:
        b = torch.randint(0x7F800001, 0x7FFFFFFF, x.shape, generator=g) - 2 ** 31 * torch.randint(0, 2, x.shape, generator=g)
        b = b.to(torch.int32)
    return torch.where(nan, b, bits(x)).view(dtype).cuda()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("start,r", RANGES)
def test_bits_beside_the_range_stay(start, r, dtype, layout):
    x = with_nans(37, 3, 128, dtype, start + r)
    before = bits(x).clone()
    pos = torch.arange(37, dtype=torch.int32, device="cuda")
    abi.csa2_rope(x, x, pos, table_of(r), start=start, layout=abi.ROPE_HALF if layout == "half" else abi.ROPE_INTERLEAVED)
    assert torch.equal(bits(x)[:, :, :start], before[:, :, :start])
    assert torch.equal(bits(x)[:, :, start + r:], before[:, :, start + r:])
    assert abi.csa2_get_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cut", [62, 66, 4, 124])
def test_neighbouring_ranges_on_two_streams(cut, dtype):
    n, heads, d = 512, 8, 128
    g = torch.Generator().manual_seed(cut)
    x = torch.randn(n, heads, d, generator=g).to(dtype).cuda()
    pos = torch.randint(0, 1 << 16, (n,), generator=g).int().cuda()
    parts = [(0, cut, table_of(cut)), (cut, d - cut, table_of(d - cut))]
    want = x.clone()
    for start, r, table in parts:
        abi.csa2_rope(want, want, pos, table, start=start, layout=abi.ROPE_INTERLEAVED)
    y = torch.empty_like(x)
    streams = [torch.cuda.Stream() for _ in parts]
    for _ in range(100):
        y.copy_(x)
        torch.cuda.synchronize()
        for s, (start, r, table) in zip(streams, parts):
            with torch.cuda.stream(s):
                abi.csa2_rope(y, y, pos, table, start=start, layout=abi.ROPE_INTERLEAVED)
        torch.cuda.synchronize()
        assert torch.equal(bits(y), bits(want))
    assert abi.csa2_get_status() == 0
