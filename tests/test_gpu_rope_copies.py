"""Channels that a rotation copies keep their bits (NaN payloads too) where x and y have the same type."""
import pytest
import torch

from compressed_sparse_attention_05_gb300 import abi, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    abi.lib()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,start,r", [(128, 64, 64), (128, 8, 0), (128, 0, 62), (128, 66, 62), (128, 2, 4), (128, 3, 10), (127, 5, 20), (64, 6, 4)])
@pytest.mark.parametrize("odd", [False, True])
def test_copied_bits(d, start, r, odd, dtype, layout):
    n, heads = 45, 3
    g = torch.Generator().manual_seed(d + start + r)
    kind, bits = (torch.int16, 16) if dtype == torch.bfloat16 else (torch.int32, 32)
    any_bits = torch.randint(-2 ** (bits - 1), 2 ** (bits - 1), (n, heads, d), generator=g).to(kind)   # every pattern, NaN among them
    nan = 0x7F81 if bits == 16 else 0x7F800123
    any_bits[::2, :, ::3] = nan
    extra = 1 if odd else 8                                # rows that start on 16 bytes, or on none
    x = torch.zeros(n, heads, d + extra, dtype=kind, device="cuda")[:, :, :d]
    x.copy_(any_bits)
    y = torch.zeros(n, heads, d + extra, dtype=kind, device="cuda")[:, :, :d]
    table = torch.empty(max(r // 2, 1), dtype=torch.int64, device="cuda")[:r // 2]
    abi.csa2_rope_table(abi.RopeSpec(scaling=abi.ROPE_PLAIN, base=10000.0, factor=1.0), r, table)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    abi.csa2_rope(x.view(dtype), y.view(dtype), pos, table, start=start, layout=abi.ROPE_HALF if layout == "half" else abi.ROPE_INTERLEAVED)
    assert torch.equal(y[:, :, :start], x[:, :, :start])
    assert torch.equal(y[:, :, start + r:], x[:, :, start + r:])
    assert abi.csa2_get_status() == 0
