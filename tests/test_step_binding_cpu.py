"""The binding refuses small operands of the wrong type or size before anything is launched (no GPU needed)."""
import pytest
import torch

from compressed_sparse_attention_05_gb300 import abi

i32, i64, f32, u8 = torch.int32, torch.int64, torch.float32, torch.uint8


def zeros(*n, t=f32):
    return torch.zeros(*n, dtype=t)


@pytest.mark.parametrize("positions,table,match", [
    (zeros(4, t=i64), zeros(32, t=i64), "positions"),             # torch's default type
    (zeros(4), zeros(32, t=i64), "positions"),
    (zeros(3, t=i32), zeros(32, t=i64), "positions"),             # too short
    (zeros(5, t=i32), zeros(32, t=i64), "positions"),
    (zeros(4, 2, t=i32), zeros(32, t=i64), "positions"),
    (zeros(4, t=i32), zeros(32, t=i32), "table"),
    (zeros(4, t=i32), zeros(32, t=torch.float64), "table"),
])
def test_rope(positions, table, match):
    x = zeros(4, 2, 64)
    with pytest.raises(ValueError, match=match):
        abi.csa2_rope(x, x, positions, table)


def test_rope_table():
    for t in (zeros(32, t=f32), zeros(32, t=i32), zeros(31, t=i64)):
        with pytest.raises(ValueError, match="table"):
            abi.csa2_rope_table(abi.RopeSpec(scaling=abi.ROPE_PLAIN, base=10000.0, factor=1.0), 64, t)


@pytest.mark.parametrize("codes,scales,match", [
    (zeros(4, 144), zeros(4, 2), "codes"),                        # four bytes a code
    (zeros(4, 144, t=torch.float16), zeros(4, 2), "codes"),
    (zeros(4, 144, t=u8), zeros(4, 1), "scales"),
    (zeros(4, 144, t=u8), zeros(2, 4), "scales"),
    (zeros(4, 144, t=u8), zeros(9), "scales"),
    (zeros(4, 144, t=u8), zeros(4, 2, t=torch.bfloat16), "scales"),
    (zeros(4, 144, t=u8), zeros(4, 2, t=torch.float64), "scales"),
])
def test_pack(codes, scales, match):
    with pytest.raises(ValueError, match=match):
        abi.csa2_pack_fp8_blocks(zeros(4, 144), codes, scales)


@pytest.mark.parametrize("kw,match", [
    (dict(A=zeros(4, 144)), "A must"), (dict(Bw=zeros(300, 144, t=torch.bfloat16)), "Bw must"),
    (dict(a_scales=zeros(2, 4)), "a_scales"), (dict(a_scales=zeros(4, 1)), "a_scales"), (dict(a_scales=zeros(4, 2, t=torch.bfloat16)), "a_scales"),
    (dict(b_scales=zeros(2, 3)), "b_scales"), (dict(b_scales=zeros(300, 2)), "b_scales"), (dict(b_scales=zeros(3, 2, t=torch.float64)), "b_scales"),
])
def test_matmul(kw, match):
    a = dict(A=zeros(4, 144, t=u8), a_scales=zeros(4, 2), Bw=zeros(300, 144, t=u8), b_scales=zeros(3, 2), out=zeros(4, 300))
    a.update(kw)
    with pytest.raises(ValueError, match=match):
        abi.csa2_matmul_fp8(**a)


def test_what_is_right_gets_as_far_as_the_device():
    e4m3 = torch.float8_e4m3fn
    for codes in (zeros(4, 144, t=u8), zeros(4, 144).to(e4m3)):
        for scales in (zeros(4, 2), zeros(8)):
            with pytest.raises(ValueError, match="CUDA"):
                abi.csa2_pack_fp8_blocks(zeros(4, 144), codes, scales)
        with pytest.raises(ValueError, match="CUDA"):
            abi.csa2_matmul_fp8(codes, zeros(4, 2), zeros(300, 144, t=u8), zeros(3, 2), zeros(4, 300))
    x = zeros(4, 2, 64)
    for table in (zeros(32, t=i64), zeros(32, t=torch.uint64)):
        for positions in (zeros(4, t=i32), zeros(2, 2, t=i32)):
            with pytest.raises(ValueError, match="CUDA"):
                abi.csa2_rope(x, x, positions, table)
