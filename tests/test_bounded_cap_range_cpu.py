"""The logit cap is refused where the kernels could not represent it (no GPU needed)."""
import pytest

from compressed_sparse_attention_05_gb300 import abi
from test_bounded_abi_cpu import attn, dims, err, lib, weights  # noqa: F401


@pytest.mark.parametrize("call", [attn, weights], ids=["attn", "weights"])
def test_caps_at_both_ends(lib, call):  # noqa: F811
    for cap in (3e38, 2.0 ** 127 * (1 + 2.0 ** -23), 2.0 ** -127, 1e-45):     # times log2(e), or its reciprocal, overflows
        assert call(lib, mods=abi.ScoreMods(logit_cap=cap)) == 1 and "logit_cap" in err(), cap
    for cap in (0.0, 2.0 ** -126, 1e-30, 50.0, 1e38, 2.0 ** 127):             # accepted: the workspace is what is missing
        assert call(lib, mods=abi.ScoreMods(logit_cap=cap), dm=dims(Tq=40), ws=None) == 4, cap
