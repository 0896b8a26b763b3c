"""Values that the whole-cache kernels must carry through or keep apart: NaN, infinite lse, scales at the end of
their range, a long tail beside a peak."""

import pytest
import torch

from bounded_case import Case
from compressed_sparse_attention_05_gb300 import abi, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    abi.lib()


def status():
    torch.cuda.synchronize()
    return abi.csa2_get_status()


def two_tokens(**kw):
    """Two tokens of one tile; entries below 295 and window rows below 1180 are hidden from the second."""
    return Case(**{**dict(seed=11, Tq=2, Hq=8, lens=(300,), W=16, q_pos=[[1170, 1199]], docs=[[0, 1180]]), **kw})


# ---- NaN window rows at d = 64 ---------------------------------------------------------
@pytest.mark.parametrize("bad", ["scale", "code"])
def test_nan_window_rows_of_the_small_kernel(bad):
    c = two_tokens(d=64)
    at = 1165 - int(c.pos0[0])
    if bad == "scale":
        c.t["wscales"][0, at] = float("nan")
    else:
        c.t["wcodes"][0, at, 5] = 0x7F
    c.attend()
    assert status() == 0
    assert c.lse[0, 0].isnan().all() and c.O[0, 0].isnan().all()
    c.check_attention([(0, 1)])
