"""Positions or slots that are wanted, but have no column: a sequence with new ones waits, as with too few columns."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_05_gb300 import abi, build

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B", [3, 100])
@pytest.mark.parametrize("wanted", ["q_pos", "slots", "neither"])
def test_no_columns(wanted, B):
    build.build()
    new = np.array([0, 4, -4] + [0] * (B - 3))
    n_pages = B + 4
    length, held = i32([8] * B), i32([1] * B)
    table, free, n_free = i32(np.arange(B)[:, None]), i32(list(range(B, n_pages)) + [-1] * B), i32([4])
    dims = abi.Dims(B=B, Tq=0, max_pages=1)
    pool = abi.PagePool(page_table=table.data_ptr(), held=held.data_ptr(), free_pages=free.data_ptr(), n_free=n_free.data_ptr(), n_pages=n_pages)
    n_entries, first, granted = (i32([-9] * B) for _ in range(3))
    ws = torch.empty(abi.csa2_page_plan_workspace_size(dims), dtype=torch.uint8, device="cuda")
    q_pos = torch.empty(B, 0, dtype=torch.int32, device="cuda") if wanted == "q_pos" else None
    slots = torch.empty(B, 0, dtype=torch.int64, device="cuda") if wanted == "slots" else None
    abi.csa2_page_plan(dims, pool, length, i32(new), length, n_entries, first, ws, q_pos=q_pos, slots=slots, granted=granted)
    torch.cuda.synchronize()
    waits = wanted != "neither"
    assert abi.csa2_get_status() == (abi.STATUS_BAD_COUNT if waits else 0)
    assert granted.tolist() == [1, 0 if waits else 1, 1] + [1] * (B - 3)
    assert length.tolist() == [8, 8 if waits else 12, 4] + [8] * (B - 3)
    assert n_entries.tolist() == [2, 2 if waits else 3, 1] + [2] * (B - 3)
