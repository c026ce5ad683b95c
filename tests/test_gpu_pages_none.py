"""Compacting a pool without pages: no moves, and the outputs say so."""
import pytest
import torch

from tests.test_gpu_pages import i32, status, vc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,room", [(0, 0), (0, 4), (3, 0), (3, 2000)])
def test_no_pages(rows, room):
    m = vc()
    none = m.PageMap.allocate(0, rows, 2)
    src, dst, moves, st = i32([9] * room), i32([9] * room), i32([9]), status()
    m.pages_compact(none, src, dst, moves, i32([]), torch.empty(m.pages_workspace_bytes(none), dtype=torch.uint8, device="cuda"),
                    status=st)
    torch.cuda.synchronize()
    assert moves.item() == 0 and st.item() == 0 and src.tolist() == dst.tolist() == [-1] * room
