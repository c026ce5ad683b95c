"""GPU page operations on maps that contradict themselves: a row that names a
page nobody holds is refused, whatever the call does with that page."""
import pytest
import torch

from tests.test_gpu_pages import Both, i32, vc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("at", [2, 31, 40, 1024, 1025, 2500])
def test_reserve_refuses_a_page_that_the_same_call_hands_out(at):
    """Row 0 gets page 1 in place of one that it shares; row `at` names page 1 although it was free."""
    rows = at + 3
    table = [[-1] * 3 for _ in range(rows)]
    table[0][0] = table[1][0] = 0
    table[at][0] = 1
    held = [int(b in (0, 1, at)) for b in range(rows)]
    b = Both(table, held, [2, 0, 0, 0, 0, 0])
    want = [0] * rows
    want[0], want[at], want[at + 1] = 6, 33, 20
    b.reserve([5 * h for h in held], want)
    assert b.o.bad and b.o.blocks[at] == 1 and b.o.blocks[at + 1] == 2


@pytest.mark.parametrize("n", [1, 17, 300])
def test_fork_refuses_a_page_that_nobody_holds(n):
    """Page n + 2 of row 0 is free by its count; it stays so, however many pairs name it, and page 1 of
    row 1, also in row 0, is shared by the pairs of row 1 alone."""
    pages = list(range(n + 2)) + [n + 2]
    table = [pages, [1] + [-1] * (n + 2)] + [[-1] * (n + 3) for _ in range(2 * n)]
    refs = [1] * (n + 2) + [0, 0]
    refs[1] = 2
    b = Both(table, [n + 3, 1] + [0] * (2 * n), refs)
    lens = [16 * (n + 3) - 4, 9] + [0] * (2 * n)
    b.fork(lens, [0, 1] * n, list(range(2, 2 * n + 2)))
    assert b.o.bad and b.o.refs[n + 2] == 0 and b.o.refs[1] == 2 + n and b.o.refs[0] == 1
    b.st.zero_()
    b.o.bad = False
    lens[0] = 16 * (n + 2)                       # without that page the row can be shared
    b.fork(lens, [0], [2])
    assert not b.o.bad and lens[2] == lens[0]


@pytest.mark.parametrize("rows,refs", [(3, 2), (40, 2), (1500, 700)])
def test_reserve_of_a_page_that_more_rows_give_up_than_hold_it(rows, refs):
    """Every row gets a page of its own; the count of the one that they held ends at none and is reported."""
    b = Both([[0]] * rows, [1] * rows, [refs] + [0] * rows)
    g, s, d = (i32([7] * rows) for _ in range(3))
    vc().pages_reserve(b.m, i32([5] * rows), i32([6] * rows), g, s, d, b.ws, status=b.st)
    torch.cuda.synchronize()
    assert b.st.item() == 3 and g.tolist() == [1] * rows and s.tolist() == [0] * rows
    assert d.tolist() == b.m.table[:, 0].tolist() == list(range(1, rows + 1))
    assert b.m.refs.tolist() == [0] + [1] * rows
