"""GPU page operations on maps that contradict themselves: a row that names a
page nobody holds is refused, whatever the call does with that page."""
import pytest

from tests.test_gpu_pages import Both

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
