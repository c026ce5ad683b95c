"""The page operations' sequential definitions where a map contradicts itself:
what is refused follows from the state that a call finds."""
from oracle import pages as P


def test_reserve_refuses_a_page_that_the_same_call_hands_out():
    m = P.Map([[0, -1, -1], [0, -1, -1], [1, -1, -1]], [1, 1, 1], [2, 0, 0, 0, 0])
    granted, src, dst = m.reserve([5, 5, 5], [6, 0, 33])
    assert m.bad and granted == [1, 1, 0] and (src, dst) == ([0, -1, -1], [1, -1, -1])
    assert m.blocks.tolist() == [1, 1, 1] and m.table.tolist() == [[1, -1, -1], [0, -1, -1], [1, -1, -1]]
    assert m.refs.tolist() == [1, 1, 0, 0, 0]


def test_fork_refuses_a_page_that_nobody_holds():
    m = P.Map([[0, 1], [2, -1], [-1, -1], [-1, -1]], [2, 1, 0, 0], [1, 0, 1])
    lens = [20, 5, 0, 0]
    m.fork(lens, [0, 1], [2, 3])
    assert m.bad and m.refs.tolist() == [1, 0, 2] and m.blocks.tolist() == [2, 1, 0, 1] and lens == [20, 5, 0, 5]
